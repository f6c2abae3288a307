"""The paged calls on the CPU: the oracle's own pins, and what the library and
the binding refuse before anything reaches a device."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import oracle
import sequence_depth_attention_moda_b200 as moda
from sequence_depth_attention_moda_b200 import build as moda_build
from paged_cases import Tree, make_tree, mask_words, oracle_tree, random_parents

FAKE = 0x10000   # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    moda_build.build()
    return moda.load()


# ---------------------------------------------------------------- oracle pins --
def test_tree_oracle_chain_is_the_operator():
    """A chain over nothing held is the causal operator; one new token over a
    cache is decoding."""
    rng = np.random.default_rng(3)
    T, Hq, Hk, d, L = 9, 4, 2, 8, 3
    q, k, v = (rng.standard_normal((T, h, d)) for h in (Hq, Hk, Hk))
    kd, vd = (rng.standard_normal((T, Hk, L, d)) for _ in range(2))
    P = 4
    table = np.array([[2, 0, 3]])
    kc, vc = np.full((4, Hk, P, d), np.nan), np.full((4, Hk, P, d), np.nan)
    for t in range(T):
        kc[table[0][t // P], :, t % P], vc[table[0][t // P], :, t % P] = k[t], v[t]
    o, lse = oracle.tree_decode(q, kc, vc, kd, vd, table, [0], [0, T])
    flat = lambda x: x.transpose(1, 0, 2, 3).reshape(1, Hk, T * L, d)  # noqa: E731
    O, LSE = oracle.fwd(q.transpose(1, 0, 2)[None], k.transpose(1, 0, 2)[None], v.transpose(1, 0, 2)[None],
                        flat(kd), flat(vd))
    np.testing.assert_allclose(o, O[0].transpose(1, 0, 2), atol=1e-12)
    np.testing.assert_allclose(lse, LSE[0].T, atol=1e-12)
    o1, l1 = oracle.tree_decode(q[-1:], kc, vc, kd[-1:], vd[-1:], table, [T - 1], [0, 1], [np.ones((1, 1), bool)])
    O1, L1 = oracle.decode(q[-1][None], k.transpose(1, 0, 2)[None], v.transpose(1, 0, 2)[None], kd[-1][None],
                           vd[-1][None])
    np.testing.assert_allclose(o1, O1, atol=1e-12)
    np.testing.assert_allclose(l1, L1, atol=1e-12)


def test_tree_oracle_branch_is_its_own_chain():
    """Each token of a tree sees what it would as the last token of a chain of
    its ancestors."""
    c = Tree(held=(5, 0), new=(6, 3), Hq=2, Hk=1, d=64, L=2, page=8)
    x, see, _ = make_tree(c)
    o, lse = oracle_tree(c, x, see)
    cu = x["cu"].numpy()
    for b in range(2):
        for i in range(c.new[b]):
            path = np.nonzero(see[b][i])[0]
            assert path[-1] == i
            key = np.concatenate([np.arange(c.held[b]), c.held[b] + path])
            page = x["table"].numpy()[b][key // c.page].astype(np.int64)
            k = x["kc"].double().numpy()[page, 0, key % c.page]
            v = x["vc"].double().numpy()[page, 0, key % c.page]
            row = cu[b] + i
            for h in range(c.Hq):
                kk = np.concatenate([k, x["Kd"][row, 0].double().numpy()])
                vv = np.concatenate([v, x["Vd"][row, 0].double().numpy()])
                s = kk @ x["q"][row, h].double().numpy() / 8.0
                p = np.exp(s - s.max())
                np.testing.assert_allclose(o[row, h], p @ vv / p.sum(), atol=1e-12)
                np.testing.assert_allclose(lse[row, h], s.max() + np.log(p.sum()), atol=1e-12)


def test_tree_oracle_empty_row():
    c = Tree(held=(0,), new=(3,), Hq=2, Hk=1, d=64, L=0, page=8)
    see = [np.array([[0, 0, 0], [1, 0, 0], [0, 0, 1]], dtype=bool)]
    x, see, _ = make_tree(c, see)
    o, lse = oracle_tree(c, x, see)
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all() and np.isfinite(lse[1:]).all()


def test_mask_oracle():
    see, pos = oracle.tree_mask([-1, 0, 0, 2, -1, -1, 0], [0, 5, 7], [10, 20])
    assert see[0].tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 0, 1, 1, 0], [0, 0, 0, 0, 1]]
    assert pos.tolist() == [10, 11, 11, 12, 10, 20, 21]
    m = mask_words([np.eye(33, dtype=bool)], 2)
    assert m[31, 0] == -2 ** 31 and m[32, 1] == 1 and m[32, 0] == 0


def test_plan_oracle_gives_back_what_it_took():
    rng = np.random.default_rng(5)
    P = 8
    held = rng.integers(0, 60, 6)
    pages = [-(-int(h) // P) for h in held]
    order = list(map(int, rng.permutation(80)))
    rows, at = [], 0
    for n in pages:
        rows.append(order[at:at + n])
        at += n
    free = order[at:]
    want = held + rng.integers(0, 20, 6)
    cu, granted, slots, rows2, free2 = oracle.page_plan(held, want, {"rows": rows, "max_pages": 20}, free, P, 200)
    assert granted == want.tolist() and cu[-1] == int((want - held).sum())
    used = [p for r in rows2 for p in r] + free2
    assert sorted(used) == list(range(80))
    cu3, back, slots3, rows3, free3 = oracle.page_plan(granted, held, {"rows": rows2, "max_pages": 20}, free2, P, 4)
    assert rows3 == rows and free3 == free and back == held.tolist() and set(slots3) == {-1}


def test_plan_oracle_drops_what_names_no_page():
    P = 8
    table = {"rows": [[5, 2, -1, 99], [], [7]], "max_pages": 6}
    cu, granted, slots, rows, free = oracle.page_plan([32, 0, 3], [0, 17, 5], table, [3, 1], P, 20, n_pages=10)
    # pages 5 and 2 come back, the other two entries do not; three pages are asked for
    assert granted == [0, 17, 5] and cu == [0, 0, 17, 19] and free == [3]
    assert rows == [[], [5, 2, 1], [7]]
    assert slots == [5 * P + i for i in range(8)] + [2 * P + i for i in range(8)] + [P] + [7 * P + 3, 7 * P + 4, -1]
    # an entry of the list that names none is entered as -1, and its tokens have no slot
    cu, granted, slots, rows, free = oracle.page_plan([0], [9], {"rows": [[]], "max_pages": 6}, [4, -3, 6], P, 9, n_pages=10)
    assert granted == [9] and rows == [[6, -1]] and slots == [6 * P + i for i in range(8)] + [-1] and free == [4]


# ------------------------------------------------------------------- refusals --
def base(**kw):
    b = dict(B=2, N=8, Hq=8, Hk=2, d=128, L=4, page_size=16, n_pages=10, max_pages=4, mask_words=1)
    b.update(kw)
    return moda.make_paged_shape(**b)


PAGE_ERRORS = [(dict(B=-1), 1), (dict(N=-1), 1), (dict(page_size=24), 1), (dict(page_size=4), 1),
               (dict(page_size=2048), 1), (dict(page_size=0), 1), (dict(n_pages=0), 1), (dict(max_pages=0), 1),
               (dict(page_size=1024, max_pages=1 << 22), 3), (dict(B=1 << 20, max_pages=1 << 12), 3)]
CACHE_ERRORS = [(dict(d=96), 3), (dict(Hk=0), 1), (dict(dtype=5), 1), (dict(n_pages=1 << 30, Hk=4), 3)]
TREE_ERRORS = [(dict(Hq=9), 1), (dict(Hq=0), 1), (dict(Hq=130, Hk=2), 3), (dict(L=-1), 1), (dict(depth_window=5), 1),
               (dict(depth_window=-1), 1), (dict(softmax_scale=float("nan")), 1), (dict(softmax_scale=-1.0), 1),
               (dict(softmax_scale=float("inf")), 1), (dict(mask_words=-1), 1), (dict(mask_words=65), 1),
               (dict(N=1 << 29, Hq=8), 3)]


def call(lib, name, sh, n, *tail):
    return getattr(lib, name)(ctypes.byref(sh) if sh is not None else None, *([FAKE] * n), *tail, None)


@pytest.mark.parametrize("kw,status", PAGE_ERRORS + CACHE_ERRORS + TREE_ERRORS)
def test_tree_decode_rejects_bad_shapes(lib, kw, status):
    sh = base(**kw)
    assert call(lib, "moda_tree_decode", sh, 12, 1 << 40) == status, moda.moda_last_error_message()
    assert moda.moda_last_error_message()
    assert lib.moda_tree_decode_workspace_size(ctypes.byref(sh)) == ctypes.c_size_t(-1).value
    with pytest.raises(moda.MoDAError) as err:
        moda.moda_tree_decode_workspace_size(sh)
    assert err.value.status == status


@pytest.mark.parametrize("kw,status", PAGE_ERRORS + [(dict(B=16385, max_pages=2), 3)])
def test_plan_rejects_bad_shapes(lib, kw, status):
    # distinct fake addresses: held and granted must not alias
    sh = base(**kw)
    ptrs = [FAKE + 256 * i for i in range(8)]
    assert lib.moda_page_plan(ctypes.byref(sh), *ptrs, None) == status, moda.moda_last_error_message()


@pytest.mark.parametrize("kw,status", PAGE_ERRORS + CACHE_ERRORS)
def test_append_rejects_bad_shapes(lib, kw, status):
    assert call(lib, "moda_cache_append", base(**kw), 5) == status, moda.moda_last_error_message()


@pytest.mark.parametrize("kw,status", PAGE_ERRORS + [(dict(mask_words=0), 1), (dict(mask_words=65), 1)])
def test_mask_rejects_bad_shapes(lib, kw, status):
    assert call(lib, "moda_tree_mask", base(**kw), 5) == status, moda.moda_last_error_message()


@pytest.mark.parametrize("B", [2 ** 31 - 1, 2 ** 31 - 1023])
def test_too_many_requests(lib, B):
    """A thread's share of them is rounded up in 32 bits."""
    sh = base(B=B, max_pages=1, Hq=1, Hk=1)
    assert call(lib, "moda_tree_decode", sh, 12, 1 << 40) == moda.MODA_ERR_UNSUPPORTED
    assert lib.moda_tree_decode_workspace_size(ctypes.byref(sh)) == ctypes.c_size_t(-1).value
    assert call(lib, "moda_tree_mask", sh, 5) == moda.MODA_ERR_UNSUPPORTED
    assert lib.moda_tree_decode_workspace_size(ctypes.byref(base(B=2 ** 28, max_pages=1, N=64))) > 0


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 512, 1024])
def test_table_length_leaves_room_for_a_tile(lib, page):
    """Positions up to a tile behind the longest request fit 32 bits."""
    most = (2 ** 31 - 1024) // page
    for pages, ok in ((most, True), (most + 1, False), (2 ** 31 // page - 1, page == 1024)):
        sh = base(B=1, Hq=2, Hk=1, page_size=page, max_pages=pages)
        assert (lib.moda_tree_decode_workspace_size(ctypes.byref(sh)) != ctypes.c_size_t(-1).value) == ok
        if ok:
            continue
        assert call(lib, "moda_tree_decode", sh, 12, 1 << 40) == moda.MODA_ERR_UNSUPPORTED
        assert lib.moda_page_plan(ctypes.byref(sh), *[FAKE + 256 * i for i in range(8)], None) == moda.MODA_ERR_UNSUPPORTED


@pytest.mark.parametrize("scale", [-1.0, float("inf"), float("nan")])
def test_refused_scale_says_what_is_accepted(lib, scale):
    assert call(lib, "moda_tree_decode", base(softmax_scale=scale), 12, 1 << 40) == moda.MODA_ERR_INVALID_ARG
    assert ">= 0 and finite" in moda.moda_last_error_message()


def test_null_shape_and_pointers(lib):
    for name, n in (("moda_page_plan", 8), ("moda_cache_append", 5), ("moda_tree_mask", 5)):
        assert call(lib, name, None, n) == 1
        for k in range(n):
            if (name, k) == ("moda_tree_mask", 2):
                continue                       # held_len may be NULL
            ptrs = [FAKE + 256 * i for i in range(n)]
            ptrs[k] = None
            assert getattr(lib, name)(ctypes.byref(base()), *ptrs, None) == 1, (name, k)
            ptrs[k] = FAKE + 8
            assert getattr(lib, name)(ctypes.byref(base()), *ptrs, None) == 2, (name, k)
    assert call(lib, "moda_tree_decode", None, 12, 1 << 40) == 1
    for k in range(12):
        ptrs = [FAKE] * 12
        ptrs[k] = None
        assert lib.moda_tree_decode(ctypes.byref(base()), *ptrs, 1 << 40, None) == 1, k
        ptrs[k] = FAKE + 4
        assert lib.moda_tree_decode(ctypes.byref(base()), *ptrs, 1 << 40, None) == 2, k
    # a mask where the shape says chain
    assert call(lib, "moda_tree_decode", base(mask_words=0), 12, 1 << 40) == 1


def test_plan_rejects_aliased_lengths(lib):
    for alias in (0, 1):
        ptrs = [FAKE + 256 * i for i in range(8)]
        ptrs[6] = ptrs[alias]
        assert lib.moda_page_plan(ctypes.byref(base()), *ptrs, None) == 1
        assert "alias" in moda.moda_last_error_message()


def test_empty_calls_are_noops(lib):
    for kw in (dict(B=0), dict(N=0)):
        sh = base(**kw)
        assert lib.moda_tree_decode(ctypes.byref(sh), *([None] * 12), 0, None) == 0
        assert lib.moda_tree_mask(ctypes.byref(sh), *([None] * 5), None) == 0
        assert moda.moda_tree_decode_workspace_size(sh) == 0
    assert lib.moda_cache_append(ctypes.byref(base(N=0)), *([None] * 5), None) == 0


def test_workspace_does_not_grow_with_lengths(lib):
    """The records are two slots a CTA, whatever the cache holds."""
    small = moda.moda_tree_decode_workspace_size(base(max_pages=4))
    assert small == moda.moda_tree_decode_workspace_size(base(max_pages=1 << 20, n_pages=1 << 20)) > 0
    assert moda.moda_tree_decode_workspace_size(base(N=1 << 16)) < 1 << 27


def test_binding_rejects_bad_tensors(lib):
    sh = base()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    good = dict(q=bf(8, 8, 128), kc=bf(10, 2, 16, 128), vc=bf(10, 2, 16, 128), Kd=bf(8, 2, 4, 128), Vd=bf(8, 2, 4, 128),
                table=i32(2, 4), held=i32(2), cu=i32(3), mask=i32(8, 1), o=bf(8, 8, 128), lse=torch.zeros(8, 8),
                ws=torch.zeros(64, dtype=torch.uint8))
    for k, v, msg in (("q", bf(7, 8, 128), "q holds"), ("q", torch.zeros(8, 8, 128), "q has dtype"),
                      ("kc", bf(9, 2, 16, 128), "k_cache holds"), ("Vd", bf(8, 2, 3, 128), "Vd holds"),
                      ("table", i32(1, 4), "block_table holds"), ("held", torch.zeros(2, dtype=torch.int64), "held_len has"),
                      ("cu", i32(2), "cu_new holds"), ("mask", i32(7, 1), "mask holds"), ("lse", bf(8, 8), "lse has"),
                      ("ws", torch.zeros(63, dtype=torch.uint8), "ws holds"), ("o", bf(8, 8, 128), "not a CUDA device")):
        a = dict(good)
        a[k] = v
        with pytest.raises(moda.MoDAError) as err:
            moda.moda_tree_decode(sh, *a.values(), 64)
        want = msg if k != "o" else "not a CUDA device"
        assert err.value.status == moda.MODA_ERR_INVALID_ARG and want in str(err.value), str(err.value)
    with pytest.raises(moda.MoDAError, match="slot_map has dtype"):
        moda.moda_page_plan(sh, i32(2), i32(2), i32(2, 4), i32(10), i32(1), i32(3), i32(2), i32(8))
    with pytest.raises(moda.MoDAError, match="k_new holds"):
        moda.moda_cache_append(sh, bf(7, 2, 128), bf(8, 2, 128), torch.zeros(8, dtype=torch.int64), good["kc"], good["vc"])
    with pytest.raises(moda.MoDAError, match="parent holds"):
        moda.moda_tree_mask(sh, i32(7), i32(3), i32(2), i32(8, 1), i32(8))


def test_dependent_launches_read_what_the_grid_before_wrote():
    """A kernel that starts while the grid before it runs must not read that
    grid's results (a plan's table, a mask) by read-only loads."""
    names = [f for f in sorted(os.listdir(moda_build.CSRC)) if f.endswith((".cu", ".cuh"))]
    text = {f: re.sub(r"//[^\n]*", "", open(os.path.join(moda_build.CSRC, f)).read()) for f in names}
    waits = [f for f in names if "griddep_wait()" in text[f] and f != "moda_ptx.cuh"]
    assert {"moda_paged.cu", "moda_tree_simt.cu", "moda_tree_sm100.cu"} <= set(waits)
    for f in waits + ["moda_tree.cuh", "moda_ptx.cuh"]:
        assert not re.search(r"__ldg|ld\.global\.nc", text[f]), f


def test_random_parents_come_before():
    p = random_parents((5, 1, 40), np.random.default_rng(0))
    i = np.concatenate([np.arange(5), np.arange(1), np.arange(40)])
    assert (p < i).all() and (p >= -1).all()

"""The paged calls on the GPU against the oracle: page plans, appends, tree
masks, the attention of drafted tokens, and a run of them together."""
import dataclasses
import threading

import numpy as np
import pytest
import torch

import oracle
import sequence_depth_attention_moda_b200 as moda
from moda_cases import Guarded
from paged_cases import (Tree, check_tree, make_tree, mask_words, out_bound, random_parents, to_device, torch_dtype)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    yield
    moda.moda_check_status()


# ----------------------------------------------------------------------- plan --
def dev_i32(v):
    return torch.as_tensor(np.asarray(v, dtype=np.int32), device=DEV)


def run_plan(P, N, held, want, table, free, count, n_pages):
    """The call on guarded outputs; table and free are updated in place."""
    B = len(held)
    sh = moda.make_paged_shape(B, N, 1, 1, 128, 0, P, n_pages, table.shape[1])
    gd = Guarded()
    cu, granted = (gd.empty(n, (k,), torch.int32, DEV, output=False) for n, k in (("cu", B + 1), ("granted", B)))
    slots = gd.empty("slots", (N,), torch.int64, DEV, output=False)
    moda.moda_page_plan(sh, dev_i32(held), dev_i32(want), table, free, count, cu, granted, slots)
    gd.check()
    return cu.tolist(), granted.tolist(), slots.tolist()


def table_of(rows, max_pages):
    t = np.full((len(rows), max_pages), -1, dtype=np.int32)
    for b, r in enumerate(rows):
        t[b, : len(r)] = r
    return dev_i32(t)


def start_pages(rng, held, P, n_pages):
    order = list(map(int, rng.permutation(n_pages)))
    rows = []
    for h in held:
        k = -(-int(h) // P)
        rows.append(order[:k])
        order = order[k:]
    return rows, order


PLANS = [  # B, P, most held, most added, spare pages
    (1, 8, 0, 1, 1), (1, 64, 1, 0, 0), (7, 16, 100, 40, 100), (300, 8, 50, 20, 2000), (513, 32, 10, 3, 900),
    (4, 16, 5000, 9000, 4000), (64, 128, 3000, 700, 5), (40, 8, 100, 100, 0), (1000, 1024, 5000, 3, 700),
    (4500, 8, 10, 1, 100),      # more requests than tokens
]


@pytest.mark.parametrize("case", PLANS, ids=lambda c: "B%d_P%d_h%d_n%d_s%d" % c)
@pytest.mark.parametrize("kind", ["grow", "mixed"])
def test_plan(case, kind):
    B, P, most, add, spare = case
    rng = np.random.default_rng(sum(case) + (kind == "grow"))
    held = rng.integers(0, most + 1, B)
    if kind == "grow":
        want = held + rng.integers(0, add + 1, B)
    else:      # some end, some shrink, some grow, some stay
        how = rng.integers(0, 4, B)
        want = np.where(how == 0, 0, np.where(how == 1, rng.integers(0, held + 1), held + (how == 2) * rng.integers(0, add + 1, B)))
    rows, free = start_pages(rng, held, P, sum(-(-int(h) // P) for h in held) + spare)
    n_pages = sum(map(len, rows)) + len(free)
    max_pages = max(1, -(-(most + add // 2) // P))       # some do not fit their row
    max_pages = max(max_pages, max(map(len, rows)))
    N = int(np.maximum(want - held, 0).sum()) + 5
    table = table_of(rows, max_pages)
    fl = dev_i32((free + [-7] * n_pages)[:max(n_pages, 1)])
    count = dev_i32([len(free)])
    n_pages = max(n_pages, 1)
    ref = oracle.page_plan(held, want, {"rows": rows, "max_pages": max_pages}, free, P, N)
    cu, granted, slots = run_plan(P, N, held, want, table, fl, count, n_pages)
    assert granted == ref[1]
    assert cu == ref[0]
    assert slots == ref[2]
    assert torch.equal(table, table_of(ref[3], max_pages))
    assert count.tolist() == [len(ref[4])] and fl.tolist()[: len(ref[4])] == ref[4]
    # giving back what the call took restores table and list, when it only took
    if kind == "grow":
        cu, back, slots = run_plan(P, 3, granted, held, table, fl, count, n_pages)
        assert back == held.tolist() and cu == [0] * (B + 1) and slots == [-1] * 3
        assert torch.equal(table, table_of(rows, max_pages))
        assert count.tolist() == [len(free)] and fl.tolist()[: len(free)] == free


def test_plan_no_requests():
    sh = moda.make_paged_shape(0, 4, 1, 1, 128, 0, 16, 3, 2)
    fl, count, cu = dev_i32([2, 0, 1]), dev_i32([3]), dev_i32([9])
    slots = torch.zeros(4, dtype=torch.int64, device=DEV)
    moda.moda_page_plan(sh, None, None, None, fl, count, cu, None, slots)
    assert cu.tolist() == [0] and count.tolist() == [3] and slots.tolist() == [-1] * 4


def bad_status():
    with pytest.raises(moda.MoDAError) as err:
        moda.moda_check_status()
    assert err.value.status == moda.MODA_ERR_INVALID_ARG and "out of range" in str(err.value)
    moda.moda_check_status()                       # the report clears it


def test_plan_out_of_range_lengths():
    """Lengths outside the table are cut, too many tokens for N get no slot;
    both are reported and nothing outside the arrays is touched."""
    P, mp = 8, 3
    table = table_of([[0, 1, 2], []], mp)
    fl, count = dev_i32([5, 4, 3, -1, -1, -1]), dev_i32([3])
    cu, granted, slots = run_plan(P, 4, [100, -5], [24, 10], table, fl, count, 6)
    bad_status()
    assert granted == [24, 10] and cu == [0, 0, 10]          # held 100 counts as 24, -5 as 0
    assert slots == [3 * 8, 3 * 8 + 1, 3 * 8 + 2, 3 * 8 + 3]
    assert table.tolist() == [[0, 1, 2], [3, 4, -1]] and count.tolist() == [1]
    # a free count beyond the cache counts as all its pages
    table, fl, count = table_of([[]], mp), dev_i32([0, 1]), dev_i32([1 << 30])
    cu, granted, slots = run_plan(P, 8, [0], [8], table, fl, count, 2)
    bad_status()
    assert granted == [8] and slots == list(range(8, 16)) and count.tolist() == [1]


def test_plan_bad_pages_do_not_reach_the_list():
    """A held length beyond the pages a request has: the entries that name no
    page are reported and not given back, so the next call gets pages only."""
    P, mp = 8, 6
    table = table_of([[5, 2, -1, 1 << 30], [7]], mp)
    fl, count = dev_i32([3, 1, -9, -9, -9, -9, -9, -9]), dev_i32([2])
    cu, granted, slots = run_plan(P, 0, [32, 3], [0, 3], table, fl, count, 8)
    bad_status()
    assert granted == [0, 3] and count.tolist() == [4] and fl.tolist()[:4] == [3, 1, 2, 5]
    assert table.tolist() == [[-1] * mp, [7] + [-1] * 5]
    cu, granted, slots = run_plan(P, 40, [0, 3], [32, 8], table, fl, count, 8)
    moda.moda_check_status()
    assert granted == [32, 8] and table.tolist() == [[5, 2, 1, 3, -1, -1], [7] + [-1] * 5] and count.tolist() == [0]
    assert slots == [p * P + i for p in (5, 2, 1, 3) for i in range(P)] + [7 * P + i for i in range(3, 8)] + [-1] * 3


def test_plan_list_entry_that_names_no_page():
    P, mp = 8, 4
    for bad in (-1, 6, 1 << 30):
        table, fl, count = table_of([[], []], mp), dev_i32([0, bad, 4, -1, -1, -1]), dev_i32([3])
        cu, granted, slots = run_plan(P, 30, [0, 0], [9, 2], table, fl, count, 6)
        bad_status()
        assert granted == [9, 2] and count.tolist() == [0] and table.tolist() == [[4, -1, -1, -1], [0, -1, -1, -1]]
        assert slots == [4 * P + i for i in range(8)] + [-1, 0, 1] + [-1] * 19
    # tokens added to a last page that is none
    table, fl, count = table_of([[3, -1]], mp), dev_i32([0, 1, 2, -1, -1, -1]), dev_i32([3])
    cu, granted, slots = run_plan(P, 12, [10], [18], table, fl, count, 6)
    bad_status()
    assert granted == [18] and table.tolist() == [[3, -1, 2, -1]]
    assert slots == [-1] * 6 + [16, 17] + [-1] * 4


@pytest.mark.parametrize("B,N", [(40, 3000), (900, 40), (900, 400000), (4500, 60000)])
def test_plan_random_bad_pages(B, N):
    """One CTA and the cluster, slots in the plan and apart."""
    P, mp = 8, 12
    rng = np.random.default_rng(B + N)
    held = rng.integers(0, P * mp + 1, B)
    want = np.where(rng.random(B) < 0.5, 0, rng.integers(0, P * mp + 9, B))
    n_pages = sum(-(-int(h) // P) for h in held) + 50
    rows, free = start_pages(rng, held, P, n_pages)
    rows = [[p if rng.random() > 0.1 else int(rng.choice([-1, n_pages, -2 ** 31, 2 ** 31 - 1])) for p in r] for r in rows]
    table, fl, count = table_of(rows, mp), dev_i32(free + [-7] * (n_pages - len(free))), dev_i32([len(free)])
    ref = oracle.page_plan(held, want, {"rows": rows, "max_pages": mp}, free, P, N, n_pages=n_pages)
    cu, granted, slots = run_plan(P, N, held, want, table, fl, count, n_pages)
    bad_status()
    assert granted == ref[1] and cu == ref[0] and slots == ref[2]
    assert torch.equal(table, table_of(ref[3], mp))
    assert count.tolist() == [len(ref[4])] and fl.tolist()[: len(ref[4])] == ref[4]


# --------------------------------------------------------------------- append --
@pytest.mark.parametrize("N,Hk,d,P,dtype", [(1, 1, 64, 8, "bf16"), (5, 3, 64, 16, "fp32"), (257, 2, 128, 64, "bf16"),
                                            (1000, 8, 128, 8, "fp32"), (4099, 5, 64, 1024, "bf16")])
def test_append(N, Hk, d, P, dtype):
    g = torch.Generator().manual_seed(N)
    dt = torch_dtype(dtype)
    n_pages = -(-N // P) + 3
    k, v = (torch.randn(N, Hk, d, generator=g).to(dt) for _ in range(2))
    k.view(-1)[0], v.view(-1)[-1] = float("nan"), float("-inf")        # bytes, whatever they say
    slots = torch.randperm(n_pages * P, generator=g)[:N]
    slots[::7] = -1
    gd = Guarded()
    kc, vc = (gd.empty(n, (n_pages, Hk, P, d), dt, DEV, output=False) for n in ("kc", "vc"))
    kc.fill_(7.0), vc.fill_(-7.0)
    sh = moda.make_paged_shape(1, N, Hk, Hk, d, 0, P, n_pages, 1, dtype=moda.MODA_FP32 if dtype == "fp32" else 0)
    moda.moda_cache_append(sh, k.to(DEV), v.to(DEV), slots.to(DEV), kc, vc)
    gd.check()
    rk, rv = torch.full((n_pages, Hk, P, d), 7.0, dtype=dt), torch.full((n_pages, Hk, P, d), -7.0, dtype=dt)
    at = slots >= 0
    rk[slots[at] // P, :, slots[at] % P] = k[at]
    rv[slots[at] // P, :, slots[at] % P] = v[at]
    raw = torch.int32 if dtype == "fp32" else torch.int16
    assert torch.equal(kc.cpu().view(raw), rk.view(raw)) and torch.equal(vc.cpu().view(raw), rv.view(raw))


def test_append_out_of_range_slots():
    sh = moda.make_paged_shape(1, 4, 1, 1, 64, 0, 8, 2, 1)
    gd = Guarded()
    kc, vc = (gd.empty(n, (2, 1, 8, 64), torch.bfloat16, DEV, output=False) for n in ("kc", "vc"))
    kc.zero_(), vc.zero_()
    k = torch.ones(4, 1, 64, dtype=torch.bfloat16, device=DEV)
    moda.moda_cache_append(sh, k, k, torch.tensor([16, 1 << 40, -2, 15], device=DEV), kc, vc)
    gd.check()
    bad_status()
    assert float(kc.float().sum()) == 64.0 and bool((kc[1, 0, 7] == 1).all())


# ----------------------------------------------------------------------- mask --
def run_mask(parent, cu, held, words, N):
    B = len(cu) - 1
    sh = moda.make_paged_shape(B, N, 1, 1, 128, 0, 16, 1, 1, words)
    gd = Guarded()
    mask, pos = gd.empty("mask", (N, words), torch.int32, DEV, output=False), gd.empty("pos", (N,), torch.int32, DEV, output=False)
    mask.fill_(-9), pos.fill_(-9)
    moda.moda_tree_mask(sh, dev_i32(parent), dev_i32(cu), None if held is None else dev_i32(held), mask, pos)
    gd.check()
    return mask.cpu(), pos.cpu()


@pytest.mark.parametrize("new,words,pad", [((1,), 1, 0), ((32, 0, 33, 1), 2, 3), ((5, 7, 300), 10, 0), ((2048,), 64, 1),
                                           ((0, 0), 1, 2), (tuple(range(64)), 3, 0)])
@pytest.mark.parametrize("kind", ["random", "chain", "flat"])
def test_mask(new, words, pad, kind):
    rng = np.random.default_rng(len(new))
    cu = np.concatenate([[0], np.cumsum(new)])
    N = int(cu[-1]) + pad
    parent = {"random": random_parents(new, rng),
              "chain": np.concatenate([np.arange(-1, n - 1) for n in new] + [[]]),
              "flat": np.full(int(cu[-1]), -1)}[kind]
    parent = np.concatenate([parent, np.full(pad, 77)]).astype(np.int32)
    held = rng.integers(0, 1000, len(new))
    see, rpos = oracle.tree_mask(parent, cu, held)
    mask, pos = run_mask(parent, cu, held, words, N)
    n = int(cu[-1])
    assert torch.equal(mask[:n], mask_words(see, words)) and pos[:n].tolist() == rpos.tolist()
    assert bool((mask[n:] == -9).all()) and bool((pos[n:] == -9).all())
    _, pos0 = run_mask(parent, cu, None, words, N)
    assert pos0[:n].tolist() == oracle.tree_mask(parent, cu)[1].tolist()


def test_mask_out_of_range():
    # a parent that is not earlier counts as the root; tokens behind 32*words get no row
    mask, pos = run_mask([-1, 1, 0, -2, 5], [0, 5], [10], 1, 5)
    bad_status()
    assert mask[:, 0].tolist() == [1, 2, 5, 8, 16] and pos.tolist() == [10, 10, 11, 10, 10]
    mask, pos = run_mask(list(range(-1, 39)), [0, 40], None, 1, 40)
    bad_status()
    assert pos[:32].tolist() == list(range(32)) and pos[32:].tolist() == [-9] * 8 and mask[32:].eq(-9).all()


# ----------------------------------------------------------------------- tree --
def run_tree(x, sh, stream=None, ws=None):
    gd = Guarded()
    n = moda.moda_tree_decode_workspace_size(sh)
    if ws is None:
        ws = gd.empty("ws", (max(n, 16),), torch.uint8, DEV, output=False)
    o = gd.empty("o", tuple(x["q"].shape), x["q"].dtype, DEV, output=False)
    lse = gd.empty("lse", tuple(x["q"].shape[:2]), torch.float32, DEV, output=False)
    o.fill_(float("nan")), lse.fill_(float("nan"))
    moda.moda_tree_decode(sh, x["q"], x["kc"], x["vc"], x["Kd"], x["Vd"], x["table"], x["held"], x["cu"], x["mask"],
                          o, lse, ws, n, stream=stream)
    gd.check()
    return o, lse


TREES = [
    Tree(held=(1000,), new=(1,), chain=True),
    Tree(held=(0,), new=(1,), L=0, chain=True),                        # nothing held: the token sees itself
    Tree(held=(0, 5, 17), new=(3, 1, 9), L=3),
    Tree(held=(127, 128, 129), new=(1, 2, 1), page=128),               # around a tile's end
    Tree(held=(63, 64, 65, 200), new=(1, 1, 64, 0), page=64, chain=True),
    Tree(held=(100, 0, 30), new=(0, 0, 5), L=48),                      # requests without new tokens
    Tree(held=(300,), new=(33,), Hq=4, Hk=4, L=1),                     # G = 1
    Tree(held=(300, 12), new=(33, 65), Hq=16, Hk=2, L=8, page=8),      # G = 8: several row tiles
    Tree(held=(77,), new=(40,), Hq=6, Hk=2, L=5),                      # G = 3
    Tree(held=(77, 3), new=(7, 2), Hq=64, Hk=1, L=6),                  # G = 64
    Tree(held=(50,), new=(3,), Hq=40, Hk=2, L=2, d=64),                # G = 20
    Tree(held=(700, 20, 4), new=(17, 31, 100), d=64, L=16, page=32),
    Tree(held=(200, 50), new=(6, 10), L=130),                          # more depth rows than a tile
    Tree(held=(200, 50), new=(6, 10), L=300, window=257, d=64),
    Tree(held=(40, 9), new=(12, 3), L=48, window=5),
    Tree(held=(2000,), new=(200,), chain=True, L=2, Hq=4, Hk=1),       # a chunk of a prompt
    Tree(held=(0, 1), new=(150, 90), chain=True, L=0, page=8),         # prompts from nothing
    Tree(held=(33, 500), new=(5, 8), pad=7, extra_words=2),
    Tree(held=tuple(range(0, 400, 7)), new=tuple(1 + k % 3 for k in range(58)), Hq=4, Hk=2, L=4),
    Tree(held=(3000, 10), new=(2, 2), page=1024, scale=0.3),
    Tree(held=(513,), new=(64,), Hq=32, Hk=8, L=16),
    Tree(held=(100, 20), new=(5, 9), dtype="fp32"),
    Tree(held=(1000, 0, 64), new=(1, 1, 1), dtype="fp32", chain=True, d=64),
    Tree(held=(300, 12), new=(33, 65), Hq=16, Hk=2, L=8, page=8, dtype="fp32"),
    Tree(held=(200, 50), new=(6, 10), L=70, window=66, d=64, dtype="fp32"),
    Tree(held=(50,), new=(9,), Hq=64, Hk=1, L=0, dtype="fp32", pad=2),
]


@pytest.mark.parametrize("c", TREES, ids=str)
def test_tree(c):
    x, see, sh = make_tree(c)
    o, lse = run_tree(to_device(x), sh)
    check_tree(c, x, see, o, lse)


# bf16 jobs of two row tiles run when requests fill more than one and the cache is
# several times L2: the same cases with a cache (and a table) that large
TWO_TILES = [
    Tree(held=(300, 12), new=(33, 65), Hq=16, Hk=2, L=8, page=8),      # G = 8: 16 tokens a row tile
    Tree(held=(2000,), new=(200,), chain=True, L=2, Hq=4, Hk=1),
    Tree(held=(0, 1), new=(150, 90), chain=True, L=0, page=8),
    Tree(held=(513, 4, 700), new=(64, 1, 40), Hq=32, Hk=8, L=16, window=9),
    Tree(held=(200, 50), new=(70, 33), L=130),
    Tree(held=tuple(range(0, 2000, 97)), new=tuple(20 + 3 * k for k in range(21)), Hq=8, Hk=2, L=5, pad=3),
    Tree(held=(3000, 10), new=(128, 200), Hq=2, Hk=2, page=1024, L=1),
]


def in_large_cache(y, sh, c):
    """The case in a cache of 360 MB of NaN and a table with as many columns."""
    n_big = 180_000_000 // (c.Hk * c.page * c.d * 2)
    for k in ("kc", "vc"):
        big = torch.full((n_big, *y[k].shape[1:]), float("nan"), dtype=y[k].dtype, device=DEV)
        big[: sh.n_pages] = y[k]
        y[k] = big
    cols = -(-n_big // sh.B)
    table = torch.full((sh.B, cols), 1 << 30, dtype=torch.int32, device=DEV)
    table[:, : sh.max_pages] = y["table"]
    y["table"] = table
    sh.n_pages, sh.max_pages = n_big, cols
    return y


@pytest.mark.parametrize("c", TWO_TILES, ids=str)
def test_tree_two_row_tiles(c):
    x, see, sh = make_tree(c)
    small = moda.moda_tree_decode_workspace_size(sh)
    y = in_large_cache(to_device(x), sh, c)
    assert moda.moda_tree_decode_workspace_size(sh) > small       # records of 256 rows
    o, lse = run_tree(y, sh)
    check_tree(c, x, see, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Hk,chain", [(385, 1, False), (800, 2, True), (1000, 1, False), (2100, 1, True)])
def test_tree_more_requests_than_threads(B, Hk, chain, dtype):
    """Several requests a thread in the schedule (384 or 256 threads add them up),
    some without new tokens, some long enough to be cut."""
    rng = np.random.default_rng(B)
    held = tuple(int(h) for h in np.where(rng.random(B) < 0.02, rng.integers(500, 2000, B), rng.integers(0, 40, B)))
    new = tuple(int(n) for n in np.where(rng.random(B) < 0.01, 20, rng.integers(0, 3, B)))
    c = Tree(held=held, new=new, Hq=2 * Hk, Hk=Hk, d=64, L=1, page=16, chain=chain, dtype=dtype, pad=2)
    x, see, sh = make_tree(c)
    o, lse = run_tree(to_device(x), sh)
    check_tree(c, x, see, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("held,L,n", [(0, 0, 40), (5, 0, 40), (0, 3, 9), (200, 2, 70)])
def test_tree_any_mask(dtype, held, L, n):
    """Masks that are no trees: rows without themselves, rows that see nothing
    (with nothing held and no depth rows: o = 0, lse = -inf)."""
    rng = np.random.default_rng(n)
    c = Tree(held=(held,), new=(n,), L=L, dtype=dtype)
    see = [rng.random((n, n)) < 0.2]
    see[0][3] = False
    see[0][n - 1] = False
    x, see, sh = make_tree(c, see)
    o, lse = run_tree(to_device(x), sh)
    check_tree(c, x, see, o, lse)
    if held == 0 and L == 0:
        assert bool((o[3] == 0).all()) and bool(torch.isneginf(lse[3]).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tree_not_finite_where_masked(dtype):
    """Infinities and NaN in a drafted token's key and value, and in a token's
    depth rows, reach the rows that see them and no others."""
    inf, nan = float("inf"), float("nan")
    c = Tree(held=(150, 20), new=(20, 9), L=4, dtype=dtype)
    x, see, sh = make_tree(c)
    at = lambda b, j: (int(x["table"][b][(c.held[b] + j) // c.page]), (c.held[b] + j) % c.page)  # noqa: E731
    p, s = at(0, 7)
    x["vc"][p, :, s, 3], x["vc"][p, 0, s, 90] = inf, nan
    p, s = at(0, 11)
    x["vc"][p, :, s, 3] = -inf
    p, s = at(1, 4)
    x["kc"][p, :, s] = nan                          # NaN scores where it is seen
    x["Vd"][5, 1, 2, 10] = -inf
    x["Kd"][25, 0, 1, 0] = nan
    o, lse = run_tree(to_device(x), sh)
    ref_finite = torch.isfinite(o[:29].float())
    assert not bool(ref_finite.all()) and bool(ref_finite.any())
    # rows with NaN scores are NaN in both; the others are compared
    check_rows_not_finite(c, x, see, o, lse)


def test_tree_not_finite_two_row_tiles():
    c = Tree(held=(150, 20), new=(70, 40), L=4)
    x, see, sh = make_tree(c)
    for b, j, v in ((0, 7, float("inf")), (0, 40, float("nan")), (1, 33, float("-inf"))):
        key = c.held[b] + j
        x["vc"][int(x["table"][b][key // c.page]), :, key % c.page, 3] = v
    x["Vd"][50, 1, 2, 10] = -float("inf")
    o, lse = run_tree(in_large_cache(to_device(x), sh, c), sh)
    check_rows_not_finite(c, x, see, o, lse)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "bf16"), (128, "fp32"), (64, "fp32")])
def test_tree_not_finite_in_a_long_chain(d, dtype):
    """Infinities and a NaN among a prompt's values: in the rows that see them and
    nowhere else, every other bit as without them, and in the time of a few clean
    calls (not of a walk over all keys for every column)."""
    n, Hq, Hk, P = 4096, 32, 8, 64
    g = torch.Generator().manual_seed(d)
    dt = torch_dtype(dtype)
    sh = moda.make_paged_shape(1, n, Hq, Hk, d, 0, P, n // P + 1, n // P + 1, 0, moda.MODA_FP32 if dtype == "fp32" else 0)
    q, kc, vc = (torch.randn(*s, generator=g).to(dt).to(DEV) for s in ((n, Hq, d), *[(n // P + 1, Hk, P, d)] * 2))
    x = dict(q=q, kc=kc, vc=vc, Kd=None, Vd=None, table=torch.arange(n // P + 1, dtype=torch.int32, device=DEV)[None].contiguous(),
             held=dev_i32([17]), cu=dev_i32([0, n]), mask=None)
    bad = ((900, 2, 5, float("inf")), (2501, 2, 5, float("-inf")), (30, 0, d - 1, float("nan")), (4000, 7, 0, float("inf")))
    y = dict(x, vc=vc.clone())
    for t, hk, col, v in bad:
        x["vc"][(17 + t) // P, hk, (17 + t) % P, col] = 0
        y["vc"][(17 + t) // P, hk, (17 + t) % P, col] = v
    nws = moda.moda_tree_decode_workspace_size(sh)
    ws = torch.empty(nws, dtype=torch.uint8, device=DEV)
    outs, best = [], []
    for z in (x, y):
        o, lse = torch.empty_like(q), torch.empty(n, Hq, device=DEV)
        times = []
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            moda.moda_tree_decode(sh, z["q"], z["kc"], z["vc"], None, None, z["table"], z["held"], z["cu"], None, o, lse, ws, nws)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        outs.append((o, lse))
        best.append(min(times))
    (o, lse), (o2, lse2) = outs
    ref = o.clone()
    for t, hk, col, v in bad:
        ref[t:, hk * 4:hk * 4 + 4, col] += v
    assert torch.equal(lse, lse2)
    assert torch.equal(o2.isnan(), ref.isnan()) and int(ref.isnan().sum()) > 0 and int(ref.isinf().sum()) > 0
    assert torch.equal(o2.nan_to_num(nan=0.0), ref.nan_to_num(nan=0.0))
    print("clean %.3f ms, with infinities %.3f ms" % tuple(best))
    assert best[1] < 10 * best[0], best


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("c", [
    Tree(held=tuple(range(0, 400, 2)), new=tuple(1 + k % 3 for k in range(200)), Hq=4, Hk=2, L=2),      # whole jobs
    Tree(held=(33,), new=(70,), L=40, window=33, page=8, d=64),
    Tree(held=(2, 900), new=(45, 20), Hq=2, Hk=2, L=1, chain=True, d=64),
    Tree(held=(70,), new=(5,), Hq=64, Hk=1, L=130, window=129),
], ids=["whole_jobs", "window", "chain", "G64"])
def test_tree_not_finite_anywhere(c, dtype):
    """Infinities and NaN strewn over the new keys' values and the depth rows, those
    outside the window among them."""
    c = dataclasses.replace(c, dtype=dtype)
    x, see, sh = make_tree(c)
    rng = np.random.default_rng(7)
    n = int(x["cu"][-1])
    for i in range(30):
        v = (float("inf"), float("-inf"), float("nan"))[i % 3]
        b = int(rng.integers(len(c.held)))
        key = c.held[b] + int(rng.integers(c.new[b]))
        x["vc"][int(x["table"][b][key // c.page]), rng.integers(c.Hk), key % c.page, rng.integers(c.d)] = v
        if c.L:
            x["Vd"][rng.integers(n), rng.integers(c.Hk), rng.integers(c.L), rng.integers(c.d)] = v
    o, lse = run_tree(to_device(x), sh)
    assert not bool(torch.isfinite(o[:n].float()).all())
    check_rows_not_finite(c, x, see, o, lse)


def check_rows_not_finite(c, x, see, o, lse):
    from paged_cases import oracle_tree
    ref, rlse = oracle_tree(c, x, see)
    clean = {k: (v.clone() if v is not None else None) for k, v in x.items()}
    for k in ("vc", "Vd"):
        clean[k][~torch.isfinite(clean[k].float())] = 0
    a, _ = oracle_tree(c, clean, see, absolute=True)
    n = int(x["cu"][-1])
    o, lse = o.double().cpu().numpy()[:n], lse.double().cpu().numpy()[:n]
    ref, rlse, a = ref[:n], rlse[:n], a[:n]
    np.testing.assert_array_equal(np.isnan(o), np.isnan(ref))
    np.testing.assert_array_equal(np.where(np.isinf(o), o, 0), np.where(np.isinf(ref), ref, 0))
    fine = np.isfinite(ref)
    assert (np.abs(o[fine] - ref[fine]) <= out_bound(c.dtype, ref[fine], a[fine])).all()
    np.testing.assert_array_equal(np.isnan(lse), np.isnan(rlse))
    seen = np.isfinite(rlse)
    assert np.abs(lse[seen] - rlse[seen]).max() <= 1e-3


def test_tree_bad_table_reads_as_zeros():
    """A table entry that names no page: reported, read as zeros."""
    c = Tree(held=(40,), new=(2,), L=0, chain=True)
    x, see, sh = make_tree(c)
    page = int(x["table"][0][1])
    for bad in (-1, 1 << 30, sh.n_pages):
        y = dict(x)
        y["table"] = x["table"].clone()
        y["table"][0][1] = bad
        o, lse = run_tree(to_device(y), sh)
        bad_status()
        z = {k: (v.clone() if v is not None else None) for k, v in x.items()}
        z["kc"][page], z["vc"][page] = 0, 0
        check_tree(c, z, see, o, lse)


def test_tree_out_of_range_lengths():
    """Lengths beyond the table, N or the mask are cut and reported."""
    c = Tree(held=(10, 10), new=(2, 2), L=0, page=16, chain=True)
    x, see, sh = make_tree(c)
    for held, cu in (([1 << 30, 10], [0, 2, 4]), ([10, -3], [0, 2, 4]), ([10, 10], [0, 2, 400]), ([10, 10], [0, 9, 4]),
                     ([10, 10], [-4, 2, 4])):
        y = dict(x)
        y["table"] = y["table"].clamp(max=sh.n_pages - 1)
        y["kc"], y["vc"] = torch.nan_to_num(x["kc"].float()).to(x["kc"].dtype), torch.nan_to_num(x["vc"].float()).to(x["vc"].dtype)
        y["held"], y["cu"] = torch.tensor(held, dtype=torch.int32), torch.tensor(cu, dtype=torch.int32)
        run_tree(to_device(y), sh)
        bad_status()
    c = Tree(held=(10,), new=(33,), L=0)
    x, see, sh = make_tree(c)
    sh.mask_words = 1
    x["mask"] = x["mask"][:, :1].contiguous()
    o, lse = run_tree(to_device(x), sh)
    bad_status()
    assert bool(torch.isnan(o[32]).all()) and not bool(torch.isnan(o[:32]).any())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("chain", [True, False])
def test_tree_starts_that_descend(dtype, chain):
    """Requests that claim the same rows: reported, and no row is written."""
    c = Tree(held=(10, 5, 7), new=(3, 2, 4), L=2, chain=chain, dtype=dtype)
    x, see, sh = make_tree(c)
    for cu in ([0, 9, 0, 9], [0, 3, 2, 9], [9, 5, 3, 0], [0, 3, 2 ** 31 - 1, -2 ** 31]):
        x["cu"] = torch.tensor(cu, dtype=torch.int32)
        o, lse = run_tree(to_device(x), sh)
        bad_status()
        assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tree_starts_outside_the_rows(dtype):
    """Starts before the first row or behind the last: each request keeps its own rows."""
    c = Tree(held=(10, 5, 7), new=(3, 2, 4), L=2, chain=True, dtype=dtype)
    x, see, sh = make_tree(c)
    for cu in ([-4, 3, 5, 9], [0, 3, 5, 40], [-2 ** 31, 3, 5, 2 ** 31 - 1]):
        y = dict(x)
        y["cu"] = torch.tensor(cu, dtype=torch.int32)
        o, lse = run_tree(to_device(y), sh)
        bad_status()
        check_tree(c, x, see, o, lse)


def test_mask_starts_out_of_range():
    mask, pos = run_mask([-1, 0, -1, 0], [-3, 2, 9], [10, 20], 1, 4)
    bad_status()
    assert mask[:, 0].tolist() == [1, 3, 1, 3] and pos.tolist() == [10, 11, 20, 21]


def test_tree_equals_decode():
    """One new token a request over equal lengths: moda_decode's result."""
    B, Hq, Hk, d, L, T, P = 3, 16, 4, 128, 5, 200, 16
    c = Tree(held=(T - 1,) * B, new=(1,) * B, Hq=Hq, Hk=Hk, d=d, L=L, page=P, chain=True)
    x, see, sh = make_tree(c)
    y = to_device(x)
    o, lse = run_tree(y, sh)
    t = x["table"][:, : -(-T // P)].long()
    K, V = (x[k][t].transpose(1, 2).reshape(B, Hk, -1, d)[:, :, :T].contiguous().to(DEV) for k in ("kc", "vc"))
    ds = moda.make_shape(B, Hq, Hk, T, d, L, 0)
    n = moda.moda_decode_workspace_size(ds)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    moda.moda_decode(ds, y["q"], K, V, y["Kd"], y["Vd"], o2, lse2, torch.empty(n, dtype=torch.uint8, device=DEV), n)
    assert (o.float() - o2.float()).abs().max() <= 2 ** -6 and (lse - lse2).abs().max() <= 1e-4


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tree_deterministic_and_replayed(dtype):
    """Equal bits again, in a graph, and in a graph replayed with other lengths."""
    c = Tree(held=(900, 70, 333), new=(9, 30, 2), dtype=dtype, L=4)
    x, see, sh = make_tree(c)
    y = to_device(x)
    o, lse = run_tree(y, sh)
    o2, lse2 = run_tree(y, sh)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    n = moda.moda_tree_decode_workspace_size(sh)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    og, lg = torch.empty_like(o), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moda.moda_tree_decode(sh, y["q"], y["kc"], y["vc"], y["Kd"], y["Vd"], y["table"], y["held"], y["cu"], y["mask"],
                              og, lg, ws, n)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, og) and torch.equal(lse, lg)
    c2 = Tree(held=(20, 800, 5), new=(9, 30, 2), dtype=dtype, L=4)
    x2 = dict(x)
    x2["held"] = torch.tensor(c2.held, dtype=torch.int32)
    # the pages of request 1 as request 0 of the longer case: any pages do, if both sides read them
    rows = torch.randint(0, sh.n_pages, x["table"].shape, generator=torch.Generator().manual_seed(4)).to(torch.int32)
    x2["table"] = rows
    x2["kc"], x2["vc"] = (torch.nan_to_num(x[k].float(), nan=0.5).to(x[k].dtype) for k in ("kc", "vc"))
    for k in ("held", "table", "kc", "vc"):
        y[k].copy_(x2[k])
    og.fill_(float("nan")), lg.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    check_tree(c2, x2, see, og, lg)


def test_tree_side_stream():
    c = Tree(held=(400,), new=(12,))
    x, see, sh = make_tree(c)
    y = to_device(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n = moda.moda_tree_decode_workspace_size(sh)
    with torch.cuda.stream(s):
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        o, lse = torch.full_like(y["q"], float("nan")), torch.full(y["q"].shape[:2], float("nan"), device=DEV)
    moda.moda_tree_decode(sh, y["q"], y["kc"], y["vc"], y["Kd"], y["Vd"], y["table"], y["held"], y["cu"], y["mask"], o, lse,
                          ws, n, stream=s)
    s.synchronize()
    check_tree(c, x, see, o, lse)


def test_tree_workspace_too_small():
    c = Tree(held=(40,), new=(2,))
    x, _, sh = make_tree(c)
    y = to_device(x)
    n = moda.moda_tree_decode_workspace_size(sh)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    with pytest.raises(moda.MoDAError) as err:
        moda.moda_tree_decode(sh, y["q"], y["kc"], y["vc"], y["Kd"], y["Vd"], y["table"], y["held"], y["cu"], y["mask"],
                              torch.empty_like(y["q"]), torch.empty(y["q"].shape[:2], device=DEV), ws, n - 1)
    assert err.value.status == moda.MODA_ERR_WORKSPACE


# fp32 keeps blocks of 4, 16 or 64 rows, for requests of that many on average, and
# tiles of 32 keys
FP32 = [
    Tree(held=(700, 33, 0), new=(1, 1, 1), Hq=8, Hk=2, L=0),
    Tree(held=(9000,), new=(1,), Hq=4, Hk=1, L=31, page=64, chain=True),          # cut over many CTAs
    Tree(held=(31, 32, 33), new=(1, 1, 1), L=48, chain=True),                     # more depth rows than a tile
    Tree(held=(95, 96), new=(4, 4), Hq=2, Hk=2, L=33, d=64),                      # G = 1
    Tree(held=(64, 200), new=(1, 1), Hq=6, Hk=2, L=32, d=64, window=7),           # G = 3
    Tree(held=(500, 31), new=(4, 2), Hq=8, Hk=2, L=31),                           # 16 rows
    Tree(held=(40, 160), new=(3, 3), Hq=10, Hk=2, L=32, d=64, chain=True),        # G = 5: 3 tokens in 15 rows
    Tree(held=(77, 3), new=(1, 1), Hq=16, Hk=1, L=2),                             # G = 16
    Tree(held=(1, 1, 1, 1), new=(16, 0, 0, 0), Hq=4, Hk=1, L=3, d=64),            # one request has all: 4 of 4 rows
    Tree(held=(333,), new=(40,), Hq=8, Hk=2, L=5, page=8),                        # 64 rows
    Tree(held=(2500, 70), new=(17, 50), Hq=12, Hk=2, L=40, d=64, page=16, pad=4), # G = 6
]


@pytest.mark.parametrize("c", FP32, ids=str)
def test_tree_fp32_blocks(c):
    c = dataclasses.replace(c, dtype="fp32")
    x, see, sh = make_tree(c)
    o, lse = run_tree(to_device(x), sh)
    check_tree(c, x, see, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tree_outputs_at_any_16_bytes(dtype):
    """Inputs, outputs and workspace that begin on odd multiples of 16 bytes."""
    c = Tree(held=(300, 20), new=(9, 2), L=5, dtype=dtype)
    x, see, sh = make_tree(c)
    y = to_device(x)

    def shifted(t):
        n = 16 // t.element_size()
        flat = torch.zeros(t.numel() + 2 * n, dtype=t.dtype, device=DEV)
        at = flat[n:n + t.numel()] if flat.data_ptr() % 32 == 0 else flat[2 * n:2 * n + t.numel()]
        assert at.data_ptr() % 32 == 16
        return at.view(t.shape).copy_(t)
    y = {k: (None if t is None else shifted(t)) for k, t in y.items()}
    n = moda.moda_tree_decode_workspace_size(sh)
    ws = shifted(torch.zeros(n, dtype=torch.uint8, device=DEV))
    o, lse = shifted(torch.full_like(y["q"], float("nan"))), shifted(torch.full(y["q"].shape[:2], float("nan"), device=DEV))
    moda.moda_tree_decode(sh, y["q"], y["kc"], y["vc"], y["Kd"], y["Vd"], y["table"], y["held"], y["cu"], y["mask"], o, lse,
                          ws, n)
    check_tree(c, x, see, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_and_tree_past_32_bit_offsets(dtype):
    """Pages whose elements begin behind 2^32."""
    c = Tree(held=(1500, 40), new=(5, 3), Hq=4, Hk=2, L=2, page=1024, dtype=dtype)
    x, see, sh = make_tree(c)
    n_big = 2 ** 32 // (c.Hk * c.page * c.d) + sh.n_pages
    y = to_device(x)
    new_k, new_v, slots = [], [], []
    used = [int(p) for b, (h, n) in enumerate(zip(c.held, c.new)) for p in x["table"][b, : -(-(h + n) // c.page)]]
    for k, rows in (("kc", new_k), ("vc", new_v)):
        big = torch.empty((n_big, *x[k].shape[1:]), dtype=x[k].dtype, device=DEV)
        for p in used:
            big[n_big - 1 - p] = y[k][p]
        for b in range(2):
            for t in range(c.held[b], c.held[b] + c.new[b]):
                p = n_big - 1 - int(x["table"][b, t // c.page])
                rows.append(big[p, :, t % c.page].clone())
                big[p, :, t % c.page] = float("nan")
                if k == "kc":
                    slots.append(p * c.page + t % c.page)
        y[k] = big
    y["table"] = torch.where(y["table"] < sh.n_pages, n_big - 1 - y["table"], y["table"]).to(torch.int32)
    sh.n_pages = n_big
    moda.moda_cache_append(sh, torch.stack(new_k), torch.stack(new_v), torch.tensor(slots, device=DEV), y["kc"], y["vc"])
    o, lse = run_tree(y, sh)
    check_tree(c, x, see, o, lse)


def test_plan_past_32_bit_slots():
    P, n_pages = 1024, 3 << 20
    fl, count = torch.arange(n_pages, dtype=torch.int32, device=DEV), dev_i32([n_pages])
    table = table_of([[], []], 3)
    cu, granted, slots = run_plan(P, 1030, [0, 0], [1025, 2], table, fl, count, n_pages)
    assert cu == [0, 1025, 1027] and granted == [1025, 2] and int(count) == n_pages - 3
    top = n_pages - 1
    assert table.tolist() == [[top, top - 1, -1], [top - 2, -1, -1]]
    assert slots == ([top * P + i for i in range(1024)] + [(top - 1) * P] + [(top - 2) * P, (top - 2) * P + 1] + [-1] * 3)


def test_plan_most_requests():
    B, P = 16384, 8
    rng = np.random.default_rng(5)
    held = rng.integers(0, 30, B)
    want = np.where(rng.random(B) < 0.2, 0, held + rng.integers(0, 5, B))
    rows, free = start_pages(rng, held, P, sum(-(-int(h) // P) for h in held) + 1000)
    n_pages = sum(map(len, rows)) + len(free)
    N = int(np.maximum(want - held, 0).sum()) + 1
    table, fl, count = table_of(rows, 5), dev_i32(free + [-7] * (n_pages - len(free))), dev_i32([len(free)])
    ref = oracle.page_plan(held, want, {"rows": rows, "max_pages": 5}, free, P, N)
    cu, granted, slots = run_plan(P, N, held, want, table, fl, count, n_pages)
    assert granted == ref[1] and cu == ref[0] and slots == ref[2]
    assert torch.equal(table, table_of(ref[3], 5)) and fl.tolist()[: len(ref[4])] == ref[4]


def test_tree_two_graphs_at_once():
    """Two captured calls, a workspace each, replayed on two streams at the same time."""
    cases = [Tree(held=(900, 70, 333), new=(9, 30, 2), L=4), Tree(held=(50,) * 40, new=(3,) * 40, L=2, seed=2)]
    runs = []
    for c in cases:
        x, see, sh = make_tree(c)
        y = to_device(x)
        n = moda.moda_tree_decode_workspace_size(sh)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        o, lse = torch.full_like(y["q"], float("nan")), torch.full(y["q"].shape[:2], float("nan"), device=DEV)
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            for _ in range(20):
                moda.moda_tree_decode(sh, y["q"], y["kc"], y["vc"], y["Kd"], y["Vd"], y["table"], y["held"], y["cu"],
                                      y["mask"], o, lse, ws, n)
        runs.append((c, x, see, graph, s, o, lse, y, ws))
    torch.cuda.synchronize()
    for _ in range(5):
        for r in runs:
            with torch.cuda.stream(r[4]):
                r[3].replay()
    torch.cuda.synchronize()
    for c, x, see, _, _, o, lse, *_ in runs:
        check_tree(c, x, see, o, lse)


def test_step_captured_over_two_streams():
    """Append on a side stream beside the mask, joined before the attention, as one graph."""
    c = Tree(held=(200, 31), new=(12, 5), L=3)
    rng = np.random.default_rng(3)
    parent = random_parents(c.new, rng)
    see, pos_ref = oracle.tree_mask(parent, np.concatenate([[0], np.cumsum(c.new)]), list(c.held))
    x, see, sh = make_tree(c, see)
    y = to_device(x)
    slots = [int(x["table"][b, t // c.page]) * c.page + t % c.page
             for b in range(2) for t in range(c.held[b], c.held[b] + c.new[b])]
    at = torch.tensor(slots)
    k, v = (x[n][at // c.page, :, at % c.page].contiguous().to(DEV) for n in ("kc", "vc"))
    y["kc"][at // c.page, :, at % c.page] = float("nan")
    y["vc"][at // c.page, :, at % c.page] = float("nan")
    par, mask, pos = dev_i32(parent), torch.zeros_like(y["mask"]), torch.zeros(len(slots), dtype=torch.int32, device=DEV)
    at = at.to(DEV)
    n = moda.moda_tree_decode_workspace_size(sh)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    o, lse = torch.full_like(y["q"], float("nan")), torch.full(y["q"].shape[:2], float("nan"), device=DEV)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        moda.moda_cache_append(sh, k, v, at, y["kc"], y["vc"], stream=side)
        moda.moda_tree_mask(sh, par, y["cu"], y["held"], mask, pos)
        main.wait_stream(side)
        moda.moda_tree_decode(sh, y["q"], y["kc"], y["vc"], y["Kd"], y["Vd"], y["table"], y["held"], y["cu"], mask, o, lse,
                              ws, n)
    graph.replay()
    torch.cuda.synchronize()
    assert pos.tolist() == pos_ref.tolist()
    check_tree(c, x, see, o, lse)


def test_tree_from_several_threads():
    """Calls of four host threads, each on its own stream with its own buffers."""
    cases = [Tree(held=(900, 70), new=(9, 30), L=4), Tree(held=(50,) * 30, new=(3,) * 30, L=2, seed=2),
             Tree(held=(300,), new=(70,), Hq=4, Hk=2, d=64, L=1, chain=True), Tree(held=(20, 400), new=(5, 8), dtype="fp32")]
    made = [make_tree(c) for c in cases]
    todo = [(c, x, see, sh, to_device(x)) for c, (x, see, sh) in zip(cases, made)]
    torch.cuda.synchronize()
    errors, outs = [], [None] * len(todo)

    def work(i):
        try:
            c, x, see, sh, y = todo[i]
            s = torch.cuda.Stream()
            n = moda.moda_tree_decode_workspace_size(sh)
            with torch.cuda.stream(s):
                ws = torch.empty(n, dtype=torch.uint8, device=DEV)
                for _ in range(60):
                    o, lse = torch.full_like(y["q"], float("nan")), torch.full(y["q"].shape[:2], float("nan"), device=DEV)
                    moda.moda_tree_decode(sh, y["q"], y["kc"], y["vc"], y["Kd"], y["Vd"], y["table"], y["held"], y["cu"], y["mask"],
                                          o, lse, ws, n)
            s.synchronize()
            outs[i] = o, lse
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(todo))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for (c, x, see, _, _), (o, lse) in zip(todo, outs):
        check_tree(c, x, see, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tree_no_new_tokens(dtype):
    """Requests without new tokens and rows that belong to none: nothing is written."""
    c = Tree(held=(40, 0, 900), new=(0, 0, 0), L=2, pad=5, dtype=dtype)
    x, see, sh = make_tree(c)
    o, lse = run_tree(to_device(x), sh)
    assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_steps_back_to_back(dtype):
    """Steps that move pages, one behind the other in a graph, each kernel set up while
    the one before runs: the bits of the same calls with a wait after each."""
    rng = np.random.default_rng(5)
    g = torch.Generator().manual_seed(5)
    dt = torch_dtype(dtype)
    B, Hq, Hk, d, L, P, n_pages, mp = 40, 8, 2, 64, 2, 8, 900, 20
    N = 3 * B
    sh = moda.make_paged_shape(B, N, Hq, Hk, d, L, P, n_pages, mp, 1, moda.MODA_FP32 if dtype == "fp32" else 0)
    nws = moda.moda_tree_decode_workspace_size(sh)
    ws = torch.empty(nws, dtype=torch.uint8, device=DEV)
    state0 = dict(kc=torch.randn(n_pages, Hk, P, d, generator=g).to(dt), vc=torch.randn(n_pages, Hk, P, d, generator=g).to(dt),
                  table=torch.full((B, mp), -1, dtype=torch.int32), free=torch.randperm(n_pages, generator=g).to(torch.int32),
                  count=torch.tensor([n_pages], dtype=torch.int32))
    state = to_device(state0)
    held, steps = rng.integers(0, 120, B), []
    big = moda.make_paged_shape(B, int(held.sum()), Hq, Hk, d, L, P, n_pages, mp)
    moda.moda_page_plan(big, dev_i32([0] * B), dev_i32(held), state["table"], state["free"], state["count"], dev_i32([0] * (B + 1)),
                        dev_i32([0] * B), torch.zeros(big.N, dtype=torch.int64, device=DEV))
    state0 = {n: t.clone() for n, t in state.items()}
    for _ in range(8):       # lengths wander up and down
        back = np.where(rng.random(B) < 0.3, rng.integers(0, held + 1), held)
        want = np.minimum(back + rng.integers(0, 4, B), mp * P)
        steps.append(dict(held=dev_i32(held), back=dev_i32(back), want=dev_i32(want),
                          parent=dev_i32(np.full(N, -1)), q=torch.randn(N, Hq, d, generator=g).to(dt).to(DEV),
                          k=torch.randn(N, Hk, d, generator=g).to(dt).to(DEV), v=torch.randn(N, Hk, d, generator=g).to(dt).to(DEV),
                          kd=torch.randn(N, Hk, L, d, generator=g).to(dt).to(DEV), vd=torch.randn(N, Hk, L, d, generator=g).to(dt).to(DEV)))
        held = want
    for s in steps:
        for n, shape, t in (("cu", (B + 1,), torch.int32), ("cu2", (B + 1,), torch.int32), ("granted", (B,), torch.int32),
                            ("granted2", (B,), torch.int32), ("slots", (N,), torch.int64), ("mask", (N, 1), torch.int32),
                            ("pos", (N,), torch.int32), ("o", (N, Hq, d), dt), ("lse", (N, Hq), torch.float32)):
            s[n] = torch.zeros(shape, dtype=t, device=DEV)

    def run(wait):
        y = state
        for s in steps:
            for call in (
                lambda: moda.moda_page_plan(sh, s["held"], s["back"], y["table"], y["free"], y["count"], s["cu2"], s["granted2"], s["slots"]),
                lambda: moda.moda_page_plan(sh, s["back"], s["want"], y["table"], y["free"], y["count"], s["cu"], s["granted"], s["slots"]),
                lambda: moda.moda_cache_append(sh, s["k"], s["v"], s["slots"], y["kc"], y["vc"]),
                lambda: moda.moda_tree_mask(sh, s["parent"], s["cu"], s["back"], s["mask"], s["pos"]),
                lambda: moda.moda_tree_decode(sh, s["q"], y["kc"], y["vc"], s["kd"], s["vd"], y["table"], s["back"], s["cu"], s["mask"],
                                              s["o"], s["lse"], ws, nws),
            ):
                call()
                if wait:
                    torch.cuda.synchronize()

    names = ("granted", "slots", "mask", "pos", "o", "lse")
    run(True)
    moda.moda_check_status()
    ref = [{n: s[n].clone() for n in names} for s in steps]
    end = {n: t.clone() for n, t in state.items()}
    assert all(torch.equal(s["granted"], s["want"]) for s in steps) and int(end["count"]) < n_pages - 2 * B
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(False)
    for _ in range(10):
        for n, t in state.items():
            t.copy_(state0[n])
        for s in steps:
            for n in names:
                s[n].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for s, r in zip(steps, ref):
            for n in names:
                assert torch.equal(s[n], r[n]), n
        assert all(torch.equal(state[n], end[n]) for n in state)


# ------------------------------------------------------------------- together --
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_speculative_steps(dtype):
    """Prompts, then steps of draft, attention and acceptance over one cache:
    plan, append, mask and attention of every step against the dense rows that
    the accepted tokens leave."""
    rng = np.random.default_rng(11)
    g = torch.Generator().manual_seed(11)
    dt = torch_dtype(dtype)
    B, Hq, Hk, d, L, P, n_pages, max_pages = 3, 8, 2, 64, 3, 8, 60, 20
    kc, vc = (torch.full((n_pages, Hk, P, d), float("nan"), dtype=dt, device=DEV) for _ in range(2))
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    fl, count = torch.randperm(n_pages, generator=g).to(torch.int32).to(DEV), dev_i32([n_pages])
    held = dev_i32([0] * B)
    dense = [[torch.zeros(0, Hk, d, dtype=dt) for _ in range(2)] for _ in range(B)]     # accepted keys, values
    for step in range(5):
        new = [int(n) for n in (rng.integers(20, 50, B) if step == 0 else rng.integers(0, 12, B))]
        chain = step == 0
        N = sum(new) + 2
        parent = random_parents(new, rng)
        cu_ref = np.concatenate([[0], np.cumsum(new)])
        words = 0 if chain else 1
        sh = moda.make_paged_shape(B, N, Hq, Hk, d, L, P, n_pages, max_pages, words,
                                   moda.MODA_FP32 if dtype == "fp32" else moda.MODA_BF16)
        cu, granted = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)
        slots = torch.empty(N, dtype=torch.int64, device=DEV)
        moda.moda_page_plan(sh, held, held + dev_i32(new), table, fl, count, cu, granted, slots)
        assert cu.tolist() == cu_ref.tolist() and granted.tolist() == (held + dev_i32(new)).tolist()
        q, k, v = (torch.randn(N, h, d, generator=g).to(dt) for h in (Hq, Hk, Hk))
        kd, vd = (torch.randn(N, Hk, L, d, generator=g).to(dt) for _ in range(2))
        moda.moda_cache_append(sh, k.to(DEV), v.to(DEV), slots, kc, vc)
        mask = None
        see, pos_ref = oracle.tree_mask(parent, cu_ref, held.tolist())
        if chain:
            see = [np.tril(np.ones((n, n), bool)) for n in new]
        else:
            mask, pos = torch.zeros(N, 1, dtype=torch.int32, device=DEV), torch.zeros(N, dtype=torch.int32, device=DEV)
            moda.moda_tree_mask(sh, dev_i32(np.concatenate([parent, [0, 0]])), cu, held, mask, pos)
            assert pos.tolist()[: sum(new)] == pos_ref.tolist()
        x = dict(q=q, kc=kc, vc=vc, Kd=kd, Vd=vd, table=table, held=held, cu=cu, mask=mask)
        o, lse = run_tree(to_device(x), sh)
        keep = []                      # the branch accepted of each request
        for b in range(B):
            c0 = int(cu_ref[b])
            for i in range(new[b]):
                path = c0 + np.nonzero(see[b][i])[0]
                kk, vv = (torch.cat([dense[b][j], t[path]]).transpose(0, 1)[None] for j, t in ((0, k), (1, v)))
                r, rl = oracle.decode(q[c0 + i][None].double(), kk.double(), vv.double(), kd[c0 + i][None].double(),
                                      vd[c0 + i][None].double())
                a, _ = oracle.decode(q[c0 + i][None].double(), kk.double(), vv.double().abs(), kd[c0 + i][None].double(),
                                     vd[c0 + i][None].double().abs())
                assert (np.abs(o[c0 + i].double().cpu().numpy() - r[0]) <= out_bound(dtype, r[0], a[0])).all()
                assert np.abs(lse[c0 + i].double().cpu().numpy() - rl[0]).max() <= 1e-3
            last = int(rng.integers(0, new[b])) if new[b] else -1
            keep.append(np.arange(new[b]) if chain else (np.nonzero(see[b][last])[0] if new[b] else np.zeros(0, int)))
        # the accepted tokens' rows again, at the slots of the positions they keep; the rest given back
        order = torch.zeros(N, dtype=torch.int64)
        at = slots.cpu().clone()
        sl = torch.full((N,), -1, dtype=torch.int64)
        for b in range(B):
            c0 = int(cu_ref[b])
            for j, i in enumerate(keep[b]):
                order[c0 + j], sl[c0 + j] = c0 + int(i), at[c0 + j]
            dense[b] = [torch.cat([dense[b][0], k[c0 + keep[b]]]), torch.cat([dense[b][1], v[c0 + keep[b]]])]
        moda.moda_cache_append(sh, k[order].to(DEV), v[order].to(DEV), sl.to(DEV), kc, vc)
        kept = held + dev_i32([len(p) for p in keep])
        held2 = torch.empty_like(held)
        moda.moda_page_plan(sh, granted, kept, table, fl, count, cu, held2, slots)
        held = held2
        assert held.tolist() == [x[0].shape[0] for x in dense]
        assert int(count) == n_pages - sum(-(-h // P) for h in held.tolist())

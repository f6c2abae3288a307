"""Inputs of the paged calls and the bound their outputs are held to.

The caches are NaN wherever no key of the case lives (free pages, slots behind
a request's last key) and the block table names no page behind a request's
last one, so a read of what a row does not see shows in the results or in the
status word.
"""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

import oracle
import sequence_depth_attention_moda_b200 as moda


@dataclasses.dataclass(frozen=True)
class Tree:
    held: tuple
    new: tuple
    Hq: int = 8
    Hk: int = 2
    d: int = 128
    L: int = 4
    page: int = 16
    window: int = 0
    dtype: str = "bf16"
    chain: bool = False
    pad: int = 0             # token rows behind the last request
    extra_words: int = 0     # mask words beyond those the trees need
    scale: float = 0.0
    seed: int = 1

    def __str__(self):
        return "held%s_new%s_Hq%d_Hk%d_d%d_L%d_P%d%s%s_%s" % (
            "-".join(map(str, self.held)), "-".join(map(str, self.new)), self.Hq, self.Hk, self.d, self.L, self.page,
            "_w%d" % self.window if self.window else "", "_chain" if self.chain else "", self.dtype)


def torch_dtype(dtype):
    return torch.float32 if dtype == "fp32" else torch.bfloat16


def mask_words(see, words):
    """int32 mask rows from per-request bool matrices."""
    rows = []
    for m in see:
        bits = np.zeros((m.shape[0], 32 * words), dtype=np.uint64)
        bits[:, : m.shape[1]] = m
        rows.append((bits.reshape(-1, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32))
    return torch.from_numpy(np.concatenate(rows).view(np.int32)) if rows else torch.zeros(0, words, dtype=torch.int32)


def random_parents(new, rng):
    return np.concatenate([np.array([rng.integers(-1, i) if i else -1 for i in range(n)], dtype=np.int32)
                           for n in new] + [np.zeros(0, np.int32)])


def make_tree(c: Tree, see=None):
    """CPU tensors of a case; `see` replaces the trees' ancestor matrices."""
    rng = np.random.default_rng(c.seed)
    g = torch.Generator().manual_seed(c.seed)
    dt, P, B = torch_dtype(c.dtype), c.page, len(c.held)
    cu = np.concatenate([[0], np.cumsum(c.new)]).astype(np.int32)
    N = int(cu[-1]) + c.pad
    need = [-(-(h + n) // P) for h, n in zip(c.held, c.new)]
    n_pages = sum(need) + 5
    max_pages = max(need + [1]) + 2
    order = rng.permutation(n_pages)
    table = np.full((B, max_pages), 1 << 30, dtype=np.int32)
    at = 0
    x = {}
    kc = torch.full((n_pages, c.Hk, P, c.d), float("nan"))
    vc = torch.full_like(kc, float("nan"))
    for b in range(B):
        table[b, : need[b]] = order[at:at + need[b]]
        at += need[b]
        key = np.arange(c.held[b] + c.new[b])
        pg, off = torch.from_numpy(table[b][key // P].astype(np.int64)), torch.from_numpy(key % P)
        kc[pg, :, off] = torch.randn(len(key), c.Hk, c.d, generator=g)
        vc[pg, :, off] = torch.randn(len(key), c.Hk, c.d, generator=g)
    x["kc"], x["vc"] = kc.to(dt), vc.to(dt)
    x["q"] = torch.randn(N, c.Hq, c.d, generator=g).to(dt)
    x["Kd"] = torch.randn(N, c.Hk, c.L, c.d, generator=g).to(dt) if c.L else None
    x["Vd"] = torch.randn(N, c.Hk, c.L, c.d, generator=g).to(dt) if c.L else None
    x["table"], x["held"], x["cu"] = (torch.from_numpy(np.ascontiguousarray(v)) for v in
                                      (table, np.array(c.held, np.int32), cu))
    words = 0
    if not c.chain:
        if see is None:
            see, _ = oracle.tree_mask(random_parents(c.new, rng), cu)
        words = max(1, -(-max(list(c.new) + [1]) // 32)) + c.extra_words
        m = mask_words(see, words)
        # bits of tokens a request does not have mean nothing: set them
        for b in range(B):
            for j in range(c.new[b], 32 * words):
                m[cu[b]:cu[b + 1], j // 32] |= int(np.uint32(1 << (j % 32)).view(np.int32))
        x["mask"] = torch.cat([m, torch.full((c.pad, words), -1, dtype=torch.int32)])
    else:
        x["mask"] = None
    shape = moda.make_paged_shape(B, N, c.Hq, c.Hk, c.d, c.L, P, n_pages, max_pages, words,
                                  moda.MODA_FP32 if c.dtype == "fp32" else moda.MODA_BF16, c.scale, c.window)
    return x, (None if c.chain else see), shape


def to_device(x, dev="cuda"):
    return {k: (v.to(dev) if v is not None else None) for k, v in x.items()}


def oracle_tree(c: Tree, x, see, absolute=False):
    """The oracle's rows; `absolute`: with |V| for V, the scale of the bound."""
    f = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    vc, vd = f(x["vc"]), f(x["Vd"])
    if absolute:
        vc, vd = np.abs(vc), (None if vd is None else np.abs(vd))
    return oracle.tree_decode(f(x["q"]), f(x["kc"]), vc, f(x["Kd"]), vd, x["table"].numpy(), x["held"].numpy(),
                              x["cu"].numpy(), see, window=c.window, scale=c.scale)


def out_bound(dtype, o, a):
    """Elementwise bound on |o - oracle|, with a = sum p |v| (>= |o|).

    bf16: each weight p is rounded once (half a step, 2^-8 of p, so 2^-8 a in
    all) and the output once (2^-8 of |o|).  Both types: a score is a sum of d
    products in fp32, off by at most d 2^-24 sum|q k| scale, with sum|q k| about
    2/pi d for N(0,1) values: 128 * 2^-24 * 82 * 128^-1/2 = 5.5e-5 at worst over the
    orders of summation; that changes p and l by that fraction each, and exp2
    and the sums over up to a few thousand keys add 2^-22-sized fractions whose
    errors do not line up.  2e-4 a covers them (the framework's fp32 bound, 1e-4
    absolute, is kept beside it for fp32)."""
    if dtype == "fp32":
        return np.minimum(2e-4 * a + 1e-7, 1e-4)
    return 2.0 ** -8 * (a + np.abs(o)) * (1 + 2.0 ** -7) + 2e-4 * a + 1e-7


def check_tree(c: Tree, x, see, o, lse, lse_tol=1e-3):
    ref, rlse = oracle_tree(c, x, see)
    a, _ = oracle_tree(c, x, see, absolute=True)
    n = int(x["cu"][-1])
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    # padding is left as it was (the tests fill outputs with NaN)
    assert np.isnan(o[n:]).all() and np.isnan(lse[n:]).all(), "rows behind the last request were written"
    o, lse, ref, rlse, a = o[:n], lse[:n], ref[:n], rlse[:n], a[:n]
    fine = np.isfinite(ref)
    np.testing.assert_array_equal(np.isnan(o), np.isnan(ref))
    np.testing.assert_array_equal(np.isposinf(o), np.isposinf(ref))
    np.testing.assert_array_equal(np.isneginf(o), np.isneginf(ref))
    if fine.any():
        b = out_bound(c.dtype, ref[fine], np.where(np.isfinite(a[fine]), a[fine], 0))
        off = np.abs(o[fine] - ref[fine])
        assert (off <= b).all(), "off by %.3g, %.3g of the bound" % (off.max(), (off / b).max())
    empty = np.isneginf(rlse)
    np.testing.assert_array_equal(np.isneginf(lse), empty)
    if (~empty).any():
        d = np.abs(lse[~empty] - rlse[~empty]).max()
        assert d <= lse_tol, d

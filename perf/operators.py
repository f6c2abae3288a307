"""Cases of the operators that serve drafted tokens over a paged KV cache.

plan    moda_page_plan: pages and cache slots for the tokens a step adds, then
        the roll-back of a draft of which nothing was accepted (which returns
        the tables to what they were, so a pass can be repeated);
append  moda_cache_append: the step's new keys and values into their slots;
mask    moda_tree_mask: ancestor bits and positions of drafted trees;
tree    moda_tree_decode: attention of drafted tokens (a tree, or a chain) over
        the paged cache and each token's own depth rows.

Lengths are a fixed function of the case; values come from the seed.
"""
import math

import torch

own = False

DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_GOLD = 0.6180339887498949


# ------------------------------------------------------------------ cases ---
def _plan(name, **kw):
    return {"name": name, "op": "plan", **kw}


def _append(name, **kw):
    return {"name": name, "op": "append", "dtype": "bf16", **kw}


def _mask(name, **kw):
    return {"name": name, "op": "mask", **kw}


def _tree(name, **kw):
    return {"name": name, "op": "tree", "dtype": "bf16", "window": 0, "ragged": False, "chain": False, **kw}


def listed():
    return [
        # a decoding step of a busy server: every request drafts a few tokens
        _plan("plan_step_B256", B=256, page=64, T=8192, n=8),
        # prompts arriving together, small pages: a quarter of a million slots
        _plan("plan_prompts_B64", B=64, page=16, T=0, n=8192),
        # the keys and values of one step's drafted trees, one layer
        _append("append_trees_N128", N=128, Hk=4, d=128, page=64),
        # the keys and values of a batch of prompts
        _append("append_prompts_N32k", N=32768, Hk=8, d=128, page=16),
        # a few requests with small trees
        _mask("mask_B8_n32", B=8, n=32),
        # many requests, trees of up to 256 drafted tokens
        _mask("mask_B256_n256", B=256, n=256),
        # one chat, one token, a short history: latency
        _tree("tree_B1_n1_T1000", B=1, Hq=16, Hk=4, d=128, L=16, page=64, T=1000, n=1),
        # plain decoding, the repository's decoding workload in pages
        _tree("tree_B8_n1_T32k", B=8, Hq=32, Hk=8, d=128, L=48, page=64, T=32767, n=1, chain=True),
        # long contexts, a tree of 32 tokens each
        _tree("tree_B8_n32_T32k", B=8, Hq=32, Hk=8, d=128, L=48, page=64, T=32768, n=32),
        # a mixed batch: uneven lengths and trees, pages smaller than a tile
        _tree("tree_B48_n64_T4k_ragged", B=48, Hq=16, Hk=4, d=128, L=16, page=16, T=4096, n=64, ragged=True),
        # a chunk of a prompt over what is cached already
        _tree("chunk_B2_n300_T16k", B=2, Hq=16, Hk=4, d=64, L=6, page=128, T=16001, n=300, chain=True, window=4),
        # fp32, odd sizes
        _tree("tree_fp32_B3_n13_T1500", B=3, Hq=6, Hk=2, d=64, L=8, page=8, T=1500, n=13, ragged=True, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "mask", "tree", "tree", "tree"])
    if op == "plan":
        B, n = _log(rng, 1, 512), _log(rng, 1, 8192)
        n = max(1, min(n, (64 * 4096) // B))
        return {"op": op, "B": B, "page": rng.choice([8, 16, 32, 64, 128, 256]), "T": rng.randint(0, 8192), "n": n}
    if op == "append":
        Hk, d, dtype = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128]), rng.choice(["bf16", "bf16", "fp32"])
        most = 32768 * 8 * 128 // (Hk * d * (2 if dtype == "fp32" else 1))
        return {"op": op, "dtype": dtype, "N": _log(rng, 1, min(65536, most)), "Hk": Hk, "d": d,
                "page": rng.choice([8, 16, 32, 64, 128, 256])}
    if op == "mask":
        return {"op": op, "B": _log(rng, 1, 256), "n": _log(rng, 1, 256)}
    Hk, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d, L = rng.choice([64, 128]), rng.choice([0, 1, 6, 8, 16, 32, 48])
    B, n, T = _log(rng, 1, 64), _log(rng, 1, 256), _log(rng, 16, 32768)
    # no larger than the largest listed: cached values, scores, depth rows
    T = max(16, min(T, 8 * 8 * 32768 * 128 // (B * Hk * d * (4 if dtype == "fp32" else 1))))
    n = max(1, min(n, 8 * 32 * 32 * 32768 // (B * Hk * G * T * (16 if dtype == "fp32" else 1)),
                   8 * 32 * 8 * 48 * 16 // (B * Hk * max(L, 1))))
    return {"op": op, "dtype": dtype, "B": B, "Hq": Hk * G, "Hk": Hk, "d": d, "L": L,
            "page": rng.choice([8, 16, 32, 64, 128, 256]), "T": T, "n": n, "ragged": rng.random() < 0.6,
            "chain": rng.random() < 0.3, "window": rng.choice([0, 0, (L + 1) // 2])}


# ------------------------------------------------------------ case lengths ---
def _frac(b, k):
    """A fixed spread of [0, 1) over the requests."""
    return ((b + 1) * _GOLD * (k + 1) + 0.37 * k) % 1.0


def _lengths(c):
    """(held, new) of each request."""
    B = c["B"]
    if c["op"] == "plan":
        return [int(c["T"] * _frac(b, 0)) for b in range(B)], [1 + int((c["n"] - 1) * _frac(b, 1)) for b in range(B)]
    if c["op"] == "mask":
        return [100 + b for b in range(B)], [1 + int(c["n"] * _frac(b, 0)) if b else c["n"] for b in range(B)]
    if not c["ragged"]:
        return [c["T"]] * B, [c["n"]] * B
    return ([int(c["T"] * _frac(b, 0)) if b else c["T"] for b in range(B)],
            [1 + int((c["n"] - 1) * _frac(b, 1)) if b else c["n"] for b in range(B)])


def _pages(length, page):
    return (length + page - 1) // page


def _win(c):
    return c["window"] if c["window"] > 0 else c["L"]


# ---------------------------------------------------------------- prepare ---
def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _starts(new):
    s = [0]
    for n in new:
        s.append(s[-1] + n)
    return s


def _parents(new, g):
    """Random trees: each token's parent is the root (-1) or an earlier token of its request."""
    at = torch.cat([torch.arange(n, device=DEV) for n in new])
    u = torch.rand(at.numel(), generator=g, device=DEV)
    return torch.minimum((u * (at + 1)).floor().to(torch.int32) - 1, at.to(torch.int32) - 1)


def _ancestor_words(parent, new, words):
    """Rows of ancestor bits (a token itself among them), made a level at a time."""
    N = parent.numel()
    first = torch.repeat_interleave(_int(_starts(new)[:-1], torch.int64), _int(new, torch.int64))
    rel = torch.arange(N, device=DEV) - first
    bits = torch.zeros(N, words * 32, dtype=torch.bool, device=DEV)
    walk, rows = rel.clone(), torch.arange(N, device=DEV)
    while True:
        live = walk >= 0
        if not bool(live.any()):
            break
        bits[rows[live], walk[live]] = True
        up = parent[(first + walk.clamp(min=0))].long()
        walk = torch.where(live, up, walk)
    w = (bits.view(N, words, 32).long() << torch.arange(32, device=DEV)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"c": case}
    if case["op"] == "append":
        dt, P = _TYPES[case["dtype"]], case["page"]
        s["n_pages"] = _pages(case["N"], P) * 2 + 7
        # runs of slots within pages, as requests fill them, pages in any order
        order = torch.randperm(s["n_pages"], generator=g, device=DEV)
        at = torch.arange(case["N"], device=DEV)
        s["slots"] = order[at // P] * P + at % P
        for k in ("k", "v"):
            s[k] = torch.randn(case["N"], case["Hk"], case["d"], generator=g, device=DEV).to(dt)
            s[k + "c"] = torch.zeros(s["n_pages"], case["Hk"], P, case["d"], device=DEV, dtype=dt)
        return s
    held, new = _lengths(case)
    s["held"], s["cu"], s["N"] = _int(held), _int(_starts(new)), sum(new)
    if case["op"] == "mask":
        s["words"] = (max(new) + 31) // 32
        s["parent"] = _parents(new, g)
        s["seq"] = torch.repeat_interleave(torch.arange(len(new), device=DEV), _int(new, torch.int64))
        return s
    P = case["page"]
    have, need = [_pages(h, P) for h in held], [_pages(h + n, P) for h, n in zip(held, new)]
    s["max_pages"] = max(need) + 1
    if case["op"] == "plan":
        s["n_pages"] = sum(need) + 11
        s["want"] = _int([h + n for h, n in zip(held, new)])
        cover = have
    else:
        s["n_pages"] = sum(need) + 3
        cover = need
    order = torch.randperm(s["n_pages"], generator=g, device=DEV).to(torch.int32)
    n_cover = _int(cover, torch.int64)
    col = torch.arange(s["max_pages"], device=DEV)
    inside = col < n_cover[:, None]
    s["table"] = torch.full((case["B"], s["max_pages"]), -1, dtype=torch.int32, device=DEV)
    s["table"][inside] = order[: sum(cover)]
    if case["op"] == "plan":
        s["free"] = torch.full((s["n_pages"],), -1, dtype=torch.int32, device=DEV)
        rest = order[sum(cover):]
        s["free"][: rest.numel()] = rest
        s["count"] = _int([rest.numel()])
        return s
    dt, Hk, d, L = _TYPES[case["dtype"]], case["Hk"], case["d"], case["L"]
    for k in ("kc", "vc"):
        s[k] = torch.randn(s["n_pages"], Hk, P, d, generator=g, device=DEV, dtype=dt)
    s["q"] = torch.randn(s["N"], case["Hq"], d, generator=g, device=DEV, dtype=dt)
    for k in ("kd", "vd"):
        s[k] = torch.randn(s["N"], Hk, L, d, generator=g, device=DEV, dtype=dt) if L else None
    s["nmax"] = max(new)
    s["words"] = 0 if case["chain"] else (s["nmax"] + 31) // 32
    s["mask"] = None if case["chain"] else _ancestor_words(_parents(new, g), new, s["words"])
    return s


# ------------------------------------------------------------ plain forms ---
def _plain_plan_step(held, want, table, free, count, P, N):
    """One plan in elementary operations; table, free and count are updated."""
    B, mp = table.shape
    held, want = held.long(), want.long()
    have, need = (held + P - 1) // P, (want + P - 1) // P
    fits = need <= mp
    drop = torch.where(fits, (have - need).clamp(min=0), 0)
    take = torch.where(fits, (need - have).clamp(min=0), 0)
    R = drop.sum()
    c0 = count.long()
    top = c0 + R
    served = fits & ((take == 0) | (take.cumsum(0) <= top))
    granted = torch.where(served, want, held)
    col = torch.arange(mp, device=table.device)
    # released pages onto the list, the first on top
    rel = (col >= need[:, None]) & (col < have[:, None]) & (drop > 0)[:, None]
    rank = (drop.cumsum(0) - drop)[:, None] + col - need[:, None]
    n_pages = free.numel()
    ext = torch.cat([free, free.new_zeros(1)])       # one place more, for what is not written
    ext.scatter_(0, torch.where(rel, (top - 1)[:, None] - rank, n_pages).reshape(-1), table.reshape(-1))
    free.copy_(ext[:n_pages])
    # pages for those that grow, from the top
    got = (col >= have[:, None]) & (col < need[:, None]) & (served & (take > 0))[:, None]
    q = (take.cumsum(0) - take)[:, None] + col - have[:, None]
    page = free[((top - 1)[:, None] - q).clamp(0, n_pages - 1)]
    table.copy_(torch.where(got, page, torch.where(rel, -1, table)))
    count.copy_((top - torch.where(served, take, 0).sum()).to(torch.int32))
    new = (granted - held).clamp(min=0)
    end = new.cumsum(0)
    cu = torch.cat([end.new_zeros(1), end])
    t = torch.arange(N, device=table.device)
    b = torch.searchsorted(end, t, right=True)
    inside = b < B
    b = b.clamp(max=B - 1)
    pos = held[b] + t - cu[b]
    slot = table[b, (pos // P).clamp(0, mp - 1)].long() * P + pos % P
    return cu.to(torch.int32), granted.to(torch.int32), torch.where(inside, slot, -1)


def _plain_plan(s):
    P = s["c"]["page"]
    cu, granted, slots = _plain_plan_step(s["held"], s["want"], s["table"], s["free"], s["count"], P, s["N"])
    cu2, back, slots2 = _plain_plan_step(granted, s["held"], s["table"], s["free"], s["count"], P, s["N"])
    return {"cu": cu, "granted": granted, "slots": slots, "cu2": cu2, "back": back, "slots2": slots2,
            "table": s["table"], "free": s["free"], "count": s["count"]}


def _plain_append(s):
    P = s["c"]["page"]
    page, off = s["slots"] // P, s["slots"] % P
    s["kc"][page, :, off] = s["k"]
    s["vc"][page, :, off] = s["v"]
    return {"k": s["kc"], "v": s["vc"]}


def _plain_mask(s):
    """Ancestors as the closure of "is the parent of", by squaring, a request a matrix."""
    B, n, W = s["held"].numel(), 32 * s["words"], s["words"]
    at = torch.arange(s["N"], device=DEV) - s["cu"].long()[s["seq"]]
    reach = torch.zeros(B, n, n, device=DEV)
    reach[s["seq"], at, at] = 1.0
    inner = s["parent"] >= 0
    reach[s["seq"][inner], at[inner], s["parent"][inner].long()] = 1.0
    for _ in range(max(1, (n - 1).bit_length())):
        reach = ((reach @ reach) > 0).float()
    rows = reach[s["seq"], at]
    words = (rows.view(-1, W, 32).long() << torch.arange(32, device=DEV)).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    position = s["held"][s["seq"]] + rows.sum(-1).to(torch.int32) - 1
    return {"mask": words, "position": position}


def _plain_tree(s):
    c = s["c"]
    B, Hq, Hk, d, L, P = (c[k] for k in ("B", "Hq", "Hk", "d", "L", "page"))
    G, n, dt = Hq // Hk, s["nmax"], _TYPES[c["dtype"]]
    scale = 1.0 / math.sqrt(d)
    table = s["table"].long().clamp(min=0)
    T = table.shape[1] * P
    held, cu = s["held"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    key = torch.arange(T, device=DEV)
    i = torch.arange(n, device=DEV)
    K = s["kc"][table].transpose(1, 2).reshape(B, Hk, T, d).float()
    V = s["vc"][table].transpose(1, 2).reshape(B, Hk, T, d).float()
    V = torch.where((key < (held + new)[:, None])[:, None, :, None], V, 0.0)
    real = i < new[:, None]                                            # [B, n]
    tok = torch.where(real, cu[:-1, None] + i, 0)
    q = s["q"][tok].float().view(B, n, Hk, G, d).permute(0, 2, 1, 3, 4)  # [B, Hk, n, G, d]
    rel = key - held[:, None]                                          # [B, T]
    drafted = (rel >= 0) & (rel < new[:, None])
    if s["mask"] is None:
        seen = drafted[:, None] & (rel[:, None] <= i[:, None])
    else:
        w = s["mask"][tok].gather(2, (rel.clamp(0, 32 * s["words"] - 1) // 32)[:, None].expand(B, n, T))
        seen = drafted[:, None] & ((w >> (rel % 32)[:, None].to(torch.int32)) & 1).bool()
    seen = seen | (rel < 0)[:, None]                                   # [B, n, T]
    S = (q.reshape(B, Hk, n * G, d) @ K.transpose(2, 3)).view(B, Hk, n, G, T) * scale
    S = S.masked_fill(~seen[:, None, :, None, :], -math.inf)
    m = S.amax(-1, keepdim=True)
    if L:
        lo = L - _win(c)
        kd = s["kd"][tok][:, :, :, lo:].float().transpose(1, 2)        # [B, Hk, n, L', d]
        vd = s["vd"][tok][:, :, :, lo:].float().transpose(1, 2)
        Sd = q @ kd.transpose(3, 4) * scale                            # [B, Hk, n, G, L']
        m = torch.maximum(m, Sd.amax(-1, keepdim=True))
    S = torch.exp(S - m)
    z = S.sum(-1, keepdim=True)
    o = (S.view(B, Hk, n * G, T) @ V).view(B, Hk, n, G, d)
    if L:
        Sd = torch.exp(Sd - m)
        z = z + Sd.sum(-1, keepdim=True)
        o = o + Sd @ vd
    o = (o / z).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, d)
    lse = (m + torch.log(z)).squeeze(-1).permute(0, 2, 1, 3).reshape(B, n, Hq)
    return {"o": o[real].to(dt), "lse": lse[real]}


# -------------------------------------------------------- framework's calls ---
def _own_shape(moda, s):
    c = s["c"]
    return moda.make_paged_shape(
        B=c.get("B", 1), N=s.get("N", c.get("N", 0)), Hq=c.get("Hq", c.get("Hk", 1)), Hk=c.get("Hk", 1),
        d=c.get("d", 128), L=c.get("L", 0), page_size=c.get("page", 64), n_pages=s.get("n_pages", 1),
        max_pages=s.get("max_pages", 1), mask_words=s.get("words", 0),
        dtype=moda.MODA_FP32 if c.get("dtype") == "fp32" else moda.MODA_BF16, depth_window=c.get("window", 0))


def _own(s):
    import sequence_depth_attention_moda_b200 as moda
    if "shape" not in s:
        s["shape"] = _own_shape(moda, s)
    c, sh, dev = s["c"], s["shape"], {"device": DEV}
    if c["op"] == "plan":
        cu, cu2 = (torch.empty(c["B"] + 1, dtype=torch.int32, **dev) for _ in range(2))
        granted, back = (torch.empty(c["B"], dtype=torch.int32, **dev) for _ in range(2))
        slots, slots2 = (torch.empty(s["N"], dtype=torch.int64, **dev) for _ in range(2))
        moda.moda_page_plan(sh, s["held"], s["want"], s["table"], s["free"], s["count"], cu, granted, slots)
        moda.moda_page_plan(sh, granted, s["held"], s["table"], s["free"], s["count"], cu2, back, slots2)
        return {"cu": cu, "granted": granted, "slots": slots, "cu2": cu2, "back": back, "slots2": slots2,
                "table": s["table"], "free": s["free"], "count": s["count"]}
    if c["op"] == "append":
        moda.moda_cache_append(sh, s["k"], s["v"], s["slots"], s["kc"], s["vc"])
        return {"k": s["kc"], "v": s["vc"]}
    if c["op"] == "mask":
        mask = torch.empty(s["N"], s["words"], dtype=torch.int32, **dev)
        position = torch.empty(s["N"], dtype=torch.int32, **dev)
        moda.moda_tree_mask(sh, s["parent"], s["cu"], s["held"], mask, position)
        return {"mask": mask, "position": position}
    if "ws" not in s:
        s["ws"] = torch.empty(moda.moda_tree_decode_workspace_size(sh), dtype=torch.uint8, **dev)
    o = torch.empty_like(s["q"])
    lse = torch.empty(s["N"], c["Hq"], dtype=torch.float32, **dev)
    moda.moda_tree_decode(sh, s["q"], s["kc"], s["vc"], s["kd"], s["vd"], s["table"], s["held"], s["cu"],
                          s["mask"], o, lse, s["ws"], s["ws"].numel())
    return {"o": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "append": _plain_append, "mask": _plain_mask, "tree": _plain_tree}[state["c"]["op"]](state)


# ------------------------------------------------------------------- work ---
def work(case):
    if case["op"] == "append":
        row = case["N"] * case["Hk"] * case["d"] * (4 if case["dtype"] == "fp32" else 2)
        return {"bytes": 4 * row + 8 * case["N"], "flops": 0}
    held, new = _lengths(case)
    B, N = len(held), sum(new)
    if case["op"] == "mask":
        return {"bytes": 4 * N + 8 * B + 4 * N * ((max(new) + 31) // 32 + 1), "flops": 0}
    if case["op"] == "plan":
        P = case["page"]
        grown = sum(_pages(h + n, P) - _pages(h, P) for h, n in zip(held, new))
        # twice: lengths in, starts and granted lengths out, pages between list and table, slots
        return {"bytes": 2 * (16 * B + 8 * grown + 8 * N), "flops": 0}
    e = 4 if case["dtype"] == "fp32" else 2
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    Lw = _win(case)
    keys = sum(h + n for h, n in zip(held, new))
    pairs = sum(n * h + n * (n + 1) // 2 for h, n in zip(held, new)) + N * Lw
    return {"bytes": 2 * e * d * (keys * Hk + N * Hk * Lw + N * Hq) + 4 * N * Hq, "flops": 4 * Hq * d * pairs}


# ------------------------------------------------------------------ exact ---
def _exact_tree(s):
    """Request by request in 64 bits, each from its own rows gathered out of the pages."""
    c = s["c"]
    Hq, Hk, d, L, P = (c[k] for k in ("Hq", "Hk", "d", "L", "page"))
    G, lo = Hq // Hk, c["L"] - _win(c)
    held, new = _lengths(c)
    outs, stats, t0 = [], [], 0
    for b, (h, n) in enumerate(zip(held, new)):
        pos = torch.arange(h + n, device=DEV)
        page, off = s["table"][b].long()[pos // P], pos % P
        see = torch.ones(n, h + n, dtype=torch.bool, device=DEV)
        j = torch.arange(n, device=DEV)
        if s["mask"] is None:
            see[:, h:] = j[None, :] <= j[:, None]
        else:
            words = s["mask"][t0:t0 + n].long() & 0xFFFFFFFF
            see[:, h:] = ((words[:, j // 32] >> (j % 32)) & 1) == 1
        q = s["q"][t0:t0 + n].double()
        o = torch.empty(n, Hq, d, dtype=torch.float64, device=DEV)
        lse = torch.empty(n, Hq, dtype=torch.float64, device=DEV)
        for hk in range(Hk):
            k, v = s["kc"][page, hk, off].double(), s["vc"][page, hk, off].double()
            for g in range(G):
                qh = q[:, hk * G + g]
                a = torch.where(see, qh @ k.T, -math.inf)
                if L:
                    ad = torch.einsum("nd,nld->nl", qh, s["kd"][t0:t0 + n, hk, lo:].double())
                    a = torch.cat([a, ad], 1)
                a = a / math.sqrt(d)
                z = torch.logsumexp(a, 1)
                p = torch.exp(a - z[:, None])
                r = p[:, : h + n] @ v
                if L:
                    r = r + torch.einsum("nl,nld->nd", p[:, h + n:], s["vd"][t0:t0 + n, hk, lo:].double())
                o[:, hk * G + g], lse[:, hk * G + g] = r, z
        outs.append(o)
        stats.append(lse)
        t0 += n
    return {"o": torch.cat(outs), "lse": torch.cat(stats)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s)
    if case["op"] == "append":
        P, Hk, d = case["page"], case["Hk"], case["d"]
        done = {}
        for name in ("k", "v"):
            flat = torch.zeros(s["n_pages"] * P, Hk, d, dtype=torch.float64, device=DEV)
            flat[s["slots"]] = s[name].double()
            done[name] = flat.view(s["n_pages"], P, Hk, d).transpose(1, 2).contiguous()
        return done
    return None

"""Cases for one step of speculative decoding over a tree of drafted tokens.

Five operators, in the order in which a serving program meets them.  M is the
number of nodes of a sequence's tree: node 0 is the last accepted token, the
others are drafted, each behind its parent, and their rows are the last M of the
sequence's cache.

* metadata  parents -> each node's ancestors (as bits), position and cache slot;
* rope      rotary positions on Q and K, K and V into the paged cache;
* tree      attention of the M rows: the cached context and a node's ancestors;
* verify    which drafted tokens stand, and one token more, from the target's and
            the drafter's probabilities and given random numbers;
* keep      the accepted path's rows moved together in the cache of every layer.
"""
import math

import torch

own = False

D = 128
ROW = 72                     # INT4 pages: bytes of a stored row, 64 of codes and 8 of scales
SM = 1.0 / math.sqrt(D)
E4M3, BF16, INT4 = "e4m3", "bf16", "int4"


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one sequence's tree of 12 nodes: launch latency only
        {"name": "metadata_one", "op": "metadata", "lens": "8192", "M": 12, "shape": "tree", "page": 32},
        # a large batch of wide trees
        {"name": "metadata_batch", "op": "metadata", "lens": "512x64-4096", "M": 64, "shape": "tree", "page": 32},
        # the 12 new tokens of each of 64 sequences on their way into an FP8 cache
        {"name": "rope_step", "op": "rope", "T": 768, "Hq": 72, "Hkv": 8, "page": 32, "rot": 128, "pairs": False,
         "cache": E4M3, "far": 131072, "skip": 0.0},
        # a long prompt's rows, an odd count, half of each head rotated in neighbouring pairs, INT4 pages
        {"name": "rope_prompt", "op": "rope", "T": 16381, "Hq": 72, "Hkv": 8, "page": 64, "rot": 64, "pairs": True,
         "cache": INT4, "far": 131072, "skip": 0.02},
        # one sequence's tree on a global layer, its tokens appended in the same call
        {"name": "tree_one", "op": "tree", "lens": "8192", "M": 12, "shape": "tree", "Hq": 72, "Hkv": 8, "page": 32,
         "window": -1, "cache": E4M3, "append": True},
        # a wide tree of one sequence over a BF16 cache
        {"name": "tree_wide", "op": "tree", "lens": "8192", "M": 64, "shape": "tree", "Hq": 72, "Hkv": 8, "page": 64,
         "window": -1, "cache": BF16, "append": False},
        # the trees of a serving batch whose lengths differ
        {"name": "tree_batch", "op": "tree", "lens": "64x1024-32768", "M": 12, "shape": "tree", "Hq": 72, "Hkv": 8,
         "page": 32, "window": -1, "cache": E4M3, "append": False},
        # trees of 32 nodes on a sliding-window layer, INT4 pages
        {"name": "tree_window", "op": "tree", "lens": "16x600-8192", "M": 32, "shape": "tree", "Hq": 72, "Hkv": 8,
         "page": 32, "window": 511, "cache": INT4, "append": False},
        # a chain of 11 drafts that a greedy drafter chose, one sequence
        {"name": "verify_one", "op": "verify", "B": 1, "M": 12, "shape": "chain", "V": 131072, "draft": False,
         "type": "fp32"},
        # trees drawn from the drafter's probabilities, a batch, a vocabulary of odd size
        {"name": "verify_batch", "op": "verify", "B": 64, "M": 16, "shape": "tree", "V": 100003, "draft": True,
         "type": "fp32"},
        # the path kept in the cache of one layer of one sequence
        {"name": "keep_one", "op": "keep", "lens": "200", "M": 12, "Hkv": 8, "page": 32, "layers": 1, "cache": BF16},
        # a batch's paths in the caches of 48 layers
        {"name": "keep_batch", "op": "keep", "lens": "64x40-200", "M": 12, "Hkv": 8, "page": 32, "layers": 48,
         "cache": E4M3},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["metadata", "rope", "rope", "tree", "tree", "tree", "verify", "verify", "keep"])
    Hkv, page, shape = rng.choice([1, 2, 4, 8]), rng.choice([32, 64]), rng.choice(["chain", "tree", "tree", "ragged"])
    cache = rng.choice([E4M3, BF16, INT4])
    if op == "metadata":
        B, M = _logint(rng, 1, 512), _logint(rng, 1, 64)
        return {"op": op, "lens": "%dx%d-%d" % (B, M, _logint(rng, 64, 8192)), "M": M, "shape": shape, "page": page}
    if op == "rope":
        return {"op": op, "T": _logint(rng, 1, 16384), "Hq": Hkv * rng.choice([1, 2, 4, 6, 8, 9]), "Hkv": Hkv,
                "page": page, "rot": rng.choice([8, 32, 64, 96, 128]), "pairs": rng.random() < 0.5, "cache": cache,
                "far": _logint(rng, 1024, 131072), "skip": rng.choice([0.0, 0.1])}
    if op == "tree":
        G, M, B = rng.choice([1, 2, 4, 5, 8, 9, 12]), rng.choice([1, 2, 5, 8, 12, 16, 24, 33, 64]), _logint(rng, 1, 64)
        # no more keys, nor more products, than the largest listed case
        top = _logint(rng, 64, max(64, int(1048576 // B * min(1.0, 864.0 / (M * G * Hkv)))))
        return {"op": op, "lens": "%dx%d-%d" % (B, max(1, top // 16), top), "M": M, "shape": shape, "Hq": G * Hkv,
                "Hkv": Hkv, "page": page, "window": rng.choice([-1, -1, 0, 511, _logint(rng, 1, 4096)]),
                "cache": cache, "append": rng.random() < 0.3}
    if op == "verify":
        V = _logint(rng, 1000, 200000)
        B, M = _logint(rng, 1, 64), _logint(rng, 1, 32)
        M = max(1, min(M, 100000000 // (B * V)))
        return {"op": op, "B": B, "M": M, "shape": shape, "V": V, "draft": rng.random() < 0.6,
                "type": rng.choice(["fp32", "fp32", "bf16"])}
    return {"op": op, "lens": "%dx%d-%d" % (_logint(rng, 1, 64), 64, _logint(rng, 65, 200)),
            "M": _logint(rng, 1, 64), "Hkv": Hkv, "page": page, "layers": _logint(rng, 1, 48),
            "cache": rng.choice([E4M3, BF16])}


def _rng(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _lens(case, seed):
    """The sequence lengths: "n", or "BxLO-HI", the same B lengths spread uniformly
    over the range (the longest of them HI) in an order that the seed shuffles."""
    s, M = case["lens"], case["M"]
    if "x" not in s:
        return [max(int(s), M)]
    B, r = s.split("x")
    B, lo, hi = int(B), *(int(v) for v in r.split("-"))
    hi = max(lo, hi)
    out = torch.randint(lo, hi + 1, (B,), generator=_rng(1005))
    out[0] = hi
    return [max(int(n), M) for n in out[torch.randperm(B, generator=_rng(seed))]]


def _parents(B, M, shape, seed):
    """int32 [B][M]: "chain"; "tree" (each node behind a random earlier one, no
    deeper than 11); "ragged" (trees of which some have fewer nodes: -1)."""
    g = _rng(seed + 77)
    par = torch.arange(M).repeat(B, 1) - 1
    if shape != "chain":
        pick = torch.rand((B, M), generator=g)
        depth = torch.zeros((B, M), dtype=torch.long)
        for m in range(1, M):
            # among the last 8 nodes before it, so that trees are deep as well as wide
            lo = max(0, m - 8)
            p = lo + (pick[:, m] * (m - lo)).long()
            p = torch.where(depth.gather(1, p[:, None])[:, 0] >= 11, torch.zeros_like(p), p)
            par[:, m] = p
            depth[:, m] = depth.gather(1, p[:, None])[:, 0] + 1
    if shape == "ragged":
        nodes = 1 + (torch.rand((B, 1), generator=g) * M).long()
        par = torch.where(torch.arange(M)[None] < nodes, par, torch.full_like(par, -1))
    return par.to(torch.int32).cuda()


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + 11)
    st = {"metadata": _prepare_metadata, "rope": _prepare_rope, "tree": _prepare_tree, "verify": _prepare_verify,
          "keep": _prepare_keep}[case["op"]](case, seed, g)
    st["op"] = case["op"]
    return st


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _tables(lens, page, g):
    """A block table over a shuffled pool of pages, unused entries -1, and the pool's size."""
    need = [(n + page - 1) // page for n in lens]
    perm = torch.randperm(sum(need) + 2, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(max(need), device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    bt[used] = perm[:sum(need)]
    return bt, sum(need) + 2


def _seq_lens(lens):
    return torch.tensor(lens, dtype=torch.int32, device="cuda")


def _empty_cache(cache, pages, Hkv, page):
    if cache == INT4:
        return torch.zeros((pages, Hkv, page * ROW), dtype=torch.uint8, device="cuda")
    return torch.zeros((pages, Hkv, page, D), dtype=torch.uint8 if cache == E4M3 else torch.bfloat16, device="cuda")


def _random_cache(cache, pages, Hkv, page, scale, g, into=None):
    """Pages that hold normal values."""
    out = _empty_cache(cache, pages, Hkv, page) if into is None else into
    for lo in range(0, pages, 2048):
        n = min(2048, pages - lo)
        x = _randn((n * page, Hkv, D), g)
        slots = torch.arange(lo * page, (lo + n) * page, device="cuda")
        _store(x, slots, scale, out, cache, page)
    return out


def _scales():
    return [torch.full((1,), v / 448, device="cuda") for v in (12.0, 6.0)]


def _prepare_metadata(case, seed, g):
    lens, M, page = _lens(case, seed), case["M"], case["page"]
    bt, pages = _tables(lens, page, g)
    return {"parents": _parents(len(lens), M, case["shape"], seed), "sl": _seq_lens(lens), "bt": bt, "page": page,
            "pages": pages, "top": max(lens)}


def _cos_sin(far, rot):
    """fp32 [far][rot]: cosines and sines of position * base^(-2 k / rot), positions
    stretched by 4 for the slow half of the frequencies (a long-context scaling)."""
    k = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = 1e6 ** (-2.0 * k / rot)
    f = torch.where(k >= rot // 4, f / 4.0, f)
    a = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _prepare_rope(case, seed, g):
    T, Hq, H, page = case["T"], case["Hq"], case["Hkv"], case["page"]
    pages = (T + page - 1) // page + 3
    qkv = _randn((T, Hq + 2 * H, D), g)                  # one projection's output, Q, K and V views of it
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    if case["skip"]:
        slots = torch.where(torch.rand(T, generator=g, device="cuda") < case["skip"], -1, slots)
    ks, vs = _scales()
    return {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + H], "v": qkv[:, Hq + H:], "slots": slots, "ks": ks, "vs": vs,
            "pos": torch.randint(0, case["far"], (T,), generator=g, device="cuda"), "page": page,
            "cs": _cos_sin(case["far"], case["rot"]), "pairs": case["pairs"], "cache": case["cache"],
            "kc": _empty_cache(case["cache"], pages, H, page), "vc": _empty_cache(case["cache"], pages, H, page),
            "qo": torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda"),
            "ko": torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda"),
            "vo": torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")}


def _prepare_tree(case, seed, g):
    lens, M, Hq, H, page = _lens(case, seed), case["M"], case["Hq"], case["Hkv"], case["page"]
    B = len(lens)
    bt, pages = _tables(lens, page, g)
    ks, vs = _scales()
    mask = _ancestors(_parents(B, M, case["shape"], seed))
    st = {"q": _randn((B, M, Hq, D), g), "bt": bt, "sl": _seq_lens(lens), "lens": lens, "mask": mask, "ks": ks,
          "vs": vs, "page": page, "window": case["window"], "cache": case["cache"], "append": case["append"],
          "kc": _random_cache(case["cache"], pages, H, page, ks, g),
          "vc": _random_cache(case["cache"], pages, H, page, vs, g)}
    if case["append"]:
        st["kn"], st["vn"] = _randn((B, M, H, D), g), _randn((B, M, H, D), g)
        pos = st["sl"].long()[:, None] - M + torch.arange(M, device="cuda")
        st["slots"] = (torch.gather(bt.long(), 1, pos // page) * page + pos % page).reshape(-1)
        st["ko"], st["vo"] = (torch.zeros((B * M, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if own:
        # what a serving loop keeps: the call over its fixed buffers
        from verify_attention_gb300 import fp8kv
        st["call"] = fp8kv.PreparedAttention(st["q"], st["kc"], st["vc"], bt, st["sl"], max(lens), ks, vs, SM,
                                             window_left=case["window"], k_new=st.get("kn"), v_new=st.get("vn"),
                                             tree_mask=mask)
    return st


def _prepare_verify(case, seed, g):
    B, M, V = case["B"], case["M"], case["V"]
    dt = torch.float32 if case["type"] == "fp32" else torch.bfloat16
    par = _parents(B, M, case["shape"], seed)
    p = torch.empty((B, M, V), dtype=dt, device="cuda")
    q = torch.empty_like(p)
    tok = torch.zeros((B, M), dtype=torch.int32, device="cuda")
    rows = torch.arange(M, device="cuda")
    for b in range(B):
        x = torch.randn((M, V), generator=g, device="cuda") * 2.5
        p[b] = torch.softmax(x, -1).to(dt)
        y = x + 0.7 * torch.randn((M, V), generator=g, device="cuda")       # a drafter that mostly agrees
        qb = torch.softmax(y, -1)
        q[b] = qb.to(dt)
        if case["draft"]:
            # one draw of every node's row for each node; a node takes its parent's
            take = torch.multinomial(qb.clamp(min=0), M, replacement=True, generator=g)
        else:
            # the drafter's likeliest tokens, one for each child in turn
            take = qb.topk(min(M, V), -1).indices
        up = par[b].long().clamp(min=0)
        nth = ((up[None] == up[:, None]) & (rows[None] < rows[:, None]) & (rows[None] > 0)).sum(1)
        tok[b] = (take[up, rows] if case["draft"] else take[up, nth]).to(torch.int32)
    st = {"p": p, "q": q if case["draft"] else None, "tok": tok, "par": par,
          "u": torch.rand((B, M), generator=g, device="cuda"),
          "out": torch.empty((B, M), dtype=torch.int32, device="cuda"),
          "num": torch.empty((B,), dtype=torch.int32, device="cuda"),
          "path": torch.empty((B, M), dtype=torch.int32, device="cuda")}
    return st


def _prepare_keep(case, seed, g):
    lens, M, H, page, n = _lens(case, seed), case["M"], case["Hkv"], case["page"], case["layers"]
    B = len(lens)
    bt, pages = _tables(lens, page, g)
    one = _empty_cache(case["cache"], pages, H, page)
    kc = torch.empty((n,) + one.shape, dtype=one.dtype, device="cuda")
    vc = torch.empty_like(kc)
    ks, vs = _scales()
    for i in range(n):
        _random_cache(case["cache"], pages, H, page, ks, g, kc[i])
        _random_cache(case["cache"], pages, H, page, vs, g, vc[i])
    # paths of up to 11 drafted nodes, ascending, none of them the destination of
    # another, so that a pass can be repeated: node i stays, or moves from beyond
    most = min(11, (M - 1) // 2)
    acc = torch.randint(0, most + 1, (B, 1), generator=_rng(seed + 5))
    path = torch.full((B, M), -1, dtype=torch.long)
    for b in range(B):
        a = int(acc[b])
        at = torch.randperm(M - 1 - a, generator=_rng(seed * 100 + b))[:a].sort().values + 1 + a
        path[b, :a + 1] = torch.cat([torch.zeros(1, dtype=torch.long), at])
    st = {"kc": kc, "vc": vc, "bt": bt, "sl": _seq_lens(lens), "path": path.to(torch.int32).cuda(), "page": page,
          "cache": case["cache"], "new": torch.zeros((B,), dtype=torch.int32, device="cuda")}
    if own:
        from verify_attention_gb300 import fp8kv
        st["call"] = fp8kv.PreparedKeepPath(list(kc.unbind(0)), list(vc.unbind(0)), bt, st["sl"], st["path"],
                                            max(lens), new_seq_lens=st["new"])
    return st


# ------------------------------------------------------- plain forms: cache

def _store(x, slots, c, cache, kind, page):
    """bf16 rows [T][H][128] into the slots >= 0 of one cache."""
    keep = slots >= 0
    x, at, off = x[keep], slots[keep] // page, slots[keep] % page
    if kind == BF16:
        cache[at, :, off] = x
    elif kind == E4M3:
        cache[at, :, off] = (x.float() / c).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        P, H = cache.shape[:2]
        xb = x.float().reshape(*x.shape[:-1], 8, 16)
        s = (xb.abs().amax(-1) / (c * 7.0)).clamp(max=448.0).to(torch.float8_e4m3fn).float().clamp(min=2.0 ** -9)
        n = (xb * (torch.ones_like(s) / (s * c))[..., None]).round().clamp(-7, 7)
        code = (n + 8).to(torch.uint8).reshape(x.shape)
        cache[..., :page * 64].view(P, H, page, 64)[at, :, off] = code[..., 0::2] | (code[..., 1::2] << 4)
        cache[..., page * 64:].view(P, H, page, 8)[at, :, off] = s.to(torch.float8_e4m3fn).view(torch.uint8)


def _codes_to_values(codes, scales):
    """INT4: code bytes [..., 64] and scale bytes [..., 8] -> n s in fp32 [..., 128]."""
    n = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], D).float() - 8.0
    return (n.reshape(*n.shape[:-1], 8, 16) * scales.view(torch.float8_e4m3fn).float()[..., None]).reshape(n.shape)


def _page_values(cache, ids, c, kind, page):
    """The pages `ids` in fp32 [H][len(ids) * page][128]."""
    pg = cache[ids]
    n, H = pg.shape[:2]
    if kind == BF16:
        x = pg.float()
    elif kind == E4M3:
        x = pg.view(torch.float8_e4m3fn).float() * c
    else:
        x = _codes_to_values(pg[..., :page * 64].reshape(n, H, page, 64),
                             pg[..., page * 64:].reshape(n, H, page, 8)) * c
    return x.transpose(0, 1).reshape(H, n * page, D)


def _load(slots, c, cache, kind, page):
    """The stored rows as bf16 [T][H][128], zeros where the slot is negative."""
    at, off = slots.clamp(min=0) // page, slots.clamp(min=0) % page
    P, H = cache.shape[:2]
    if kind == BF16:
        x = cache[at, :, off].float()
    elif kind == E4M3:
        x = cache[at, :, off].view(torch.float8_e4m3fn).float() * c
    else:
        x = _codes_to_values(cache[..., :page * 64].view(P, H, page, 64)[at, :, off],
                             cache[..., page * 64:].view(P, H, page, 8)[at, :, off]) * c
    return torch.where((slots >= 0)[:, None, None], x, torch.zeros_like(x)).to(torch.bfloat16)


# -------------------------------------------------- plain forms: the operators

def _reach(par):
    """parents int32 [B][M] -> [B][M][M] truth values: i is m or an ancestor of m,
    in a tree that hangs from node 0 (no node: nothing)."""
    B, M = par.shape
    at = torch.arange(M, device=par.device)
    ok = (par >= 0) & (par < at)
    a = torch.eye(M, device=par.device).repeat(B, 1, 1)
    a += (par[..., None] == at) & ok[..., None]
    for _ in range(6):                                # paths of up to 64 steps
        a = (torch.matmul(a, a) > 0).float()
    return (a > 0) & (a[..., :1] > 0)


def _ancestors(par):
    """... as the bits of int64 [B][M]."""
    a = _reach(par)
    return (a.long() << torch.arange(par.shape[1], device=par.device)).sum(-1)


def _plain_metadata(st):
    par, sl, bt, page = st["parents"], st["sl"].long(), st["bt"].long(), st["page"]
    a = _reach(par)
    M = par.shape[1]
    node, depth = a.any(-1), (a.sum(-1) - 1).clamp(min=0)
    pos = sl[:, None] - M + depth
    at = sl[:, None] - M + torch.arange(M, device=par.device)
    slot = torch.gather(bt, 1, at // page) * page + at % page
    return (a.long() << torch.arange(M, device=par.device)).sum(-1), pos, torch.where(node, slot, -1)


def _rotate(x, cs, pairs):
    """fp32 rows [T][H][128], the first rot elements of a head rotated."""
    rot = cs.shape[1]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    ra, rb = a * c - b * s, b * c + a * s
    r = torch.stack([ra, rb], -1).flatten(-2) if pairs else torch.cat([ra, rb], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_rope(st):
    cs = st["cs"][st["pos"]]
    q = _rotate(st["q"].float(), cs, st["pairs"]).to(torch.bfloat16)
    k = _rotate(st["k"].float(), cs, st["pairs"]).to(torch.bfloat16)
    _store(k, st["slots"], st["ks"], st["kc"], st["cache"], st["page"])
    _store(st["v"], st["slots"], st["vs"], st["vc"], st["cache"], st["page"])
    return (q, _load(st["slots"], st["ks"], st["kc"], st["cache"], st["page"]),
            _load(st["slots"], st["vs"], st["vc"], st["cache"], st["page"]))


def _sees(mask, L, first, window):
    """int64 [M] ancestor bits -> [M][L - first] truth values: node m sees key
    first + j.  The node itself is at the context's length and its depth."""
    M = mask.shape[0]
    bit = ((mask[:, None] >> torch.arange(M, device=mask.device)) & 1).bool()
    pos = L - M + bit.sum(-1) - 1
    key = torch.cat([torch.arange(first, L - M, device=mask.device), pos])
    see = torch.cat([(mask != 0)[:, None].expand(M, L - M - first), bit], 1)
    return see & (key >= pos[:, None] - window) if window >= 0 else see


def _plain_tree(st):
    q, page, window, kind = st["q"], st["page"], st["window"], st["cache"]
    B, M, Hq, _ = q.shape
    H = st["kc"].shape[1]
    G = Hq // H
    if st["append"]:
        _store(st["kn"].reshape(-1, H, D), st["slots"], st["ks"], st["kc"], kind, page)
        _store(st["vn"].reshape(-1, H, D), st["slots"], st["vs"], st["vc"], kind, page)
    out = torch.empty_like(q)
    for b, L in enumerate(st["lens"]):
        lo = max(0, L - M - window) // page if window >= 0 else 0
        lo = min(lo, (L - M) // page)
        ids = st["bt"][b, lo:(L + page - 1) // page].long()
        k = _page_values(st["kc"], ids, st["ks"], kind, page)[:, :L - lo * page]
        v = _page_values(st["vc"], ids, st["vs"], kind, page)[:, :L - lo * page]
        see = _sees(st["mask"][b], L, lo * page, window).repeat_interleave(G, 0)
        x = q[b].float().view(M, H, G, D).transpose(0, 1).reshape(H, M * G, D)
        s = (torch.matmul(x, k.transpose(-1, -2)) * SM).masked_fill_(~see, -math.inf)
        top = s.amax(-1, keepdim=True)
        p = (s - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp()
        den = p.sum(-1, keepdim=True)
        o = torch.matmul(p, v) / torch.where(den == 0, torch.ones_like(den), den)      # no key: zeros
        out[b] = o.view(H, M, G, D).transpose(0, 1).reshape(M, Hq, D).to(torch.bfloat16)
    if st["append"]:
        return (out, _load(st["slots"], st["ks"], st["kc"], kind, page),
                _load(st["slots"], st["vs"], st["vc"], kind, page))
    return out


def _plain_verify(st):
    """Nodes in order, all sequences at once: w is what is left of the current
    node's distribution, S its weight.  A child with token x stands when
    u S q(x) < w(x); otherwise w becomes (w - S q)+ (a drafter without
    probabilities: q is 1 at x)."""
    p, q, tok, par, u = st["p"], st["q"], st["tok"].long(), st["par"], st["u"].double()
    B, M, V = p.shape
    row = torch.arange(B, device=p.device)
    cur = torch.zeros(B, dtype=torch.long, device=p.device)
    n = torch.ones_like(cur)
    path = torch.full((B, M), -1, dtype=torch.int32, device=p.device)
    path[:, 0] = 0
    w = p[:, 0].double().clamp(min=0)
    S = torch.ones(B, dtype=torch.float64, device=p.device)
    for m in range(1, M):
        x = tok[:, m]
        child = par[:, m] == cur
        wx = w[row, x]
        qx = q[row, cur, x].double() if q is not None else torch.ones_like(S)
        stands = child & (wx > 0) & (u[:, m] * S * qx < wx)
        if q is not None:
            left = (w - S[:, None] * q[row, cur].double()).clamp(min=0)
            rest = left.sum(-1)
        else:
            left = torch.where(torch.arange(V, device=p.device) == x[:, None], torch.zeros_like(w), w)
            rest = S - wx
        w = torch.where(stands[:, None], p[:, m].double().clamp(min=0), torch.where(child[:, None], left, w))
        S = torch.where(stands, torch.ones_like(S), torch.where(child, rest, S))
        cur = torch.where(stands, torch.full_like(cur, m), cur)
        path[row, torch.where(stands, n, torch.zeros_like(n))] = torch.where(stands, cur, torch.zeros_like(cur)).int()
        n = n + stands
    # the token after them: the first whose running sum exceeds u S (nothing left: of the node's own row)
    total = w.sum(-1)
    w = torch.where((total > 0)[:, None], w, p[row, cur].double().clamp(min=0))
    run_sum = w.cumsum(-1)
    nxt = (run_sum <= (u[:, 0] * run_sum[:, -1])[:, None]).sum(-1)
    out = torch.where(path >= 0, torch.gather(tok, 1, path.long().clamp(min=0)).int(), -1)
    out = torch.cat([out[:, 1:], torch.full((B, 1), -1, dtype=torch.int32, device=p.device)], 1)
    out[row, n - 1] = nxt.int()
    return out, n.int(), path


def _values_of(cache, kind):
    """A cache as the values that it holds (E4M3: over their scale)."""
    return cache.view(torch.float8_e4m3fn) if kind == E4M3 else cache


def _plain_keep(st):
    path, sl, bt, page = st["path"].long(), st["sl"].long(), st["bt"].long(), st["page"]
    M = path.shape[1]
    to = sl[:, None] - M + torch.arange(M, device=path.device)
    frm = sl[:, None] - M + path
    moved = path >= 0
    src, dst = [(torch.gather(bt, 1, x // page) * page + x % page)[moved] for x in (frm.clamp(min=0), to)]
    sp, so, dp, do = src // page, src % page, dst // page, dst % page
    for cache in (st["kc"], st["vc"]):
        cache[:, dp, :, do] = cache[:, sp, :, so]
    st["new"].copy_(sl - M + moved.sum(-1))
    return _values_of(st["kc"], st["cache"]), _values_of(st["vc"], st["cache"]), st["new"]


def run(state):
    if own:
        return _run_own(state)
    return {"metadata": _plain_metadata, "rope": _plain_rope, "tree": _plain_tree, "verify": _plain_verify,
            "keep": _plain_keep}[state["op"]](state)


def _run_own(st):
    from verify_attention_gb300 import fp8kv
    op = st["op"]
    if op == "metadata":
        return fp8kv.fp8kv_tree_metadata(st["parents"], st["sl"], st["bt"], st["page"], st["top"], st["pages"])
    if op == "rope":
        q = fp8kv.fp8kv_rope_insert(st["q"], st["k"], st["v"], st["pos"], st["cs"], st["slots"], st["ks"], st["vs"],
                                    st["kc"], st["vc"], interleaved=st["pairs"], q_out=st["qo"])
        return (q, *fp8kv.fp8kv_cache_gather(st["slots"], st["ks"], st["vs"], st["kc"], st["vc"], st["ko"], st["vo"]))
    if op == "tree":
        out = st["call"]()
        if not st["append"]:
            return out
        return (out, *fp8kv.fp8kv_cache_gather(st["slots"], st["ks"], st["vs"], st["kc"], st["vc"], st["ko"], st["vo"]))
    if op == "verify":
        return fp8kv.fp8kv_verify_tree(st["p"], st["q"], st["tok"], st["par"], st["u"], st["out"], st["num"],
                                       st["path"])
    new = st["call"]()
    return _values_of(st["kc"], st["cache"]), _values_of(st["vc"], st["cache"]), new


# -------------------------------------------------------- work and exactness

def work(case):
    op = case["op"]
    elem = {E4M3: 128, BF16: 256, INT4: ROW}.get(case.get("cache"))      # bytes of a stored row
    if op == "metadata":
        n = len(_lens(case, 1)) * case["M"]
        return {"bytes": 32 * n + 4 * len(_lens(case, 1)), "flops": 16 * n}
    if op == "rope":
        T, Hq, H, rot = case["T"], case["Hq"], case["Hkv"], case["rot"]
        # Q in and out, K and V in, stored, read back and out; a table row, position and slot a token
        return {"bytes": T * (512 * Hq + H * 2 * (256 + 2 * elem + 256) + 4 * rot + 16),
                "flops": T * (3 * rot * (Hq + H) + 2 * D * 2 * H)}
    if op == "verify":
        # the row in which a sequence ends, of the target and of the drafter
        n = case["B"] * case["V"]
        size = 4 if case["type"] == "fp32" else 2
        return {"bytes": n * size * (2 if case["draft"] else 1) + 20 * case["B"] * case["M"], "flops": 4 * n}
    lens, M, H = _lens(case, 1), case["M"], case["Hkv"]
    if op == "keep":
        # half as many nodes as a path may have, each row read and written
        rows = len(lens) * min(11, (M - 1) // 2) / 2 * H * 2 * case["layers"]
        return {"bytes": int(2 * elem * rows) + len(lens) * (4 * M + 8), "flops": 0}
    Hq, window, byts, flops = case["Hq"], case["window"], 0, 0
    for L in lens:
        ctx = L - M if window < 0 else min(L - M, window)
        byts += (ctx + M) * H * 2 * elem + 2 * M * Hq * 256 + 8 * M + (M * H * 2 * (256 + elem + 256) if case["append"] else 0)
        flops += 4 * D * Hq * M * (ctx + min(M, 6))
    return {"bytes": byts, "flops": flops}


def _walk(par):
    """Each node's path from the root, by following the parents one after another."""
    paths = []
    for m, p in enumerate(par):
        up = [0] if m == 0 else (paths[p] + [m] if 0 <= p < m and paths[p] else [])
        paths.append(up)
    return paths


def _exact_e4m3(x):
    """The nearest E4M3 value (ties to even), at most 448, of float64 values."""
    x = x.clamp(-448.0, 448.0)
    e = torch.frexp(torch.where(x == 0, torch.ones_like(x), x)).exponent.double() - 1
    step = torch.exp2(e.clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_stored(x, c, kind):
    """What bf16 rows (as float64) become in a cache of tensor scale c, float64."""
    if kind == BF16:
        return x
    c = c.double()
    if kind == E4M3:
        return _exact_e4m3((x / c).float().double()) * c
    b = x.reshape(*x.shape[:-1], 8, 16)
    s = _exact_e4m3((b.abs().amax(-1) / (c.float() * 7).double()).float().double()).clamp(min=2.0 ** -9)
    inv = (1.0 / (s * c).float().double()).float().double()
    n = torch.round((b * inv[..., None]).float().double()).clamp(-7, 7)
    return (n * (s * c)[..., None]).reshape(x.shape)


def _exact_cache(cache, kind, page, c):
    """A whole cache as float64 [pages][page][H][128]."""
    if kind == BF16:
        return cache.double().transpose(1, 2)
    table = torch.tensor([((b & 7) / 8.0 * 2.0 ** -6 if not (b >> 3 & 15) else (1 + (b & 7) / 8.0) * 2.0 ** ((b >> 3 & 15) - 7))
                          * (-1 if b > 127 else 1) for b in range(256)], dtype=torch.float64, device=cache.device)
    if kind == E4M3:
        return (table[cache.long()] * c.double()).transpose(1, 2)
    P, H = cache.shape[:2]
    code = cache[..., :page * 64].reshape(P, H, page, 64).long()
    x = torch.stack([code % 16 - 8, code // 16 - 8], -1).reshape(P, H, page, 8, 16).double()
    s = table[cache[..., page * 64:].reshape(P, H, page, 8).long()]
    return (x * s[..., None] * c.double()).reshape(P, H, page, D).transpose(1, 2)


def _exact_metadata(st):
    par, sl, bt = st["parents"].tolist(), st["sl"].tolist(), st["bt"].tolist()
    bits, pos, slots = [], [], []
    for row, L, pages in zip(par, sl, bt):
        M, paths = len(row), _walk(row)
        word = [sum(1 << i for i in up) for up in paths]
        bits.append([w - (1 << 64) if w >> 63 else w for w in word])
        pos.append([L - M + max(0, len(up) - 1) for up in paths])
        slots.append([pages[(L - M + m) // st["page"]] * st["page"] + (L - M + m) % st["page"] if up else -1
                      for m, up in enumerate(paths)])
    return tuple(torch.tensor(v, dtype=torch.int64, device="cuda") for v in (bits, pos, slots))


def _exact_rope(st):
    rot, T = st["cs"].shape[1], st["pos"].shape[0]
    h = rot // 2
    z = torch.complex(st["cs"][st["pos"], :h].double(), st["cs"][st["pos"], h:].double())[:, None]
    got = []
    for x in (st["q"].double(), st["k"].double()):
        r = x.clone()
        if st["pairs"]:
            y = torch.view_as_complex(x[..., :rot].reshape(T, -1, h, 2).contiguous()) * z
            r[..., :rot] = torch.view_as_real(y).reshape(T, -1, rot)
        else:
            y = torch.complex(x[..., :h], x[..., h:rot]) * z
            r[..., :h], r[..., h:rot] = y.real, y.imag
        got.append(r)
    hide = (st["slots"] < 0)[:, None, None]
    stored = [_exact_stored(x, c, st["cache"]).masked_fill(hide, 0.0)
              for x, c in ((got[1].to(torch.bfloat16).double(), st["ks"]), (st["v"].double(), st["vs"]))]
    return (got[0], *stored)


def _exact_tree(st):
    q, page, window, kind = st["q"].double(), st["page"], st["window"], st["cache"]
    B, M, Hq, _ = q.shape
    H = st["kc"].shape[1]
    G = Hq // H
    out = torch.zeros_like(q)
    new = ()
    if st["append"]:
        new = tuple(_exact_stored(st[x].reshape(-1, H, D).double(), st[c], kind) for x, c in (("kn", "ks"), ("vn", "vs")))
    words = st["mask"].tolist()
    for b, L in enumerate(st["lens"]):
        nodes = [[i for i in range(M) if w >> i & 1] for w in words[b]]
        at = torch.tensor([L - M + len(up) - 1 for up in nodes], device="cuda")
        see = torch.zeros((M, L), dtype=torch.bool, device="cuda")
        for m, up in enumerate(nodes):
            if up:
                see[m, :L - M] = True
                see[m, [L - M + i for i in up]] = True
        if window >= 0:
            key = torch.arange(L, device="cuda")
            key[L - M:] = at
            see &= key[None] + window >= at[:, None]
        first = (int(see.any(0).nonzero()[0]) if see.any() else 0) // page
        ids = st["bt"][b, first:(L + page - 1) // page].long()
        k, v = (_exact_cache(st[c][ids], kind, page, st[s]).reshape(-1, H, D)[:L - first * page]
                for c, s in (("kc", "ks"), ("vc", "vs")))
        if new:
            k[L - M - first * page:], v[L - M - first * page:] = (n[b * M:(b + 1) * M] for n in new)
        for h in range(Hq):
            e = (k[:, h // G] @ q[b, :, h].T).T / math.sqrt(128.0)
            e = e.masked_fill(~see[:, first * page:], -math.inf)
            out[b, :, h] = torch.nan_to_num(torch.softmax(e, -1)) @ v[:, h // G]
    return (out, *new) if new else out


def _exact_verify(st):
    """One sequence after another, with normalised distributions."""
    tok, par, u = st["tok"].tolist(), st["par"].tolist(), st["u"].double().tolist()
    B, M, V = st["p"].shape
    outs, nums, paths = [], [], []
    for b in range(B):
        cur, path, scale = 0, [0], 1.0
        r = st["p"][b, 0].double()                     # the distribution is r / scale
        m = 1
        while m < M:
            if par[b][m] == cur:
                x = tok[b][m]
                qd = st["q"][b, cur].double() if st["q"] is not None else None
                qx = float(qd[x]) if qd is not None else 1.0
                if 0 < float(r[x]) and u[b][m] * qx < float(r[x]) / scale:
                    cur, scale = m, 1.0
                    path.append(m)
                    r = st["p"][b, m].double()
                elif qd is not None:
                    r = torch.relu(r / scale - qd)
                    scale = float(r.sum())
                else:
                    scale -= float(r[x])
                    r = r.clone()
                    r[x] = 0.0
            m += 1
        if float(r.sum()) == 0:
            r = st["p"][b, cur].double()
        c = torch.cumsum(r, 0)
        t = u[b][0] * float(c[-1])
        nxt = int(torch.searchsorted(c, torch.tensor([t], dtype=torch.float64, device="cuda"), right=True)[0])
        got = [tok[b][m] for m in path[1:]] + [nxt]
        outs.append(got + [-1] * (M - len(got)))
        nums.append(len(got))
        paths.append(path + [-1] * (M - len(path)))
    return tuple(torch.tensor(v, dtype=torch.int32, device="cuda") for v in (outs, nums, paths))


def _exact_keep(st):
    page, kind = st["page"], st["cache"]
    path, sl, bt = st["path"].tolist(), st["sl"].tolist(), st["bt"].tolist()
    kc, vc = st["kc"].clone(), st["vc"].clone()
    M, new = len(path[0]), []
    for row, L, pages in zip(path, sl, bt):
        kept = [m for m in row if m >= 0]
        new.append(L - M + len(kept))
        for i, m in enumerate(kept):
            (sp, so), (dp, do) = ((pages[(L - M + x) // page], (L - M + x) % page) for x in (m, i))
            for old, cache in ((st["kc"], kc), (st["vc"], vc)):
                cache[:, dp, :, do] = old[:, sp, :, so]
    return (*(_values_of(c, kind).double() for c in (kc, vc)), torch.tensor(new, dtype=torch.int32, device="cuda"))


def exact(case, seed):
    if work(case)["flops"] > 2e12 or (case["op"] == "keep" and case["layers"] * len(_lens(case, 1)) > 4000):
        return None                                    # beyond what 64 bits do in some seconds
    st = prepare(case, seed)
    return {"metadata": _exact_metadata, "rope": _exact_rope, "tree": _exact_tree, "verify": _exact_verify,
            "keep": _exact_keep}[case["op"]](st)

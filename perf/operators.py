"""Cases for the 4-bit paged KV cache and the whole-prompt attention.

Four operators, in the order in which a serving program meets them:

* prompt    causal attention of packed prompts (grouped heads, optional window)
            over the K and V rows that the projection just produced;
* insert    those K and V rows into pages held in 4 bits, and the stored rows
            read back as bf16 (what a prefix reuse or an inspection reads);
* attention decode rows (M = 1) and verifier rows (M = 12) over the 4-bit pages,
            plain or with the step's new tokens appended.

A row of a (token, KV head) is 128 elements in 8 blocks of 16.  With the tensor
scale c (fp32), everything in fp32 with the roundings written out:
    r = amax|x| / (7 c),  s = max(e4m3(r), 2^-9),  inv = 1 / (s c),
    n = clamp(rint(x inv), -7, 7),  value = n s c.
A page of one head is page_size rows of 64 code bytes (element 2i in the low
nibble of byte i, n + 8), then page_size rows of 8 scale bytes.
"""
import math

import numpy as np
import torch

own = False

D = 128
ROW = 72                     # bytes of a stored row: 64 of codes, 8 of scales
SM = 1.0 / math.sqrt(D)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the 12 new tokens of each of 64 sequences: one insert of a serving step
        {"name": "insert_step", "op": "insert", "T": 768, "Hkv": 8, "page": 32, "skip": 0.0},
        # a long prompt's rows at once, an odd count, some rows padding (slot -1)
        {"name": "insert_prompt", "op": "insert", "T": 16381, "Hkv": 8, "page": 64, "skip": 0.02},
        # the smallest decode: one short sequence, latency only
        {"name": "decode_256", "op": "attention", "lens": "256", "M": 1, "Hq": 72, "Hkv": 8, "page": 32,
         "window": -1, "append": False},
        # long-context decode of one sequence
        {"name": "decode_128k", "op": "attention", "lens": "131072", "M": 1, "Hq": 72, "Hkv": 8, "page": 64,
         "window": -1, "append": False},
        # decode of a batch whose lengths differ
        {"name": "decode_batch", "op": "attention", "lens": "64x1024-32768", "M": 1, "Hq": 72, "Hkv": 8, "page": 32,
         "window": -1, "append": False},
        # one speculative step on a global layer: 12 rows, their tokens appended
        {"name": "verify_8k", "op": "attention", "lens": "8192", "M": 12, "Hq": 72, "Hkv": 8, "page": 32,
         "window": -1, "append": True},
        # the same step on a sliding-window layer of 512 keys
        {"name": "verify_window", "op": "attention", "lens": "8192", "M": 12, "Hq": 72, "Hkv": 8, "page": 32,
         "window": 511, "append": False},
        # the verifier rows of a serving mix
        {"name": "verify_batch", "op": "attention", "lens": "64x1024-32768", "M": 12, "Hq": 72, "Hkv": 8, "page": 32,
         "window": -1, "append": False},
        # one short prompt alone
        {"name": "prompt_33", "op": "prompt", "lens": "33", "Hq": 72, "Hkv": 8, "window": -1, "pad": 0, "fused": True},
        # sixteen prompts packed, of very different lengths, padded behind the last
        {"name": "prompt_packed", "op": "prompt", "lens": "16x1-2048", "Hq": 72, "Hkv": 8, "window": -1, "pad": 77,
         "fused": True},
        # one long prompt on a global layer
        {"name": "prompt_8k", "op": "prompt", "lens": "8192", "Hq": 72, "Hkv": 8, "window": -1, "pad": 0,
         "fused": False},
        # a longer one on a sliding-window layer
        {"name": "prompt_16k_window", "op": "prompt", "lens": "16384", "Hq": 72, "Hkv": 8, "window": 511, "pad": 0,
         "fused": True},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["insert", "attention", "attention", "prompt", "prompt"])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "insert":
        return {"op": op, "T": _logint(rng, 1, 16384), "Hkv": Hkv, "page": rng.choice([32, 64]),
                "skip": rng.choice([0.0, 0.1])}
    if op == "attention":
        G, M = rng.choice([1, 2, 4, 5, 8, 9, 12]), rng.choice([1, 1, 2, 4, 7, 12])
        B = _logint(rng, 1, 64)
        hi = min(131072, 1048576 // B)                  # no more keys than the largest listed case
        top = _logint(rng, 64, hi)
        return {"op": op, "lens": "%dx%d-%d" % (B, max(M, top // 16), top), "M": M, "Hq": G * Hkv, "Hkv": Hkv,
                "page": rng.choice([32, 64]), "window": rng.choice([-1, -1, 511, _logint(rng, 1, 4096)]),
                "append": rng.random() < 0.3}
    G = rng.choice([1, 2, 3, 4, 6, 8, 9])
    B = _logint(rng, 1, 32)
    top = _logint(rng, 1, 8192 // B)
    return {"op": op, "lens": "%dx%d-%d" % (B, rng.choice([0, 1, max(1, top // 4)]) if top > 1 else 1, top),
            "Hq": G * Hkv, "Hkv": Hkv, "window": rng.choice([-1, -1, 0, 127, 511, _logint(rng, 1, 4096)]),
            "pad": rng.choice([0, 1, 130]), "fused": rng.random() < 0.5}


def _lens(case, seed):
    """The sequence lengths: "n", or "BxLO-HI", the same B lengths spread
    uniformly over the range (the longest of them HI) in an order that the seed
    shuffles."""
    s = case["lens"]
    if "x" not in s:
        return [int(s)]
    B, r = s.split("x")
    lo, hi = (int(v) for v in r.split("-"))
    out = [int(v) for v in np.random.default_rng(1005).integers(lo, hi + 1, size=int(B))]
    out[0] = hi
    return [out[i] for i in np.random.default_rng(seed).permutation(len(out))]


# ------------------------------------------------------------------ inputs

def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _scale(*ts):
    """The calibrated tensor scale: max|x| / 448, one fp32 on the device."""
    amax = torch.stack([t.float().abs().amax() for t in ts]).amax().reshape(1)
    return amax / torch.full_like(amax, 448.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + 7)
    return {"insert": _prepare_insert, "attention": _prepare_attention,
            "prompt": _prepare_prompt}[case["op"]](case, seed, g)


def _prepare_insert(case, seed, g):
    T, H, ps = case["T"], case["Hkv"], case["page"]
    pages = (T + ps - 1) // ps + 3
    k = _randn((T, H, D), g)
    k *= (0.5 + 1.5 * torch.rand((1, H, 1), generator=g, device="cuda")).to(torch.bfloat16)
    v = _randn((T, H, D), g)
    slots = torch.randperm(pages * ps, generator=g, device="cuda")[:T]
    if case["skip"]:
        slots = torch.where(torch.rand(T, generator=g, device="cuda") < case["skip"], -1, slots)
    cache = [torch.zeros((pages, H, ps * ROW), dtype=torch.uint8, device="cuda") for _ in range(2)]
    return {"op": "insert", "k": k, "v": v, "slots": slots, "ks": _scale(k), "vs": _scale(v), "kc": cache[0],
            "vc": cache[1], "ps": ps, "ko": torch.zeros_like(k), "vo": torch.zeros_like(v)}


def _prepare_attention(case, seed, g):
    lens, M, Hq, H, ps = _lens(case, seed), case["M"], case["Hq"], case["Hkv"], case["page"]
    lens = [max(L, M) for L in lens]
    B = len(lens)
    need = [(L + ps - 1) // ps for L in lens]
    perm = torch.randperm(sum(need) + 2, generator=g, device="cuda")
    kc = torch.zeros((sum(need) + 2, H, ps * ROW), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks = torch.full((1,), 12.0 / 448, device="cuda")
    vs = torch.full((1,), 6.0 / 448, device="cuda")
    bt = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
    head = 0.5 + 1.5 * torch.rand((1, H, 1), generator=g, device="cuda")
    at = 0
    for b, (L, n) in enumerate(zip(lens, need)):
        ids = perm[at:at + n]
        at += n
        bt[b, :n] = ids.to(torch.int32)
        for lo in range(0, n, 1024):
            m = min(1024, n - lo)
            for c, sc, mul in ((kc, ks, head), (vc, vs, 1.0)):
                x = (torch.randn((m * ps, H, D), generator=g, device="cuda") * mul).to(torch.bfloat16)
                c[ids[lo:lo + m]] = _pages(*_quantise(x, sc), ps)
    q = _randn((B, M, Hq, D), g)
    st = {"op": "attention", "q": q, "kc": kc, "vc": vc, "bt": bt, "lens": lens, "ks": ks, "vs": vs, "ps": ps,
          "window": case["window"], "append": case["append"],
          "sl": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    if case["append"]:
        st["kn"], st["vn"] = _randn((B, M, H, D), g), _randn((B, M, H, D), g)
        pos = st["sl"].long()[:, None] - M + torch.arange(M, device="cuda")
        st["slots"] = (torch.gather(bt.long(), 1, pos // ps) * ps + pos % ps).reshape(-1)
        st["ko"], st["vo"] = (torch.zeros((B * M, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if own:
        from verify_attention_gb300 import fp8kv
        st["call"] = fp8kv.PreparedAttention(q, kc, vc, bt, st["sl"], max(lens), ks, vs, SM, window_left=case["window"],
                                             k_new=st.get("kn"), v_new=st.get("vn"))
    return st


def _prepare_prompt(case, seed, g):
    lens, Hq, H = _lens(case, seed), case["Hq"], case["Hkv"]
    T = sum(lens) + case["pad"]
    if case["fused"]:                # three views of one projection's output
        qkv = _randn((T, Hq + 2 * H, D), g)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    else:
        q, k, v = (_randn((T, h, D), g) for h in (Hq, H, H))
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return {"op": "prompt", "q": q, "k": k, "v": v, "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"),
            "lens": lens, "window": case["window"], "out": torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")}


# ------------------------------------------------------------- plain forms

def _quantise(x, c):
    """bf16 [T][H][128] -> codes n + 8 (uint8 [T][H][128]) and scales (E4M3 [T][H][8])."""
    xb = x.float().reshape(*x.shape[:-1], 8, 16)
    r = xb.abs().amax(-1) / (c * 7.0)
    s = r.clamp(max=448.0).to(torch.float8_e4m3fn).float().clamp(min=2.0 ** -9)
    inv = torch.ones_like(s) / (s * c)
    n = (xb * inv[..., None]).round().clamp(-7, 7)
    codes = (torch.nan_to_num(n) + 8).to(torch.uint8).reshape(x.shape)
    return codes, s.to(torch.float8_e4m3fn).view(torch.uint8)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _pages(codes, scales, ps):
    """Rows of whole pages -> pages [n][H][ps * 72]."""
    n, H = codes.shape[0] // ps, codes.shape[1]
    c = _pack(codes).view(n, ps, H, 64).transpose(1, 2).reshape(n, H, ps * 64)
    return torch.cat([c, scales.view(n, ps, H, 8).transpose(1, 2).reshape(n, H, ps * 8)], -1)


def _values(codes, scales):
    """Code bytes [..., 64] and scale bytes [..., 8] -> n s in fp32 [..., 128]."""
    n = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 128).float() - 8.0
    s = scales.view(torch.float8_e4m3fn).float()
    return (n.reshape(*n.shape[:-1], 8, 16) * s[..., None]).reshape(n.shape)


def _store(x, slots, c, cache, ps):
    keep = slots >= 0
    codes, scales = _quantise(x[keep], c)
    page, off = slots[keep] // ps, slots[keep] % ps
    P, H = cache.shape[:2]
    cache[..., :ps * 64].view(P, H, ps, 64)[page, :, off] = _pack(codes)
    cache[..., ps * 64:].view(P, H, ps, 8)[page, :, off] = scales


def _load(slots, c, cache, ps):
    P, H = cache.shape[:2]
    at = slots.clamp(min=0)
    page, off = at // ps, at % ps
    x = _values(cache[..., :ps * 64].view(P, H, ps, 64)[page, :, off],
                cache[..., ps * 64:].view(P, H, ps, 8)[page, :, off]) * c
    return torch.where((slots >= 0)[:, None, None], x, torch.zeros_like(x)).to(torch.bfloat16)


def _softmax_rows(q, k, v, qpos, kpos, window):
    """q fp32 [H][R][128] at qpos [R], k and v fp32 [H][N][128] at kpos [N]."""
    s = torch.matmul(q, k.transpose(-1, -2)) * SM
    hide = kpos[None, :] > qpos[:, None]
    if window >= 0:
        hide |= kpos[None, :] < qpos[:, None] - window
    s = s.masked_fill_(hide, -math.inf)
    p = (s - s.amax(-1, keepdim=True)).exp()
    return torch.matmul(p, v) / p.sum(-1, keepdim=True)


def _plain_attention(st):
    q, ps, M, window = st["q"], st["ps"], st["q"].shape[1], st["window"]
    B, _, Hq, _ = q.shape
    P, H = st["kc"].shape[:2]
    G = Hq // H
    if st["append"]:
        _store(st["kn"].reshape(-1, H, D), st["slots"], st["ks"], st["kc"], ps)
        _store(st["vn"].reshape(-1, H, D), st["slots"], st["vs"], st["vc"], ps)
    out = torch.empty_like(q)
    for b, L in enumerate(st["lens"]):
        lo = max(0, L - M - window) // ps if window >= 0 else 0
        n = (L + ps - 1) // ps
        ids = st["bt"][b, lo:n].long()
        kv = []
        for c, sc in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
            pg = c[ids]
            x = _values(pg[..., :ps * 64].reshape(n - lo, H, ps, 64), pg[..., ps * 64:].reshape(n - lo, H, ps, 8)) * sc
            kv.append(x.transpose(0, 1).reshape(H, (n - lo) * ps, D)[:, :L - lo * ps])
        qb = q[b].float().view(M, H, G, D).transpose(0, 1).reshape(H, M * G, D)
        qpos = (L - M + torch.arange(M, device=q.device)).repeat_interleave(G)
        o = _softmax_rows(qb, kv[0], kv[1], qpos, torch.arange(lo * ps, L, device=q.device), window)
        out[b] = o.view(H, M, G, D).transpose(0, 1).reshape(M, Hq, D).to(torch.bfloat16)
    if st["append"]:
        return out, _load(st["slots"], st["ks"], st["kc"], ps), _load(st["slots"], st["vs"], st["vc"], ps)
    return out


def _plain_prompt(st):
    q, k, v, window = st["q"], st["k"], st["v"], st["window"]
    T, Hq, _ = q.shape
    H = k.shape[1]
    G = Hq // H
    out = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=q.device)
    t0 = 0
    for L in st["lens"]:
        kf = k[t0:t0 + L].float().transpose(0, 1)
        vf = v[t0:t0 + L].float().transpose(0, 1)
        for lo in range(0, L, 1024):
            hi = min(L, lo + 1024)
            first = max(0, lo - window) if window >= 0 else 0
            n = hi - lo
            qf = q[t0 + lo:t0 + hi].float().view(n, H, G, D).permute(1, 0, 2, 3).reshape(H, n * G, D)
            qpos = torch.arange(lo, hi, device=q.device).repeat_interleave(G)
            o = _softmax_rows(qf, kf[:, first:hi], vf[:, first:hi], qpos, torch.arange(first, hi, device=q.device),
                              window)
            out[t0 + lo:t0 + hi] = o.view(H, n, G, D).permute(1, 0, 2, 3).reshape(n, Hq, D).to(torch.bfloat16)
        t0 += L
    return out


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "insert":
        for x, c, cache in (("k", "ks", "kc"), ("v", "vs", "vc")):
            _store(state[x], state["slots"], state[c], state[cache], state["ps"])
        return (_load(state["slots"], state["ks"], state["kc"], state["ps"]),
                _load(state["slots"], state["vs"], state["vc"], state["ps"]))
    return _plain_attention(state) if state["op"] == "attention" else _plain_prompt(state)


def _run_own(st):
    from verify_attention_gb300 import fp8kv
    if st["op"] == "insert":
        fp8kv.fp8kv_cache_insert(st["k"], st["v"], st["slots"], st["ks"], st["vs"], st["kc"], st["vc"])
        return fp8kv.fp8kv_cache_gather(st["slots"], st["ks"], st["vs"], st["kc"], st["vc"], st["ko"], st["vo"])
    if st["op"] == "attention":
        out = st["call"]()
        if not st["append"]:
            return out
        return (out, *fp8kv.fp8kv_cache_gather(st["slots"], st["ks"], st["vs"], st["kc"], st["vc"], st["ko"], st["vo"]))
    return fp8kv.fp8kv_prompt_attention(st["q"], st["k"], st["v"], st["cu"], max(st["lens"]), SM,
                                        window_left=st["window"], out=st["out"])


# -------------------------------------------------------- work and exactness

def _pairs(L, first, window):
    """Visible (row, key) pairs of rows first .. L - 1 of a sequence of L keys."""
    if window < 0:
        return (L * (L + 1) - first * (first + 1)) // 2
    w = window + 1
    full = max(0, L - max(first, w - 1))
    short = L - first - full                    # rows that see less than a whole window
    return full * w + (short * (2 * first + short + 1)) // 2


def work(case):
    op = case["op"]
    if op == "insert":
        # rows in, stored rows written, their bf16 values out
        rows = case["T"] * case["Hkv"]
        return {"bytes": rows * (512 + 2 * ROW + 512) + 8 * case["T"], "flops": 4 * rows * 2 * D}
    lens, Hq, H, window = _lens(case, 1), case["Hq"], case["Hkv"], case["window"]
    if op == "attention":
        M, byts, flops = case["M"], 0, 0
        for L in lens:
            L = max(L, M)
            keys = L if window < 0 else min(L, M + window)
            byts += keys * H * 2 * ROW + 2 * M * Hq * D * 2 + (M * H * 4 * D * (2 if case["append"] else 0))
            flops += 4 * D * Hq * _pairs(L, L - M, window)
        return {"bytes": byts, "flops": flops}
    T = sum(lens)
    return {"bytes": 2 * D * T * (2 * Hq + 2 * H), "flops": 4 * D * Hq * sum(_pairs(L, 0, window) for L in lens)}


def _e4m3_of(r):
    """float32 array, r >= 0 -> the nearest E4M3 value (ties to even), at most 448, NaN kept."""
    r = np.minimum(r.astype(np.float64), 448.0)                    # np.minimum keeps NaN
    _, e = np.frexp(np.where(np.isnan(r) | (r == 0), 1.0, r))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(r / step) * step


def _exact_rows(x, c):
    """Definition of the stored value of bf16 rows [T][H][128], in float64."""
    x = x.float().cpu().numpy()
    c = np.float32(c.item())
    xb = x.reshape(*x.shape[:-1], 8, 16)
    s = np.maximum(_e4m3_of(np.max(np.abs(xb), -1) / np.float32(c * np.float32(7))), 2.0 ** -9)
    inv = np.float32(1) / (s.astype(np.float32) * c)
    n = np.clip(np.rint((xb.astype(np.float64) * inv[..., None].astype(np.float64)).astype(np.float32)), -7, 7)
    return torch.from_numpy((n.astype(np.float64) * s[..., None] * np.float64(c)).reshape(x.shape)).cuda()


def _exact_pages(cache, ids, c, ps):
    """Values of the pages `ids` of one cache, float64 [H][len(ids) * ps][128]."""
    pg = cache[ids]
    n, H = pg.shape[:2]
    table = torch.tensor([((b & 7) / 8.0 * 2.0 ** -6 if b < 8 else (1 + (b & 7) / 8.0) * 2.0 ** ((b >> 3) - 7))
                          for b in range(127)] + [math.nan], dtype=torch.float64, device=pg.device)
    code = pg[..., :ps * 64].reshape(n, H, ps, 64).to(torch.int32)
    x = torch.empty((n, H, ps, D), dtype=torch.float64, device=pg.device)
    x[..., 0::2] = (code % 16 - 8).double()
    x[..., 1::2] = (code // 16 - 8).double()
    x *= table[pg[..., ps * 64:].reshape(n, H, ps, 8).long()].repeat_interleave(16, -1)
    return (x * c.double()).transpose(0, 1).reshape(H, n * ps, D)


def _exact_softmax(q, k, v, see):
    """float64: q [R][128], k and v [N][128], see [R][N] truth values."""
    e = torch.einsum("rd,nd->rn", q, k) / math.sqrt(128.0)
    e = torch.where(see, e, torch.full_like(e, -math.inf))
    return torch.einsum("rn,nd->rd", torch.softmax(e, -1), v)


def exact(case, seed):
    if work(case)["flops"] > 4e12:                  # beyond what 64 bits do in some seconds
        return None
    st = prepare(case, seed)
    if case["op"] == "insert":
        out = []
        for x, c in (("k", "ks"), ("v", "vs")):
            y = _exact_rows(st[x], st[c])
            y[st["slots"] < 0] = 0.0
            out.append(y)
        return tuple(out)
    if case["op"] == "attention":
        q, ps, window = st["q"].double(), st["ps"], st["window"]
        B, M, Hq, _ = q.shape
        H = st["kc"].shape[1]
        G = Hq // H
        new = None
        if st["append"]:
            new = (_exact_rows(st["kn"].reshape(-1, H, D), st["ks"]), _exact_rows(st["vn"].reshape(-1, H, D), st["vs"]))
        out = torch.empty((B, M, Hq, D), dtype=torch.float64, device=q.device)
        for b, L in enumerate(st["lens"]):
            n = (L + ps - 1) // ps
            f = max(0, L - M - window) // ps if window >= 0 else 0
            ids = st["bt"][b, f:n].long()
            k, v = (_exact_pages(st[c], ids, st[s], ps)[:, :L - f * ps] for c, s in (("kc", "ks"), ("vc", "vs")))
            if new:
                k[:, L - M - f * ps:] = new[0][b * M:(b + 1) * M].transpose(0, 1)
                v[:, L - M - f * ps:] = new[1][b * M:(b + 1) * M].transpose(0, 1)
            j = torch.arange(f * ps, L, device=q.device)
            p = torch.arange(L - M, L, device=q.device)
            see = j[None] <= p[:, None]
            if window >= 0:
                see &= j[None] >= p[:, None] - window
            see = see.repeat(G, 1)                  # rows in the order (head, row)
            for h in range(H):
                qh = q[b, :, h * G:(h + 1) * G].transpose(0, 1).reshape(G * M, D)
                out[b, :, h * G:(h + 1) * G] = _exact_softmax(qh, k[h], v[h], see).view(G, M, D).transpose(0, 1)
        return (out, *new) if new else out
    q, k, v, window = st["q"], st["k"], st["v"], st["window"]
    T, Hq, _ = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    t0 = 0
    for L in st["lens"]:
        for h in range(Hq):
            kh, vh = k[t0:t0 + L, h // G].double(), v[t0:t0 + L, h // G].double()
            for lo in range(0, L, 2048):
                hi = min(L, lo + 2048)
                f = max(0, lo - window) if window >= 0 else 0
                p = torch.arange(lo, hi, device=q.device)[:, None]
                j = torch.arange(f, hi, device=q.device)[None]
                see = (j <= p) & (j >= p - window) if window >= 0 else j <= p
                out[t0 + lo:t0 + hi, h] = _exact_softmax(q[t0 + lo:t0 + hi, h].double(), kh[f:hi], vh[f:hi], see)
        t0 += L
    return out

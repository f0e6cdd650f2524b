"""A step over trees of drafted tokens in numpy, from the definitions in
include/fp8kv.h (test infrastructure only): ancestors, rotary positions, what a
row sees, verification and the kept path, in Python integers and float64."""
import numpy as np


def paths(parents):
    """Each node's path from the root (node 0), [] for padding."""
    out = []
    for m, p in enumerate(parents):
        p = int(p)
        out.append([0] if m == 0 else out[p] + [m] if 0 <= p < m and out[p] else [])
    return out


def metadata(parents, seq_lens, block_table, ps):
    """(mask, positions, slots) int64 [B][M] of valid inputs."""
    B, M = parents.shape
    mask, pos, slot = (np.zeros((B, M), np.int64) for _ in range(3))
    for b in range(B):
        base = int(seq_lens[b]) - M
        for m, up in enumerate(paths(parents[b])):
            word = sum(1 << i for i in up)
            mask[b, m] = word - (1 << 64) if word >> 63 else word
            pos[b, m] = base + max(0, len(up) - 1)
            slot[b, m] = int(block_table[b, (base + m) // ps]) * ps + (base + m) % ps if up else -1
    return mask, pos, slot


def bf16_round(x):
    """float32 -> the nearest bf16 (ties to even), as float32."""
    u = np.asarray(x, np.float32).view(np.uint32)
    return ((u + 0x7fff + ((u >> 16) & 1)) & np.uint32(0xffff0000)).view(np.float32)


def rope(x, cos_sin, positions, interleaved):
    """bf16 values [T][H][128] as float32 -> rotated and rounded to bf16.  The fma's
    product and sum are exact in float64 but for bits far below its rounding."""
    rot = cos_sin.shape[1]
    h = rot // 2
    cs = cos_sin[positions][:, None]
    c, s = cs[..., :h], cs[..., h:]
    i, j = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(h), np.arange(h, rot))
    a, b = x[..., i], x[..., j]
    out = x.copy()
    f = np.float64
    out[..., i] = bf16_round((a.astype(f) * c.astype(f) - (b * s).astype(f)).astype(np.float32))
    out[..., j] = bf16_round((b.astype(f) * c.astype(f) + (a * s).astype(f)).astype(np.float32))
    return out


def sees(words, M, L, window):
    """bool [M][L]: what each row of a sequence sees, from its mask words."""
    see = np.zeros((M, L), bool)
    base = L - M
    nodes = [[i for i in range(M) if int(w) >> i & 1] for w in words]
    pos = [base + max(len(n), 1) - 1 for n in nodes]
    for m in range(M):
        if not nodes[m]:
            continue
        see[m, :base] = True
        see[m, [base + i for i in nodes[m]]] = True
        if window >= 0:
            for j in range(base):
                see[m, j] &= j >= pos[m] - window
            for i in nodes[m]:
                see[m, base + i] &= pos[i] >= pos[m] - window
    return see


def attention(q, k, v, see, sm_scale):
    """One sequence: q float64 [M][Hq][128], k, v [H][L][128], see [M][L]; rows that
    see nothing are zeros."""
    M, Hq, _ = q.shape
    out = np.zeros(q.shape)
    for h in range(Hq):
        kh, vh = k[h * k.shape[0] // Hq], v[h * k.shape[0] // Hq]
        for m in range(M):
            if see[m].any():
                s = kh[see[m]] @ q[m, h] * sm_scale
                w = np.exp(s - s.max())
                out[m, h] = (w / w.sum()) @ vh[see[m]]
    return out


def verify(p, q, tokens, parents, uniforms):
    """One sequence: p, q float64 [M][V] (q None: chosen drafts); returns the emitted
    tokens, the path, and how near the closest decision was to its border, relative
    to the weight it was taken from."""
    clean = lambda x: np.where(np.isnan(x), 0.0, np.maximum(x, 0.0))  # noqa: E731
    M, V = p.shape
    n, path, near = 0, [0], np.inf
    w, S = clean(p[0]), 1.0
    for m in range(1, M):
        if int(parents[m]) != n:
            continue
        x = int(tokens[m])
        if not 0 <= x < V:
            continue
        qn = clean(q[n]) if q is not None else None
        qx = qn[x] if q is not None else 1.0
        lhs = float(uniforms[m]) * S * qx
        if w[x] > 0:
            near = min(near, abs(lhs - w[x]) / max(S, 1e-300))
        if w[x] > 0 and lhs < w[x]:
            n = m
            path.append(m)
            w, S = clean(p[m]), 1.0
        elif q is not None:
            w = np.maximum(w - S * qn, 0.0)
            S = w.sum()
        else:
            S -= w[x]
            w = w.copy()
            w[x] = 0.0
    if not w.sum() > 0:
        w = clean(p[n])
    c = np.cumsum(w)
    out = [int(tokens[m]) for m in path[1:]]
    if not (c[-1] > 0 and np.isfinite(c[-1])):
        return out, path, near
    t = float(uniforms[0]) * c[-1]
    out.append(int(np.searchsorted(c, t, side="right")))
    near = min(near, np.min(np.abs(c - t)) / c[-1])
    return out, path, near

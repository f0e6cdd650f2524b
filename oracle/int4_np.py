"""The INT4 cache and attention over it, in numpy (test infrastructure only).

encode_rows follows the definition of the INT4 cache step by step in fp32;
values and attention are float64.  Page bytes are [num_pages][Hkv][ps * 72]:
ps rows of 64 code bytes, then ps rows of 8 scale bytes, per (page, head)."""
import numpy as np

ROW = 72


def e4m3_value(code):
    """Decode E4M3FN codes (uint8) to float64."""
    c = np.asarray(code).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


_E4M3 = e4m3_value(np.arange(127))                      # increasing, 0 .. 448


def e4m3_code(r):
    """Nearest E4M3 code of r >= 0 (ties to even codes, saturating, NaN -> 0x7f)."""
    r = np.asarray(r, np.float64)
    x = np.minimum(np.where(np.isnan(r), 0.0, r), 448.0)
    hi = np.clip(np.searchsorted(_E4M3, x), 1, 126)
    lo = hi - 1
    dl, dh = x - _E4M3[lo], _E4M3[hi] - x
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(r), 127, code).astype(np.uint8)


def encode_rows(x, c):
    """fp32 rows [..., 128] (bf16 values), tensor scale c -> integers n
    [..., 128] in [-7, 7] and scale codes [..., 8]."""
    c = np.float32(c)
    xb = np.asarray(x, np.float32).reshape(*x.shape[:-1], 8, 16)
    with np.errstate(all="ignore"):
        amax = np.max(np.abs(xb), -1)                   # NaN propagates
        r = amax / np.float32(np.float32(7) * c)
        sc = np.maximum(e4m3_code(r), 1)
        s = e4m3_value(sc).astype(np.float32)
        inv = np.float32(1) / (s * c)
        y = xb * inv[..., None]
        n = np.clip(np.rint(y), -7, 7)
    n = np.where(np.isnan(s)[..., None], 0, n)
    return n.reshape(x.shape).astype(np.int8), sc


def write_rows(cache, ps, slots, n, sc):
    """Store rows n [T][Hkv][128], sc [T][Hkv][8] at their slots (< 0: skipped)."""
    codes = (n + 8).astype(np.uint8)
    by = codes[..., 0::2] | (codes[..., 1::2] << 4)
    for t, slot in enumerate(slots):
        if slot < 0:
            continue
        page, off = int(slot) // ps, int(slot) % ps
        cache[page, :, off * 64:(off + 1) * 64] = by[t]
        cache[page, :, ps * 64 + off * 8:ps * 64 + (off + 1) * 8] = sc[t]


def read_pages(cache, ps):
    """Page bytes [P][Hkv][ps * 72] -> n * s in float64 [P][Hkv][ps][128] (exact)."""
    P, H, _ = cache.shape
    by = cache[..., :ps * 64].reshape(P, H, ps, 64)
    s = e4m3_value(cache[..., ps * 64:].reshape(P, H, ps, 8))
    n = np.empty((P, H, ps, 128))
    n[..., 0::2] = (by & 15).astype(np.float64) - 8
    n[..., 1::2] = (by >> 4).astype(np.float64) - 8
    return n * np.repeat(s, 16, axis=-1)


def paged_attention(q, kc, vc, ps, block_table, seq_lens, ck, cv, sm_scale, window_left=-1):
    """q float64 [B][M][Hq][128] -> (out, mag, lmag, vsum) float64 of that
    shape, with the softmax weights w: mag = sum w |v| is what roundings of the weights act
    on; lmag = sum w a |v| + |out| sum w a, a = sm_scale sum |q_i k_i|, is what a
    relative error of the logits' partial sums acts on (the first-order change
    of sum w v when every logit moves by at most e a is at most e lmag); vsum =
    sum |v| is what an absolute error of every weight acts on."""
    B, M, Hq, D = q.shape
    H = kc.shape[1]
    G = Hq // H
    out, mag, lmag, vsum = (np.zeros(q.shape) for _ in range(4))
    for b in range(B):
        L = int(seq_lens[b])
        n = (L + ps - 1) // ps
        ids = np.asarray(block_table[b][:n])
        ok = (ids >= 0) & (ids < kc.shape[0])
        k, v = (np.where(ok[:, None, None, None], read_pages(c[np.where(ok, ids, 0)], ps), 0.0) for c in (kc, vc))
        k = k.transpose(1, 0, 2, 3).reshape(H, n * ps, D)[:, :L] * float(ck)
        v = v.transpose(1, 0, 2, 3).reshape(H, n * ps, D)[:, :L] * float(cv)
        j = np.arange(L)
        for m in range(M):
            p = L - M + m
            see = (j <= p) & ((j >= p - window_left) if window_left >= 0 else True)
            for h in range(Hq):
                s = k[h // G][see] @ q[b, m, h] * sm_scale
                w = np.exp(s - s.max())
                w /= w.sum()
                out[b, m, h] = w @ v[h // G][see]
                mag[b, m, h] = w @ np.abs(v[h // G][see])
                vsum[b, m, h] = np.abs(v[h // G][see]).sum(0)
                wa = w * (np.abs(k[h // G][see]) @ np.abs(q[b, m, h])) * sm_scale
                lmag[b, m, h] = wa @ np.abs(v[h // G][see]) + np.abs(out[b, m, h]) * wa.sum()
    return out, mag, lmag, vsum

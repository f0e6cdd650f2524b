"""fp8kv_prompt_attention: argument checks (CPU), and the GPU kernel against a
float64 softmax at the lengths, groupings, windows and strides where row tiles,
key tiles and sequences end."""
import ctypes

import numpy as np
import pytest
import torch

from verify_attention_gb300 import build, fp8kv

NULL = ctypes.c_void_p(0)
P16 = ctypes.c_void_p(1 << 20)          # fake, 16-byte aligned: never dereferenced
SM = 128 ** -0.5


def test_argument_checks():
    build.build()
    L = fp8kv.lib()
    good = dict(q=P16, qs=72 * 128, k=P16, ks=1024, v=P16, vs=1024, cu=P16, B=2, T=100, maxL=60, Hq=72, Hkv=8, D=128,
                sm=0.088, wl=-1, out=P16, stream=NULL)
    bad16 = ctypes.c_void_p((1 << 20) + 8)
    for over, want in (({"q": NULL}, 1), ({"k": NULL}, 1), ({"v": NULL}, 1), ({"cu": NULL}, 1), ({"out": NULL}, 1),
                       ({"q": bad16}, 1), ({"v": bad16}, 1), ({"out": bad16}, 1), ({"qs": 71 * 128}, 1),
                       ({"ks": 1028}, 1), ({"vs": 1000}, 1), ({"B": -1}, 1), ({"T": -1}, 1), ({"maxL": -1}, 1),
                       ({"Hq": 70}, 1), ({"Hkv": 0}, 1), ({"wl": -2}, 1), ({"sm": 0.0}, 1), ({"sm": -1.0}, 1),
                       ({"sm": float("nan")}, 1), ({"sm": float("inf")}, 1), ({"D": 64}, 2),
                       ({"Hq": 8 * 129, "qs": 8 * 129 * 128}, 2), ({"T": 2_000_000_000}, 2), ({"B": 70000}, 2),
                       ({"B": 0, "q": NULL, "out": NULL}, 0), ({"T": 0, "cu": NULL}, 0)):
        assert L.fp8kv_prompt_attention(*{**good, **over}.values()) == want, over


def test_binding_refuses_other_layouts():
    q = torch.zeros((5, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):                     # not on a GPU
        fp8kv.fp8kv_prompt_attention(q, q, q, torch.zeros(2, dtype=torch.int32), 5, SM)


# ------------------------------------------------------------------- GPU

def _inputs(seed, lens, G, H, pad=0, fused=False, head=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T = head + sum(lens) + pad
    if fused:
        x = torch.randn((T, (G + 2) * H, 128), generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = x[:, :G * H], x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:]
    else:
        q, k, v = (torch.randn((T, h, 128), generator=g, device="cuda").to(torch.bfloat16) for h in (G * H, H, H))
    cu = torch.tensor(np.concatenate([[head], head + np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    return q, k, v, cu


def _reference(q, k, v, lo, hi, window, sm=SM):
    """float64 (out, mag, lmag) of one sequence: see oracle/int4_np.py."""
    G = q.shape[1] // k.shape[1]
    n = hi - lo
    p, j = torch.arange(n, device=q.device)[:, None], torch.arange(n, device=q.device)[None]
    see = (j <= p) & (j >= p - window) if window >= 0 else j <= p
    res = [torch.empty((n, q.shape[1], 128), dtype=torch.float64, device=q.device) for _ in range(3)]
    for h in range(q.shape[1]):
        qh, kh, vh = q[lo:hi, h].double(), k[lo:hi, h // G].double(), v[lo:hi, h // G].double()
        w = torch.softmax(torch.where(see, qh @ kh.T * sm, float("-inf")), -1)
        res[0][:, h] = w @ vh
        res[1][:, h] = w @ vh.abs()
        wa = w * (qh.abs() @ kh.abs().T) * sm
        res[2][:, h] = wa @ vh.abs() + res[0][:, h].abs() * wa.sum(-1, keepdim=True)
    return res


def _check(out, q, k, v, cu, window, sm=SM):
    c = cu.tolist()
    for lo, hi in zip(c[:-1], c[1:]):
        if hi == lo:
            continue
        ref, mag, lmag = _reference(q, k, v, lo, hi, window, sm)
        # output: half a bf16 step, 2^-8 of the value.  Weights: the same half
        # step, 2^-8 of each, plus exponentials and sums (below 2^-12): of mag.
        # Logits: eight accumulating steps off by an ulp (2^-23) of a partial sum
        # each: 2^-20 lmag.
        err = (out[lo:hi].double() - ref).abs()
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -20 * lmag
        assert bool((err <= tol).all()), (lo, hi, float((err / tol).max()), float(err.max()))


CASES = [
    # lens, G, H, window, pad, fused
    ([1], 1, 1, -1, 0, False),
    ([1, 1, 1], 9, 2, -1, 5, True),
    ([33], 9, 8, -1, 0, True),
    ([14, 15, 28, 29, 27], 9, 1, -1, 0, False),         # row tiles of 14 positions, CTAs of 28
    ([127, 128, 129], 1, 2, -1, 3, False),
    ([255, 256, 257, 1], 1, 1, -1, 0, True),
    ([0, 40, 0, 0, 100, 0], 4, 2, -1, 130, False),
    ([500, 3, 77], 8, 2, -1, 0, True),
    ([1300], 9, 2, -1, 0, False),
    ([2500], 2, 1, -1, 0, False),
    ([900, 411], 9, 1, 511, 0, True),
    ([700], 3, 2, 0, 0, False),
    ([700, 50], 6, 1, 1, 0, False),
    ([1000], 1, 2, 100, 7, True),
    ([1000], 16, 1, 127, 0, False),
    ([300], 128, 1, -1, 0, False),
    ([300], 65, 1, 40, 0, False),
    ([300], 100, 1, -1, 0, False),
    ([641, 640, 639], 5, 3, 128, 1, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,G,H,window,pad,fused", CASES)
def test_matches_the_definition(lens, G, H, window, pad, fused):
    fp8kv.fp8kv_device_status(clear=True)
    q, k, v, cu = _inputs(sum(lens) + G, lens, G, H, pad, fused)
    out = torch.full((q.shape[0], G * H, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    got = fp8kv.fp8kv_prompt_attention(q, k, v, cu, max(lens), SM, window_left=window, out=out)
    assert got is out and "prompt" in fp8kv.fp8kv_last_dispatch()
    assert fp8kv.fp8kv_device_status(clear=True) == 0
    _check(out, q, k, v, cu, window)
    assert bool((out[sum(lens):] == 3.0).all())         # rows behind the last sequence


@pytest.mark.gpu
def test_many_sequences():
    rng = np.random.default_rng(7)
    lens = [int(n) for n in rng.integers(0, 40, 300)]
    q, k, v, cu = _inputs(11, lens, 4, 1)
    out = fp8kv.fp8kv_prompt_attention(q, k, v, cu, 40, SM)
    _check(out, q, k, v, cu, -1)


@pytest.mark.gpu
def test_only_empty_sequences():
    q, k, v, _ = _inputs(3, [5], 4, 1)
    out = torch.full_like(q, 3.0)
    cu = torch.tensor([2, 2, 2, 2], dtype=torch.int32, device="cuda")
    fp8kv.fp8kv_prompt_attention(q, k, v, cu, 0, SM, out=out)
    assert bool((out == 3.0).all())


@pytest.mark.gpu
def test_rows_beyond_four_gigabytes():
    """2001 sequences of up to 130 tokens, 72 heads: q and out of more than 2^32
    bytes; the first and the last sequences against the definition."""
    rng = np.random.default_rng(2)
    lens = [int(n) for n in rng.integers(120, 131, 2001)]
    q, k, v, cu = _inputs(14, lens, 9, 8)
    assert q.numel() * 2 > 2 ** 32
    out = fp8kv.fp8kv_prompt_attention(q, k, v, cu, 130, SM)
    _check(out, q, k, v, cu[:4], -1)
    _check(out, q, k, v, cu[-4:], -1)
    _check(out, q, k, v, cu[1850:1853], -1)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [-1, 60])
def test_rows_of_no_sequence_may_hold_anything(window):
    """NaN and infinities before the first sequence, behind the last one and in
    a neighbour reach no row of a clean sequence."""
    lens = [200, 50, 333]
    q, k, v, cu = _inputs(5, lens, 9, 2, pad=300, head=17)
    want = fp8kv.fp8kv_prompt_attention(q, k, v, cu, 333, SM, window_left=window)
    for x in (q, k, v):
        x[:17] = float("nan")
        x[17 + 583:] = float("inf")
        x[17 + 200:17 + 250] = float("nan")             # the whole second sequence
    out = torch.full_like(want, 3.0)
    fp8kv.fp8kv_prompt_attention(q, k, v, cu, 333, SM, window_left=window, out=out)
    for lo, hi in ((17, 217), (267, 600)):
        assert torch.equal(out[lo:hi], want[lo:hi])
    assert bool((out[:17] == 3.0).all()) and bool((out[600:] == 3.0).all())


@pytest.mark.gpu
def test_masked_keys_with_infinite_scores():
    """A later key of any size, up to infinity, does not reach earlier rows."""
    q, k, v, cu = _inputs(6, [400], 4, 1)
    want = fp8kv.fp8kv_prompt_attention(q, k, v, cu, 400, SM)
    for bad in (float("inf"), float("nan"), 3e38):
        k2 = k.clone()
        k2[300:] = bad
        out = fp8kv.fp8kv_prompt_attention(q, k2, v, cu, 400, SM)
        assert torch.equal(out[:300], want[:300])


@pytest.mark.gpu
@pytest.mark.parametrize("sm", [1e-3, 1.0, 4.0])
def test_large_and_small_logits(sm):
    q, k, v, cu = _inputs(8, [700, 90], 9, 1)
    q[::3] *= 8
    k[5::50] *= 4
    out = fp8kv.fp8kv_prompt_attention(q, k, v, cu, 700, sm)
    _check(out, q, k, v, cu, -1, sm)


@pytest.mark.gpu
def test_growing_maxima_rescale_the_output():
    """Keys sorted so that every tile raises the row maxima by more than 2^8."""
    q, k, v, cu = _inputs(9, [1200], 2, 1)
    q[:] = q.abs()
    k[:] = (k.abs() * torch.linspace(0.01, 6, 1200, device="cuda")[:, None, None]).to(torch.bfloat16)
    out = fp8kv.fp8kv_prompt_attention(q, k, v, cu, 1200, 0.5)
    _check(out, q, k, v, cu, -1, 0.5)


@pytest.mark.gpu
def test_bad_sequences_are_flagged_and_skipped():
    fp8kv.fp8kv_device_status(clear=True)
    q, k, v, cu = _inputs(10, [50, 60, 70], 9, 1, pad=20)
    want = fp8kv.fp8kv_prompt_attention(q, k, v, cu, 70, SM)
    out = torch.full_like(want, 3.0)
    fp8kv.fp8kv_prompt_attention(q, k, v, cu, 65, SM, out=out)                  # the third is too long
    assert fp8kv.fp8kv_device_status(clear=True) == fp8kv.DEV_BAD_SEQ_LEN
    assert torch.equal(out[:110], want[:110]) and bool((out[110:] == 3.0).all())
    for bad in ([0, 50, 40, 180], [-4, 50, 110, 180], [0, 50, 110, 1000], [0, 2 ** 31 - 1, 60, 90],
                [0, 50, -2 ** 31, 180]):
        out.fill_(3.0)
        c = torch.tensor(bad, dtype=torch.int32, device="cuda")
        fp8kv.fp8kv_prompt_attention(q, k, v, c, 200, SM, out=out)
        assert fp8kv.fp8kv_device_status(clear=True) == fp8kv.DEV_BAD_SEQ_LEN, bad
    out = fp8kv.fp8kv_prompt_attention(q, k, v, cu, 70, SM)
    assert torch.equal(out, want)


@pytest.mark.gpu
def test_captured_replayed_and_on_two_streams():
    q, k, v, cu = _inputs(12, [300, 41], 9, 2)
    outs = [torch.zeros_like(q) for _ in range(2)]
    side = [torch.cuda.Stream() for _ in range(2)]
    fp8kv.fp8kv_prompt_attention(q, k, v, cu, 300, SM)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for o, s in zip(outs, side):
            s.wait_stream(main)
            fp8kv.fp8kv_prompt_attention(q, k, v, cu, 300, SM, out=o, stream=s)
            main.wait_stream(s)
    q.copy_(q.roll(1, 0))
    cu.copy_(torch.tensor([0, 100, 341], dtype=torch.int32))
    want = fp8kv.fp8kv_prompt_attention(q, k, v, cu, 300, SM)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.gpu
@pytest.mark.parametrize("ps,window", [(32, -1), (64, 100)])
def test_prompt_insert_and_decode_together(ps, window):
    """A prompt through prompt attention and the 4-bit insert, then decode steps
    that append: as a serving program runs them, against the oracle's attention
    over the stored values."""
    from oracle import int4_np
    lens, G, H, steps = [70, 33], 9, 2, 3
    q, k, v, cu = _inputs(13, lens, G, H, fused=True)
    out = fp8kv.fp8kv_prompt_attention(q, k, v, cu, 70, SM, window_left=window)
    _check(out, q, k, v, cu, window)
    width = (max(lens) + steps + ps - 1) // ps
    bt = torch.randperm(2 * width, device="cuda").to(torch.int32).view(2, width)
    kc, vc = (fp8kv.fp8kv_int4_cache(2 * width, H, ps) for _ in range(2))
    ks, vs = (torch.tensor([5 / 448], device="cuda") for _ in range(2))
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    seq = torch.repeat_interleave(torch.arange(2, device="cuda"), torch.tensor(lens, device="cuda"))
    slots = bt[seq, pos // ps].long() * ps + pos % ps
    fp8kv.fp8kv_cache_insert(k.contiguous(), v.contiguous(), slots, ks, vs, kc, vc)
    got = fp8kv.fp8kv_cache_gather(slots, ks, vs, kc, vc)
    for x, y in zip((k, v), got):                       # half a step of the block's scale, and bf16's rounding
        amax = x.float().view(-1, H, 8, 16).abs().amax(-1, keepdim=True).expand(-1, -1, 8, 16).reshape(x.shape)
        assert bool(((x.float() - y.float()).abs() <= amax * (1.0625 / 14) + 2.0 ** -8 * y.float().abs()).all())
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(steps):
        sl += 1
        qd, kn, vn = (torch.randn((2, 1, h, 128), generator=g, device="cuda").to(torch.bfloat16)
                      for h in (G * H, H, H))
        o = fp8kv.fp8kv_append_paged_attention(kn, vn, qd, kc, vc, bt, sl, int(sl.max()), ks, vs, SM, window_left=window)
        ref, mag, lmag, vsum = int4_np.paged_attention(qd.double().cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy(), ps,
                                                       bt.cpu().numpy(), sl.cpu().numpy(), ks.item(), vs.item(), SM,
                                                       window)
        # the tolerance of tests/test_int4_cache.py
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag + 2.0 ** -20 * lmag + 2.0 ** -36 * vsum
        assert np.all(np.abs(o.double().cpu().numpy() - ref) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_outputs_of_a_call_on_another_stream(handle):
    """What the calls allocate is filled on their stream: here the current stream
    is busy until they are done."""
    lens = [200, 70]
    q, k, v, cu = _inputs(15, lens, 9, 2)
    want = fp8kv.fp8kv_prompt_attention(q, k, v, cu, 200, SM)
    kc, vc = (fp8kv.fp8kv_int4_cache(9, 2, 32) for _ in range(2))
    one = torch.tensor([0.01], device="cuda")
    slots = torch.arange(270, device="cuda")
    fp8kv.fp8kv_cache_insert(k, v, slots, one, one, kc, vc)
    rows = fp8kv.fp8kv_cache_gather(slots, one, one, kc, vc)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                               # about 0.1 s
    s = side.cuda_stream if handle else side
    out = fp8kv.fp8kv_prompt_attention(q, k, v, cu, 200, SM, stream=s)
    got = fp8kv.fp8kv_cache_gather(slots, one, one, kc, vc, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(got[0], rows[0]) and torch.equal(got[1], rows[1])


@pytest.mark.gpu
def test_tensors_of_another_device_are_refused(monkeypatch):
    q, k, v, cu = _inputs(16, [40], 4, 1)
    kc, vc = (fp8kv.fp8kv_int4_cache(2, 1, 32) for _ in range(2))
    one = torch.tensor([0.01], device="cuda")
    slots = torch.arange(40, device="cuda")
    bt, sl = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), torch.tensor([40], dtype=torch.int32, device="cuda")
    call = fp8kv.PreparedAttention(q[None, -1:].contiguous(), kc, vc, bt, sl, 40, one, one, SM)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for f in (lambda: fp8kv.fp8kv_prompt_attention(q, k, v, cu, 40, SM, out=torch.empty_like(q)), call,
              lambda: fp8kv.fp8kv_cache_insert(k, v, slots, one, one, kc, vc),
              lambda: fp8kv.fp8kv_cache_gather(slots, one, one, kc, vc, torch.empty_like(k), torch.empty_like(v))):
        with pytest.raises(ValueError, match="current device"):
            f()


# Items one of whose two row tiles is whole, then items with both, on every CTA:
# the two share the staging tile of the output.

def _staged_items(seed, NP, sequences, longest):
    """Lengths whose last item has a whole first row tile and a partial, a
    one-row or no second one, between sequences of whole items."""
    rng = np.random.default_rng(seed)
    ends = [NP, NP + 1, 2 * NP - 1]
    return [2 * NP * int(rng.integers(0 if e else 1, longest)) + e
            for e in (int(rng.choice([0, 0, *ends])) for _ in range(sequences))]


@pytest.mark.gpu
@pytest.mark.parametrize("G,H", [(2, 8), (1, 4), (4, 3)])
def test_output_tiles_of_items_with_one_whole_row_tile_exactly(G, H):
    """With a window of its own key alone a row's output is that key's value,
    bit for bit: items of one uncleaned key tile, far more than SMs."""
    lens = _staged_items(G, 128 // G, 300, 4)
    q, k, v, cu = _inputs(G, lens, G, H)
    want = v.repeat_interleave(G, 1)
    out = torch.empty_like(want)
    for _ in range(40):
        out.fill_(3.0)
        fp8kv.fp8kv_prompt_attention(q, k, v, cu, max(lens), SM, window_left=0, out=out)
        assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("G,H,window", [(8, 4, -1), (2, 4, 63), (16, 2, -1)])
def test_output_tiles_of_items_with_one_whole_row_tile(G, H, window):
    fp8kv.fp8kv_device_status(clear=True)
    lens = _staged_items(10 + G, 128 // G, 150, 12)
    q, k, v, cu = _inputs(20 + G, lens, G, H)
    want = fp8kv.fp8kv_prompt_attention(q, k, v, cu, max(lens), SM, window_left=window)
    _check(want, q, k, v, cu, window)
    out = torch.empty_like(want)
    for _ in range(40):
        out.fill_(3.0)
        fp8kv.fp8kv_prompt_attention(q, k, v, cu, max(lens), SM, window_left=window, out=out)
        assert torch.equal(out, want)
    assert fp8kv.fp8kv_device_status(clear=True) == 0


class _On:
    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device


@pytest.mark.parametrize("stream", [0, 1 << 20, type("S", (), {"cuda_stream": 1 << 20})()])
def test_a_given_stream_does_not_hide_another_device(monkeypatch, stream):
    """The kernels run on the current device: tensors of another one are refused
    whether the stream is given or not."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert fp8kv._stream(stream, _On(0)) == getattr(stream, "cuda_stream", stream)
    with pytest.raises(ValueError, match="current device"):
        fp8kv._stream(stream, _On(1))

"""The INT4 cache: its definition (CPU), argument checks (CPU), and insert,
append, gather and paged attention on the GPU against the numpy oracle."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import int4_np
from verify_attention_gb300 import build, fp8kv, inputs as gen

NULL = ctypes.c_void_p(0)
P16 = ctypes.c_void_p(1 << 20)          # fake, 16-byte aligned: never dereferenced
SM = 128 ** -0.5


@pytest.fixture(scope="module")
def L():
    build.build()
    return fp8kv.lib()


# ------------------------------------------------------------ definition

def _bf16(x):
    return torch.tensor(np.asarray(x, np.float32)).to(torch.bfloat16)


def test_e4m3_codec_against_the_format():
    v = int4_np.e4m3_value(np.arange(256))
    assert v[0x7e] == 448 and v[1] == 2.0 ** -9 and np.isnan(v[0x7f]) and v[0x38] == 1.0
    assert np.array_equal(int4_np.e4m3_code(v[:127]), np.arange(127))
    mid = (v[:126] + v[1:127]) / 2                       # ties go to the even code
    assert np.array_equal(int4_np.e4m3_code(mid), np.arange(126) + np.arange(126) % 2)
    assert int4_np.e4m3_code(np.array([1e9, np.inf]))[0] == 0x7e


@pytest.mark.parametrize("c", [1.0, 0.0123, 37.0])
def test_encode_is_within_half_a_step(c):
    x = _bf16(np.random.default_rng(3).normal(size=(50, 2, 128)) * c * 20).float().numpy()
    n, sc = int4_np.encode_rows(x, c)
    step = np.repeat(int4_np.e4m3_value(sc), 16, -1) * float(np.float32(c))
    # amax / step <= 7 (1 + 2^-4) < 7.5: clamping never costs more than rounding;
    # the fp32 roundings of s c, its reciprocal and the product: 3 * 2^-24 of n
    assert np.all(np.abs(x - n * step) <= step * (0.5 + 8 * 2.0 ** -22))


def test_page_bytes_round_trip():
    rng = np.random.default_rng(5)
    n = rng.integers(-7, 8, (40, 3, 128)).astype(np.int8)
    sc = rng.integers(1, 127, (40, 3, 8)).astype(np.uint8)
    cache = np.zeros((2, 3, 32 * 72), np.uint8)
    slots = rng.permutation(64)[:40]
    int4_np.write_rows(cache, 32, slots, n, sc)
    got = int4_np.read_pages(cache, 32)[slots // 32, :, slots % 32]
    assert np.array_equal(got, n * np.repeat(int4_np.e4m3_value(sc), 16, -1))


# ------------------------------------------------------- argument checks

def test_int4_entry_points_check_their_arguments(L):
    ins = [P16, P16, P16, 4, 8, 128, P16, P16, P16, P16, 16, 32, 2, NULL]
    for at, bad, want in ((0, NULL, 1), (6, NULL, 1), (7, NULL, 1), (5, 96, 2), (11, 48, 2), (3, -1, 1), (3, 0, 0),
                          (8, ctypes.c_void_p((1 << 20) + 8), 1), (12, 3, 1)):
        assert L.fp8kv_cache_insert(*[bad if i == at else a for i, a in enumerate(ins)]) == want, at
    gat = [P16, 4, 8, 128, P16, P16, P16, P16, 16, 32, 2, P16, P16, NULL]
    for at, bad, want in ((0, NULL, 1), (4, NULL, 1), (6, NULL, 1), (11, NULL, 1), (3, 64, 2), (9, 16, 2), (10, 5, 1),
                          (1, 0, 0), (1, -1, 1), (12, ctypes.c_void_p((1 << 20) + 4), 1)):
        for dt in (0, 2):
            a = [bad if i == at else (dt if i == 10 else x) for i, x in enumerate(gat)]
            assert L.fp8kv_cache_gather(*a) == want, (at, dt)
    att = dict(q=P16, k=P16, v=P16, dt=2, bt=P16, mpps=4, sl=P16, maxL=100, B=1, M=1, Hq=72, Hkv=8, D=128, ps=32, P=16,
               ks=P16, vs=P16, sm=0.088, wl=-1, split=32, ws=P16, wsb=1 << 30, out=P16, stream=NULL)
    for over, want in (({"ks": NULL}, 1), ({"vs": NULL}, 1), ({"M": 17, "split": 0}, 2), ({"D": 64}, 2),
                       ({"M": 16, "Hq": 80, "split": 0}, 2), ({"ws": NULL}, 3), ({"wsb": 16}, 3), ({"maxL": 200}, 1),
                       ({"ps": 16, "split": 0}, 2), ({"wl": -2}, 1), ({"B": 0}, 0),
                       ({"k": ctypes.c_void_p((1 << 20) + 8)}, 1)):
        assert L.fp8kv_paged_attention(*{**att, **over}.values()) == want, over
    layers = (fp8kv.fp8kv_layer * 1)()
    assert L.fp8kv_paged_attention_layers(ctypes.byref(layers), 1, 1, 12, 72, 8, 128, 32, 2, P16, 1 << 30, NULL) in (1, 2)


def test_int4_attention_refuses_grids_that_do_not_exist(L):
    att = dict(q=P16, k=P16, v=P16, dt=2, bt=P16, mpps=4, sl=P16, maxL=100, B=1, M=1, Hq=72, Hkv=8, D=128, ps=32, P=16,
               ks=P16, vs=P16, sm=0.088, wl=-1, split=0, ws=P16, wsb=1 << 62, out=P16, stream=NULL)
    for over in ({"B": 65536}, {"Hq": 65536, "Hkv": 65536}, {"M": 16, "Hq": 2 * 33000, "Hkv": 33000}):
        assert L.fp8kv_paged_attention(*{**att, **over}.values()) == 2, over


def test_binding_refuses_other_shapes():
    assert fp8kv._cache_dtype(torch.zeros((2, 8, 32 * 72), dtype=torch.uint8)) == fp8kv.FP8KV_CACHE_INT4
    assert fp8kv._cache_dtype(torch.zeros((2, 8, 32, 128), dtype=torch.uint8)) == fp8kv.FP8KV_CACHE_E4M3
    c = torch.zeros((2, 8, 32 * 72), dtype=torch.uint8)
    assert fp8kv._cache_shape(c, c, 2) == (2, 8, 32)
    with pytest.raises(ValueError):
        fp8kv._cache_shape(torch.zeros((2, 8, 100), dtype=torch.uint8), c, 2)
    with pytest.raises(ValueError):
        fp8kv._cache_shape(c, torch.zeros((3, 8, 32 * 72), dtype=torch.uint8), 2)


# --------------------------------------------------------------- GPU: rows

def _scale(c):
    return torch.tensor([c], dtype=torch.float32, device="cuda")


def _insert(k, v, slots, pages, ps, ck, cv, poison=0xA5):
    kc = torch.full((pages, k.shape[1], ps * 72), poison, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    fp8kv.fp8kv_cache_insert(k.cuda(), v.cuda(), slots.cuda(), _scale(ck), _scale(cv), kc, vc)
    return kc, vc


def _special(rng, T, H):
    """Rows with zeros, signed zeros, tiny and huge values, infinities and NaN."""
    x = rng.normal(size=(T, H, 128)).astype(np.float32)
    for i, val in enumerate((0.0, -0.0, 1e-38, -3e38, np.inf, -np.inf, np.nan, 1e-5, 7.5, 2.0 ** -20)):
        x[i % T, i % H, (13 * i) % 128] = val
        x[(i + 3) % T, (i + 1) % H, 16 * (i % 8):16 * (i % 8) + 16] = val
    return _bf16(x)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,ps,ck,cv", [(1, 1, 32, 1.0, 1.0), (7, 2, 64, 0.01, 2.0), (97, 8, 32, 12 / 448, 6 / 448),
                                          (300, 3, 64, 1e-3, 1e4), (33, 5, 32, 2.0 ** -100, 2.0 ** 100)])
def test_insert_is_bit_exact(T, H, ps, ck, cv):
    rng = np.random.default_rng(T)
    k, v = _special(rng, T, H), _special(rng, T, H)
    pages = T // ps + 2
    slots = torch.from_numpy(rng.permutation(pages * ps)[:T].copy())
    if T > 2:
        slots[T // 2] = -1
        slots[1] = -7
    kc, vc = _insert(k, v, slots, pages, ps, ck, cv)
    for x, c, got in ((k, ck, kc), (v, cv, vc)):
        want = np.full((pages, H, ps * 72), 0xA5, np.uint8)
        int4_np.write_rows(want, ps, slots.numpy(), *int4_np.encode_rows(x.float().numpy(), c))
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.gpu
def test_every_bf16_value_in_one_block():
    """Each of the 65536 bf16 patterns as a block of its own beside a 1.0."""
    bits = np.arange(65536, dtype=np.uint32)
    x = np.full((512, 1, 128), 1.0, np.float32).reshape(-1, 16)
    x = np.concatenate([x] * 16)                          # 65536 blocks
    x[:, 5] = (bits << 16).view(np.float32)
    x = torch.from_numpy(x.reshape(8192, 1, 128)).to(torch.bfloat16)
    slots = torch.arange(8192)
    kc, _ = _insert(x, x, slots, 256, 32, 0.037, 0.037)
    want = np.zeros((256, 1, 32 * 72), np.uint8)
    int4_np.write_rows(want, 32, slots.numpy(), *int4_np.encode_rows(x.float().numpy(), 0.037))
    assert np.array_equal(kc.cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["int4", "e4m3", "bf16"])
@pytest.mark.parametrize("T,H,ps", [(1, 1, 64), (45, 8, 32), (130, 3, 64)])
def test_gather_reads_back_what_is_stored(dt, T, H, ps):
    rng = np.random.default_rng(T + H)
    k, v = _special(rng, T, H).cuda(), _bf16(rng.normal(size=(T, H, 128))).cuda()
    pages = T // ps + 2
    if dt == "int4":
        kc = fp8kv.fp8kv_int4_cache(pages, H, ps)
    else:
        kc = torch.zeros((pages, H, ps, 128), dtype=torch.uint8 if dt == "e4m3" else torch.bfloat16, device="cuda")
    vc = kc.clone()
    slots = torch.from_numpy(rng.permutation(pages * ps)[:T].copy()).cuda()
    ks, vs = _scale(0.02), _scale(0.013)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    read = torch.cat([slots, slots[:1], torch.tensor([-1], device="cuda")])          # a slot twice, one skipped
    ko = torch.full((T + 2, H, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    fp8kv.fp8kv_cache_gather(read, ks, vs, kc, vc, ko, vo)
    for c, s, o in ((kc, ks, ko), (vc, vs, vo)):
        if dt == "int4":
            x = torch.from_numpy(int4_np.read_pages(c.cpu().numpy(), ps)).float()
        elif dt == "e4m3":
            x = torch.from_numpy(int4_np.e4m3_value(c.cpu().numpy())).float()
        else:
            x = c.float().cpu()
        x = x if dt == "bf16" else x * s.cpu()
        at = read.cpu()[:-1]
        want = x[at // ps, :, at % ps].to(torch.bfloat16)
        assert torch.equal(torch.nan_to_num(o[:-1].cpu(), nan=99.0), torch.nan_to_num(want, nan=99.0))
        assert bool((o[-1] == 3.0).all())


@pytest.mark.gpu
def test_bad_slots_are_flagged_and_skipped():
    fp8kv.fp8kv_device_status(clear=True)
    k = _bf16(np.ones((3, 2, 128)))
    slots = torch.tensor([5, 64, 1 << 40])
    kc, vc = _insert(k, k, slots, 2, 32, 1.0, 1.0)
    assert fp8kv.fp8kv_device_status(clear=True) == fp8kv.DEV_BAD_SLOT
    rest = torch.cat([kc[0, :, :5 * 64].flatten(), kc[0, :, 6 * 64:32 * 64].flatten(), kc[1].flatten()])
    assert bool((rest == 0xA5).all())
    o = torch.full((3, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8kv.fp8kv_cache_gather(slots.cuda(), _scale(1.0), _scale(1.0), kc, vc, o, o.clone())
    assert fp8kv.fp8kv_device_status(clear=True) == fp8kv.DEV_BAD_SLOT
    # a block of ones with tensor scale 1: s is the E4M3 value nearest to 1/7 =
    # 0.142857..., between 9/64 = 0.140625 and 10/64 the former, n = rint(64/9) = 7,
    # and the row reads as 7 * 9/64 = 0.984375 (exact in bf16)
    assert bool((o[0] == 0.984375).all()) and bool((o[1:] == 7.0).all())


# ---------------------------------------------------------- GPU: attention

def _case(seed, lens, M, G, H, ps, extra=1):
    g = gen.generator(seed)
    lay = gen.paged_layout(lens, ps, g, extra_pages=extra)
    B = len(lens)
    q = torch.randn((B, M, G * H, 128), generator=g).to(torch.bfloat16).cuda()
    # stale bytes everywhere (NaN scales, arbitrary codes) behind what is written
    kc = torch.full((lay.num_pages, H, ps * 72), 0x7F, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    ks, vs = _scale(6 / 448), _scale(5 / 448)
    x = [torch.randn((sum(lens), H, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    slots = torch.cat([lay.slots(b, range(n)) for b, n in enumerate(lens)]).cuda()
    return lay, q, kc, vc, ks, vs, x[0], x[1], slots


def _attend(lay, q, kc, vc, ks, vs, window=-1, **kw):
    return fp8kv.fp8kv_paged_attention(q, kc, vc, lay.block_table.cuda(), lay.seq_lens.cuda(), int(lay.seq_lens.max()),
                                       ks, vs, SM, window_left=window, **kw)


def _check(out, lay, q, kc, vc, ks, vs, ps, window=-1, rows=None):
    ref, mag, lmag, vsum = int4_np.paged_attention(q.double().cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy(), ps,
                                                   lay.block_table.numpy(), lay.seq_lens.numpy(), ks.item(), vs.item(),
                                                   SM, window)
    # bf16 output: half a step, 2^-8 of the value.  Softmax weights: f16 of 2^11
    # times the weight against a maximum that lags at most 2^4 behind, off by
    # 2^-11 of itself (with exponentials, sums and the f32 product with the scale
    # below 2^-14 more: under 2^-10 of mag) or, below f16's normal range, by
    # 2^-25, that is 2^-36 of the row's sum, which is at least 2^11: times vsum.
    # Logits: a sum of 128 products is eight accumulating steps of 16, each off by
    # at most an ulp (2^-23) of the partial sum, whose size is at most a:
    # 8 * 2^-23 a, which moves the output by at most 2^-20 lmag.  (That term
    # matters only where |q| |k| is in the hundreds: with a = 560, 2 * 560 * 2^-20
    # is already 2^-10.)  Partials of more than 16 rows: f16, 2^-11 of each, so at
    # most 2^-11 of mag.
    err = np.abs(out.double().cpu().numpy() - ref)
    many = q.shape[1] * q.shape[2] // kc.shape[1] > 16
    tol = (2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + many * 2.0 ** -11) * mag + 2.0 ** -20 * lmag + 2.0 ** -36 * vsum)
    assert np.all(err <= tol), (float((err / tol).max()), float(err.max()))


ATTENTION = [
    # lens, M, G, H, ps, window, split_tokens
    ([1], 1, 1, 1, 32, -1, 0),
    ([256], 1, 9, 8, 32, -1, 0),
    ([33, 1, 64, 500], 1, 4, 2, 64, -1, 64),
    ([31, 32, 33, 63, 65], 1, 12, 1, 32, -1, 32),
    ([5000], 1, 9, 2, 64, -1, 0),
    ([3001, 2, 1024], 2, 8, 2, 32, -1, 256),
    ([1500, 700], 1, 16, 2, 32, 99, 0),
    ([400, 90], 1, 9, 2, 64, 0, 0),
    ([12, 300], 12, 9, 2, 32, -1, 0),
    ([1000], 12, 9, 2, 64, -1, 0),
    ([1000], 12, 9, 2, 32, -1, 96),
    ([2100, 13, 640], 12, 9, 1, 32, 511, 0),
    ([777, 40], 7, 5, 3, 64, 20, 0),
    ([2500, 130], 16, 9, 1, 64, -1, 0),
    ([600], 16, 1, 2, 32, 100, 64),
    ([300, 17], 3, 6, 2, 32, -1, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,M,G,H,ps,window,split", ATTENTION)
def test_attention_matches_the_oracle(lens, M, G, H, ps, window, split):
    fp8kv.fp8kv_device_status(clear=True)
    lay, q, kc, vc, ks, vs, k, v, slots = _case(sum(lens) + M, lens, M, G, H, ps)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    out = _attend(lay, q, kc, vc, ks, vs, window, split_tokens=split)
    assert "int4" in fp8kv.fp8kv_last_dispatch()
    _check(out, lay, q, kc, vc, ks, vs, ps, window)
    assert fp8kv.fp8kv_device_status(clear=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("lens,M,G,H,ps,window", [([1, 70], 1, 9, 2, 32, -1), ([12, 95, 1000], 12, 9, 2, 32, -1),
                                                  ([2000], 12, 9, 2, 64, 127), ([64, 65], 4, 4, 3, 64, -1)])
def test_append_equals_insert_then_attention(lens, M, G, H, ps, window):
    lay, q, kc, vc, ks, vs, k, v, slots = _case(7 * sum(lens), lens, M, G, H, ps)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    want = _attend(lay, q, kc, vc, ks, vs, window)
    _check(want, lay, q, kc, vc, ks, vs, ps, window)
    new = torch.cat([torch.arange(sum(lens[:b + 1]) - M, sum(lens[:b + 1])) for b in range(len(lens))]).cuda()
    kc2, vc2 = kc.clone(), vc.clone()
    old = torch.ones(len(slots), dtype=torch.bool, device="cuda")
    old[new] = False
    zero = torch.zeros_like(k)
    fp8kv.fp8kv_cache_insert(zero, zero, torch.where(old, -1, slots), ks, vs, kc2, vc2)     # new rows wiped
    shape = (len(lens), M, H, 128)
    out = fp8kv.fp8kv_append_paged_attention(k[new].view(shape), v[new].view(shape), q, kc2, vc2,
                                             lay.block_table.cuda(), lay.seq_lens.cuda(), max(lens), ks, vs, SM,
                                             window_left=window)
    assert torch.equal(kc2, kc) and torch.equal(vc2, vc)
    assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,M,G,H,ps,window,split", [
    ([130, 257, 12, 640], 12, 9, 2, 32, -1, 128), ([130, 128, 1], 1, 9, 3, 32, -1, 128), ([518], 16, 1, 2, 64, -1, 128),
    ([4100], 12, 9, 1, 64, -1, 1024), ([300, 261], 8, 16, 2, 64, 100, 128), ([1030], 16, 8, 2, 32, 40, 256),
    ([513, 100], 16, 9, 2, 64, -1, 128), ([40, 700], 3, 9, 1, 32, -1, 0)])
def test_appended_tokens_on_either_side_of_a_partition(lens, M, G, H, ps, window, split):
    """New tokens that begin in one partition and end in the next, several times
    over, with other bytes in their rows before each call."""
    lay, q, kc, vc, ks, vs, k, v, slots = _case(11 * sum(lens), lens, M, G, H, ps)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    want = _attend(lay, q, kc, vc, ks, vs, window, split_tokens=split)
    _check(want, lay, q, kc, vc, ks, vs, ps, window)
    new = torch.cat([torch.arange(sum(lens[:b + 1]) - M, sum(lens[:b + 1])) for b in range(len(lens))]).cuda()
    old = torch.ones(len(slots), dtype=torch.bool, device="cuda")
    old[new] = False
    other = torch.full_like(k, float("nan"))
    kc2, vc2 = kc.clone(), vc.clone()
    shape = (len(lens), M, H, 128)
    call = fp8kv.PreparedAttention(q, kc2, vc2, lay.block_table.cuda(), lay.seq_lens.cuda(), max(lens), ks, vs, SM,
                                   window_left=window, split_tokens=split, k_new=k[new].view(shape).contiguous(),
                                   v_new=v[new].view(shape).contiguous())
    for _ in range(20):
        fp8kv.fp8kv_cache_insert(other, other, torch.where(old, -1, slots), ks, vs, kc2, vc2)
        out = call()
        assert torch.equal(kc2, kc) and torch.equal(vc2, vc)
        assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [-1, 200])
@pytest.mark.parametrize("L", [12, 128, 129, 700, 1000, 1001, 5])
def test_one_sequence_shorter_than_its_partitions(L, window):
    """Eight partitions that combine in a cluster, of which the sequence fills
    some; lengths that are refused leave the output as it was."""
    lay, q, kc, vc, ks, vs, k, v, slots = _case(L, [1100], 12, 9, 2, 32)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    lay = gen.PagedLayout(32, lay.num_pages, lay.block_table, torch.tensor([L], dtype=torch.int32))
    out = torch.full_like(q, 3.0)
    fp8kv.fp8kv_device_status(clear=True)
    fp8kv.fp8kv_paged_attention(q, kc, vc, lay.block_table.cuda(), lay.seq_lens.cuda(), 1000, ks, vs, SM, out=out,
                                window_left=window, split_tokens=128)
    text = fp8kv.fp8kv_last_dispatch()
    # the 212 keys that 12 rows see through the window touch at most ceil(212 / 32) + 1 = 8 pages, two partitions
    assert ("cluster=8" if window < 0 else "cluster=2") in text and "reduce=0" in text
    if 12 <= L <= 1000:
        _check(out, lay, q, kc, vc, ks, vs, 32, window)
        assert fp8kv.fp8kv_device_status(clear=True) == 0
    else:
        assert bool((out == 3.0).all()) and fp8kv.fp8kv_device_status(clear=True) != 0


@pytest.mark.gpu
@pytest.mark.parametrize("lens,M,G,H,ps,window,want", [
    ([2000, 30, 1, 900], 1, 9, 2, 32, -1, "cluster"), ([400, 700], 2, 8, 3, 64, -1, "cluster"),
    ([3000, 12, 500], 12, 9, 2, 64, -1, "cluster"), ([3000, 2500], 1, 4, 4, 32, 1500, "cluster"),
    ([5000], 1, 12, 1, 64, -1, "cluster"), ([2500, 12] + [300] * 18, 12, 9, 8, 32, -1, "longest_first"),
    ([2000, 12] + [300] * 18, 12, 9, 8, 32, -1, "splits=1 "),
    ([100] * 39 + [500], 1, 9, 8, 32, -1, "threads=128"), ([6000] + [40] * 31, 1, 5, 8, 64, -1, "longest_first")])
def test_automatic_partitions(lens, M, G, H, ps, window, want):
    """Calls that are cut in the different ways: clusters of partitions some of
    which are empty, one partition longest first, small CTAs.  A sequence whose
    length is refused keeps its output rows and leaves the others' alone."""
    lay, q, kc, vc, ks, vs, k, v, slots = _case(sum(lens), lens, M, G, H, ps)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    out = _attend(lay, q, kc, vc, ks, vs, window)
    assert want in fp8kv.fp8kv_last_dispatch()
    _check(out, lay, q, kc, vc, ks, vs, ps, window)
    fp8kv.fp8kv_device_status(clear=True)
    sl = lay.seq_lens.clone()
    sl[-1] = M - 1
    again = torch.full_like(q, 3.0)
    fp8kv.fp8kv_paged_attention(q, kc, vc, lay.block_table.cuda(), sl.cuda(), max(lens), ks, vs, SM, out=again,
                                window_left=window)
    assert fp8kv.fp8kv_device_status(clear=True) != 0
    assert torch.equal(again[:-1], out[:-1]) and bool((again[-1] == 3.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 12])
def test_append_to_pages_outside_the_pool(M):
    """Flagged; those tokens are written nowhere, and their keys read as zeros."""
    lay, q, kc, vc, ks, vs, k, v, slots = _case(3 + M, [70, 40], M, 9, 2, 32, extra=2)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    before = kc.clone(), vc.clone()
    bt = lay.block_table.clone()
    bt[0, 2], bt[1, 1] = lay.num_pages, -1
    new = torch.full((2, M, 2, 128), 100.0, dtype=torch.bfloat16, device="cuda")
    fp8kv.fp8kv_device_status(clear=True)
    out = fp8kv.fp8kv_append_paged_attention(new, new, q, kc, vc, bt.cuda(), lay.seq_lens.cuda(), 70, ks, vs, SM)
    assert fp8kv.fp8kv_device_status(clear=True) != 0
    changed = [(a != b).any(-1).any(-1).nonzero()[:, 0].tolist() for a, b in zip((kc, vc), before)]
    # M = 12: tokens 58 .. 63 and 28 .. 31 still lie in good pages
    good = sorted(int(lay.block_table[b, p]) for b, p in ((0, 1), (1, 0))) if M == 12 else []
    assert changed == [good, good]
    zero = gen.PagedLayout(32, lay.num_pages + 1, torch.where((bt < 0) | (bt >= lay.num_pages), lay.num_pages, bt),
                           lay.seq_lens)
    pad = [torch.cat([c, torch.zeros_like(c[:1])]) for c in (kc, vc)]
    _check(out, zero, q, pad[0], pad[1], ks, vs, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 12])
def test_extreme_scales_logits_and_values(M):
    """Block scales up to 448 (a tensor scale far below the calibrated one) and
    at the smallest step, queries of very different sizes, one dominant key."""
    lay, q, kc, vc, ks, vs, k, v, slots = _case(91 + M, [700], M, 9, 2, 32)
    k[::7] *= 100
    k[3::7] *= 1e-4
    k[123] *= 5
    v[::5] *= 300
    q[:, :, ::2] *= 2.0 ** -30
    q[:, :, 5] = 0
    ks, vs = _scale(2e-2), _scale(1e-2)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    assert int(kc[:, :, 32 * 64:].max()) >= 0x70
    out = _attend(lay, q, kc, vc, ks, vs)
    _check(out, lay, q, kc, vc, ks, vs, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 12])
@pytest.mark.parametrize("sm", [-0.3, 0.0])
def test_negative_and_zero_softmax_scale(M, sm):
    lay, q, kc, vc, ks, vs, k, v, slots = _case(43, [400, 20], M, 9, 2, 32)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    bt, sl = lay.block_table.cuda(), lay.seq_lens.cuda()
    out = fp8kv.fp8kv_paged_attention(q, kc, vc, bt, sl, 400, ks, vs, sm)
    neg = fp8kv.fp8kv_paged_attention(-q if sm else torch.zeros_like(q), kc, vc, bt, sl, 400, ks, vs, abs(sm) or 1.0)
    assert torch.equal(out, neg) if sm else bool((out.float() - neg.float()).abs().max() < 2.0 ** -8)


@pytest.mark.gpu
@pytest.mark.parametrize("M,split", [(1, 0), (1, 128), (12, 0), (12, 128)])
def test_bad_pages_read_zeros_and_bad_lengths_leave_the_output(M, split):
    fp8kv.fp8kv_device_status(clear=True)
    lens = [200, 90, 150]
    lay, q, kc, vc, ks, vs, k, v, slots = _case(17, lens, M, 9, 2, 32)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    lay.block_table[0, 2] = lay.num_pages + 5
    lay.block_table[0, 3] = -3
    out = _attend(lay, q, kc, vc, ks, vs, split_tokens=split)
    _check(out, lay, q, kc, vc, ks, vs, 32)
    assert fp8kv.fp8kv_device_status(clear=True) == 0
    sl = lay.seq_lens.cuda()
    sl[1] = M - 1                                       # fewer keys than rows
    sl[2] = 201                                         # above max_seq_len
    out2 = torch.full_like(q, 3.0)
    fp8kv.fp8kv_paged_attention(q, kc, vc, lay.block_table.cuda(), sl, 200, ks, vs, SM, split_tokens=split, out=out2)
    assert fp8kv.fp8kv_device_status(clear=True) == fp8kv.DEV_BAD_SEQ_LEN
    assert torch.equal(out2[0], out[0]) and bool((out2[1:] == 3.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 12])
def test_noalloc_prepared_and_captured_calls(M):
    lay, q, kc, vc, ks, vs, k, v, slots = _case(29, [1500, 800], M, 9, 2, 32)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    bt, sl = lay.block_table.cuda(), lay.seq_lens.cuda()
    want = _attend(lay, q, kc, vc, ks, vs)
    out = torch.empty_like(q)
    fp8kv.fp8kv_paged_attention_noalloc(q, kc, vc, bt, sl, 1500, ks, vs, SM, out)
    assert torch.equal(out, want)
    # two prepared calls captured into one graph, on two side streams, each
    # with its own workspace; replayed with other queries in place
    calls = [fp8kv.PreparedAttention(q, kc, vc, bt, sl, 1500, ks, vs, SM) for _ in range(2)]
    side = [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for c, s in zip(calls, side):
            s.wait_stream(main)
            with torch.cuda.stream(s):
                c()
            main.wait_stream(s)
    q.copy_(q.flip(0))
    want = _attend(lay, q, kc, vc, ks, vs)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(c.out, want) for c in calls)


@pytest.mark.gpu
def test_binding_refuses_what_the_library_cannot_see():
    lay, q, kc, vc, ks, vs, k, v, slots = _case(37, [100, 50], 1, 9, 2, 32)
    bt, sl = lay.block_table.cuda(), lay.seq_lens.cuda()
    good = dict(q=q, k_cache=kc, v_cache=vc, block_table=bt, seq_lens=sl, max_seq_len=100, k_scale=ks, v_scale=vs,
                sm_scale=SM)
    for over in ({"k_scale": ks.cpu()}, {"v_scale": vs.double()}, {"k_scale": ks.repeat(2)}, {"seq_lens": sl[:1]},
                 {"block_table": bt[:1]}, {"out": torch.empty_like(q)[:1]}, {"out": torch.empty_like(q).float()},
                 {"num_pages": kc.shape[0] + 1}, {"v_cache": vc[:1]}, {"q": q.float()}):
        with pytest.raises(ValueError):
            fp8kv.fp8kv_paged_attention(**{**good, **over})
        with pytest.raises(ValueError):
            fp8kv.PreparedAttention(**{**good, **over})
    for bad in ((k[:, :1], v[:, :1], slots), (k, v[:5], slots), (k, v, slots[:5])):
        with pytest.raises(ValueError):
            fp8kv.fp8kv_cache_insert(bad[0].contiguous(), bad[1].contiguous(), bad[2], ks, vs, kc, vc)
    with pytest.raises(ValueError):
        fp8kv.fp8kv_cache_gather(slots, ks, vs, kc, vc, k_out=k[:3])
    with pytest.raises(fp8kv.Fp8kvError):                       # 17 rows per sequence
        fp8kv.fp8kv_paged_attention(**{**good, "q": q.repeat(1, 17, 1, 1)})


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 12])
def test_pages_beyond_four_gigabytes(M):
    """A pool of more than 2^32 bytes; the sequence's pages at both ends of it."""
    ps, H, G = 64, 8, 9
    pages = 2 ** 32 // (H * ps * 72) + 64
    kc = torch.empty((pages, H, ps * 72), dtype=torch.uint8, device="cuda")
    vc = torch.empty_like(kc)
    ids = torch.tensor([[pages - 1, 0, pages - 3, 1]], dtype=torch.int32)
    for i in ids[0].tolist():
        kc[i], vc[i] = 0x7F, 0x7F
    g = torch.Generator(device="cuda").manual_seed(M)
    L = 250
    k, v = (torch.randn((L, H, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((1, M, G * H, 128), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(L)
    slots = (ids[0].long()[pos // ps] * ps + pos % ps).cuda()
    ks, vs = _scale(6 / 448), _scale(5 / 448)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    ko, vo = fp8kv.fp8kv_cache_gather(slots, ks, vs, kc, vc)
    n, sc = int4_np.encode_rows(k.float().cpu().numpy(), ks.item())
    want = torch.from_numpy(n * np.repeat(int4_np.e4m3_value(sc), 16, -1)).float() * ks.cpu()
    assert torch.equal(ko.cpu(), want.to(torch.bfloat16))
    sl = torch.tensor([L], dtype=torch.int32, device="cuda")
    out = fp8kv.fp8kv_paged_attention(q, kc, vc, ids.cuda(), sl, L, ks, vs, SM)
    small = gen.PagedLayout(ps, 4, torch.arange(4, dtype=torch.int32)[None], sl.cpu())
    _check(out, small, q, kc[ids[0].long().cuda()], vc[ids[0].long().cuda()], ks, vs, ps)


@pytest.mark.gpu
def test_page_order_does_not_matter():
    lay, q, kc, vc, ks, vs, k, v, slots = _case(31, [900], 12, 9, 2, 32)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    want = _attend(lay, q, kc, vc, ks, vs)
    perm = torch.randperm(lay.num_pages)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(lay.num_pages)
    lay.block_table = inv[lay.block_table.long()].to(torch.int32)
    assert torch.equal(_attend(lay, q, kc[perm.cuda()], vc[perm.cuda()], ks, vs), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [fp8kv.FP8KV_CACHE_E4M3, fp8kv.FP8KV_CACHE_BF16, fp8kv.FP8KV_CACHE_INT4])
@pytest.mark.parametrize("T,H", [(1200, 16), (4999, 5)])
def test_gather_of_few_and_many_rows(dt, T, H):
    """Either side of the number of rows above which a thread takes 16 elements:
    the rows of a slot are the same wherever and however they are read."""
    ps, ks, vs = 64, _scale(0.02), _scale(0.03)
    pages = T // ps + 2
    if dt == fp8kv.FP8KV_CACHE_INT4:
        kc, vc = (fp8kv.fp8kv_int4_cache(pages, H, ps) for _ in range(2))
    else:
        kc, vc = (torch.zeros((pages, H, ps, 128), device="cuda",
                              dtype=torch.uint8 if dt == fp8kv.FP8KV_CACHE_E4M3 else torch.bfloat16) for _ in range(2))
    g = gen.generator(T)
    k, v = (torch.randn((T, H, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    slots = torch.randperm(pages * ps, generator=g)[:T].cuda()
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    ko, vo = fp8kv.fp8kv_cache_gather(slots, ks, vs, kc, vc)
    some = torch.randperm(T, generator=g)[:100].cuda()
    k1, v1 = fp8kv.fp8kv_cache_gather(slots[some], ks, vs, kc, vc)
    assert torch.equal(ko[some], k1) and torch.equal(vo[some], v1)
    if dt == fp8kv.FP8KV_CACHE_BF16:
        assert torch.equal(ko, k) and torch.equal(vo, v)
    elif dt == fp8kv.FP8KV_CACHE_INT4:
        n, sc = int4_np.encode_rows(v.float().cpu().numpy(), vs.item())
        want = torch.from_numpy(n * np.repeat(int4_np.e4m3_value(sc), 16, -1)).float() * vs.cpu()
        assert torch.equal(vo.cpu(), want.to(torch.bfloat16))
    else:
        # E4M3: half a step, 2^-4 of the value or 2^-10 scale units; then fp32 and bf16 roundings, under 2^-7 of it
        err = (vo.float() - v.float()).abs()
        assert bool((err <= v.float().abs() * (2.0 ** -4 + 2.0 ** -7) + 0.03 * 2.0 ** -10).all())


@pytest.mark.gpu
def test_calls_on_several_streams_at_once():
    """Decode, verifier rows in a cluster and through partials, insert and gather
    on streams of their own, each over its own cache, repeated."""
    work = []
    for seed, lens, M, split in ((1, [2000, 300], 1, 0), (2, [900], 12, 0), (3, [3000, 40], 12, 256), (4, [5000], 1, 512)):
        lay, q, kc, vc, ks, vs, k, v, slots = _case(seed, lens, M, 9, 4, 32)
        fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
        call = fp8kv.PreparedAttention(q, kc, vc, lay.block_table.cuda(), lay.seq_lens.cuda(), max(lens), ks, vs, SM,
                                       split_tokens=split)
        rows = fp8kv.fp8kv_cache_gather(slots, ks, vs, kc, vc)
        work.append((call, call().clone(), (slots, ks, vs, kc, vc), rows, (k, v, slots, ks, vs, kc, vc),
                     [torch.empty_like(r) for r in rows], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(30):
        for call, _, g, _, ins, got, stream in work:
            with torch.cuda.stream(stream):
                fp8kv.fp8kv_cache_insert(*ins)
                call()
                fp8kv.fp8kv_cache_gather(*g, *got)
    torch.cuda.synchronize()
    for call, want, _, rows, _, got, _ in work:
        assert torch.equal(call.out, want)
        assert torch.equal(got[0], rows[0]) and torch.equal(got[1], rows[1])
    assert fp8kv.fp8kv_device_status(clear=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("ps", [32, 64])
def test_tiles_of_bad_pages_between_good_ones(ps):
    """Whole key tiles, single pages and runs of them outside the pool, each slot
    of the staging ring used several times with either, called again and again:
    zeros where a page is bad, over what the slot held before and before what it
    holds next."""
    L, M = 40 * 128, 12
    lay, q, kc, vc, ks, vs, k, v, slots = _case(ps, [L], M, 9, 1, ps, extra=3)
    fp8kv.fp8kv_cache_insert(k * 8, v * 8, slots, ks, vs, kc, vc)
    per = 128 // ps
    rng = np.random.default_rng(ps)
    bad = np.repeat(rng.integers(0, 3, 40) == 0, per)           # a third of the tiles, whole
    bad |= rng.integers(0, 8, 40 * per) == 0                    # and pages anywhere
    bad[-per:] = False
    outside = torch.from_numpy(np.where(rng.integers(0, 2, len(bad)), -1 - rng.integers(0, 9, len(bad)),
                                        lay.num_pages + rng.integers(0, 9, len(bad))).astype(np.int32))
    lay.block_table[0, :len(bad)] = torch.where(torch.from_numpy(bad), outside, lay.block_table[0, :len(bad)])
    out = _attend(lay, q, kc, vc, ks, vs, split_tokens=L)
    assert "attention_int4_tc" in fp8kv.fp8kv_last_dispatch() and "splits=1 " in fp8kv.fp8kv_last_dispatch()
    bt = lay.block_table
    zero = gen.PagedLayout(ps, lay.num_pages + 1, torch.where((bt < 0) | (bt >= lay.num_pages), lay.num_pages, bt),
                           lay.seq_lens)
    pad = [torch.cat([c, torch.zeros_like(c[:1])]) for c in (kc, vc)]
    _check(out, zero, q, pad[0], pad[1], ks, vs, ps)
    for _ in range(30):
        assert torch.equal(_attend(lay, q, kc, vc, ks, vs, split_tokens=L), out)


# ---------------------------------- GPU: every way of combining partitions

def _check_route(out, text, lay, q, kc, vc, ks, vs, ps, window=-1):
    """_check with the rounding of the partitions' partial outputs taken from the
    route that the call reports, in place of the row count; NaN where the
    definition has it, and nowhere else."""
    ref, mag, lmag, vsum = int4_np.paged_attention(q.double().cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy(), ps,
                                                   lay.block_table.numpy(), lay.seq_lens.numpy(), ks.item(), vs.item(),
                                                   SM, window)
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    # The terms of _check, and: partials through the reduce kernel, and those of
    # the tcgen05 kernel's clusters, are f16 of the partition's mean of n s: off
    # by 2^-11 of it, which the partitions' weights (their sum is 1) turn into
    # 2^-11 of mag at most, or below f16's normal range by 2^-25, v_scale times
    # that in the output.  Clusters of the decode kernel exchange fp32.
    f16 = "reduce=1" in text or ("int4_tc" in text and "cluster=1 " not in text)
    tol = (2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + f16 * 2.0 ** -11) * mag + 2.0 ** -20 * lmag + 2.0 ** -36 * vsum
           + f16 * 2.0 ** -25 * vs.item())
    ok = np.isnan(ref) | (np.abs(got - ref) <= tol)
    assert ok.all(), float(np.nanmax(np.abs(got - ref) / tol))


ROUTES = [
    # lens, M, split_tokens, what the call reports (G = 9, H = 2, pages of 32)
    ([257], 1, 512, "splits=1 "), ([257], 12, 512, "splits=1 "),
    ([257], 1, 128, "cluster=3 "), ([257], 12, 128, "cluster=3 "),
    ([1025], 1, 128, "reduce=1"), ([1025], 12, 128, "reduce=1"),           # 9 partitions: the reduce kernel's short form
    ([2561], 1, 128, "reduce=1"), ([2561], 12, 128, "reduce=1"),           # 21: its long one
    ([2561, 130, 1665, 13], 2, 128, "reduce=1"), ([2561, 130, 1665, 13], 12, 128, "reduce=1"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,M,split,route", ROUTES)
def test_every_route_against_the_definition(lens, M, split, route):
    lay, q, kc, vc, ks, vs, k, v, slots = _case(5 * sum(lens) + M, lens, M, 9, 2, 32)
    v[::3] *= 2.0 ** -12                                        # small values beside large ones
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    out = _attend(lay, q, kc, vc, ks, vs, split_tokens=split)
    text = fp8kv.fp8kv_last_dispatch()
    assert route in text and ("int4_tc" in text) == (M * 9 > 16)
    _check_route(out, text, lay, q, kc, vc, ks, vs, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["last", "partition", "first"])
@pytest.mark.parametrize("lens,M,split,route", ROUTES)
def test_a_nan_key_is_seen_however_the_keys_are_cut(lens, M, split, route, where):
    """The newest token alone in the last partition, a whole partition, or the
    oldest token, with a NaN in K of head 0: the rows that see it are NaN, the
    others (earlier rows, the other head) as they were."""
    lay, q, kc, vc, ks, vs, k, v, slots = _case(9 * sum(lens) + M, lens, M, 9, 2, 32)
    at = 0
    for n in lens:
        lo, hi = {"last": (n - 1, n), "partition": (128, min(256, n)), "first": (0, 1)}[where]
        k[at + lo:at + hi, 0, 77] = float("nan")
        at += n
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    out = _attend(lay, q, kc, vc, ks, vs, split_tokens=split)
    text = fp8kv.fp8kv_last_dispatch()
    assert route in text
    assert bool(out[0, -1, 0].isnan().all()) and not bool(out[..., 9:, :].isnan().any())
    _check_route(out, text, lay, q, kc, vc, ks, vs, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["e4m3", "int4"])
def test_gather_refuses_scales_per_head(cache):
    """It reads caches with one scale per tensor: a scale for each head would be
    read as its first head's."""
    kc, vc = (fp8kv.fp8kv_int4_cache(2, 4, 32) if cache == "int4" else
              torch.zeros((2, 4, 32, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.arange(10, device="cuda")
    one, heads = _scale(0.5), torch.full((4,), 0.5, device="cuda")
    fp8kv.fp8kv_cache_gather(slots, one, one, kc, vc)
    for ks, vs in ((heads, one), (one, heads), (heads, heads), (one, one[:0])):
        with pytest.raises(ValueError):
            fp8kv.fp8kv_cache_gather(slots, ks, vs, kc, vc)


@pytest.mark.parametrize("c", [1.0, 0.0123, 37.0, 2.0 ** -100, 2.0 ** 100])
def test_error_of_a_stored_value_over_all_block_scales(c):
    """Blocks whose largest element is anything from far below the smallest block
    scale to the largest: constant ones just below every border between two
    scales, where the rounding of s costs most, and random ones."""
    c32 = float(np.float32(c))
    s = int4_np.e4m3_value(np.arange(127))[1:]                  # 2^-9 .. 448
    border = (s[:-1] + s[1:]) / 2
    rng = np.random.default_rng(11)
    amax = np.concatenate([7 * c32 * border * 0.999, 7 * c32 * border * 1.001, 7 * c32 * s,
                           7 * c32 * 2.0 ** rng.uniform(-14, np.log2(448), 2000)])
    x = amax[:, None] * np.where(np.arange(16) % 2, rng.uniform(-1, 1, (len(amax), 16)), 1.0)
    # bf16 rounded towards zero: above 448 * 7 c the value would saturate
    bits = np.asarray(x, np.float32).view(np.uint32) & np.uint32(0xffff0000)
    x = bits.view(np.float32).reshape(-1, 1, 16).repeat(8, 1).reshape(-1, 1, 128)
    n, sc = int4_np.encode_rows(x, c)
    assert sc.min() == 1 and sc.max() == 0x7e
    step = np.repeat(int4_np.e4m3_value(sc), 16, -1) * c32
    err = np.abs(x.astype(np.float64) - n * step)
    # r = amax / (7 c).  s rounded down: r - s <= 2^-10 where s is subnormal (and
    # s >= 2^-9 > r - 2^-10 below), 2^-4 s where it is normal, so clamping at 7 s c
    # costs at most 7 * 2^-10 c or 7/16 of a step; rounding n costs half a step.
    # r, s c and the reciprocal are fp32, each off by at most 2^-23 of itself, and
    # r is at most 1.5 s: 7 * 1.5 * 3 * 2^-23 < 2^-18 of a step.
    bound = np.where(step >= 7 * 2.0 ** -9 * c32, step / 2, np.maximum(step / 2, 7 * 2.0 ** -10 * c32))
    assert np.all(err <= bound + 2.0 ** -18 * step)
    # the second bound is needed: at s = 2^-9 more than three steps are reached
    low = np.repeat(sc, 16, -1) == 1
    assert err[low].max() > 3.3 * 2.0 ** -9 * c32


@pytest.mark.gpu
@pytest.mark.parametrize("M,split", [(1, 0), (1, 128), (12, 0), (12, 128)])
def test_a_nan_value_stays_with_its_head_and_sequence(M, split):
    lay, q, kc, vc, ks, vs, k, v, slots = _case(71, [300, 257], M, 9, 2, 32)
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    want = _attend(lay, q, kc, vc, ks, vs, split_tokens=split)
    v[-1, 1, 5] = float("nan")                                  # the newest token of the second sequence
    fp8kv.fp8kv_cache_insert(k, v, slots, ks, vs, kc, vc)
    out = _attend(lay, q, kc, vc, ks, vs, split_tokens=split)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1, :, :9], want[1, :, :9])
    # the whole block of 16 elements of the row that sees it
    assert bool(out[1, -1, 9:, :16].isnan().all()) and not bool(out[1, :, 9:, 16:].isnan().any())

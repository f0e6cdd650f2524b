"""A step over trees of drafted tokens: argument checks (CPU), and metadata, rotary
insert, attention, verification and the kept path on the GPU against float64."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import draft_tree_np as tree_np, int4_np
from verify_attention_gb300 import build, fp8kv

NULL = ctypes.c_void_p(0)
P16 = ctypes.c_void_p(1 << 20)          # fake, 16-byte aligned: never dereferenced
Q16 = ctypes.c_void_p(1 << 24)
SM = 128 ** -0.5
CACHES = ("e4m3", "bf16", "int4")


@pytest.fixture(scope="module")
def L():
    build.build()
    return fp8kv.lib()


# ------------------------------------------------------- argument checks

def _refusals(fn, args, cases):
    """fn(**args) with each override refused (or accepted) with its status."""
    for over, want in cases:
        unknown = set(over) - set(args)
        assert not unknown, unknown
        assert fn(*{**args, **over}.values()) == want, over


def test_metadata_checks_its_arguments(L):
    args = dict(par=P16, sl=P16, bt=P16, mpps=4, maxL=100, B=2, M=12, P=16, ps=32, mask=P16, pos=P16, slot=P16, s=NULL)
    _refusals(L.fp8kv_tree_metadata, args, [
        ({"par": NULL}, 1), ({"sl": NULL}, 1), ({"bt": NULL}, 1), ({"mask": NULL}, 1), ({"pos": NULL}, 1),
        ({"slot": NULL}, 1), ({"B": -1}, 1), ({"M": 0}, 1), ({"M": 65}, 2), ({"ps": 16}, 2), ({"P": 0}, 1),
        ({"maxL": 11}, 1), ({"maxL": 129}, 1), ({"mpps": 0}, 1), ({"B": 0, "par": NULL}, 0)])


def test_rope_insert_checks_its_arguments(L):
    args = dict(q=P16, qs=9216, k=P16, ks_=1024, v=P16, vs_=1024, pos=P16, cs=P16, maxp=64, rot=128, il=0, qo=Q16,
                slot=P16, T=4, Hq=72, Hkv=8, D=128, ks=P16, vs=P16, kc=P16, vc=P16, P=16, ps=32, dt=0, s=NULL)
    odd = ctypes.c_void_p((1 << 20) + 8)
    _refusals(L.fp8kv_rope_insert, args, [
        ({"q": NULL}, 1), ({"k": NULL}, 1), ({"v": NULL}, 1), ({"pos": NULL}, 1), ({"cs": NULL}, 1), ({"qo": NULL}, 1),
        ({"slot": NULL}, 1), ({"kc": NULL}, 1), ({"vc": NULL}, 1), ({"ks": NULL}, 1), ({"vs": NULL, "dt": 2}, 1),
        ({"qo": P16}, 1), ({"qo": ctypes.c_void_p((1 << 20) + 4 * 18432 - 16)}, 1),
        ({"k": ctypes.c_void_p((1 << 24) + 4 * 18432 - 16)}, 1), ({"v": ctypes.c_void_p((1 << 24) - 4 * 2048 + 16)}, 1),
        ({"q": odd}, 1), ({"cs": odd}, 1), ({"kc": odd}, 1), ({"qs": 9208}, 1), ({"qs": 9220}, 1),
        ({"ks_": 1016}, 1), ({"vs_": 1028}, 1), ({"rot": 0}, 1), ({"rot": 136}, 1), ({"rot": 63}, 1), ({"rot": 12}, 2),
        ({"D": 64, "rot": 64}, 2), ({"ps": 48}, 2), ({"dt": 3}, 1), ({"T": -1}, 1), ({"maxp": 0}, 1), ({"Hq": 0}, 1),
        ({"T": 0, "q": NULL}, 0)])


def test_tree_attention_checks_its_arguments(L):
    args = dict(kn=NULL, vn=NULL, q=P16, k=P16, v=P16, dt=0, bt=P16, mpps=4, sl=P16, maxL=100, mask=P16, B=1, M=12,
                Hq=72, Hkv=8, D=128, ps=32, P=16, ks=P16, vs=P16, sm=0.088, wl=-1, split=0, ws=P16, wsb=1 << 30,
                out=Q16, s=NULL)
    _refusals(L.fp8kv_tree_attention, args, [
        ({"out": P16}, 1), ({"out": ctypes.c_void_p((1 << 20) + 12 * 18432 - 16)}, 1),
        ({"mask": NULL}, 1), ({"q": NULL}, 1), ({"out": NULL}, 1), ({"M": 65, "maxL": 128}, 2), ({"M": 0}, 1),
        ({"D": 64}, 2), ({"ps": 16}, 2), ({"wl": -2}, 1), ({"Hq": 70}, 1), ({"kn": P16}, 1), ({"ks": NULL}, 1),
        ({"split": 96}, 2), ({"split": 64, "dt": 1}, 2), ({"split": 32, "dt": 2}, 2), ({"dt": 5}, 1),
        ({"maxL": 11}, 1), ({"B": 0, "q": NULL}, 0), ({"sm": float("nan")}, 1)])
    # the shapes that plain calls refuse on these caches are a tree's
    assert L.fp8kv_tree_attention(*{**args, "dt": 2, "M": 64, "ws": NULL, "maxL": 16384, "mpps": 512, "B": 1}.values()) == 3
    assert L.fp8kv_tree_attention(*{**args, "dt": 1, "M": 64, "ws": NULL, "maxL": 16384, "mpps": 512, "B": 1}.values()) == 3


def test_verify_checks_its_arguments(L):
    args = dict(p=P16, ps=1000, q=P16, qs=1000, dt=0, tok=P16, par=P16, u=P16, B=2, M=12, V=1000, out=P16, num=P16,
                path=P16, s=NULL)
    _refusals(L.fp8kv_verify_tree, args, [
        ({"p": NULL}, 1), ({"tok": NULL}, 1), ({"par": NULL}, 1), ({"u": NULL}, 1), ({"out": NULL}, 1),
        ({"num": NULL}, 1), ({"path": NULL}, 1), ({"ps": 999}, 1), ({"qs": 999}, 1), ({"dt": 2}, 1), ({"M": 0}, 1),
        ({"M": 65}, 2), ({"V": 0}, 1), ({"B": -1}, 1), ({"p": ctypes.c_void_p((1 << 20) + 2)}, 1),
        ({"B": 0, "p": NULL}, 0)])


def test_outputs_that_overlap_are_refused(L):
    """Whole or by their last bytes; addresses a MiB apart otherwise."""
    at = lambda i, back=0: ctypes.c_void_p((i << 20) - back)  # noqa: E731
    B, M, V = 2, 12, 1000
    meta = dict(par=at(1), sl=at(2), bt=at(3), mpps=4, maxL=100, B=B, M=M, P=16, ps=32, mask=at(4), pos=at(5),
                slot=at(6), s=NULL)
    over = [{n: at(i, d)} for n, own in (("mask", 4), ("pos", 5), ("slot", 6)) for i, size in
            ((1, 96), (2, 8), (3, 32), (4, 192), (5, 192), (6, 192)) if i != own for d in (0, 184, 4 - size)]
    _refusals(L.fp8kv_tree_metadata, meta, [(o, 1) for o in over])
    ver = dict(p=at(1), ps=V, q=at(2), qs=V, dt=0, tok=at(3), par=at(4), u=at(5), B=B, M=M, V=V, out=at(6), num=at(7),
               path=at(8), s=NULL)
    rows, whole = 4 * B * M, 4 * B * M * V
    _refusals(L.fp8kv_verify_tree, ver, [
        *(({n: at(i, d)}, 1) for n in ("out", "path") for i in (1, 2) for d in (0, rows - 4, 4 - whole)),
        *(({n: at(i, d)}, 1) for n in ("out", "path") for i in (3, 4, 5) for d in (rows - 4, 4, -4, 4 - rows)),
        *(({"num": at(i, d)}, 1) for i in (1, 2, 3, 4, 5, 6, 8) for d in (0, 4, -4)),
        ({"out": at(8)}, 1), ({"path": at(6, 4)}, 1), ({"path": at(7)}, 1), ({"out": at(7, rows - 4)}, 1),
        ({"q": NULL, "out": at(1, 4)}, 1), ({"dt": 1, "out": at(1, 4 - whole // 2)}, 1)])
    att = dict(kn=at(1), vn=at(2), q=at(3), k=at(16), v=at(17), dt=0, bt=at(18), mpps=4, sl=at(19), maxL=100, mask=at(20),
               B=1, M=M, Hq=72, Hkv=8, D=128, ps=32, P=16, ks=at(21), vs=at(22), sm=0.088, wl=-1, split=0, ws=at(23),
               wsb=1 << 30, out=at(30), s=NULL)
    out = M * 72 * 256
    _refusals(L.fp8kv_tree_attention, att, [({"out": at(i, d)}, 1) for i in (1, 2, 3, 20) for d in (0, out - 16, -16)])


def test_keep_path_checks_its_arguments(L):
    two = (ctypes.c_void_p * 2)(1 << 20, 1 << 21)
    odd = (ctypes.c_void_p * 2)(1 << 20, (1 << 21) + 8)
    none = (ctypes.c_void_p * 2)(1 << 20, None)
    other = (ctypes.c_void_p * 2)(1 << 22, 1 << 23)
    half = (ctypes.c_void_p * 2)(1 << 22, (1 << 22) + 16 * 8 * 32 * 128 - 16)
    args = dict(k=two, v=other, n=2, dt=0, bt=P16, mpps=4, sl=P16, maxL=100, path=P16, B=2, M=12, Hkv=8, D=128, P=16,
                ps=32, new=Q16, s=NULL)
    _refusals(L.fp8kv_cache_keep_path, args, [
        ({"k": NULL}, 1), ({"v": none}, 1), ({"v": odd}, 1), ({"v": two}, 1), ({"v": half}, 1), ({"bt": NULL}, 1), ({"sl": NULL}, 1), ({"path": NULL}, 1),
        ({"new": NULL}, 1), ({"new": P16}, 1), ({"new": ctypes.c_void_p((1 << 20) + 4)}, 1), ({"n": 0}, 1),
        ({"n": 65}, 2), ({"M": 65, "maxL": 128}, 2), ({"dt": 9}, 1), ({"D": 64}, 2), ({"ps": 16}, 2), ({"maxL": 11}, 1),
        ({"Hkv": 0}, 1), ({"B": 0, "k": NULL}, 0)])


def test_binding_refuses_what_the_library_cannot_see():
    t = torch.zeros
    with pytest.raises(ValueError):
        fp8kv.fp8kv_tree_metadata(t(2, 4, dtype=torch.int32), t(2, dtype=torch.int32), t(2, 4, dtype=torch.int32), 32, 64, 8)
    with pytest.raises(ValueError):
        fp8kv.fp8kv_verify_tree(t(2, 4, 10), None, t(2, 4, dtype=torch.int32), t(2, 4, dtype=torch.int32), t(2, 4))
    with pytest.raises(ValueError):
        fp8kv.PreparedKeepPath([], [], t(2, 4), t(2), t(2, 4), 64)
    with pytest.raises(ValueError):
        fp8kv._tree_rows(t(2, 4), "path", torch.int32, 2, 4)


class _Shapes:
    """CUDA tensors without memory, their pointers null: what the binding lets through,
    the library refuses (Fp8kvError) before anything could be launched."""

    def __init__(self, kind, D=128, row=128, heads=2, v_heads=2, v_ps=32):
        z = lambda *shape, t=torch.bfloat16: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
        i32, i64, f32 = torch.int32, torch.int64, torch.float32
        T, H, B, M = 6, 2, 2, 3
        if kind == "int4":
            self.kc, self.vc = z(8, heads, 32 * 72, t=torch.uint8), z(8, v_heads, v_ps * 72, t=torch.uint8)
        else:
            t = torch.uint8 if kind == "e4m3" else torch.bfloat16
            self.kc, self.vc = z(8, heads, 32, row, t=t), z(8, v_heads, v_ps, row, t=t)
        k, v, q, slots, pos, s = z(T, H, D), z(T, H, D), z(T, 4, D), z(T, t=i64), z(T, t=i64), z(1, t=f32)
        cs, w, hs = z(64, D, t=f32), z(D), z(H, t=f32)
        qb, bt, sl, mask, new = z(B, M, 4, D), z(B, 4, t=i32), z(B, t=i32), z(B, M, t=i64), z(B, M, H, D)
        c, sm = (self.kc, self.vc), D ** -0.5
        self.calls = {
            "insert": lambda: fp8kv.fp8kv_cache_insert(k, v, slots, s, s, *c),
            "rope": lambda: fp8kv.fp8kv_rope_insert(q, k, v, pos, cs, slots, s, s, *c, q_out=z(T, 4, D)),
            "attention": lambda: fp8kv.fp8kv_paged_attention(qb, *c, bt, sl, 100, s, s, sm),
            "append": lambda: fp8kv.fp8kv_append_paged_attention(new, new, qb, *c, bt, sl, 100, s, s, sm),
            "noalloc": lambda: fp8kv.fp8kv_paged_attention_noalloc(qb, *c, bt, sl, 100, s, s, sm, out=z(B, M, 4, D)),
            "tree": lambda: fp8kv.fp8kv_tree_attention(qb, *c, bt, sl, mask, 100, s, s, sm),
            "prepared": lambda: fp8kv.PreparedAttention(qb, *c, bt, sl, 100, s, s, sm, tree_mask=mask)(),
        }
        if kind == "e4m3":
            self.calls["head insert"] = lambda: fp8kv.fp8kv_cache_insert_per_head(k, v, slots, hs, hs, *c)
            self.calls["head attention"] = lambda: fp8kv.fp8kv_paged_attention_per_head(qb, *c, bt, sl, 100, hs, hs, sm)
            self.calls["norm"] = lambda: fp8kv.fp8kv_qk_norm_rope_insert(q, k, v, pos, w, w, 1e-6, cs, z(T, 4, D), slots, s,
                                                                         s, *c)


@pytest.mark.parametrize("kind", CACHES)
def test_binding_compares_the_caches_with_the_call(L, kind, monkeypatch):
    """Rows of another length, another number of heads, a V cache of another shape: the
    kernels would write and read beyond the caches."""
    from torch._subclasses import FakeTensorMode
    monkeypatch.setattr(fp8kv, "_stream", lambda stream, t=None: 0)
    monkeypatch.setattr(fp8kv._Owned, "__init__", lambda self, tensors: None)
    monkeypatch.setattr(fp8kv._Owned, "before_call", lambda self, stream, handle: None)
    with FakeTensorMode():
        for name, call in _Shapes(kind).calls.items():
            with pytest.raises(fp8kv.Fp8kvError):               # null pointers
                call()
        bad = [dict(v_heads=1), dict(v_ps=64)]
        if kind != "int4":
            bad += [dict(row=64), dict(row=256), dict(D=64, row=128)]
        for over in bad:
            for name, call in _Shapes(kind, **over).calls.items():
                with pytest.raises(ValueError):
                    call()
                    raise AssertionError((name, over))
        for name in ("insert", "rope", "head insert", "norm"):
            call = _Shapes(kind, heads=1, v_heads=1).calls.get(name)
            if call:
                with pytest.raises(ValueError):
                    call()


# ----------------------------------------------------------------- inputs

def _tree(rng, B, M, shape):
    """parents int32 [B][M]."""
    par = np.tile(np.arange(M) - 1, (B, 1))
    if shape == "star":
        par[:, 1:] = 0
    elif shape in ("tree", "ragged"):
        for b in range(B):
            par[b, 1:] = [rng.integers(max(0, m - 6), m) for m in range(1, M)]
            if shape == "ragged":
                par[b, int(rng.integers(1, M + 1)):] = -1
                if M > 6:
                    par[b, 3] = -1                      # padding in the middle; its children are padding too
    return par.astype(np.int32)


def _layout(rng, lens, ps, spare=3):
    need = [(n + ps - 1) // ps for n in lens]
    ids = rng.permutation(sum(need) + spare)
    bt = np.full((len(lens), max(need) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    return bt, sum(need) + spare


def _cuda(*arrays):
    out = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]
    return out[0] if len(out) == 1 else out


def _empty(kind, pages, H, ps, fill=0):
    if kind == "int4":
        return torch.full((pages, H, ps * 72), fill, dtype=torch.uint8, device="cuda")
    if kind == "e4m3":
        return torch.full((pages, H, ps, 128), fill, dtype=torch.uint8, device="cuda")
    return torch.full((pages, H, ps, 128), float(fill), dtype=torch.bfloat16, device="cuda")


def _values(cache, kind, ps, c):
    """float64 [pages][H][ps][128]."""
    if kind == "bf16":
        return cache.double().cpu().numpy()
    x = cache.cpu().numpy()
    return (int4_np.read_pages(x, ps) if kind == "int4" else int4_np.e4m3_value(x)) * float(c)


def _scale(v):
    return torch.tensor([v], dtype=torch.float32, device="cuda")


def _status(want=0):
    assert fp8kv.fp8kv_device_status(clear=True) == want


# --------------------------------------------------------------- metadata

@pytest.mark.gpu
@pytest.mark.parametrize("B,M,shape,ps", [(1, 1, "chain", 32), (1, 12, "tree", 32), (3, 64, "chain", 64),
                                          (5, 64, "star", 32), (7, 33, "ragged", 64), (700, 64, "tree", 32),
                                          (153, 2, "ragged", 32)])
def test_metadata(B, M, shape, ps):
    rng = np.random.default_rng(B * 100 + M)
    lens = [int(n) for n in rng.integers(M, M + 200, B)]
    lens[0] = M                                         # no context
    bt, pages = _layout(rng, lens, ps)
    par = _tree(rng, B, M, shape)
    got = fp8kv.fp8kv_tree_metadata(_cuda(par), _cuda(np.array(lens, np.int32)), _cuda(bt), ps, max(lens), pages)
    for g, w, what in zip(got, tree_np.metadata(par, lens, bt, ps), ("mask", "positions", "slots")):
        assert np.array_equal(g.cpu().numpy(), w), what
    _status()


@pytest.mark.gpu
def test_metadata_flags_bad_input():
    par = np.array([[5, 0, 1, 2], [0, 0, 2, 7], [-1, -2, 0, 2], [-1, 0, 0, 1]], np.int32)
    lens = np.array([40, 40, 40, 3], np.int32)          # the last is shorter than its tree
    bt = np.array([[0, 1], [2, 9], [3, 4], [5, 6]], np.int32)   # page 9 is outside the pool
    mask, pos, slot = fp8kv.fp8kv_tree_metadata(_cuda(par), _cuda(lens), _cuda(bt), 32, 64, 8)
    assert mask.tolist() == [[1, 3, 7, 15], [1, 3, 0, 0], [1, 0, 5, 13], [0] * 4]
    assert pos.tolist() == [[36, 37, 38, 39], [36, 37, 36, 36], [36, 36, 37, 38], [0] * 4]
    assert slot.tolist() == [[36, 37, 38, 39], [-1, -1, -1, -1], [132, -1, 134, 135], [-1] * 4]
    _status(fp8kv.DEV_BAD_TREE | fp8kv.DEV_BAD_SEQ_LEN | fp8kv.DEV_BAD_SLOT)


# ------------------------------------------------------------ rotary insert

@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("T,Hq,H,rot,pairs,ps", [(1, 1, 1, 128, False, 32), (3, 72, 8, 128, True, 64),
                                                 (37, 6, 2, 64, False, 32), (37, 5, 5, 8, False, 32),
                                                 (513, 9, 1, 96, True, 64), (300, 72, 8, 24, False, 32),
                                                 (33, 4, 2, 120, True, 32)])
def test_rope_insert(kind, T, Hq, H, rot, pairs, ps):
    rng = np.random.default_rng(T + rot)
    g = torch.Generator().manual_seed(T * 7 + rot)
    qkv = torch.randn((T, Hq + 2 * H, 128), generator=g).to(torch.bfloat16)
    far = 131072
    pos = rng.integers(0, far, T)
    pos[0] = far - 1
    ang = np.arange(far)[:, None] * 1e6 ** (-2.0 * np.arange(rot // 2) / rot)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pages = (T + ps - 1) // ps + 2
    slots = rng.permutation(pages * ps)[:T]
    slots[rng.random(T) < 0.1] = -1
    ks, vs = _scale(0.0271), _scale(0.0131)
    kc, vc, kc2, vc2 = (_empty(kind, pages, H, ps, 5) for _ in range(4))
    d = qkv.cuda()
    q, k, v = d[:, :Hq], d[:, Hq:Hq + H], d[:, Hq + H:]      # views of one projection
    out = fp8kv.fp8kv_rope_insert(q, k, v, _cuda(pos), _cuda(cs), _cuda(slots), ks, vs, kc, vc, interleaved=pairs)
    x = qkv.float().numpy()
    want_q = tree_np.rope(x[:, :Hq], cs, pos, pairs)
    want_k = tree_np.rope(x[:, Hq:Hq + H], cs, pos, pairs)
    assert np.array_equal(out.float().cpu().numpy(), want_q)         # bit for bit: the roundings are the definition's
    # the stored rows are those that an insert of the rotated rows writes
    fp8kv.fp8kv_cache_insert(torch.from_numpy(want_k).to(torch.bfloat16).cuda(), v.contiguous(), _cuda(slots), ks, vs,
                             kc2, vc2)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)
    _status()


@pytest.mark.gpu
def test_rope_insert_matches_the_fused_norm_insert():
    """A row of norm 1 with weights 1 passes the norm unchanged: same bits as
    fp8kv_qk_norm_rope_insert."""
    T, rng = 20, np.random.default_rng(3)
    x = torch.from_numpy(rng.choice([-1.0, 1.0], (T, 4, 128))).to(torch.bfloat16).cuda()
    q, k, v = x[:, :2].contiguous(), x[:, 2:3].contiguous(), x[:, 3:].contiguous()
    ang = np.arange(64)[:, None] * 1e4 ** (-np.arange(64) / 64)
    cs = _cuda(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
    pos, slots, s = _cuda(np.arange(T)), _cuda(np.arange(T)), _scale(0.01)
    one = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    caches = [_empty("e4m3", 1, 1, 32) for _ in range(4)]
    q1 = fp8kv.fp8kv_rope_insert(q, k, v, pos, cs, slots, s, s, *caches[:2])
    q2 = torch.empty_like(q)
    fp8kv.fp8kv_qk_norm_rope_insert(q, k, v, pos, one, one, 0.0, cs, q2, slots, s, s, *caches[2:])
    assert torch.equal(q1, q2) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
def test_rope_insert_skips_bad_tokens(kind):
    T, H = 6, 2
    x = torch.randn((T, 3 * H, 128), device="cuda").to(torch.bfloat16)
    cs = torch.ones((10, 64), device="cuda")
    pos = torch.tensor([0, -1, 10, 9, 3, 2 ** 40], device="cuda")
    slots = torch.tensor([0, 1, 2, 64, -5, 3], device="cuda")       # slot 64 is outside the pool of 2 pages
    kc, vc = _empty(kind, 2, H, 32, 7), _empty(kind, 2, H, 32, 7)
    before = kc.clone(), vc.clone()
    qo = torch.full((T, H, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    s = _scale(0.02)
    fp8kv.fp8kv_rope_insert(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], pos, cs, slots, s, s, kc, vc, q_out=qo)
    untouched = (qo == 3.0).all(-1).all(-1).tolist()
    assert untouched == [False, True, True, False, False, True]
    ref = before[0].clone(), before[1].clone()
    fp8kv.fp8kv_rope_insert(x[:1, :H], x[:1, H:2 * H], x[:1, 2 * H:], pos[:1], cs, slots[:1], s, s, *ref)
    assert torch.equal(kc, ref[0]) and torch.equal(vc, ref[1])
    _status(fp8kv.DEV_BAD_POSITION | fp8kv.DEV_BAD_SLOT)
    none = torch.empty((0, H, 128), dtype=torch.bfloat16, device="cuda")
    assert fp8kv.fp8kv_rope_insert(none, none, none, pos[:0], cs, slots[:0], s, s, kc, vc).shape == (0, H, 128)


# --------------------------------------------------------------- attention

class Case:
    def __init__(self, seed, kind, lens, M, Hq, H, ps, shape="tree", spread=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.kind, self.lens, self.M, self.ps, self.H = kind, [max(n, M) for n in lens], M, ps, H
        B = len(lens)
        self.bt, self.pages = _layout(rng, self.lens, ps)
        self.par = _tree(rng, B, M, shape)
        self.mask = tree_np.metadata(self.par, self.lens, self.bt, ps)[0]
        self.q = (torch.randn((B, M, Hq, 128), generator=g) * spread).to(torch.bfloat16)
        self.ks, self.vs = _scale(0.03), _scale(0.02)
        # whatever lies in rows that no sequence owns: NaN (E4M3 0x7f, bf16 NaN, INT4 scales 0x7f)
        self.kc, self.vc = (_empty(kind, self.pages, H, ps, 0x7f if kind != "bf16" else float("nan")) for _ in range(2))
        rows = [(b, j) for b, n in enumerate(self.lens) for j in range(n)]
        slots = np.array([self.bt[b, j // ps] * ps + j % ps for b, j in rows], np.int64)
        k, v = (torch.randn((len(rows), H, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        fp8kv.fp8kv_cache_insert(k, v, _cuda(slots), self.ks, self.vs, self.kc, self.vc)

    def run(self, window=-1, split=0, **kw):
        kw.setdefault("tree_mask", _cuda(self.mask))
        return fp8kv.fp8kv_tree_attention(self.q.cuda(), self.kc, self.vc, _cuda(self.bt),
                                          _cuda(np.array(self.lens, np.int32)), max_seq_len=max(self.lens),
                                          k_scale=self.ks, v_scale=self.vs, sm_scale=SM, window_left=window,
                                          split_tokens=split, **kw)

    def want(self, window=-1, mask=None):
        """(float64 outputs, tolerance).  With vmax = max |v|: the weights are rounded
        (f16 2^-11, bf16 2^-8; half a step relative to each), an INT4 or E4M3
        partial is rounded to f16 (2^-11), the output to bf16 (2^-8 of its value).  Q
        is held to 2^-17 of its row's maximum (E4M3, INT4), so a score moves by at
        most e = 128 2^-17 qmax kmax sm, the weights by a factor in 1 +- e, the mean
        by 2 e vmax; sums and exponentials in fp32 are far below (2^-16 vmax)."""
        out = np.zeros(self.q.shape)
        kk, vv = _values(self.kc, self.kind, self.ps, self.ks), _values(self.vc, self.kind, self.ps, self.vs)
        q = self.q.double().numpy()
        vmax = kmax = 0.0
        for b, n in enumerate(self.lens):
            ids = self.bt[b, :(n + self.ps - 1) // self.ps]
            k, v = (x[ids].transpose(1, 0, 2, 3).reshape(self.H, -1, 128)[:, :n] for x in (kk, vv))
            vmax, kmax = max(vmax, np.abs(v).max()), max(kmax, np.abs(k).max())
            see = tree_np.sees((self.mask if mask is None else mask)[b], self.M, n, window)
            out[b] = tree_np.attention(q[b], k, v, see, SM)
        if self.kind == "bf16":
            tol = (2.0 ** -8 + 2.0 ** -16) * vmax
        else:
            e = 128 * 2.0 ** -17 * np.abs(q).max() * kmax * SM
            tol = (2.0 ** -11 + 2.0 ** -11 + 2 * e + 2.0 ** -16) * vmax
        return out, tol + 2.0 ** -8 * np.abs(out)

    def check(self, got, window=-1, mask=None):
        want, tol = self.want(window, mask)
        g = got.double().cpu().numpy()
        assert np.isfinite(g).all()
        assert np.all(np.abs(g - want) <= tol), np.abs(g - want).max()
        hidden = (self.mask if mask is None else mask) == 0
        assert np.all(g[hidden] == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("lens,M,Hq,H,ps,shape,window,split", [
    ([1], 1, 1, 1, 32, "chain", -1, 0),                 # one node, no context
    ([300], 2, 9, 1, 32, "tree", -1, 0),                # 16-row kernels: 18 rows a head below, 2 here
    ([300, 8, 45], 8, 4, 2, 64, "ragged", -1, 0),
    ([2500, 3], 3, 8, 2, 32, "tree", 100, 0),           # several partitions, a window
    ([700], 16, 2, 2, 32, "star", 0, 0),                # a window of the row itself
    ([12, 13, 200], 12, 18, 2, 32, "tree", -1, 0),      # 108 rows a head; no context, one key of it
    ([1000], 12, 18, 2, 64, "ragged", -1, 128),         # a cluster of 8
    ([3000], 12, 9, 1, 32, "tree", 511, 0),
    ([3000, 150, 2000], 12, 18, 2, 32, "tree", -1, 0),  # partitions longest first
    ([130, 64, 65], 64, 18, 2, 64, "tree", -1, 0),      # five row tiles
    ([2100, 500], 64, 9, 1, 32, "ragged", 200, 0),
    ([900], 33, 12, 2, 32, "chain", 3, 0),              # a window shorter than the tree is deep
    ([777], 64, 2, 1, 64, "chain", 20, 128),            # 128 rows a head, nodes over two tiles
    ([3000], 64, 18, 2, 64, "ragged", -1, 512),         # five row tiles of one sequence, six partitions each
    ([5003], 40, 9, 1, 32, "tree", -1, 8192),           # one partition of forty key tiles
    ([4100], 34, 4, 1, 32, "star", 4000, 0),            # a second row tile of eight rows
])
def test_tree_attention(kind, lens, M, Hq, H, ps, shape, window, split):
    c = Case(M * 1000 + len(lens), kind, lens, M, Hq, H, ps, shape)
    c.check(c.run(window, split), window)
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("ns", [2, 5, 8])
def test_row_tiles_combine_in_clusters(kind, ns):
    """Partitions of one sequence are a cluster for each KV head and row tile."""
    c = Case(ns, kind, [128 * ns - 5], 50, 6, 2, 32, "tree")
    c.check(c.run(split=128))
    assert f"cluster={ns} reduce=0" in fp8kv.fp8kv_last_dispatch()
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("M,Hq,window,split", [(33, 10, -1, 0), (40, 18, -1, 0), (64, 6, 50, 0), (33, 10, -1, 256),
                                                 (33, 10, 100, 0), (40, 18, 130, 0), (33, 10, 150, 128)])
def test_several_row_tiles_a_cta_end_inside_a_warp(M, Hq, window, split):
    """INT4 pages: the last row tile has 37, 104, 64 rows; with a window, which leaves
    64 sequences of 2 KV heads the same keys, a CTA takes several row tiles."""
    rng = np.random.default_rng(M)
    c = Case(M + 1, "int4", [int(n) for n in rng.integers(M, 300, 63)] + [300], M, Hq, 2, 32, "ragged")
    c.check(c.run(window, split), window)
    tiles = (M * Hq // 2 + 127) // 128
    dispatch = fp8kv.fp8kv_last_dispatch()
    rows = int(dispatch.split("grid=")[1].split("x")[1])
    assert f"row_tiles={tiles} " in dispatch and (window < 0 or rows < 2 * tiles), dispatch
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("M,Hq", [(2, 4), (12, 18), (16, 18)])
def test_a_chain_is_the_plain_call(kind, M, Hq):
    c = Case(11 + M, kind, [400, 90], M, Hq, 2, 32, "chain")
    if kind != "e4m3" and M * Hq // 2 > 144:
        pytest.skip("shape of tree calls only")
    plain = fp8kv.fp8kv_paged_attention(c.q.cuda(), c.kc, c.vc, _cuda(c.bt), _cuda(np.array(c.lens, np.int32)), 400,
                                        c.ks, c.vs, SM)
    c.check(plain)                                      # the same values, hence tolerance, whatever the kernel
    got = c.run()
    c.check(got)
    if kind == "int4" or M * Hq // 2 <= 16:
        assert torch.equal(got, plain)                  # the same kernel, the same order of operations


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("lens,M,Hq,H,window", [([200, 40], 4, 8, 2, -1), ([1500], 12, 18, 2, -1),
                                                ([300, 2000], 24, 18, 2, 100), ([200], 64, 2, 1, -1),
                                                ([160, 90], 40, 6, 2, -1)])
def test_appended_nodes(kind, lens, M, Hq, H, window):
    """Rows written by the call itself: cache bytes of an insert, output of the call after it."""
    c = Case(M, kind, lens, M, Hq, H, 32, "tree")
    B = len(c.lens)
    want = c.run(window)
    whole = c.kc.clone(), c.vc.clone()
    pos = np.array([[n - M + m for m in range(M)] for n in c.lens])
    slots = _cuda(np.take_along_axis(c.bt, pos // 32, 1).astype(np.int64) * 32 + pos % 32).reshape(-1)
    g = torch.Generator().manual_seed(5)
    kn, vn = (torch.randn((B, M, H, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    fp8kv.fp8kv_cache_insert(kn.view(-1, H, 128), vn.view(-1, H, 128), slots, c.ks, c.vs, *whole)
    got = c.run(window, k_new=kn, v_new=vn)
    a, b = _values(c.kc, kind, 32, c.ks), _values(whole[0], kind, 32, c.ks)
    assert np.array_equal(a, b, equal_nan=True)
    assert np.array_equal(_values(c.vc, kind, 32, c.vs), _values(whole[1], kind, 32, c.vs), equal_nan=True)
    c.check(got, window)
    assert not torch.equal(got, want)
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("M,Hq,lens", [(4, 4, [200, 34]), (12, 18, [200, 100]), (40, 6, [150, 70]), (40, 18, [150, 70])])
def test_appended_nodes_on_pages_outside_the_pool(kind, M, Hq, lens):
    """They are not written, and read as zeros, as after an insert of the others."""
    c = Case(M + 5, kind, lens, M, Hq, 2, 32, "tree")
    for b, n in enumerate(c.lens):
        c.bt[b, (n - 1) // 32] = (-1, c.pages)[b]       # the last page, on which nodes are
    pos = np.array([[n - M + m for m in range(M)] for n in c.lens])
    page = np.take_along_axis(c.bt, pos // 32, 1).astype(np.int64)
    good = (page >= 0) & (page < c.pages)
    slots = _cuda(np.where(good, page * 32 + pos % 32, -1)).reshape(-1)
    g = torch.Generator().manual_seed(7)
    kn, vn = (torch.randn((len(lens), M, 2, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    whole = c.kc.clone(), c.vc.clone()
    fp8kv.fp8kv_cache_insert(kn.view(-1, 2, 128), vn.view(-1, 2, 128), slots, c.ks, c.vs, *whole)
    got = c.run(k_new=kn, v_new=vn)
    for a, w, s in ((c.kc, whole[0], c.ks), (c.vc, whole[1], c.vs)):
        assert np.array_equal(_values(a, kind, 32, s), _values(w, kind, 32, s), equal_nan=True)
    _status(fp8kv.DEV_BAD_SLOT)
    assert torch.equal(got, c.run())
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
def test_masks_of_any_kind(kind):
    """Words that are no ancestor sets (a node that sees a later one, not itself),
    bits beyond M, and none."""
    c = Case(3, kind, [70, 12, 300], 12, 18, 2, 32)
    rng = np.random.default_rng(9)
    words = rng.integers(0, 1 << 12, (3, 12))
    words[:, 4] = 0
    words[1, 5] = 1 << 11                               # no context, a later node only
    high = words | (rng.integers(0, 1 << 40, (3, 12)) << 12)
    high[:, 4] = 0
    high[0, 6] = words[0, 6] = 0
    high[0, 6] |= 3 << 50                               # nothing but bits beyond M: padding
    for window in (-1, 5):
        c.check(c.run(window, tree_mask=_cuda(high)), window, mask=words)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("M,Hq", [(8, 4), (16, 14), (31, 10)])
@pytest.mark.parametrize("window", [0, 1, 3])
def test_masks_of_any_kind_behind_a_short_window(kind, M, Hq, window):
    """A node's position is its number of bits, not its index: nodes far below a row's
    own position by their index are seen, in the half of a key tile before the others."""
    rng = np.random.default_rng(M + window)
    c = Case(M, kind, [int(x) for x in 64 * rng.integers(1, 9, 12) - rng.integers(1, M, 12) + M], M, Hq, 2, 64)
    words = rng.integers(0, 1 << M, (12, M))
    words[:, :M // 2] = (1 << M) - 1 - (rng.integers(0, 1 << M, (12, M // 2)) & rng.integers(0, 1 << M, (12, M // 2)))
    c.check(c.run(window, tree_mask=_cuda(words)), window, mask=words)
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("M,Hq", [(4, 4), (12, 18), (24, 18)])
def test_bad_sequences_leave_their_rows(kind, M, Hq):
    c = Case(21, kind, [100, 60, 90], M, Hq, 2, 32)
    c.lens[1] = M - 1                                   # shorter than its tree
    out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got = fp8kv.fp8kv_tree_attention(c.q.cuda(), c.kc, c.vc, _cuda(c.bt), _cuda(np.array(c.lens, np.int32)),
                                     _cuda(c.mask), 100, c.ks, c.vs, SM, out=out)
    assert (got[1] == 7.0).all() and not (got[0] == 7.0).all() and not (got[2] == 7.0).all()
    _status(fp8kv.DEV_BAD_SEQ_LEN)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,M,Hq", [("bf16", 12, 18), ("bf16", 4, 4), ("e4m3", 12, 18), ("int4", 12, 18)])
def test_negative_scale_and_large_logits(kind, M, Hq):
    """Logits of up to some hundreds, either sign of the scale: the running maximum
    and the rescaling of O."""
    c = Case(8, kind, [900], M, Hq, 2, 32, spread=8.0)
    got = c.run()
    c.check(got)
    if kind != "e4m3":
        c.q = -c.q
        neg = fp8kv.fp8kv_tree_attention(c.q.cuda(), c.kc, c.vc, _cuda(c.bt), _cuda(np.array(c.lens, np.int32)),
                                         _cuda(c.mask), 900, c.ks, c.vs, -SM)
        assert torch.equal(neg, got)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("lens,M,Hq,split", [([900], 4, 4, 0), ([900, 70], 12, 18, 0), ([500], 40, 18, 0),
                                             ([900], 12, 18, 128)])
def test_a_negative_scale_is_that_of_negated_queries(kind, lens, M, Hq, split):
    """-sm_scale with -q: the same logits, hence the same bits in every kernel (negation
    is exact in every type that holds q), and the values of the oracle."""
    c = Case(18, kind, lens, M, Hq, 2, 32, "ragged")
    got = c.run(split=split)
    c.check(got)
    neg = fp8kv.fp8kv_tree_attention(-c.q.cuda(), c.kc, c.vc, _cuda(c.bt), _cuda(np.array(c.lens, np.int32)),
                                     _cuda(c.mask), max(c.lens), c.ks, c.vs, -SM, split_tokens=split)
    assert torch.equal(neg, got)
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
def test_nan_stays_with_the_rows_that_see_it(kind):
    """A NaN key among the nodes reaches its descendants and no sibling's row."""
    c = Case(31, kind, [200], 12, 18, 2, 32, "star")
    base = 200 - 12
    slot = int(c.bt[0, (base + 5) // 32]), (base + 5) % 32
    if kind == "int4":
        c.kc[slot[0], :, 32 * 64 + slot[1] * 8:32 * 64 + slot[1] * 8 + 8] = 0x7f
    else:
        c.kc[slot[0], :, slot[1]] = 0x7f if kind == "e4m3" else float("nan")
    got = c.run().float().cpu()
    assert torch.isnan(got[0, 5]).all()
    keep = [m for m in range(12) if m != 5]
    assert torch.isfinite(got[0, keep]).all()


def _poison(cache, kind, page, off, ps):
    """The row's bytes as those that Case finds in rows of no sequence: NaN."""
    if kind == "int4":
        cache[page, :, off * 64:off * 64 + 64] = 0x7f
        cache[page, :, ps * 64 + off * 8:ps * 64 + off * 8 + 8] = 0x7f
    else:
        cache[page, :, off] = 0x7f if kind == "e4m3" else float("nan")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("lens,M,Hq,H,ps,window,split", [
    ([300, 45, 8], 8, 4, 2, 32, -1, 0),                 # up to 16 rows a head
    ([8, 100], 8, 4, 2, 64, -1, 0),                     # nodes from key 0 on
    ([2500], 15, 2, 2, 64, 700, 0),                     # several partitions
    ([260, 31, 90], 12, 18, 2, 32, -1, 0),              # one row tile; nodes over two key tiles
    ([1000], 12, 18, 2, 64, -1, 128),                   # a cluster
    ([1029, 517], 12, 18, 2, 32, -1, 128),              # nodes over two partitions, longest first
    ([777], 12, 18, 2, 32, 5, 0),                       # a first tile with keys before the window, holes and an end
    ([400, 130, 64], 64, 18, 2, 32, -1, 0),             # several row tiles; trees over two key tiles, from key 0 on
    ([160], 60, 9, 1, 32, -1, 128),                     # nodes over two partitions
    ([700] * 40, 33, 20, 4, 32, 300, 0),                # INT4: several row tiles a CTA
    ([1301], 50, 18, 2, 64, -1, 256),
])
def test_stale_rows_of_padding_nodes_reach_no_output(kind, lens, M, Hq, H, ps, window, split):
    """Nobody writes the rows of padding nodes (slot -1): whatever is there."""
    c = Case(M * 100 + len(lens), kind, lens, M, Hq, H, ps, "ragged")
    if not (c.mask == 0).any():
        c.mask[:, M // 2] = 0
    want, tol = c.want(window)
    for b, m in zip(*np.nonzero(c.mask == 0)):
        at = c.lens[b] - M + m
        for cache in (c.kc, c.vc):
            _poison(cache, kind, int(c.bt[b, at // ps]), int(at % ps), ps)
    got = c.run(window, split).double().cpu().numpy()
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - want) <= tol), np.abs(got - want).max()
    assert np.all(got[c.mask == 0] == 0)
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("lens,M,Hq,H", [([200, 40], 8, 4, 2), ([1500], 12, 18, 2), ([300, 2000], 24, 18, 2),
                                         ([160, 90], 40, 6, 2), ([260], 30, 8, 2)])
def test_appended_rows_of_padding_nodes_reach_no_output(kind, lens, M, Hq, H):
    """With k_new the rows of padding nodes are written too, NaN here."""
    c = Case(M, kind, lens, M, Hq, H, 32, "ragged")
    c.mask[:, M // 2] = 0
    pos = np.array([[n - M + m for m in range(M)] for n in c.lens])
    slots = _cuda(np.take_along_axis(c.bt, pos // 32, 1).astype(np.int64) * 32 + pos % 32).reshape(-1)
    g = torch.Generator().manual_seed(6)
    kn, vn = (torch.randn((len(lens), M, H, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    fp8kv.fp8kv_cache_insert(kn.view(-1, H, 128), vn.view(-1, H, 128), slots, c.ks, c.vs, c.kc, c.vc)
    want, tol = c.want()
    pad = torch.from_numpy(c.mask == 0).cuda()
    kn[pad] = float("nan")
    vn[pad] = float("nan")
    got = c.run(k_new=kn, v_new=vn).double().cpu().numpy()
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - want) <= tol), np.abs(got - want).max()
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("M,Hq", [(8, 4), (12, 18), (40, 18)])
def test_ragged_trees_over_an_uninitialised_cache(kind, M, Hq):
    """Metadata, rotary insert of the context and of the nodes, attention: rows that the
    insert skips hold NaN."""
    H, ps, lens = 2, 32, [70, 45, 200]
    rng = np.random.default_rng(M)
    bt_np, pages = _layout(rng, lens, ps)
    par = _tree(rng, 3, M, "ragged")
    par[0, 2] = par[1, M - 1] = -1
    fill = float("nan") if kind == "bf16" else 0x7f
    kc, vc = _empty(kind, pages, H, ps, fill), _empty(kind, pages, H, ps, fill)
    x = torch.randn((sum(lens), Hq + 2 * H, 128), generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    ang = np.arange(256)[:, None] * 1e4 ** (-np.arange(64) / 64)
    cs, s = _cuda(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)), _scale(0.03)
    bt, sl = _cuda(bt_np, np.array(lens, np.int32))
    mask, pos, slot = fp8kv.fp8kv_tree_metadata(_cuda(par), sl, bt, ps, max(lens), pages)
    q, first = [], 0
    for b, n in enumerate(lens):
        y = x[first:first + n]
        first += n
        p = torch.cat([torch.arange(n - M, device="cuda"), pos[b]])
        at = torch.from_numpy(bt_np[b, np.arange(n - M) // ps].astype(np.int64) * ps + np.arange(n - M) % ps).cuda()
        q.append(fp8kv.fp8kv_rope_insert(y[:, :Hq], y[:, Hq:Hq + H], y[:, Hq + H:], p, cs, torch.cat([at, slot[b]]), s,
                                         s, kc, vc)[n - M:])
    got = fp8kv.fp8kv_tree_attention(torch.stack(q), kc, vc, bt, sl, mask, max(lens), s, s, SM).double().cpu().numpy()
    assert np.isfinite(got).all()
    words = mask.cpu().numpy()
    assert np.all(got[words == 0] == 0) and (words == 0).any()
    kk, vv = _values(kc, kind, ps, s), _values(vc, kind, ps, s)
    qmax = max(float(t.abs().max()) for t in q)
    for b, n in enumerate(lens):
        ids = bt_np[b, :(n + ps - 1) // ps]
        k, v = (a[ids].transpose(1, 0, 2, 3).reshape(H, -1, 128)[:, :n] for a in (kk, vv))
        want = tree_np.attention(q[b].double().cpu().numpy(), k, v, tree_np.sees(words[b], M, n, -1), SM)
        # the bounds of Case.want, of the rows that are held
        vmax, kmax = np.nanmax(np.abs(v)), np.nanmax(np.abs(k))
        e = 0 if kind == "bf16" else 128 * 2.0 ** -17 * qmax * kmax * SM
        tol = ((2.0 ** -8 if kind == "bf16" else 2.0 ** -10) + 2 * e + 2.0 ** -16) * vmax + 2.0 ** -8 * np.abs(want)
        assert np.all(np.abs(got[b] - want) <= tol), (b, np.abs(got[b] - want).max())
    _status()


# -------------------------------------------------------------- verification

def _probs(rng, B, M, V, sharp=2.0, zero=0.0):
    x = rng.normal(size=(B, M, V)) * sharp
    y = x + rng.normal(size=(B, M, V)) * 0.7
    out = []
    for z in (x, y):
        p = np.exp(z - z.max(-1, keepdims=True))
        if zero:
            p *= rng.random((B, M, V)) >= zero          # what a truncated distribution leaves
            p[..., 0] += 1e-3
        out.append((p / p.sum(-1, keepdims=True)).astype(np.float32))
    return out


def _draws(rng, q, par):
    """A token for each node from its parent's row, independently."""
    B, M, V = q.shape
    c = np.cumsum(q.astype(np.float64), -1)
    up = np.maximum(par, 0)
    t = rng.random((B, M)) * c[np.arange(B)[:, None], up, -1]
    return np.array([[min(V - 1, int(np.searchsorted(c[b, up[b, m]], t[b, m], side="right"))) for m in range(M)]
                     for b in range(B)], np.int32)


def _check_verify(p, q, tok, par, u, got, margin=2.0 ** -40):
    """Whole numbers are equal wherever no decision is nearer to its border than the
    sums' error: 2^-45 of a weight a step, 64 steps at most, 2^-39 at the very worst;
    2^-40 here, for trees of few rejections.  (Such a case would be skipped, and
    counted: with 2^17 tokens one in 2^22.)"""
    out, num, path = (t.cpu().numpy() for t in got)
    B, M, _ = p.shape
    near = 0
    for b in range(B):
        w_out, w_path, d = tree_np.verify(p[b].astype(np.float64), None if q is None else q[b].astype(np.float64),
                                          tok[b], par[b], u[b])
        if d < margin:
            near += 1
            continue
        assert num[b] == len(w_out), (b, num[b], w_out)
        assert out[b].tolist() == w_out + [-1] * (M - len(w_out)), b
        assert path[b].tolist() == w_path + [-1] * (M - len(w_path)), b
    assert near <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,M,V,shape", [(1, 1, 1, "chain"), (2, 3, 7, "star"), (1, 12, 50001, "chain"),
                                         (3, 64, 999, "star"), (5, 16, 4099, "tree"), (70, 9, 2500, "ragged"),
                                         (200, 6, 300, "tree"), (2, 5, 131072, "star"), (1, 20, 33000, "tree")])
def test_verify(dtype, draft, B, M, V, shape):
    rng = np.random.default_rng(V + M)
    p, q = _probs(rng, B, M, V)
    tp, tq = (torch.from_numpy(x).to(torch.float32 if dtype == "fp32" else torch.bfloat16) for x in (p, q))
    p, q = tp.float().numpy(), tq.float().numpy()
    par = _tree(rng, B, M, shape)
    tok = _draws(rng, q, par)
    u = rng.random((B, M)).astype(np.float32)
    u = np.minimum(u, np.float32(1 - 2.0 ** -24))
    u[0, 0] = 0.0
    if B > 1:
        u[1, 0] = 1 - 2.0 ** -24
    got = fp8kv.fp8kv_verify_tree(tp.cuda(), tq.cuda() if draft else None, _cuda(tok), _cuda(par), _cuda(u))
    _check_verify(p, q if draft else None, tok, par, u, got)
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_verify_truncated_rows_and_strided_views(draft):
    """Rows with many zeros, views of a padded vocabulary whose rows start anywhere."""
    rng = np.random.default_rng(4)
    B, M, V = 6, 8, 3001
    p, q = _probs(rng, B, M, V, zero=0.95)
    par = _tree(rng, B, M, "tree")
    tok = _draws(rng, q, par)
    u = rng.random((B, M)).astype(np.float32)
    wide = [torch.full((B, M, V + w), float("nan"), device="cuda") for w in (7, 12)]
    views = [w[..., 3 + i:3 + i + V] for i, w in enumerate(wide)]     # p and q on different boundaries
    views[0].copy_(torch.from_numpy(p))
    views[1].copy_(torch.from_numpy(q))
    got = fp8kv.fp8kv_verify_tree(views[0], views[1] if draft else None, _cuda(tok), _cuda(par), _cuda(u))
    _check_verify(p, q if draft else None, tok, par, u, got)
    # the same in bf16, rows of both on odd boundaries of their own
    halves = [v.to(torch.bfloat16) for v in wide]
    views = [w[..., 3 + i:3 + i + V] for i, w in enumerate(halves)]
    p, q = (v.float().cpu().numpy() for v in views)
    got = fp8kv.fp8kv_verify_tree(views[0], views[1] if draft else None, _cuda(tok), _cuda(par), _cuda(u))
    _check_verify(p, q if draft else None, tok, par, u, got)
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_chosen_drafts_at_every_boundary_of_a_row(dtype):
    """Rows that start at each place of a 16-byte group, in CTAs of many whole chunks;
    without draft_probs its stride means nothing."""
    rng = np.random.default_rng(15)
    B, M, V = 300, 3, 50001
    p, _ = _probs(rng, 1, 2 * M, V)
    pick = rng.integers(0, 2 * M, (B, M))
    tp = torch.from_numpy(p[0]).to(torch.float32 if dtype == "fp32" else torch.bfloat16)
    rows = tp.cuda()[_cuda(pick)]
    p = tp.float().numpy()[pick]
    par = _tree(rng, B, M, "tree")
    tok = _draws(rng, p, par)
    u = np.minimum(rng.random((B, M)).astype(np.float32), np.float32(1 - 2.0 ** -24))
    dev = _cuda(tok, par, u)
    got = fp8kv.fp8kv_verify_tree(rows, None, *dev)
    _check_verify(p, None, tok, par, u, got)
    for stride in (1, V + 2):
        again = [torch.empty_like(t) for t in got]
        rc = fp8kv.lib().fp8kv_verify_tree(rows.data_ptr(), V, 0, stride, 0 if dtype == "fp32" else 1,
                                           *(t.data_ptr() for t in dev), B, M, V,
                                           *(t.data_ptr() for t in again), torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and all(torch.equal(a, b) for a, b in zip(got, again))
    _status()


def _after_falls(p, q, k):
    """What k falls leave of p, exact up to a common factor."""
    w = [max(a - b, 0) for a, b in zip(p, q)]
    for _ in range(k - 1):
        S = sum(w)
        w = [max(a - S * b, 0) for a, b in zip(w, q)]
        while 0 < sum(w) < 1:
            w = [2 * a for a in w]
    return w


@pytest.mark.gpu
def test_verify_draws_what_little_many_falls_leave():
    """A drafter that is the target but for a little weight on a token which the target
    does not have; every sibling drew that one and falls, each fall leaving that little
    of the weights, so that what is left are differences of their last bits.  A weight
    is off by 2^-45 of the one before the fall, and p and q differ by 2^-24 of
    themselves where anything is left: 2^-21 in all, and the draws keep 2^-16 of the
    sum from every border."""
    drawn = 0
    for seed in range(60):
        rng = np.random.default_rng(seed)
        A = int(rng.integers(4, 40))
        share = rng.random(A) + 0.5
        share /= share.sum()
        extra = 2.0 ** -float(rng.integers(5, 10))
        p = np.concatenate([share, [0]]).astype(np.float32)
        q = np.concatenate([share * (1 - extra), [extra]]).astype(np.float32)
        pf, qf = ([Fraction(float(x)) for x in r] for r in (p, q))
        for k in range(2, 10):
            w = _after_falls(pf, qf, k)
            ends, total = np.cumsum(np.array(w, object)), sum(w)
            if total == 0:
                continue
            u0, want = [], []
            for i, x in enumerate(w):
                u = np.float32(float((ends[i] - x / 2) / total))
                t = Fraction(float(u)) * total
                if min(t - ends[i] + x, ends[i] - t) > total / 2 ** 16:
                    u0.append(u)
                    want.append(i)
            B, M = len(u0), k + 1
            u = np.full((B, M), 0.5, np.float32)
            u[:, 0] = u0
            rows = [torch.from_numpy(r).cuda().expand(B, M, A + 1).contiguous() for r in (p, q)]
            par, tok = np.zeros((B, M), np.int32), np.full((B, M), A, np.int32)
            out, num, _ = fp8kv.fp8kv_verify_tree(*rows, *_cuda(tok, par, u))
            assert num.tolist() == [1] * B and out[:, 0].tolist() == want, (seed, k)
            drawn += B
    assert drawn > 2000
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_verify_sums_of_many_small_weights(draft):
    """Four million tokens a CTA, a few of weight 1 or some at the start of every warp's
    run and then 2^-26 (1 + 2^-13) each: a thread's sum of those is multiples of 2^-39 beside its
    1, so every sum is exact in a pair whose parts are in order (a low part that only
    grows loses 2^-39 a token behind 2^-14: tens of tokens by the end of a run).  The
    draw t is the product of u and the sum, off by 2^-47 of it: 2^-37, and a token's
    width is 2^-26; draws nearer than 2^-30 to a border are left out."""
    B, V, one = 257, 1 << 22, 1 << 39
    w = np.full(V, (1 << 13) + 1, np.int64)             # units of 2^-39
    run = V // 8
    for i in range(8):
        for lane in range(32):
            w[i * run + 4 * lane:i * run + 4 * lane + 2] = one
    rng = np.random.default_rng(2)
    w[2:4096:4] = rng.integers(1 << 21, 1 << 22, 1024) << 16       # (so that draws fall anywhere in a token)
    ends = np.cumsum(w)
    total = int(ends[-1])
    u, want = [], []
    for _ in range(4 * B):
        v = int(rng.integers(7)) * run + int(rng.integers(run // 2, run))
        x = np.float32(int(ends[v]) / total)
        t = Fraction(float(x)) * total
        at = int(np.searchsorted(ends, int(t), side="right"))
        if min(t - int(ends[at]) + int(w[at]), int(ends[at]) - t) > 512:
            u.append([x])
            want.append(at)
    u, want = u[:B], want[:B]
    assert len(u) == B
    row = torch.from_numpy((w / one).astype(np.float32)).cuda()
    assert np.array_equal(row.double().cpu().numpy() * one, w)
    p = row.expand(B, 1, V).contiguous()
    none = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    out, num, _ = fp8kv.fp8kv_verify_tree(p, p if draft else None, none, none, _cuda(np.array(u, np.float32)))
    assert num.tolist() == [1] * B and out[:, 0].tolist() == want
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("B,V", [(1, 70000), (40, 9000), (300, 500)])
def test_verify_writes_over_the_rows_that_it_read(B, V):
    """out_tokens and path may be [B][M] inputs: a sequence's CTAs have read their rows."""
    rng = np.random.default_rng(B)
    M = 7
    p, q = _probs(rng, B, M, V)
    par = _tree(rng, B, M, "tree")
    tok = _draws(rng, q, par)
    u = np.minimum(rng.random((B, M)).astype(np.float32), np.float32(1 - 2.0 ** -24))
    args = _cuda(p, q, tok, par, u)
    want = fp8kv.fp8kv_verify_tree(*args)
    got = fp8kv.fp8kv_verify_tree(*args, out_tokens=args[2], path=args[3])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    _status()


@pytest.mark.gpu
def test_verify_a_greedy_target_and_certain_cases():
    """Rows of one 1: the path follows the target's tokens whatever the numbers."""
    rng = np.random.default_rng(6)
    B, M, V = 9, 12, 5000
    best = rng.integers(0, 4, (B, M))
    p = np.zeros((B, M, V), np.float32)
    np.put_along_axis(p, best[..., None], 1.0, -1)
    par = _tree(rng, B, M, "tree")
    tok = rng.integers(0, 4, (B, M)).astype(np.int32)
    u = rng.random((B, M)).astype(np.float32)
    got = fp8kv.fp8kv_verify_tree(_cuda(p), None, _cuda(tok), _cuda(par), _cuda(u))
    out, num, path = (t.tolist() for t in got)
    for b in range(B):
        n, want, at = 0, [], [0]
        while True:
            t = int(best[b, n])
            want.append(t)
            kids = [m for m in range(1, M) if par[b, m] == n and tok[b, m] == t]
            if not kids:
                break
            n = kids[0]
            at.append(n)
        assert out[b][:num[b]] == want and path[b][:num[b]] == at


@pytest.mark.gpu
def test_verify_distributes_tokens_as_the_target():
    """The first token of 20000 sequences of one distribution, drafts drawn from the
    drafter's: each token's count is binomial, 6 sigma."""
    rng = np.random.default_rng(12)
    B, M, V = 20000, 4, 12
    p, q = (np.repeat(x, B, 0) for x in _probs(rng, 1, M, V, sharp=1.0))
    par = np.tile(np.array([-1, 0, 0, 0], np.int32), (B, 1))
    tok = _draws(rng, q, par)
    u = rng.random((B, M)).astype(np.float32)
    out, num, _ = fp8kv.fp8kv_verify_tree(_cuda(p), _cuda(q), _cuda(tok), _cuda(par), _cuda(u))
    count = np.bincount(out[:, 0].cpu().numpy(), minlength=V)
    e = p[0, 0].astype(np.float64) * B
    assert np.all(np.abs(count - e) <= 6 * np.sqrt(e * (1 - e / B)) + 1)
    assert 1.3 < float(num.float().mean()) < 2.01


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_verify_distributes_the_second_token_too(draft):
    """Behind each first token that stands, the counts of the second: binomial, 6 sigma
    (chosen drafts: two tokens that the drafter likes best, at either node)."""
    rng = np.random.default_rng(13)
    B, V = 200000, 6
    p, q = (np.repeat(x, B, 0) for x in _probs(rng, 1, 5, V, sharp=1.0))
    par = np.tile(np.array([-1, 0, 0, 1, 1], np.int32), (B, 1))
    tok = _draws(rng, q, par) if draft else np.tile(np.array([0, 2, 4, 1, 3], np.int32), (B, 1))
    u = np.minimum(rng.random((B, 5)).astype(np.float32), np.float32(1 - 2.0 ** -24))
    out, num, path = (t.cpu().numpy() for t in fp8kv.fp8kv_verify_tree(
        _cuda(p), _cuda(q) if draft else None, _cuda(tok), _cuda(par), _cuda(u)))

    def binomial(tokens, row):
        e = row.astype(np.float64) * len(tokens)
        assert np.all(np.abs(np.bincount(tokens, minlength=V) - e) <= 6 * np.sqrt(e * (1 - e / len(tokens))) + 1)

    binomial(out[:, 0], p[0, 0])
    behind = path[:, 1] == 1
    assert behind.sum() > 5000
    # (the tree's second token hangs on node 1: its row)
    binomial(out[behind, 1], p[0, 1])
    assert num.min() >= 1 and (num[behind] >= 2).all()


@pytest.mark.gpu
def test_verify_flags_bad_input():
    V, M = 40, 4
    p = torch.full((6, M, V), 1.0 / V, device="cuda")
    q = p.clone()
    par = torch.tensor([[-1, 0, 1, 2]] * 6, dtype=torch.int32, device="cuda")
    tok = torch.tensor([[0, 5, 6, 7]] * 6, dtype=torch.int32, device="cuda")
    u = torch.zeros((6, M), device="cuda")
    u[:, 0] = 0.5
    par[0, 2] = 3                                       # behind itself
    tok[1, 2] = V                                       # outside the vocabulary
    p[2, 3] = 0.0                                       # nothing to draw from
    p[3, 3, 9] = float("inf")
    p[4, 0] = float("nan")                              # no token stands, none is drawn
    out, num, path = fp8kv.fp8kv_verify_tree(p, q, tok, par, u)
    assert out.tolist() == [[5, 20, -1, -1], [5, 20, -1, -1], [5, 6, 7, -1], [5, 6, 7, -1], [-1] * 4, [5, 6, 7, 20]]
    assert num.tolist() == [2, 2, 3, 3, 0, 4]
    assert path.tolist() == [[0, 1, -1, -1]] * 2 + [[0, 1, 2, 3]] * 2 + [[0, -1, -1, -1], [0, 1, 2, 3]]
    _status(fp8kv.DEV_BAD_TREE | fp8kv.DEV_BAD_PROBS)


@pytest.mark.gpu
def test_verify_when_nothing_is_left():
    """p = q with sums below 1 (what bf16 leaves): a fallen token takes all of w with
    it, and the next is drawn from the node's own row."""
    V = 64
    p = torch.full((1, 2, V), 1.0 / 128, dtype=torch.bfloat16, device="cuda")
    q = torch.full((1, 2, V), 1.0 / 64, dtype=torch.bfloat16, device="cuda")
    par = torch.tensor([[-1, 0]], dtype=torch.int32, device="cuda")
    tok = torch.tensor([[0, 3]], dtype=torch.int32, device="cuda")
    u = torch.tensor([[0.25, 0.75]], device="cuda")
    out, num, path = fp8kv.fp8kv_verify_tree(p, q, tok, par, u)
    assert out.tolist() == [[16, -1]] and num.tolist() == [1] and path.tolist() == [[0, -1]]
    _status()


# ---------------------------------------------------------------- kept path

@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("layers,B,M,H,ps", [(1, 1, 12, 8, 32), (3, 5, 64, 2, 64), (48, 2, 7, 1, 32), (2, 40, 1, 4, 32),
                                             (2, 3, 33, 40, 32), (64, 40, 5, 1, 32)])
def test_keep_path(kind, layers, B, M, H, ps):
    rng = np.random.default_rng(M + layers)
    lens = [int(n) for n in rng.integers(M, M + 150, B)]
    lens[0] = M
    bt, pages = _layout(rng, lens, ps)
    g = torch.Generator(device="cuda").manual_seed(M)
    caches = []
    for _ in range(2 * layers):
        c = torch.randint(0, 120, _empty(kind, pages, H, ps).shape, generator=g, device="cuda")
        caches.append(c.to(torch.bfloat16) if kind == "bf16" else c.to(torch.uint8))
    path = np.full((B, M), -1, np.int32)
    for b in range(B):
        # sources that are destinations of others among them: 0 1 2 3 ... 2 3 5 6 ...
        n = int(rng.integers(1, M + 1))
        path[b, :n] = np.concatenate([[0], np.sort(rng.choice(np.arange(1, M), n - 1, replace=False))])
    want = [c.cpu().numpy() if kind != "bf16" else c.float().cpu().numpy() for c in caches]
    for w in want:
        old = w.copy()
        for b, n in enumerate(lens):
            for i, m in enumerate(path[b][path[b] >= 0]):
                (sp, so), (dp, do) = ((bt[b, (n - M + x) // ps], (n - M + x) % ps) for x in (m, i))
                if kind == "int4":
                    w[dp, :, do * 64:do * 64 + 64] = old[sp, :, so * 64:so * 64 + 64]
                    e, f = ps * 64 + do * 8, ps * 64 + so * 8
                    w[dp, :, e:e + 8] = old[sp, :, f:f + 8]
                else:
                    w[dp, :, do] = old[sp, :, so]
    new = fp8kv.fp8kv_cache_keep_path(caches[:layers], caches[layers:], _cuda(bt), _cuda(np.array(lens, np.int32)),
                                      _cuda(path), max(lens))
    for c, w in zip(caches, want):
        assert np.array_equal(c.cpu().numpy() if kind != "bf16" else c.float().cpu().numpy(), w)
    assert new.tolist() == [n - M + int((path[b] >= 0).sum()) for b, n in enumerate(lens)]
    _status()
    with pytest.raises(ValueError):
        fp8kv.fp8kv_cache_keep_path(caches[:layers], caches[:layers], _cuda(bt), _cuda(np.array(lens, np.int32)),
                                    _cuda(path), max(lens))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
def test_keep_path_leaves_bad_sequences(kind):
    M, ps = 8, 32
    lens = np.array([40, 40, 40, 40, 40, 7, 40], np.int32)
    bt = np.arange(14, dtype=np.int32).reshape(7, 2)
    bt[6] = [12, 99]                                    # its tree is on a page outside the pool
    path = np.full((7, M), -1, np.int32)
    path[:, :3] = [0, 2, 5]
    path[0, :3] = [1, 2, 5]                             # does not begin with the root
    path[1, :3] = [0, 5, 2]                             # does not ascend
    path[2, :3] = [0, 2, 8]                             # beyond M
    path[3, 5] = 7                                      # a gap
    kc, vc = (torch.randint(0, 120, _empty(kind, 14, 2, ps).shape, device="cuda").to(
        torch.bfloat16 if kind == "bf16" else torch.uint8) for _ in range(2))
    before = kc.clone()
    new = fp8kv.fp8kv_cache_keep_path([kc], [vc], _cuda(bt), _cuda(lens), _cuda(path), 64)
    assert new.tolist() == [40, 40, 40, 40, 35, 7, 35]
    changed = (kc != before).flatten(1).any(1).tolist()
    assert changed == [False] * 9 + [True] + [False] * 4
    _status(fp8kv.DEV_BAD_TREE | fp8kv.DEV_BAD_SEQ_LEN | fp8kv.DEV_BAD_SLOT)


# ------------------------------------------------------------- the whole step

class Step:
    """A small model-free step: metadata, rotary insert, attention, verification and
    the kept path over fixed buffers."""

    def __init__(self, seed, kind="e4m3", lens=(300, 45, 130), M=12, Hq=18, H=2, ps=32, V=5000, layers=2):
        rng = np.random.default_rng(seed)
        self.kind, self.M, self.ps, self.H, self.layers = kind, M, ps, H, layers
        self.lens = list(lens)
        B = len(lens)
        self.bt_np, self.pages = _layout(rng, self.lens, ps)
        self.par_np = _tree(rng, B, M, "tree")
        g = torch.Generator().manual_seed(seed)
        self.qkv = torch.randn((layers, B * M, Hq + 2 * H, 128), generator=g).to(torch.bfloat16).cuda()
        self.p_np, q = _probs(rng, B, M, V)
        self.q_np = q
        self.tok_np = _draws(rng, q, self.par_np)
        self.u_np = rng.random((B, M)).astype(np.float32)
        self.bt, self.par, self.p, self.q, self.tok, self.u = _cuda(self.bt_np, self.par_np, self.p_np, q, self.tok_np,
                                                                    self.u_np)
        self.sl = _cuda(np.array(lens, np.int32))
        ang = np.arange(512)[:, None] * 1e4 ** (-np.arange(64) / 64)
        self.cs_np = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        self.cs = _cuda(self.cs_np)
        self.ks, self.vs = _scale(0.03), _scale(0.03)
        self.caches = [_empty(kind, self.pages, H, ps) for _ in range(2 * layers)]
        for i in range(layers):
            n = self.pages * ps
            k, v = (torch.randn((n, H, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
            fp8kv.fp8kv_cache_insert(k, v, torch.arange(n, device="cuda"), self.ks, self.vs, self.caches[i],
                                     self.caches[layers + i])
        self.keep = fp8kv.PreparedKeepPath(self.caches[:layers], self.caches[layers:], self.bt, self.sl,
                                           torch.zeros((B, M), dtype=torch.int32, device="cuda"), self.bt.shape[1] * ps)
        self.path = self.keep._keep[4]
        self.Hq = Hq

    def run(self, stream=None):
        B, M = len(self.lens), self.M
        mask, pos, slots = fp8kv.fp8kv_tree_metadata(self.par, self.sl, self.bt, self.ps, max(self.lens), self.pages,
                                                     stream=stream)
        outs = []
        for i in range(self.layers):
            x = self.qkv[i]
            q = fp8kv.fp8kv_rope_insert(x[:, :self.Hq], x[:, self.Hq:self.Hq + self.H], x[:, self.Hq + self.H:],
                                        pos.view(-1), self.cs, slots.view(-1), self.ks, self.vs, self.caches[i],
                                        self.caches[self.layers + i], stream=stream)
            outs.append(fp8kv.fp8kv_tree_attention(q.view(B, M, self.Hq, 128), self.caches[i],
                                                   self.caches[self.layers + i], self.bt, self.sl, mask,
                                                   max(self.lens), self.ks, self.vs, SM, stream=stream))
        out, num, _ = fp8kv.fp8kv_verify_tree(self.p, self.q, self.tok, self.par, self.u, path=self.path, stream=stream)
        new = self.keep(stream)
        return outs, out, num, new


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
def test_a_step_leaves_the_cache_of_the_accepted_tokens(kind):
    """After the step, a decode over the kept rows is that over a cache into which only
    the accepted tokens were inserted, at their positions."""
    s = Step(4, kind)
    B, M = len(s.lens), s.M
    fresh = [c.clone() for c in s.caches]
    outs, out, num, new = s.run()
    paths = []
    for b in range(B):
        w_out, w_path, d = tree_np.verify(s.p_np[b].astype(np.float64), s.q_np[b].astype(np.float64), s.tok_np[b],
                                          s.par_np[b], s.u_np[b])
        assert d > 2.0 ** -40
        assert out[b].tolist()[:int(num[b])] == w_out
        paths.append(w_path)
    assert new.tolist() == [n - M + len(p) for n, p in zip(s.lens, paths)]
    assert max(len(p) for p in paths) > 2               # something was accepted
    # the accepted chain alone, inserted at its positions
    idx = [b * M + m for b, p in enumerate(paths) for m in p]
    at = [(b, n - M + i) for b, (n, p) in enumerate(zip(s.lens, paths)) for i in range(len(p))]
    slots = _cuda(np.array([s.bt_np[b, j // s.ps] * s.ps + j % s.ps for b, j in at], np.int64))
    pos = _cuda(np.array([j for _, j in at], np.int64))
    for i in range(s.layers):
        x = s.qkv[i][idx]
        fp8kv.fp8kv_rope_insert(x[:, :s.Hq], x[:, s.Hq:s.Hq + s.H], x[:, s.Hq + s.H:], pos, s.cs, slots, s.ks, s.vs,
                                fresh[i], fresh[s.layers + i])
        for a, f, c in ((s.caches[i], fresh[i], s.ks), (s.caches[s.layers + i], fresh[s.layers + i], s.vs)):
            got = fp8kv.fp8kv_cache_gather(slots, c, c, a, a)[0]
            want = fp8kv.fp8kv_cache_gather(slots, c, c, f, f)[0]
            assert torch.equal(got, want)
        q1 = torch.randn((B, 1, s.Hq, 128), device="cuda").to(torch.bfloat16)
        d1, d2 = (fp8kv.fp8kv_paged_attention(q1, c[i], c[s.layers + i], s.bt, new, max(s.lens), s.ks, s.vs, SM)
                  for c in (s.caches, fresh))
        assert torch.equal(d1, d2)
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
def test_a_step_in_a_graph_with_new_contents(kind):
    """The whole step captured once; replayed with other trees, lengths and numbers in
    the same buffers it gives what eager calls give."""
    s = Step(7, kind)
    other = Step(8, kind, lens=(200, 100, 260))
    stream = torch.cuda.Stream()
    saved = [c.clone() for c in s.caches]
    with torch.cuda.stream(stream):
        s.run()                                         # first use outside of the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    s.lens = [300, 300, 300]                            # the largest length that a replay may have
    with torch.cuda.graph(graph, stream=stream):
        outs, out, num, new = s.run()
    for a, b in ((s.par, other.par), (s.tok, other.tok), (s.u, other.u), (s.p, other.p), (s.q, other.q),
                 (s.qkv, other.qkv)):
        a.copy_(b)
    s.sl.copy_(torch.tensor([290, 40, 100], device="cuda"))
    for c, v in zip(s.caches, saved):
        c.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs], out.clone(), num.clone(), new.clone(), [c.clone() for c in s.caches]
    for c, v in zip(s.caches, saved):
        c.copy_(v)
    want = s.run()
    for a, b in zip(got[0], want[0]):
        assert torch.equal(a, b)
    assert all(torch.equal(a, b) for a, b in zip(got[1:4], want[1:]))
    assert all(torch.equal(a, b) for a, b in zip(got[4], s.caches))
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("M,Hq", [(4, 8), (12, 72)])
def test_pages_beyond_four_gigabytes(kind, M, Hq):
    """The last pages of caches of 5 GiB: the same bytes and outputs as those of small ones."""
    H, ps, n = 8, 64, 200
    page = H * ps * {"bf16": 256, "e4m3": 128, "int4": 72}[kind]
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((n, Hq + 2 * H, 128), generator=g, device="cuda").to(torch.bfloat16)
    cs = torch.randn((256, 64), generator=g, device="cuda")
    s, pos, sl = _scale(0.03), torch.arange(n, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    par = _cuda(_tree(np.random.default_rng(M), 1, M, "tree"))
    path = torch.tensor([[0] + list(range(2, M)) + [-1]], dtype=torch.int32, device="cuda")
    got = []
    for pages in (4, (5 << 30) // page):
        kc, vc = (torch.empty_like(_empty(kind, 1, H, ps)).new_empty((pages, *_empty(kind, 1, H, ps).shape[1:]))
                  for _ in range(2))
        kc[-4:].zero_(), vc[-4:].zero_()
        bt = torch.arange(pages - 1, pages - 5, -1, dtype=torch.int32, device="cuda")[None]
        slots = bt[0, pos // ps].long() * ps + pos % ps
        q = fp8kv.fp8kv_rope_insert(x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], pos, cs, slots, s, s, kc, vc)
        mask, _, node_slots = fp8kv.fp8kv_tree_metadata(par, sl, bt, ps, n, pages)
        assert torch.equal(node_slots[0], slots[n - M:])
        out = fp8kv.fp8kv_tree_attention(q[n - M:][None].contiguous(), kc, vc, bt, sl, mask, n, s, s, SM)
        new = fp8kv.fp8kv_cache_keep_path([kc], [vc], bt, sl, path, n)
        got.append((q, out, new, *fp8kv.fp8kv_cache_gather(slots, s, s, kc, vc), kc[-4:].clone(), vc[-4:].clone()))
        del kc, vc
    for a, b in zip(*got):
        assert torch.equal(a, b)
    _status()


@pytest.mark.gpu
def test_steps_on_several_streams_at_once():
    """Steps of their own buffers on four streams give what they give alone."""
    steps = [Step(20 + i, CACHES[i % 3]) for i in range(4)]
    saved = [[c.clone() for c in s.caches] for s in steps]
    alone = [s.run() for s in steps]
    torch.cuda.synchronize()
    for s, v in zip(steps, saved):
        for c, x in zip(s.caches, v):
            c.copy_(x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [s.run(st) for s, st in zip(steps, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a[0], b[0])) and all(torch.equal(x, y) for x, y in zip(a[1:], b[1:]))
    _status()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", CACHES)
def test_prepared_tree_call(kind):
    c = Case(77, kind, [500], 12, 18, 2, 32)
    sl = _cuda(np.array(c.lens, np.int32))
    call = fp8kv.PreparedAttention(c.q.cuda(), c.kc, c.vc, _cuda(c.bt), sl, 500, c.ks, c.vs, SM,
                                   tree_mask=_cuda(c.mask))
    assert torch.equal(call(), c.run())
    with pytest.raises(ValueError):
        fp8kv.PreparedAttention(c.q.cuda(), c.kc, c.vc, _cuda(c.bt), sl, 500, c.ks, c.vs, SM,
                                tree_mask=_cuda(c.mask[:, :5]))

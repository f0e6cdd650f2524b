"""What a call on another stream allocates for itself: the memory is that
stream's, not work's still queued on the current one."""
import pytest
import torch

from verify_attention_gb300 import build, fp8kv, inputs as gen

pytestmark = pytest.mark.gpu
SM = 128 ** -0.5
BUSY = 200_000_000          # cycles, about 0.1 s: longer than the host needs for all that follows


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def _tensors(cache, M, lens=(1500, 700), H=4, G=9, ps=32):
    g = gen.generator(sum(lens) + M)
    lay = gen.paged_layout(list(lens), ps, g)
    B = len(lens)
    q = torch.randn((B, M, G * H, 128), generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn((sum(lens), H, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    slots = torch.cat([lay.slots(b, range(n)) for b, n in enumerate(lens)]).cuda()
    s = torch.tensor([0.01], device="cuda")
    if cache == "int4":
        kc, vc = (fp8kv.fp8kv_int4_cache(lay.num_pages, H, ps) for _ in range(2))
    else:
        kc, vc = (torch.zeros((lay.num_pages, H, ps, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    fp8kv.fp8kv_cache_insert(k, v, slots, s, s, kc, vc)
    call = dict(q=q, k_cache=kc, v_cache=vc, block_table=lay.block_table.cuda(), seq_lens=lay.seq_lens.cuda(),
                max_seq_len=max(lens), k_scale=s, v_scale=s, sm_scale=SM)
    return call, (k, v, slots, s)


def _calls():
    """name -> (shape, bytes of one output, call(stream) -> outputs)"""
    out = {}
    for cache in ("int4", "e4m3"):
        for M in (1, 12):
            c, (k, v, slots, s) = _tensors(cache, M)
            out[f"{cache} M={M}"] = lambda st, c=c: (fp8kv.fp8kv_paged_attention(**c, stream=st),)
            new = [x[:2 * M].view(2, M, 4, 128).contiguous() for x in (k, v)]
            d = {**c, "k_cache": c["k_cache"].clone(), "v_cache": c["v_cache"].clone()}
            out[f"append {cache} M={M}"] = (
                lambda st, d=d, new=new: (fp8kv.fp8kv_append_paged_attention(*new, **d, stream=st),))
            if M == 1:
                out[f"gather {cache}"] = lambda st, c=c, slots=slots, s=s: fp8kv.fp8kv_cache_gather(
                    slots, s, s, c["k_cache"], c["v_cache"], stream=st)
                keep = torch.empty_like(k)
                out[f"gather {cache}, k_out given"] = lambda st, c=c, slots=slots, s=s, keep=keep: fp8kv.fp8kv_cache_gather(
                    slots, s, s, c["k_cache"], c["v_cache"], k_out=keep, stream=st)[1:]
            if cache == "e4m3":
                e = {**c, "k_scale": s.repeat(4), "v_scale": s.repeat(4)}
                out[f"per head M={M}"] = lambda st, e=e: (fp8kv.fp8kv_paged_attention_per_head(**e, stream=st),)
    g = gen.generator(9)
    q, k, v = (torch.randn((900, h, 128), generator=g).to(torch.bfloat16).cuda() for h in (18, 2, 2))
    cu = torch.tensor([0, 500, 900], dtype=torch.int32, device="cuda")
    out["prompt"] = lambda st: (fp8kv.fp8kv_prompt_attention(q, k, v, cu, 500, SM, stream=st),)
    return out


NAMES = [f"{a}{c} M={m}" for a in ("", "append ") for c in ("int4", "e4m3") for m in (1, 12)] + [
    f"gather {c}{x}" for c in ("int4", "e4m3") for x in ("", ", k_out given")] + ["per head M=1", "per head M=12", "prompt"]


@pytest.fixture(scope="module")
def calls():
    return _calls()


@pytest.mark.parametrize("name", NAMES)
def test_an_output_takes_no_memory_that_queued_work_still_writes(calls, name):
    """Blocks of the output's size, written by work queued on the current stream
    and dropped, while the call runs at once on a side stream."""
    call = calls[name]
    want = [o.clone() for o in call(None)]
    sizes = [o.untyped_storage().nbytes() for o in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(BUSY)
    for n in sizes:
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(7)       # queued behind the sleep, then free again
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_a_dropped_output_is_not_handed_out_while_the_call_runs(calls, name):
    call = calls[name]
    sizes = [o.untyped_storage().nbytes() for o in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    call(side)                                                          # its outputs are dropped here
    others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    assert all(bool((o == 7).all()) for o in others)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("cache,M", [("int4", 1), ("int4", 12), ("e4m3", 12)])
def test_prepared_call_on_another_stream_than_it_was_made_on(cache, M, raw):
    """Its own output and workspace were allocated from a block that work queued
    before still writes."""
    c, _ = _tensors(cache, M)
    want = fp8kv.fp8kv_paged_attention(**c, split_tokens=256).clone()
    n = want.untyped_storage().nbytes()
    need = fp8kv.fp8kv_paged_attention_workspace_size(2, M, 36, 4, 128, 32, 1500, -1, 256)
    assert need > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(BUSY)
    blocks = [torch.empty(b, dtype=torch.uint8, device="cuda").fill_(7) for b in (n, need)]
    del blocks
    call = fp8kv.PreparedAttention(**c, split_tokens=256)
    got = call(side.cuda_stream if raw else side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_prepared_call_dropped_while_it_runs_on_another_stream():
    c, _ = _tensors("int4", 12)
    call = fp8kv.PreparedAttention(**c, split_tokens=256)
    sizes = [call.out.untyped_storage().nbytes(), call._keep[7].numel()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        call()
    del call
    others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    assert all(bool((o == 7).all()) for o in others)


def test_prepared_call_captured_on_another_stream():
    c, _ = _tensors("int4", 1)
    want = fp8kv.fp8kv_paged_attention(**c).clone()
    call = fp8kv.PreparedAttention(**c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call()
    call.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(call.out, want)
    assert torch.equal(call(), want)


@pytest.mark.parametrize("raw", [False, True])
def test_layers_call_on_another_stream_than_it_was_made_on(raw):
    """The counters of its workspace are zero before the call, whatever was in
    the block and whatever the current stream still has to do."""
    layers = []
    for window in (-1, 511, -1):
        c, (k, v, _, _) = _tensors("e4m3", 12)
        new = [x[:24].view(2, 12, 4, 128).contiguous() for x in (k, v)]
        layers.append({**c, "window_left": window, "k_new": new[0], "v_new": new[1], "out": torch.empty_like(c["q"])})
    n = fp8kv.fp8kv_paged_attention_layers(layers).ws_bytes
    torch.cuda.synchronize()
    want = [d["out"].clone() for d in layers]
    for d in layers:
        d["out"].fill_(3.0)
    fp8kv.fp8kv_device_status(clear=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(BUSY)
    torch.empty(n, dtype=torch.uint8, device="cuda").fill_(7)
    fp8kv.fp8kv_paged_attention_layers(layers, stream=side.cuda_stream if raw else side)
    side.synchronize()
    torch.cuda.synchronize()
    assert fp8kv.fp8kv_device_status(clear=True) == 0
    assert all(torch.equal(d["out"], w) for d, w in zip(layers, want))

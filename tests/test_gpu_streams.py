"""GPU tests of calls with stream=: what a call allocates belongs to the stream it runs on, so that it shares no
memory with work still queued on another one."""
import pytest
import torch

from fp8_block_scaled_scales_b200 import binding

import plain_train as plain

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def segments_of(stream):
    """Address ranges that the allocator holds for this stream."""
    return [(s["address"], s["address"] + s["total_size"]) for s in torch.cuda.memory_snapshot()
            if s["stream"] == stream.cuda_stream]


def fresh_stream():
    """A side stream without cached memory, everything done before."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    return torch.cuda.Stream()


def route(T, k, G, seed):
    return torch.randint(0, G, (T, k), generator=torch.Generator().manual_seed(seed)).cuda()


def quantized(R, C, seed):
    x = torch.randn((R, C), generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()
    return binding.quantize_blockwise(x)


def sort_case(seed):
    ids, G = route(5000, 8, 64, seed), 64
    return lambda out, stream: binding.moe_sort(ids, G, *out, stream=stream)


def sort_masked_case(seed):
    ids, G = route(5000, 8, 64, seed), 64
    return lambda out, stream: binding.moe_sort_masked(ids, G, 700, *out, stream=stream)


def dispatch_case(seed, T=1100, k=8, G=16, H=7696):
    assert binding.lib().dg_moe_dispatch_workspace(T, k, H, plain.cap_of(T, k, G)) > 0
    x = torch.randn((T, H), generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()
    off, row, slot = binding.moe_sort(route(T, k, G, seed), G)
    cap = slot.numel()
    # rows past the last expert are not written: outputs of known content
    base = torch.zeros((cap, H), dtype=torch.uint8, device="cuda"), torch.zeros((cap // 128, -(-H // 128)), device="cuda")

    def call(out, stream):
        q, s = binding.moe_dispatch_quantize(x, slot, off, k, None, *out, stream=stream)
        used = int(off[-1]) if stream is None and not out else None
        return (q, s) if used is None else (torch.cat([q[:used], base[0][used:]]), torch.cat([s[:used // 128], base[1][used // 128:]]))
    call.base = base
    return call


def wgrad_case(seed, M=4096, N=272, K=400):
    assert binding.lib().dg_fp8_wgrad_workspace(M, N, K) > 0
    a = (*quantized(M, N, seed), *quantized(M, K, seed + 100))
    return lambda out, stream: (binding.wgrad_blockscaled(*a, *out, stream=stream),)


def dgrad_case(seed, M=37, N=4096, K=784):
    assert binding.lib().dg_fp8_dgrad_workspace(M, N, K) > 0
    a = (*quantized(M, N, seed), *quantized(N, K, seed + 100))
    return lambda out, stream: (binding.dgrad_blockscaled(*a, *out, stream=stream),)


WORKSPACE = [sort_case, sort_masked_case, dispatch_case, wgrad_case, dgrad_case]


@pytest.mark.parametrize("case", WORKSPACE)
def test_workspaces_belong_to_the_calls_stream(case):
    """With every output passed the workspace is all that the call allocates."""
    call = case(1)
    out = call((), None)
    side = fresh_stream()
    assert not segments_of(side)
    call(out, side)
    torch.cuda.synchronize()
    assert segments_of(side)


@pytest.mark.parametrize("first", WORKSPACE)
@pytest.mark.parametrize("second", WORKSPACE)
def test_calls_on_the_current_stream_and_on_another_at_once(first, second):
    """Calls on the current stream, then at once, with nothing waited for, others with stream=: each as if alone."""
    calls = [first(1), first(2), second(3), second(4)]
    want = [c((), None) for c in calls]
    outs = [[tuple(o.clone() for o in getattr(c, "base", w)) for _ in range(6)] for c, w in zip(calls, want)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(6):
        for c, o in zip(calls[:2], outs[:2]):
            c(o[i], None)
        for c, o in zip(calls[2:], outs[2:]):
            c(o[i], side)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for got in o:
            assert all(torch.equal(a, b) for a, b in zip(got, w))
    assert binding.last_device_status() == 0


def test_a_forked_stream_inside_a_capture():
    """A call with stream= on a stream forked into a captured graph, beside one on the capturing stream."""
    G, ids = 64, [route(5000, 8, 64, s) for s in (1, 2)]
    live = [t.clone() for t in ids]
    outs = [binding.moe_sort(t, G) for t in live]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        binding.moe_sort(live[0], G, *outs[0])
        binding.moe_sort(live[1], G, *outs[1], stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for a, b in ((0, 1), (1, 0)):
        live[0].copy_(ids[a])
        live[1].copy_(ids[b])
        graph.replay()
        torch.cuda.synchronize()
        for t, out in zip(live, outs):
            for x, y in zip(out, binding.moe_sort(t.clone(), G)):
                assert torch.equal(x, y)


def expert_layer_calls():
    """Every expert-layer and gradient call on a small problem: name -> call(stream)."""
    T, k, G, H, F = 40, 2, 3, 256, 128
    ids, x = route(T, k, G, 5), torch.randn((T, H)).to(BF16).cuda()
    off, row, slot = binding.moe_sort(ids, G)
    m, row_m, slot_m = binding.moe_sort_masked(ids, G, 40)
    cap = slot.numel()
    y, h = torch.zeros((cap, H), dtype=BF16, device="cuda"), torch.zeros((cap, 2 * F), dtype=BF16, device="cuda")
    hm = torch.zeros((G, 40, 2 * F), dtype=BF16, device="cuda")
    q, s, h8, sh = binding.swiglu_quantize(h, checkpoint=True)
    da = torch.zeros((cap, F), dtype=BF16, device="cuda")
    dy, dx, w = quantized(cap, H, 1), quantized(cap, F, 2), quantized(H, F, 3)
    wg = torch.zeros((G, H, F), dtype=torch.uint8, device="cuda"), torch.ones((G, H // 128, F // 128), device="cuda")
    return {
        "moe_sort": lambda st: binding.moe_sort(ids, G, stream=st),
        "moe_sort_masked": lambda st: binding.moe_sort_masked(ids, G, 40, stream=st),
        "moe_dispatch_quantize": lambda st: binding.moe_dispatch_quantize(x, slot, off, k, stream=st),
        "moe_dispatch_quantize_masked": lambda st: binding.moe_dispatch_quantize_masked(x, slot_m, m, k, stream=st),
        "moe_combine": lambda st: binding.moe_combine(y, row, stream=st),
        "moe_combine_backward": lambda st: binding.moe_combine_backward(x, y, row, stream=st),
        "swiglu_quantize": lambda st: binding.swiglu_quantize(h, off, checkpoint=True, stream=st),
        "swiglu_quantize_masked": lambda st: binding.swiglu_quantize_masked(hm, m, stream=st),
        "swiglu_quantize_backward": lambda st: binding.swiglu_quantize_backward(h8, sh, da, off, stream=st),
        "dgrad_blockscaled": lambda st: binding.dgrad_blockscaled(*dy, *w, stream=st),
        "wgrad_blockscaled": lambda st: binding.wgrad_blockscaled(*dy, *dx, stream=st),
        "grouped_dgrad_contiguous": lambda st: binding.grouped_dgrad_contiguous(*dy, *wg, off, stream=st),
        "grouped_wgrad_contiguous": lambda st: binding.grouped_wgrad_contiguous(*dy, *dx, off, stream=st),
    }


def assert_on(out, stream):
    for t in out if isinstance(out, tuple) else (out,):
        assert any(a <= t.data_ptr() < b for a, b in segments_of(stream)), "allocated for another stream"


def test_new_outputs_belong_to_the_calls_stream():
    calls = expert_layer_calls()
    side, here = fresh_stream(), torch.cuda.current_stream()
    for name, call in calls.items():
        assert_on(call(side), side)
        assert_on(call(None), here)
        assert torch.cuda.current_stream() == here, name
    torch.cuda.synchronize()


def test_the_current_stream_is_restored_after_a_refusal():
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    with pytest.raises(binding.DGError):
        binding.moe_sort(route(4, 2, 3, 1), 2000, stream=side)
    with pytest.raises(ValueError):
        binding.moe_sort(route(4, 2, 3, 1).float(), 3, stream=side)
    with pytest.raises(AttributeError):
        binding.moe_sort(route(4, 2, 3, 1), 3, stream=object())
    assert torch.cuda.current_stream() == here


def product_and_quantizer_calls():
    """The forward products and the quantizers on a small problem: name -> call(stream)."""
    x, xs = torch.randn((40, 256)).to(BF16).cuda(), torch.randn((3, 40, 256)).to(BF16).cuda()
    m = torch.tensor([40, 0, 7], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 128, 128, 384], dtype=torch.int32, device="cuda")
    a, b, a1 = quantized(40, 256, 1), quantized(128, 256, 2), binding.quantize_1x128(x)
    rows, masked = quantized(384, 256, 3), binding.quantize_blockwise_masked(xs, m)
    wg = torch.zeros((3, 128, 256), dtype=torch.uint8, device="cuda"), torch.ones((3, 1, 2), device="cuda")
    return {
        "quantize_blockwise": lambda st: binding.quantize_blockwise(x, stream=st),
        "quantize_blockwise_masked": lambda st: binding.quantize_blockwise_masked(xs, m, stream=st),
        "quantize_1x128": lambda st: binding.quantize_1x128(x, stream=st),
        "gemm_blockscaled": lambda st: binding.gemm_blockscaled(*a, *b, stream=st),
        "gemm_blockscaled_bf16a": lambda st: binding.gemm_blockscaled_bf16a(x, *b, stream=st),
        "gemm_1x128": lambda st: binding.gemm_1x128(*a1, *b, stream=st),
        "grouped_gemm_contiguous": lambda st: binding.grouped_gemm_contiguous(*rows, *wg, off, stream=st),
        "grouped_gemm_masked": lambda st: binding.grouped_gemm_masked(*masked, *wg, m, stream=st),
    }


def test_new_outputs_of_products_and_quantizers_belong_to_the_calls_stream():
    calls = product_and_quantizer_calls()
    side, here = fresh_stream(), torch.cuda.current_stream()
    for name, call in calls.items():
        assert_on(call(side), side)
        assert_on(call(None), here)
        assert torch.cuda.current_stream() == here, name
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["quantize_blockwise_masked", "grouped_gemm_masked"])
def test_zero_fill_comes_before_the_kernel(name):
    """The masked calls fill a new output before their kernel writes the tokens' rows, also while the current
    stream is busy."""
    call = product_and_quantizer_calls()[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # about 10 ms of work queued on the current stream
    got = call(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want) if isinstance(want, tuple) else ((got, want),):
        assert torch.equal(a, b)


def test_a_stream_of_another_library():
    """Anything with a cuda_stream handle is a stream."""
    class Handle:
        cuda_stream = torch.cuda.Stream().cuda_stream
    x = torch.randn((40, 256)).to(BF16).cuda()
    want = binding.quantize_blockwise(x)
    torch.cuda.synchronize()
    got = binding.quantize_blockwise(x, stream=Handle())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

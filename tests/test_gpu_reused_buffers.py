"""GPU tests of calls queued back to back that read a buffer, write it anew and read it again: a kernel may start
before the one ahead of it has finished, and has to see what that one wrote all the same."""
import pytest
import torch

from fp8_block_scaled_scales_b200 import binding

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
ROUNDS = 40


def run(produce, consume, sets, outs):
    """For each output in turn: produce from a set into the shared buffers, consume from them into the output."""
    for i, out in enumerate(outs):
        produce(sets[i % len(sets)])
        consume(out)


def check(produce, consume, sets, new_out):
    """Queued one after another, and captured and replayed: every output is what its own set gives alone."""
    want = []
    for s in sets:
        produce(s)
        out = new_out()
        consume(out)
        torch.cuda.synchronize()
        want.append(out)
    outs = [new_out() for _ in range(ROUNDS)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    for repeat in range(3):
        if repeat < 2:
            run(produce, consume, sets, outs)
        else:
            with torch.cuda.graph(graph):
                run(produce, consume, sets, outs)
            graph.replay()
        torch.cuda.synchronize()
        for i, out in enumerate(outs):
            for a, b in zip(out, want[i % len(sets)]):
                assert torch.equal(a, b), (repeat, i)
                a.zero_()
        torch.cuda.synchronize()


def routes(T, k, G, n=3):
    return [torch.randint(0, G, (T, k), generator=torch.Generator().manual_seed(s)).cuda() for s in range(n)]


@pytest.mark.parametrize("T,k,G,H", [(16, 8, 64, 2048), (64, 8, 64, 7168), (300, 2, 8, 4096), (3000, 2, 8, 1024)])
def test_sort_then_dispatch(T, k, G, H):
    ids, x = routes(T, k, G), torch.randn((T, H)).to(BF16).cuda()
    off, row, slot = binding.moe_sort(ids[0], G)
    cap = slot.numel()

    def new_out():
        return torch.zeros((cap, H), dtype=torch.uint8, device="cuda"), torch.zeros((cap // 128, -(-H // 128)), device="cuda")

    check(lambda s: binding.moe_sort(s, G, off, row, slot),
          lambda out: binding.moe_dispatch_quantize(x, slot, off, k, None, *out), ids, new_out)


@pytest.mark.parametrize("T,k,G,H,m_max", [(1, 8, 64, 7168, 128), (64, 8, 64, 2048, 64), (300, 2, 8, 4096, 300)])
def test_masked_sort_then_dispatch(T, k, G, H, m_max):
    ids, x = routes(T, k, G), torch.randn((T, H)).to(BF16).cuda()
    m, row, slot = binding.moe_sort_masked(ids[0], G, m_max)

    def new_out():
        return (torch.zeros((G, m_max, H), dtype=torch.uint8, device="cuda"),
                torch.zeros((G, -(-m_max // 128), -(-H // 128)), device="cuda"))

    check(lambda s: binding.moe_sort_masked(s, G, m_max, m, row, slot),
          lambda out: binding.moe_dispatch_quantize_masked(x, slot, m, k, *out), ids, new_out)


@pytest.mark.parametrize("T,k,G,H", [(16, 8, 64, 2048), (300, 2, 8, 4096), (3000, 2, 8, 1024)])
def test_sort_then_combine(T, k, G, H):
    ids = routes(T, k, G)
    off, row, slot = binding.moe_sort(ids[0], G)
    y = torch.randn((slot.numel(), H)).to(BF16).cuda()
    check(lambda s: binding.moe_sort(s, G, off, row, slot), lambda out: binding.moe_combine(y, row, out=out[0]), ids,
          lambda: (torch.zeros((T, H), dtype=BF16, device="cuda"),))


@pytest.mark.parametrize("M,F", [(64, 1024), (300, 2048), (2000, 1024)])
def test_swiglu_then_its_backward(M, F):
    hs = [(torch.randn((M, 2 * F), generator=torch.Generator().manual_seed(s))).to(BF16).cuda() for s in range(3)]
    da = torch.randn((M, F)).to(BF16).cuda()
    q, s, h8, sh = binding.swiglu_quantize(hs[0], checkpoint=True)
    check(lambda h: binding.swiglu_quantize(h, None, True, q, s, h8, sh),
          lambda out: binding.swiglu_quantize_backward(h8, sh, da, None, *out), hs,
          lambda: (torch.zeros((M, 2 * F), dtype=torch.uint8, device="cuda"), torch.zeros((-(-M // 128), 2 * F // 128), device="cuda")))


@pytest.mark.parametrize("M,N,K", [(128, 512, 256), (1000, 528, 784), (4096, 256, 256)])
def test_quantizer_then_gradient_products(M, N, K):
    xs = [torch.randn((M, N), generator=torch.Generator().manual_seed(s)).to(BF16).cuda() for s in range(3)]
    q, s = binding.quantize_blockwise(xs[0])
    x, w = (binding.quantize_blockwise(torch.randn(n, K).to(BF16).cuda()) for n in (M, N))
    check(lambda v: binding.quantize_blockwise(v, q, s), lambda out: binding.wgrad_blockscaled(q, s, *x, C=out[0]), xs,
          lambda: (torch.zeros((N, K), device="cuda"),))
    check(lambda v: binding.quantize_blockwise(v, q, s), lambda out: binding.dgrad_blockscaled(q, s, *w, C=out[0]), xs,
          lambda: (torch.zeros((M, K), dtype=BF16, device="cuda"),))

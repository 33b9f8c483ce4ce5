"""A mixture-of-experts layer's training step and decode step through the calls together, as
a user makes them: against a float64 layer, captured and replayed, and the two layouts
against each other."""
import numpy as np
import pytest
import torch

from fp8_block_scaled_scales_b200 import binding as dg

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


class Layer:
    """Weights quantized once: W1 [G][2F][H], W2 [G][H][F]."""

    def __init__(self, G, H, F, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.G, self.H, self.F = G, H, F
        self.w1 = (torch.randn((G, 2 * F, H), generator=g, device="cuda") * H ** -0.5).to(BF16)
        self.w2 = (torch.randn((G, H, F), generator=g, device="cuda") * F ** -0.5).to(BF16)
        q, s = dg.quantize_blockwise(self.w1.view(G * 2 * F, H))
        self.q1, self.s1 = q.view(G, 2 * F, H), s.view(G, 2 * F // 128, -1)
        q, s = dg.quantize_blockwise(self.w2.view(G * H, F))
        self.q2, self.s2 = q.view(G, H, F), s.view(G, H // 128, -1)

    def forward(self, x, ids, weights):
        k = ids.shape[1]
        off, row, slot = dg.moe_sort(ids, self.G)
        xq, sx = dg.moe_dispatch_quantize(x, slot, off, k)
        h = dg.grouped_gemm_contiguous(xq, sx, self.q1, self.s1, off)
        aq, sa, h8, sh = dg.swiglu_quantize(h, off, checkpoint=True)
        y = dg.grouped_gemm_contiguous(aq, sa, self.q2, self.s2, off)
        out = dg.moe_combine(y, row, weights)
        return out, (off, row, slot, xq, sx, aq, sa, h8, sh, y, weights)

    def backward(self, dout, saved, dw1=None, dw2=None):
        off, row, slot, xq, sx, aq, sa, h8, sh, y, weights = saved
        k = row.shape[1]
        dweights = dg.moe_combine_backward(dout, y, row)
        dyq, sdy = dg.moe_dispatch_quantize(dout, slot, off, k, weights=weights)
        acc = dw1 is not None
        dw2 = dg.grouped_wgrad_contiguous(dyq, sdy, aq, sa, off, C=dw2, accumulate=acc)
        da = dg.grouped_dgrad_contiguous(dyq, sdy, self.q2, self.s2, off)
        dhq, sdh = dg.swiglu_quantize_backward(h8, sh, da, off)
        dw1 = dg.grouped_wgrad_contiguous(dhq, sdh, xq, sx, off, C=dw1, accumulate=acc)
        dxr = dg.grouped_dgrad_contiguous(dhq, sdh, self.q1, self.s1, off)
        return dg.moe_combine(dxr, row), dweights, dw1, dw2

    def decode(self, x, ids, weights, m_max):
        k = ids.shape[1]
        m, row, slot = dg.moe_sort_masked(ids, self.G, m_max)
        xq, sx = dg.moe_dispatch_quantize_masked(x, slot, m, k)
        h = dg.grouped_gemm_masked(xq, sx, self.q1, self.s1, m)
        aq, sa = dg.swiglu_quantize_masked(h, m)
        return dg.moe_combine(dg.grouped_gemm_masked(aq, sa, self.q2, self.s2, m), row, weights)

    def exact(self, x, ids, weights, dout):
        """(out, dx, dweights, dW1, dW2) of the unquantized layer, float64, by differentiation."""
        x, w = x.double().requires_grad_(True), weights.double().requires_grad_(True)
        w1, w2 = self.w1.double().requires_grad_(True), self.w2.double().requires_grad_(True)
        out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for e in range(self.G):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if t.numel():
                h = x[t] @ w1[e].t()
                a = torch.nn.functional.silu(h[:, :self.F]) * h[:, self.F:]
                out = out.index_add(0, t, (a @ w2[e].t()) * w[t, j][:, None])
        return (out.detach(), *torch.autograd.grad(out, (x, w, w1, w2), dout.double()))


def batch(T, H, G, k, seed, drop=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, H), generator=g, device="cuda").to(BF16)
    ids = torch.rand((T, G), generator=g, device="cuda").topk(k, 1)[1]
    if drop:
        ids[torch.rand((T, k), generator=g, device="cuda") < drop] = -1
    w = torch.rand((T, k), generator=g, device="cuda") + 0.1
    dout = (torch.randn((T, H), generator=g, device="cuda") * 1e-3).to(BF16)
    return x, ids, w, dout


@pytest.mark.parametrize("T,k,G,H,F,drop", [(300, 2, 6, 512, 256, 0.0), (1, 1, 3, 128, 128, 0.0), (700, 4, 9, 384, 384, 0.2),
                                            (40, 2, 64, 256, 128, 0.0)])
def test_training_step_against_the_unquantized_layer(T, k, G, H, F, drop):
    layer = Layer(G, H, F)
    x, ids, w, dout = batch(T, H, G, k, T + G, drop)
    out, saved = layer.forward(x, ids, w)
    dx, dw, dw1, dw2 = layer.backward(dout, saved)
    assert dg.last_device_status() == 0
    want = layer.exact(x, ids, w, dout)
    # A quantization moves a value by at most 2^-4 of itself (2^-10 of its block's scale below
    # E4M3's normal range, smaller still in the norm).  Along the longest path to each result:
    # out 4 of them (x, W1, a, W2); dweights the same; dW2 5 (dout, and a's three and its own);
    # dx and dW1 7 (dout, W2, h's two and its checkpoint, dh, and W1 or x); the SwiGLU between
    # stretches an error at most twice here.  Independent errors add up far below the sum.
    for got, ref, n, what in zip((out, dx, dw, dw1, dw2), want, (4, 7, 4, 7, 5), ("out", "dx", "dweights", "dW1", "dW2")):
        err = float((got.double() - ref).norm() / ref.norm().clamp_min(1e-300))
        assert err <= 2 * n * 2.0 ** -4, f"{what}: relative error {err:.3g}"
    # accumulation: a second step's gradients on top
    first1, first2 = dw1.clone(), dw2.clone()
    layer.backward(dout, saved, dw1, dw2)
    assert torch.equal(dw1, 2 * first1) and torch.equal(dw2, 2 * first2)


def test_training_step_captured_and_replayed():
    """A step captured once and replayed on other tokens and routing equals the eager calls, bit for bit."""
    layer = Layer(8, 512, 256)
    x, ids, w, dout = batch(1500, 512, 8, 2, 1)  # past one CTA's slots: the sort has a workspace

    def step():
        out, saved = layer.forward(x, ids, w)
        return (out, *layer.backward(dout, saved))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = step()
    for seed in (2, 3):
        for a, b in zip((x, ids, w, dout), batch(1500, 512, 8, 2, seed, 0.1 * seed)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in static]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    assert dg.last_device_status() == 0


@pytest.mark.parametrize("T,k,G,m_max", [(1, 1, 4, 128), (1, 4, 8, 128), (37, 2, 8, 128), (400, 2, 4, 384)])
def test_decode_step_equals_the_contiguous_layout_bitwise(T, k, G, m_max):
    """The same tokens through the masked slabs: an expert's rows form the same 128-row blocks."""
    layer = Layer(G, 256, 128)
    x, ids, w, _ = batch(T, 256, G, k, T)
    out, saved = layer.forward(x, ids, w)
    got = layer.decode(x, ids, w, m_max)
    assert dg.last_device_status() == 0
    assert int((saved[0][1:] - saved[0][:-1]).max()) <= m_max  # nothing was dropped
    assert torch.equal(out, got)


def test_decode_step_drops_what_does_not_fit():
    """A slab of 16 rows: the first 16 slots of an expert are computed, the others add nothing."""
    layer = Layer(2, 128, 128)
    x, _, w, _ = batch(40, 128, 2, 1, 5)
    ids = torch.zeros((40, 1), dtype=torch.int32, device="cuda")
    got = layer.decode(x, ids, w, 16)
    full = layer.decode(x[:16].contiguous(), ids[:16], w[:16].contiguous(), 16)
    assert torch.equal(got[:16], full) and not bool(got[16:].any())


def test_a_batch_without_tokens():
    layer = Layer(3, 128, 128)
    x, w = torch.empty((0, 128), dtype=BF16, device="cuda"), torch.empty((0, 2), device="cuda")
    out, saved = layer.forward(x, torch.empty((0, 2), dtype=torch.int64, device="cuda"), w)
    dx, dw, dw1, dw2 = layer.backward(x, saved)
    assert out.shape == (0, 128) and dx.shape == (0, 128) and dw.shape == (0, 2)
    assert not bool(dw1.any()) and not bool(dw2.any())
    assert dg.last_device_status() == 0


def test_all_slots_dropped():
    layer = Layer(3, 128, 128)
    x, ids, w, dout = batch(50, 128, 3, 2, 9)
    out, saved = layer.forward(x, torch.full_like(ids, -1), w)
    dx, dw, dw1, dw2 = layer.backward(dout, saved)
    assert not any(bool(t.any()) for t in (out, dx, dw, dw1, dw2))
    assert dg.last_device_status() == 0


def test_two_steps_on_two_streams():
    """Independent steps at once, each on its own stream, equal the same steps one after the other."""
    layer = Layer(4, 256, 128)
    data = [batch(2100, 256, 4, 2, s) for s in (1, 2)]
    alone = []
    for x, ids, w, dout in data:
        out, saved = layer.forward(x, ids, w)
        alone.append((out, *layer.backward(dout, saved)))
    torch.cuda.synchronize()
    got = []
    for x, ids, w, dout in data:
        with torch.cuda.stream(torch.cuda.Stream()):
            out, saved = layer.forward(x, ids, w)
            got.append((out, *layer.backward(dout, saved), saved))
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        for s, t in zip(a, b):
            assert torch.equal(s, t)


def test_offsets_without_an_expert_are_refused():
    """An empty tensor has no address; it must not be taken for "no offsets", which means all rows."""
    codes = torch.zeros((128, 128), dtype=torch.uint8, device="cuda")
    one = torch.ones((1, 1), device="cuda")
    h = torch.zeros((128, 256), dtype=torch.bfloat16, device="cuda")
    for n in (0, 1):
        off = torch.zeros(n, dtype=torch.int32, device="cuda")
        with pytest.raises(ValueError):
            dg.swiglu_quantize(h, offsets=off)
        with pytest.raises(ValueError):
            dg.swiglu_quantize_backward(h.to(torch.float8_e4m3fn), torch.ones((2, 128), device="cuda"),
                                        h[:, :128].contiguous(), offsets=off)
        with pytest.raises(ValueError):
            dg.grouped_dgrad_contiguous(codes, one, codes, one, off)
        with pytest.raises(ValueError):
            dg.grouped_wgrad_contiguous(codes, one, codes, one, off)

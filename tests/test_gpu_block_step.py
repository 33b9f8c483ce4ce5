"""A block's training and decode steps through the calls together, as a user makes them: the norm
before it, routing, the expert layer, the norm after it with its gate and residual, the gradients
of all of these and their clipping; against float64 differentiation, and captured and replayed."""
import pytest
import torch

from fp8_block_scaled_scales_b200 import binding as dg

import plain_step as plain
from plain_step import BF, U
from test_gpu_expert_layer import Layer

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPS, ALPHA, SCALE, COEF = 1e-6, 0.5, 1.5, 0.01


class Block:
    """An expert layer between its norms: the residual stream x0 and the layer before's y0 come in."""

    def __init__(self, G, H, F, k, score="sigmoid"):
        g = torch.Generator(device="cuda").manual_seed(G + H)

        def vector(mean):
            return mean + 0.1 * torch.randn((H,), generator=g, device="cuda")

        self.layer, self.k, self.score = Layer(G, H, F), k, score
        self.router = torch.randn((G, H), generator=g, device="cuda") * H ** -0.5
        self.bias = (torch.rand((G,), generator=g, device="cuda") - 0.5) * 0.2
        self.before, self.after, self.post, self.gate = vector(1.0), vector(1.0), vector(1.0), vector(0.5)

    def logits(self, n):
        return (n.float()[:, None, :] * self.router).sum(2)  # the same bits in a graph and out of it

    def route(self, z, **kw):
        return dg.moe_route(z, self.k, score=self.score, bias=self.bias, scale=SCALE, **kw)

    def forward(self, x0, y0, mask=None):
        n0, r0, rstd0, _ = dg.rmsnorm_residual(x0, self.before, y=y0, alpha=ALPHA, eps=EPS)
        z = self.logits(n0)
        ids, w, counts, loss, dprob = self.route(z, mask=mask, balance=True)
        out, saved = self.layer.forward(n0, ids, w)
        n1, r1, rstd1, rstd_y = dg.rmsnorm_residual(r0, self.after, y=out, gate=self.gate, post_weight=self.post, eps=EPS)
        return n1, r1, loss, counts, (n0, r0, rstd0, z, ids, w, dprob, out, saved, r1, rstd1, rstd_y)

    def backward(self, dn1, dr1, dloss, kept, y0):
        n0, r0, rstd0, z, ids, w, dprob, out, saved, r1, rstd1, rstd_y = kept
        dr0, dout, dafter, dgate, dpost = dg.rmsnorm_residual_backward(
            dn1, r1, rstd1, self.after, dr=dr1, y=out, rstd_y=rstd_y, gate=self.gate, post_weight=self.post)
        dn0, dw, dw1, dw2 = self.layer.backward(dout, saved)
        dz = dg.moe_route_backward(z, ids, dw, dprob, dloss, score=self.score, scale=SCALE)
        drouter = (dz[:, :, None] * n0.float()[:, None, :]).sum(0)
        dn0 = (dn0.float() + (dz[:, :, None] * self.router).sum(1)).to(BF16)
        dx0, dy0, dbefore, _, _ = dg.rmsnorm_residual_backward(dn0, r0, rstd0, self.before, dr=dr0, y=y0, alpha=ALPHA)
        return dx0, dy0, dout, dw, dz, [dafter, dgate, dpost, dbefore, drouter, dw1, dw2]

    def step(self, x0, y0, dn1, dr1, dloss, max_norm, mask=None):
        n1, r1, loss, counts, kept = self.forward(x0, y0, mask)
        dx0, dy0, _, _, _, grads = self.backward(dn1, dr1, dloss, kept, y0)
        norm = dg.clip_grad_norm(grads, max_norm)
        return n1, r1, loss, counts, dx0, dy0, norm, *grads


def batch(T, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(std):
        return (torch.randn((T, H), generator=g, device="cuda") * std).to(BF16)

    return rand(1.5), rand(0.7), rand(1e-3), rand(1e-3)


@pytest.mark.parametrize("T,G,H,F,k,score", [(300, 6, 256, 128, 2, "sigmoid"), (1, 3, 128, 128, 1, "softmax"),
                                             (517, 40, 384, 128, 4, "softmax")])
def test_training_step_against_differentiation(T, G, H, F, k, score):
    """From the expert rows y on: combination, norm, loss and routing in float64, differentiated at the
    BF16 numbers that the calls passed on."""
    b = Block(G, H, F, k, score)
    x0, y0, dn1, dr1 = batch(T, H, T)
    mask = torch.arange(T, device="cuda") % 9 != 5
    dloss = torch.tensor(COEF, device="cuda")
    n1, r1, loss, counts, kept = b.forward(x0, y0, mask)
    n0, r0, rstd0, z, ids, w, dprob, out, saved, _, rstd1, rstd_y = kept
    dx0, dy0, dout, dw, dz, grads = b.backward(dn1, dr1, dloss, kept, y0)
    row, y = saved[1], saved[9]
    assert not bool((ids[~mask] >= 0).any()) and not bool(w[~mask].any()) and not bool(out[~mask].any())
    assert torch.equal(counts.cpu().long(), plain.balance(z.double().cpu(), ids.cpu().long(), score)[0])

    ok = (ids >= 0)
    rows = torch.where(ok[:, :, None], y.double()[row.long().clamp_min(0)], torch.zeros((), dtype=torch.float64, device="cuda"))

    def at(value, given):  # value's derivative at the number that was passed on
        return value + (given.double() - value).detach()

    with torch.enable_grad():
        z64 = z.double().requires_grad_(True)
        rows.requires_grad_(True)
        x64, gate, post, after = (t.double().requires_grad_(True) for t in (r0, b.gate, b.post, b.after))
        w64 = plain.weights(z64, ids.long(), score, True, SCALE)
        w_given = at(w64, w)
        o = at((rows * w_given[:, :, None]).sum(1), out)
        o.retain_grad()
        w_given.retain_grad()
        rsy = (o.pow(2).mean(1, keepdim=True) + EPS).pow(-0.5)
        r = at(x64 + gate * (o * rsy * post), r1)
        n = r * (r.pow(2).mean(1, keepdim=True) + EPS).pow(-0.5) * after
        p = plain.probabilities(z64, score)[1] * ok.any(1, keepdim=True)
        routed = int(ok.any(1).sum())
        balance = (p * (counts.double() * G / (k * routed * routed))).sum()
        ((n * dn1.double()).sum() + (r * dr1.double()).sum() + COEF * balance).backward()
    balance = balance.detach()
    assert abs(float(loss) - float(balance)) <= (2 * float(plain.spread(z.double()).max()) + 128 + T / 16) * U * float(balance)

    # the norm's gradient: its own bounds, the row's rstd taken from r before its rounding to BF16,
    # which moves it by half a step at most, as that moves r
    want = plain.norm_backward(dn1.double(), dr1.double(), r1.double(), rstd1.double(), out.double(), rstd_y.double(),
                               b.after.double(), b.post.double(), b.gate.double(), 1.0)
    shift = 4 * BF  # three factors of rstd in the correction term, one in the other
    for got, name, exact in ((grads[0], "dweight", after.grad), (grads[1], "dgate", gate.grad), (grads[2], "dpost_weight", post.grad),
                             (dout, "dy", o.grad)):
        ref, bound = want[name]
        half = BF if got.dtype == BF16 else U
        assert ((got.double() - ref).abs() <= bound * (1 + half) + half * ref.abs() + 2.0 ** -126).all(), name
        assert float((got.double() - exact).norm()) <= (shift + half) * float(exact.norm()) + 2.0 ** -126, name
    # dout enters the weights' gradient after its rounding, and with what the norm's gradient was off by
    off = (dout.double() - o.grad).abs()
    wbound = (off[:, None, :] * rows.detach().abs()).sum(2) + H * U * (dout.double()[:, None, :] * rows.detach()).abs().sum(2)
    assert ((dw.double() - w_given.grad).abs()[ok] <= wbound[ok] + 2.0 ** -126).all()
    # and these the logits' gradient: through its linear form, whose magnitudes bound it
    ids64 = ids.cpu().long()
    through = plain.route_backward(z.double().cpu(), ids64, wbound.detach().cpu(), None, None, score, True, SCALE)[1]
    mag = plain.route_backward(z.double().cpu(), ids64, dw.double().cpu(), dprob.double().cpu(), dloss.double().cpu(), score,
                               True, SCALE)[1]
    rel = (4 * plain.spread(z.double().cpu()) + 192) * U
    assert ((dz.cpu().double() - z64.grad.cpu()).abs() <= through + rel * mag + U * z64.grad.cpu().abs() + 2.0 ** -126).all()

    # all gradients clipped together
    norm64 = sum(float((t.double() ** 2).sum()) for t in grads) ** 0.5
    before = [t.clone() for t in grads]
    norm = dg.clip_grad_norm(grads, norm64 / 3)
    assert abs(float(norm) - norm64) <= 20 * U * norm64
    for t, first in zip(grads, before):
        assert ((t.double() - first.double() / 3).abs() <= 24 * U * first.double().abs() + 2.0 ** -126).all()
    assert dg.last_device_status() == 0


@pytest.mark.parametrize("T,k", [(900, 2), (64, 3)])
def test_training_step_captured_and_replayed(T, k):
    """A step captured once and replayed on other tokens, padding and gradients equals the eager
    calls, bit for bit; eager steps run between the replays."""
    b = Block(8, 256, 128, k)
    x0, y0, dn1, dr1 = batch(T, 256, 1)
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    dloss = torch.tensor(COEF, device="cuda")

    def step():
        return b.step(x0, y0, dn1, dr1, dloss, 1e-3, mask)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = step()
    for seed in (2, 3):
        for a, fresh in zip((x0, y0, dn1, dr1), batch(T, 256, seed)):
            a.copy_(fresh)
        mask.copy_(torch.arange(T, device="cuda") < T - 7 * seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in static]
        for a, want in zip(got, step()):
            assert torch.equal(a, want)
        assert float(got[6]) > 1e-3  # clipped
    assert dg.last_device_status() == 0


@pytest.mark.parametrize("T", [1, 5, 130])
def test_decode_step_gives_the_training_steps_tokens(T):
    """Single tokens through the masked layout, routed without counts: the same bits as the training form."""
    G, H, F, k = 16, 256, 128, 4
    b = Block(G, H, F, k)
    x0, y0, _, _ = batch(T, H, T)
    n1, r1, _, _, kept = b.forward(x0, y0)
    n0, r0, _, _ = dg.rmsnorm_residual(x0, b.before, y=y0, alpha=ALPHA, eps=EPS)
    ids, w = b.route(b.logits(n0))
    out = b.layer.decode(n0, ids, w, 256)
    r = torch.empty_like(r0)
    n, _, _, _ = dg.rmsnorm_residual(r0, b.after, y=out, gate=b.gate, post_weight=b.post, eps=EPS, r=r)
    for a, want in ((ids, kept[4]), (w, kept[5]), (out, kept[7]), (n, n1), (r, r1)):
        assert torch.equal(a, want)
    # the next block's dense projection from the codes of the same norm
    q, s, r2 = dg.rmsnorm_residual_quantize(r0, b.after, y=out, gate=b.gate, post_weight=b.post, eps=EPS)
    assert torch.equal(r2, r1)
    wq, ws = dg.quantize_blockwise(b.layer.w1[0])
    c = dg.gemm_1x128(q, s, wq, ws)
    ref = (q.view(torch.float8_e4m3fn).double() * s.double().t().repeat_interleave(128, 1)) @ (
        wq.view(torch.float8_e4m3fn).double() * ws.double().repeat_interleave(128, 0).repeat_interleave(128, 1)).t()
    assert float((c.double() - ref).abs().max()) <= float(BF * ref.abs().max() + 1e-3 * ref.pow(2).mean().sqrt())
    assert dg.last_device_status() == 0

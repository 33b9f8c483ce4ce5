"""GPU tests of routing, the norms around a block and clipping where a call is allowed but unusual:
few experts beside other work, rows that reach no expert, extreme magnitudes, gradients given by
an iterator."""
import math
import weakref

import pytest
import torch

from fp8_block_scaled_scales_b200 import binding

import plain_step as plain
from plain_step import BF, U
from test_gpu_route import check, check_backward

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


def logits(T, G, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, G), generator=g) * 1.5 + torch.randn((G,), generator=g) * 0.5


@pytest.mark.parametrize("G", [1, 8, 32, 33, 64, 256, 300])
def test_balance_loss_of_few_experts_beside_other_work(G):
    """Most CTAs of the cluster that adds up the parts have no expert, and other kernels keep the SMs busy, so that
    its CTAs begin apart: the loss of every call is the same and that of the definition."""
    T, k = 4096, min(G, 2)
    z = logits(T, G, G)
    zc, other = z.cuda(), torch.randn((2048, 2048), device="cuda")
    beside, s = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    with torch.cuda.stream(beside):
        for _ in range(40):
            other = (other @ other).clamp_(-1, 1)
    for _ in range(40):
        outs.append(binding.moe_route(zc, k, balance=True, stream=s))
    torch.cuda.synchronize()
    ids = outs[0][0].cpu().long()
    counts, loss, dprob = plain.balance(z.double(), ids, "softmax")
    # numerator and denominator: exponentials off by 2 + 1.2 |x| whole steps, the denominator's 40 additions; a
    # reciprocal; then up to 2 + 32 additions of positive terms in float32 (148 CTAs of 28 warps), the rest in float64
    top = float(plain.spread(z.double()).max())
    for out in outs:
        for a, b in zip(out, outs[0]):
            assert torch.equal(a, b)
    assert torch.equal(outs[0][2].cpu().long(), counts)
    assert ((outs[0][4].cpu().double() - dprob).abs() <= 2 * U * dprob).all()
    assert abs(float(outs[0][3]) - float(loss)) <= (2 * (2.4 * top + 4) + 40 + 2 + 34 + 2) * U * float(loss)


class WatchedStream:
    """A stream that counts, when a call asks for its handle, which of some tensors are still there."""

    def __init__(self, stream):
        self.stream, self.made, self.alive = stream, [], None

    def yielding(self, tensors):
        for t in tensors:
            t = t.clone()
            self.made.append(weakref.ref(t))
            yield t
            del t
        self.stream.wait_stream(torch.cuda.current_stream())

    @property
    def cuda_stream(self):
        self.alive = sum(r() is not None for r in self.made)
        return self.stream.cuda_stream


def test_gradients_that_only_an_iterator_holds():
    """The call keeps them: their memory is neither its workspace nor its outputs, on any stream."""
    g = torch.Generator(device="cuda").manual_seed(1)
    # some as large as the workspace, some as the norm
    grads = [torch.randn((n,), generator=g, device="cuda") for n in [1184] * 30 + [1, 128] * 10 + [300000]]
    norm = binding.grad_norm(grads)
    clipped = [torch.empty_like(t) for t in grads]
    binding.clip_grad_norm(grads, 0.5, out=clipped)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (torch.cuda.current_stream(), side):
        for _ in range(5):
            outs = [torch.zeros_like(t) for t in grads]
            torch.cuda.synchronize()
            w = WatchedStream(stream)
            assert torch.equal(binding.grad_norm(w.yielding(grads), stream=w).cpu(), norm.cpu())
            assert w.alive == len(grads) and all(r() is None for r in w.made)
            stream.synchronize()
            w = WatchedStream(stream)
            binding.clip_grad_norm(w.yielding(grads), 0.5, out=(t for t in outs), stream=w)
            assert w.alive == len(grads)
            stream.synchronize()
            for a, b in zip(outs, clipped):
                assert torch.equal(a, b)
            outs = [t.clone() for t in grads]
            torch.cuda.synchronize()
            binding.grad_clip(iter(outs), norm, 0.5, stream=stream)  # in place
            stream.synchronize()
            for a, b in zip(outs, clipped):
                assert torch.equal(a, b)


def test_an_iterator_that_changes_the_other_sequence():
    grads = [torch.ones(8, device="cuda"), torch.ones(3, device="cuda")]
    outs = [torch.zeros(8, device="cuda"), torch.zeros(3, device="cuda")]

    def dropping():
        for t in outs:
            grads.clear()
            yield t

    with pytest.raises(ValueError):
        binding.clip_grad_norm(grads, 1.0, out=dropping())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,G", [(40, 40), (60, 24), (3000, 40), (2500, 200), (700, 300), (300, 600)])
def test_tokens_that_reach_no_expert_stay_out_of_the_balance_loss(T, G, score):
    """Rows of nothing but NaN and -inf, and rows whose finite logits are those of experts that the bias takes out: no
    expert, no share in the loss, no gradient; in one cluster and over the whole GPU."""
    k = 6
    z = logits(T, G, T + G)
    gone = torch.arange(G) % 5 == 2        # by their bias
    z[3] = NAN
    z[5, ::2], z[5, 1::2] = NAN, -INF
    z[7] = -INF
    z[9, ~gone] = -INF                     # finite only where the bias takes the expert out
    z[11, ~gone] = -INF
    z[11, 2] = 80.0                        # a large share of one expert
    z[13, ~gone] = -INF
    z[13, 4] = 0.25                        # one expert is left
    z[15, gone] = -INF
    bias = (torch.rand((G,), generator=torch.Generator().manual_seed(G)) - 0.5) * 0.3
    bias[gone] = -INF
    bias[7] = NAN
    mask = torch.arange(T) % 11 != 4
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(T))
    for kw in (dict(), dict(renormalize=False, mask=mask), dict(bias=bias), dict(bias=bias, mask=mask, renormalize=False, scale=2.5)):
        ids = check(z, k, score, **kw)
        none = [3, 5, 7] + ([9, 11] if "bias" in kw else [])
        assert (ids.cpu()[none] == -1).all()
        dz = check_backward(z, k, score, kw.get("renormalize", True), dw, mask=kw.get("mask"), ids=ids)
        assert not dz.cpu()[none].any()
    # nothing but such rows
    lost = z[[3, 5, 7, 9, 11]].repeat(T // 5, 1)
    ids, w, counts, loss, dprob = binding.moe_route(lost.cuda(), k, score=score, bias=bias.cuda(), balance=True)
    assert bool((ids == -1).all()) and not w.any() and not counts.any() and not dprob.any() and float(loss) == 0.0
    # a softmax's sum is NaN with a single NaN, and with a bias so are all keys
    if score == "softmax":
        one = z.clone()
        one[20, 1] = NAN
        got = binding.moe_route(one.cuda(), k, bias=bias.cuda(), balance=True)
        without = torch.arange(T) != 20
        want = binding.moe_route(z.cuda(), k, bias=bias.cuda(), mask=without.cuda(), balance=True)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert (got[0][20] == -1).all() and bool(torch.isfinite(got[3]))
    # a row that reaches an expert and has a NaN: by the definition the loss has one too
    z[20, 1] = NAN
    ids, _, _, loss, _ = binding.moe_route(z.cuda(), k, score=score, balance=True)
    assert int(ids[20, 0]) >= 0 and bool(torch.isnan(loss))


@pytest.mark.parametrize("norm,limit", [(2e38, 1e-3), (1e38, 1e-8), (3e30, 2e-9), (1e20, 1e-30), (1e25, 1e-40), (1e-3, 1e-42),
                                        (2e38, 1e-38), (1e38, 0.0), (1e38, 2.0)])
def test_clipping_by_factors_beyond_float32(norm, limit):
    """max_norm / norm below the smallest normal number: the clipped gradients are ordinary numbers all the same."""
    g = torch.Generator(device="cuda").manual_seed(5)
    sizes = [9000, 1, 300000, 4099, 64]
    ts = [torch.randn((n + 1,), generator=g, device="cuda") for n in sizes]
    ts = [t * (norm / math.sqrt(sum(sizes))) for t in ts]
    ts = [t.to(torch.bfloat16) if i % 2 else t for i, t in enumerate(ts)]
    ts = [t[1:] if i == 3 else t[:-1] for i, t in enumerate(ts)]
    want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))
    coef = min(1.0, float(torch.tensor(limit)) / want)  # the limit as float32
    outs = [torch.full_like(t, 7.0) for t in ts]
    n = binding.clip_grad_norm(ts, limit, out=outs)
    # 32 squares are added in float32, a root of these, a rounding
    assert abs(float(n) - want) <= 20 * U * want
    for t, o in zip(ts, outs):
        ref = t.double() * coef
        half, least = (BF, 2.0 ** -134) if t.dtype == torch.bfloat16 else (U, 2.0 ** -150)  # least: half a subnormal step
        assert ((o.double() - ref).abs() <= (20 * U + 3 * U + half) * ref.abs() + 2 * least).all()
    mine, again = [t.clone() for t in ts], [t.clone() for t in ts]
    binding.clip_grad_norm(mine, limit)
    binding.grad_clip(again, n, limit)
    for a, b, c in zip(outs, mine, again):
        assert torch.equal(a, b) and torch.equal(a, c)


NORM_FORMS = [(False, False, False), (True, False, False), (True, True, False), (True, False, True), (True, True, True)]


@pytest.mark.parametrize("H", [16, 256, 784, 4096, 8192, 16384])
@pytest.mark.parametrize("y,post,gate", NORM_FORMS)
@pytest.mark.parametrize("grad", [1.0, 1e-6])
@pytest.mark.parametrize("small", [True, False])
def test_norm_gradient_of_rows_of_any_magnitude(H, y, post, gate, grad, small):
    """Rows whose mean square float32 holds: rstd^3 does not have to lie in float32, nor rstd^2 times a small gradient."""
    T, alpha, eps = 44, 0.5 if y else 1.0, 0.0 if small else 1e-6
    g = torch.Generator().manual_seed(H)
    sign = -1 if small else 1
    powers = torch.tensor([0, 6, 10, 12, 13, 14, 15, 15.5, 16, 16.5, 17])
    scale_r = 10.0 ** (sign * powers.repeat_interleave(4))
    scale_y = 10.0 ** (sign * powers.repeat(4))

    def rows(std, scale):
        return (torch.randn((T, H), generator=g) * std * scale[:, None]).to(torch.bfloat16).cuda()

    def vector(mean):
        return (mean + 0.3 * torch.randn((H,), generator=g)).cuda()

    one = torch.ones(T)
    # without a norm of its own y is no larger than the rest
    r, Y = rows(1.0, scale_r), rows(0.7, scale_y if post else one) if y else None
    dn, dr = rows(grad, one), rows(grad, one / scale_r.double()) if H % 3 else None
    w, P, A = vector(1.0), vector(1.0) if post else None, vector(0.5) if gate else None

    def rstd_of(v):
        return ((v.double() ** 2).mean(1) + eps).pow(-0.5).float()

    rstd, rstd_y = rstd_of(r), rstd_of(Y) if post else None
    got = binding.rmsnorm_residual_backward(dn, r, rstd, w, dr=dr, y=Y, rstd_y=rstd_y, gate=A, post_weight=P, alpha=alpha)

    def d(t):
        return None if t is None else t.double()

    want = plain.norm_backward(d(dn), d(dr), d(r), d(rstd), d(Y), d(rstd_y), d(w), d(P), d(A), alpha)
    for name, t in zip(("dx", "dy", "dweight", "dgate", "dpost_weight"), got):
        assert (t is not None) == (name in want), name
        if t is None:
            continue
        ref, bound = want[name]
        half, least = (BF, 2.0 ** -134) if t.dtype == torch.bfloat16 else (U, 2.0 ** -150)
        assert bool(torch.isfinite(t).all()), name
        # the bounds count roundings of normal numbers; what is subnormal in the output is rounded to its step
        assert ((t.double() - ref).abs() <= bound * (1 + half) + half * ref.abs() + least).all(), name


def test_norm_gradient_of_no_rows_is_zero_whatever_the_vectors_hold():
    x, w = torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda"), torch.ones(256, device="cuda")
    bad = torch.full((256,), INF, device="cuda")
    bad[::2] = NAN
    stat = torch.zeros(0, device="cuda")
    outs = [torch.full((256,), 7.0, device="cuda") for _ in range(3)]
    binding.rmsnorm_residual_backward(x, x, stat, bad, y=x, rstd_y=stat, gate=bad, post_weight=bad, dweight=outs[0],
                                      dgate=outs[1], dpost_weight=outs[2])
    assert not any(bool((t != 0).any()) for t in outs)

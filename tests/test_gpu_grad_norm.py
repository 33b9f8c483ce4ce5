"""GPU tests of the norm of many gradients and of clipping by it, against float64."""
import math

import pytest
import torch

from fp8_block_scaled_scales_b200 import binding

from plain_step import BF, U

pytestmark = pytest.mark.gpu


def tensors(sizes, seed, std=1e-3):
    """Every third in bfloat16; addresses at multiples of 16 bytes, and one element past that."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn((n + 1,), generator=g, device="cuda") * std
        t = t.to(torch.bfloat16) if i % 3 == 1 else t
        out.append(t[1:] if i % 4 == 2 else t[:n])
    return out


def norm64(ts):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))


# at most 32 squares are added in FP32 before FP64 takes over; the root halves that, one rounding follows
NORM = 20 * U

SIZES = [[1], [0], [], [5, 0, 3], [8192, 8191, 8193, 16384, 1], [100000, 7, 65536, 4099, 12], [3 * (1 << 20) + 5],
         list(range(1, 65)), list(range(1, 66)), [17] * 1024, [33] * 1025, [1 + i % 40 for i in range(2100)]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s, default=0)}")
def test_norm_and_clip(sizes):
    ts = tensors(sizes, len(sizes) + 1)
    want = norm64(ts)
    norm = binding.grad_norm(ts)
    assert norm.shape == () and abs(float(norm) - want) <= NORM * want
    for limit in (want * 0.3, want * 1.5, 0.0):
        coef = min(1.0, limit / want) if want else 1.0
        outs = [torch.full_like(t, 7.0) for t in ts]
        n2 = binding.clip_grad_norm(ts, limit, out=outs)
        assert torch.equal(n2, norm)
        for t, o in zip(ts, outs):
            ref = t.double() * coef
            half = BF if t.dtype == torch.bfloat16 else U
            assert ((o.double() - ref).abs() <= (NORM + 3 * U + half) * ref.abs() + 2.0 ** -126).all()
            if coef == 1.0:
                assert torch.equal(o, t)
        mine = [t.clone() for t in ts]
        n3 = binding.clip_grad_norm(mine, limit)
        assert torch.equal(n3, norm)
        for a, b in zip(mine, outs):
            assert torch.equal(a, b)
        again = [t.clone() for t in ts]
        binding.grad_clip(again, norm, limit)
        for a, b in zip(again, outs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [1e-30, 1e-42, 1e25, 3e37])
def test_squares_beyond_float32(scale):
    """Gradients whose squares over- or underflow in FP32 have a norm all the same."""
    ts = [torch.randn(5000, device="cuda") * scale, (torch.randn(300, device="cuda") * scale).to(torch.bfloat16),
          torch.zeros(70000, device="cuda"), torch.zeros(33, device="cuda")[1:]]
    want = norm64(ts)
    got = float(binding.grad_norm(ts))
    assert abs(got - want) <= NORM * want + 2.0 ** -149 if want < 3.4e38 else math.isinf(got)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_norms_that_are_not_finite_clip_nothing(bad):
    ts = tensors([9000, 20, 64], 3)
    ts[1][7] = bad
    mine = [t.clone() for t in ts]
    norm = binding.clip_grad_norm(mine, 1e-3)
    assert math.isinf(float(norm)) if math.isinf(bad) else math.isnan(float(norm))
    outs = [torch.zeros_like(t) for t in ts]
    binding.clip_grad_norm(ts, 1e-3, out=outs)
    for a, b, c in zip(mine, ts, outs):
        assert torch.equal(a.nan_to_num(1.0), b.nan_to_num(1.0)) and torch.equal(c.nan_to_num(1.0), b.nan_to_num(1.0))


def test_what_lies_beside_the_tensors_stays():
    flat = torch.full((100000,), 2.0, device="cuda")
    ts = [flat[3:5003], flat[5011:5012], flat[5020:70021]]
    spare = torch.ones(100000, dtype=torch.bool, device="cuda")
    for a, b in ((3, 5003), (5011, 5012), (5020, 70021)):
        spare[a:b] = False
    norm = binding.clip_grad_norm(ts, 1.0)
    assert bool((flat[spare] == 2.0).all()) and bool((flat[~spare] != 2.0).all())
    assert abs(float(binding.grad_norm(ts)) - 1.0) < 1e-5 and float(norm) > 100


def test_tensors_that_overlap_are_refused():
    flat = torch.ones(1000, device="cuda")
    for ts in ([flat, flat], [flat[:500], flat[499:]], [flat[10:20], flat], [flat, flat[:0], flat[5:6]]):
        with pytest.raises(binding.DGError):
            binding.clip_grad_norm(ts, 1.0)
        with pytest.raises(binding.DGError):
            binding.grad_clip(ts, torch.ones((), device="cuda"), 1.0)
        assert float(binding.grad_norm(ts)) > 0  # read only
        outs = [torch.empty_like(t) for t in ts]
        binding.clip_grad_norm(ts, 1.0, out=outs)  # written apart
        with pytest.raises(binding.DGError):  # an output over another gradient
            binding.clip_grad_norm([flat[:500], flat[500:]], 1.0, out=[flat[500:], torch.empty(500, device="cuda")])
        with pytest.raises(binding.DGError):  # or shifted over its own
            binding.clip_grad_norm([flat[:500]], 1.0, out=[flat[1:501]])
    assert bool((flat == 1).all())
    binding.clip_grad_norm([flat[:500], flat[500:]], 1.0, out=[flat[:500], flat[500:]])  # in place by name
    assert abs(float(binding.grad_norm([flat])) - 1.0) < 1e-5


def test_two_streams_and_graph():
    a, b = tensors([300000, 5, 77], 1), tensors([100, 4, 900000], 2)
    want = [binding.grad_norm(a), binding.grad_norm(b)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        got = [binding.grad_norm(a, stream=s1), binding.grad_norm(b, stream=s2)]
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    norm, outs = torch.empty((), device="cuda"), [torch.empty_like(t) for t in a]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.clip_grad_norm(a, 0.1, out=outs, norm=norm)
    for t, fresh in zip(a, tensors([300000, 5, 77], 9)):
        t.copy_(fresh)
    graph.replay()
    other = [torch.empty_like(t) for t in a]
    assert torch.equal(norm, binding.clip_grad_norm(a, 0.1, out=other))
    for x, y in zip(outs, other):
        assert torch.equal(x, y)

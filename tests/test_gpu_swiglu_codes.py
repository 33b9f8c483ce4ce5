"""GPU tests of SwiGLU's codes and scales to the width of the actual E4M3 step: a neighbouring code passes only where
the value lies within the kernel's own FP32 error of the border between the two."""
import pytest
import torch

from fp8_block_scaled_scales_b200 import binding

import plain_train as plain

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of FP32, relative
TINY = 2.0 ** -149  # a step of subnormal FP32
B = 128


def blockwise(s, R, C):
    return s.double().repeat_interleave(B, 0)[:R].repeat_interleave(B, 1)[:, :C]


def sigma_noise(g):
    """Relative error of the kernel's sigma(g) = 1 / (1 + e), e = exp(-g): the exponential's documented 2 + 1.173 |g|
    units of 2^-23 (|g| / 2 more for g itself off by a rounding) enter by the share e / (1 + e) of the denominator;
    its rounding, the reciprocal corrected by its remainder and the products on the way add less than four units."""
    return ((1 - torch.sigmoid(g)) * (2 + 1.7 * g.abs()) + 4) * 2 * U


def forward64(h):
    F = h.shape[1] // 2
    g, u = h[:, :F].double(), h[:, F:].double()
    a = g * torch.sigmoid(g) * u
    a = torch.where(torch.sigmoid(g) < 2.0 ** -126, torch.zeros_like(a), a)  # counts as 0
    return a, (sigma_noise(g) * a.abs() + TINY) * (a != 0)


def backward64(g, u, d):
    """[dg | du] and the error of each: g and u are the decoded values, off by U each in the kernel."""
    p = torch.sigmoid(g)
    p = torch.where(p < 2.0 ** -126, torch.zeros_like(p), p)
    w = 1 + g * (1 - p)
    e = sigma_noise(g)
    # 1 - p is off by p e and its rounding (by itself where e^-g is lost in 1 + e^-g: the kernel's p is 1 then); g by U;
    # the sum rounds once more
    w_off = g.abs() * torch.where(g > 18, 1 - p, p * e + (1 - p) * 2 * U) + w.abs() * U
    dg, du = d * u * p * w, d * g * p
    return torch.cat([dg, du], 1), torch.cat([(d * u * p).abs() * (w_off + w.abs() * (e + 6 * U)) + TINY * (dg != 0),
                                            du.abs() * (e + 3 * U) + TINY * (du != 0)], 1)


def check(q, s, value, noise, what):
    """scale: amax of values off by at most their noise, over 448, rounded; code: the E4M3 rounding of a quotient off by
    noise / s and one FP32 rounding: half the step at the value, and that."""
    R, C = value.shape
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            sl = (slice(i * B, min(R, i * B + B)), slice(j * B, min(C, j * B + B)))
            top, low = float((value[sl].abs() + noise[sl]).max()), float((value[sl].abs() - noise[sl]).max())
            if top == 0:
                assert s[i, j] == 1.0, (what, i, j)
            else:
                assert low / 448 * (1 - 2 * U) - TINY <= float(s[i, j]) <= top / 448 * (1 + 2 * U) + TINY, (what, i, j)
    w = blockwise(s, R, C)
    v = value / w
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    err = (plain.decode(q, s) / w - v).abs()
    bound = step / 2 + v.abs() * 2 * U + noise / w
    assert bool((err <= bound).all()), f"{what}: {int((err > bound).sum())} codes, worst by {float((err - bound).max()):.3g}"


def pre_activation(M, F, seed, scale):
    h = torch.randn((M, 2 * F), generator=torch.Generator().manual_seed(seed)) * scale
    if M > 2:
        h[M // 2] *= 20  # saturated gates of both signs
        h[M - 1] = 0
    return h.to(torch.bfloat16)


SHAPES = [(1, 128, 2.0), (7, 256, 0.1), (300, 640, 2.0), (1000, 256, 8.0), (500, 1024, 1.0)]


@pytest.mark.parametrize("M,F,scale", SHAPES)
@pytest.mark.parametrize("form", ["plain", "checkpoint", "masked"])
def test_forward(M, F, scale, form):
    h = pre_activation(M, F, M + F, scale)
    if form == "masked":
        q, s = binding.swiglu_quantize_masked(h.cuda()[None], torch.tensor([M], dtype=torch.int32, device="cuda"))
        q, s = q[0], s[0]
    else:
        q, s = binding.swiglu_quantize(h.cuda(), checkpoint=form == "checkpoint")[:2]
    check(q.cpu(), s.cpu(), *forward64(h), form)


@pytest.mark.parametrize("M,F,scale", SHAPES)
def test_backward(M, F, scale):
    h8, sh = binding.quantize_1x128(pre_activation(M, F, M + F + 1, scale).cuda())
    da = (torch.randn((M, F), generator=torch.Generator().manual_seed(2)) * 1e-3).to(torch.bfloat16)
    q, s = binding.swiglu_quantize_backward(h8, sh, da.cuda())
    v = plain.decode_rows(h8.cpu(), sh.cpu())
    check(q.cpu(), s.cpu(), *backward64(v[:, :F], v[:, F:], da.double()), "gradient")


GATES = [0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, -1.28, 1.0, -1.0, 8.0, -8.0, 17.0, -17.0, 30.0, -30.0, 60.0, -60.0, 80.0, -80.0,
         86.0, -86.0, 87.0, -87.0, 87.5, -87.5, 88.0, -88.0, 88.5, -88.5, 89.0, -89.0, 104.0, -104.0, 127.0, -127.0, 1e4, -1e4,
         3e38, -3e38]


def gates():
    return torch.tensor(GATES).to(torch.bfloat16)


def test_forward_of_each_gate_in_a_block_of_its_own():
    """From the smallest to the largest, around where the exponential overflows and sigma leaves the normal range: the
    block's scale is the activation's, so none hides behind another's."""
    g = gates()
    F = len(g) * B
    for exponent in (0, 60, 126):  # up values that bring small activations into range, and large ones near its end
        u = torch.where(g.float().abs() > 1e30, torch.tensor(0.75), torch.tensor(2.0 ** exponent))
        u = torch.where((g.float() > 1) & (g.float() < 1e30), torch.tensor(3.0), u).to(torch.bfloat16)
        h = torch.zeros((3, 2 * F), dtype=torch.bfloat16)
        h[1, 5:F:B], h[1, F + 5::B] = g, u
        for form in (False, True):
            q, s = (t.cpu() for t in binding.swiglu_quantize(h.cuda(), checkpoint=form)[:2])
            check(q, s, *forward64(h), f"up 2^{exponent}")


def test_backward_of_each_gate_in_a_block_of_its_own():
    g = gates()
    F = len(g) * B
    one = 0x38  # the code of 1
    h8 = torch.zeros((3, 2 * F), dtype=torch.uint8)
    h8[1, 5:F:B] = torch.where(g.float() < 0, one | 0x80, one).to(torch.uint8)
    h8[1, F + 5::B] = one
    sh = torch.ones((2 * F // B, 3))
    sh[:len(g), 1] = g.float().abs()
    for exponent in (0, 60, 120):
        da = torch.zeros((3, F), dtype=torch.bfloat16)
        da[1, 5::B] = torch.where(g.float() > 1, 1e-3, 2.0 ** exponent).to(torch.bfloat16)
        big = g.float().abs() > 1e30
        da[1, 5::B][big] = 0.25
        q, s = (t.cpu() for t in binding.swiglu_quantize_backward(h8.cuda(), sh.cuda(), da.cuda()))
        v = plain.decode_rows(h8, sh)
        check(q, s, *backward64(v[:, :F], v[:, F:], da.double()), f"2^{exponent}")

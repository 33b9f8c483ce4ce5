"""GPU tests of SwiGLU with its 8-bit checkpoint and of its backward pass."""
import pytest
import torch

from fp8_block_scaled_scales_b200 import binding

import plain_train as plain

pytestmark = pytest.mark.gpu


def pre_activation(M, F, seed, scale=2.0):
    h = torch.randn((M, 2 * F), generator=torch.Generator().manual_seed(seed)) * scale
    if M > 2:
        h[M // 2] *= 20   # saturated gates of both signs
        h[M - 1] = 0
    return h.to(torch.bfloat16)


def check_codes(q, s, value, noise, what):
    """Scales from the block maxima, codes within the bound of their rounding."""
    err = (plain.decode(q, s) - value).abs()
    bound = plain.code_error_bound(value, s, noise)
    assert bool((err <= bound).all()), f"{what}: worst ratio {float((err / bound.clamp_min(1e-300)).max()):.4g}"
    R, C = value.shape
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            sl = (slice(i * 128, min(R, i * 128 + 128)), slice(j * 128, min(C, j * 128 + 128)))
            top, n = float(value[sl].abs().max()), float(torch.as_tensor(noise)[sl].max())
            if top == 0 and n == 0:
                assert s[i, j] == 1.0
            else:
                assert abs(float(s[i, j]) - top / 448) <= (n / 448) * 1.01 + top / 448 * 2.0 ** -23, (what, i, j)


SHAPES = [(1, 128), (7, 256), (128, 128), (129, 384), (300, 640), (1000, 256)]


@pytest.mark.parametrize("M,F", SHAPES)
@pytest.mark.parametrize("checkpoint", [False, True])
def test_swiglu_quantize(M, F, checkpoint):
    h = pre_activation(M, F, M + F)
    out = [t.cpu() for t in binding.swiglu_quantize(h.cuda(), checkpoint=checkpoint)]
    a = plain.swiglu64(h)
    check_codes(out[0], out[1], a, plain.sigma_error(h[:, :F].double()) * a.abs(), "activation")
    if checkpoint:
        q, s = binding.quantize_1x128(h.cuda())
        assert torch.equal(out[2], q.cpu()) and torch.equal(out[3], s.cpu())


def test_checkpoint_of_arbitrary_finite_bit_patterns():
    """Rows of finite BF16 values of every exponent, and rows of subnormals: the checkpoint is still
    dg_quantize_1x128's output, bit for bit."""
    g = torch.Generator().manual_seed(6)
    bits = torch.randint(0, 65536, (512, 512), generator=g, dtype=torch.int32)
    bits[:, ::3] &= 0xBFFF      # half the exponents below 1
    bits[128:256] &= 0x807F     # zeros and subnormals
    bits[256:384] = (bits[256:384] & 0x807F) | 0x3F80  # one exponent
    bits[(bits & 0x7F80) == 0x7F80] = 0
    h = bits.to(torch.int16).view(torch.bfloat16).cuda()
    _, _, h8, sh = binding.swiglu_quantize(h, checkpoint=True)
    q, s = binding.quantize_1x128(h)
    assert torch.equal(sh.view(torch.int32), s.view(torch.int32)) and torch.equal(h8, q)


def test_swiglu_extremes():
    """Gates whose exponential overflows or underflows: the sigmoid is 0 or 1, nothing is NaN."""
    g = torch.tensor([0.0, -0.0, 88.0, -88.0, 89.0, -89.0, 104.0, -104.0, 1e4, -1e4, 3e38, -3e38, 1e-30, -1e-30, 127.0, -127.0])
    h = torch.zeros((1, 256))
    h[0, :16], h[0, 128:] = g, 1.0
    h = h.to(torch.bfloat16)
    q, s = (t.cpu() for t in binding.swiglu_quantize(h.cuda()))
    a = plain.swiglu64(h)
    err = (plain.decode(q, s) - a).abs()
    assert bool((err <= plain.code_error_bound(a, s, plain.sigma_error(h[:, :128].double()).clamp_max(1e-2) * a.abs())).all())


@pytest.mark.parametrize("counts", [[0, 0], [128, 0], [0, 256, 0, 128]])
def test_swiglu_grouped_leaves_rows_past_the_last_expert(counts):
    F, cap = 256, 512
    off = torch.tensor([0] + counts).cumsum(0).int()
    used = int(off[-1])
    h = pre_activation(cap, F, 5)
    h[used:] = float("nan")
    q = torch.full((cap, F), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((cap // 128, F // 128), -7.0, device="cuda")
    h8 = torch.full((cap, 2 * F), 0xA5, dtype=torch.uint8, device="cuda")
    sh = torch.full((2 * F // 128, cap), -7.0, device="cuda")
    binding.swiglu_quantize(h.cuda(), off.cuda(), checkpoint=True, q=q, s=s, h8=h8, sh=sh)
    assert bool((q[used:] == 0xA5).all()) and bool((s[used // 128:] == -7).all())
    assert bool((h8[used:] == 0xA5).all()) and bool((sh[:, used:] == -7).all())
    da = torch.randn((cap, F)).to(torch.bfloat16)
    da[used:] = float("inf")
    dq = torch.full((cap, 2 * F), 0xA5, dtype=torch.uint8, device="cuda")
    ds = torch.full((cap // 128, 2 * F // 128), -7.0, device="cuda")
    binding.swiglu_quantize_backward(h8, sh, da.cuda(), off.cuda(), q=dq, s=ds)
    assert bool((dq[used:] == 0xA5).all()) and bool((ds[used // 128:] == -7).all())
    if used:  # the rows that are there: as the dense call on them alone
        d = [t.cpu() for t in binding.swiglu_quantize(h[:used].cuda(), checkpoint=True)]
        assert torch.equal(q[:used].cpu(), d[0]) and torch.equal(s[:used // 128].cpu(), d[1])
        assert torch.equal(h8[:used].cpu(), d[2]) and torch.equal(sh[:, :used].cpu(), d[3])
        b = binding.swiglu_quantize_backward(d[2].cuda(), d[3].cuda(), da[:used].cuda())
        assert torch.equal(dq[:used], b[0]) and torch.equal(ds[:used // 128], b[1])


@pytest.mark.parametrize("m_max,counts", [(40, [0, 40, 1]), (300, [300, 129, -4, 1000]), (2200, [2100])])
def test_swiglu_masked(m_max, counts):
    G, F = len(counts), 256
    m = [min(max(c, 0), m_max) for c in counts]
    h = torch.stack([pre_activation(m_max, F, 10 + g) for g in range(G)])
    for g in range(G):
        h[g, m[g]:] = float("nan")
    q = torch.full((G, m_max, F), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((G, -(-m_max // 128), F // 128), -7.0, device="cuda")
    binding.swiglu_quantize_masked(h.cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda"), q=q, s=s)
    for g in range(G):
        nb = -(-m[g] // 128)
        assert bool((q[g, m[g]:] == 0xA5).all()) and bool((s[g, nb:] == -7).all())
        if m[g]:
            wq, ws = binding.swiglu_quantize(h[g, :m[g]].cuda())
            assert torch.equal(q[g, :m[g]], wq) and torch.equal(s[g, :nb], ws)


def backward64(h, da):
    """([dg | du], the kernel's error bound of each) in float64."""
    F = da.shape[1]
    g, u, d = h[:, :F], h[:, F:], da.double()
    p = torch.sigmoid(g)
    dg, du = d * u * p * (1 + g * (1 - p)), d * g * p
    e = plain.sigma_error(g)
    # 1 + g (1 - p) cancels: its error is that of its terms
    noise = torch.cat([e * (d * u * p).abs() * (2 + 2 * g.abs()), e * du.abs()], 1)
    return torch.cat([dg, du], 1), noise


@pytest.mark.parametrize("M,F", SHAPES)
def test_swiglu_backward(M, F):
    h = pre_activation(M, F, M + F + 1)
    h8, sh = binding.quantize_1x128(h.cuda())
    da = (torch.randn((M, F), generator=torch.Generator().manual_seed(2)) * 1e-3).to(torch.bfloat16)
    q, s = (t.cpu() for t in binding.swiglu_quantize_backward(h8, sh, da.cuda()))
    d, noise = backward64(plain.decode_rows(h8.cpu(), sh.cpu()), da)
    check_codes(q, s, d, noise, "gradient")


def test_swiglu_backward_against_differences():
    """The formula against central differences of the float64 forward at the checkpoint's values."""
    M, F = 64, 128
    h8, sh = binding.quantize_1x128(pre_activation(M, F, 9, 1.0).cuda())
    h = plain.decode_rows(h8.cpu(), sh.cpu())
    da = torch.randn((M, F), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    q, s = (t.cpu() for t in binding.swiglu_quantize_backward(h8, sh, da.cuda()))
    d, noise = backward64(h, da)
    e = 1e-4
    for half in range(2):
        step = torch.zeros_like(h)
        step[:, half * F:(half + 1) * F] = e
        num = (plain.swiglu64(h + step) - plain.swiglu64(h - step)) / (2 * e) * da.double()
        exact = d[:, half * F:(half + 1) * F]
        # third derivatives of g sigma(g) u are below |u| + 1: the difference is off by e^2 of that
        assert bool(((num - exact).abs() <= e * e * da.double().abs() * (h.abs().max() + 1) + 1e-9).all())
        got = plain.decode(q, s)[:, half * F:(half + 1) * F]
        bound = plain.code_error_bound(d, s, noise)[:, half * F:(half + 1) * F]
        assert bool(((got - num).abs() <= bound + 1e-6).all())


def test_swiglu_past_32_bit_offsets():
    """More than 2^32 elements of h: the last block equals the same rows alone."""
    M, F = 132_224, 16384
    h = torch.empty((M, 2 * F), dtype=torch.bfloat16, device="cuda")
    h[-256:] = pre_activation(256, F, 3).cuda()
    h8 = torch.empty((M, 2 * F), dtype=torch.uint8, device="cuda")
    q, s, h8, sh = binding.swiglu_quantize(h, checkpoint=True, h8=h8)
    a = binding.swiglu_quantize(h[-256:].contiguous(), checkpoint=True)
    assert torch.equal(q[-256:], a[0]) and torch.equal(s[-2:], a[1])
    assert torch.equal(h8[-256:], a[2]) and torch.equal(sh[:, -256:], a[3])
    da = torch.empty((M, F), dtype=torch.bfloat16, device="cuda")
    da[-256:] = torch.randn((256, F), device="cuda").to(torch.bfloat16)
    dq, ds = binding.swiglu_quantize_backward(h8, sh, da)
    b = binding.swiglu_quantize_backward(a[2], a[3], da[-256:].contiguous())
    assert torch.equal(dq[-256:], b[0]) and torch.equal(ds[-2:], b[1])


def test_swiglu_non_finite_values_stay_in_their_block():
    M, F = 256, 256
    h = pre_activation(M, F, 8)
    clean = h.clone()
    h[3, 7], h[200, F + 130] = float("nan"), float("inf")   # a gate in block (0, 0), an up in (1, 1)
    q, s = binding.swiglu_quantize(h.cuda())
    cq, cs = binding.swiglu_quantize(clean.cuda())
    assert torch.equal(torch.isfinite(s).cpu(), torch.tensor([[False, True], [True, False]]))
    assert torch.equal(q[:128, 128:], cq[:128, 128:]) and torch.equal(q[128:, :128], cq[128:, :128])
    assert s[0, 1] == cs[0, 1] and s[1, 0] == cs[1, 0]


def non_finite_input():
    """(h, F, blocks): row block and column block of each value that is not finite."""
    M, F, inf, nan = 300, 640, float("inf"), float("nan")
    h = pre_activation(M, F, 12)
    h[h == 0] = 0.5
    put = {(0, 0): [(3, 7, inf, 1.5), (90, 100, inf, -2.0)],  # gates of +infinity: infinite of both signs
           (0, 1): [(17, 130, inf, 0.0)],                     # times zero: NaN
           (0, 2): [(5, 300, 0.0, inf)], (0, 3): [(5, 400, 1.0, -inf)],
           (1, 0): [(130, 0, -inf, 1.0)], (1, 1): [(255, 255, nan, 1.0)], (1, 2): [(200, 256, 1.0, nan)],
           (2, 3): [(299, 511, inf, inf)], (2, 4): [(260, 513, inf, 2.0), (261, 514, -inf, 1.0)]}
    for places in put.values():
        for r, c, g, u in places:
            h[r, c], h[r, F + c] = g, u
    return h, F, put


@pytest.mark.parametrize("form", ["plain", "checkpoint", "masked"])
def test_swiglu_of_infinite_and_nan_gates(form):
    """g * sigma(g) * u of an infinite gate is infinite (NaN for u = 0 and for -infinity): the block's scale and
    codes are the quantizer's definition on that, and blocks of numbers stay as they are."""
    h, F, put = non_finite_input()
    clean = torch.where(torch.isfinite(h), h, torch.ones((), dtype=h.dtype))
    if form == "masked":
        def call(x):
            q, s = binding.swiglu_quantize_masked(x.cuda()[None], torch.tensor([len(x)], dtype=torch.int32, device="cuda"))
            return q[0].cpu(), s[0].cpu()
    else:
        def call(x):
            return [t.cpu() for t in binding.swiglu_quantize(x.cuda(), checkpoint=form == "checkpoint")[:2]]
    (q, s), (cq, cs) = call(h), call(clean)
    g, u = h[:, :F].float(), h[:, F:].float()
    wq, ws = plain.quantize_f32(g / (1 + torch.exp(-g)) * u)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            sl = (slice(i * 128, min(len(h), i * 128 + 128)), slice(j * 128, j * 128 + 128))
            if (i, j) not in put:
                assert s[i, j] == cs[i, j] and torch.equal(q[sl], cq[sl]), (i, j)
                continue
            assert not torch.isfinite(ws[i, j])
            assert torch.equal(s[i, j].nan_to_num(nan=-1.0), ws[i, j].nan_to_num(nan=-1.0)), (i, j)
            nan = (wq[sl] & 0x7F) == 0x7F
            assert bool(nan.any()) and torch.equal((q[sl] & 0x7F) == 0x7F, nan), (i, j)
            assert torch.equal(q[sl][~nan], wq[sl][~nan]), (i, j)


def test_checkpoint_of_non_finite_values():
    """The checkpoint is dg_quantize_1x128's output where rows hold infinities and NaN, too."""
    h = non_finite_input()[0].cuda()
    _, _, h8, sh = binding.swiglu_quantize(h, checkpoint=True)
    q, s = binding.quantize_1x128(h)
    assert torch.equal(sh.nan_to_num(nan=-1.0), s.nan_to_num(nan=-1.0)) and torch.equal(h8, q)
    assert not bool(torch.isfinite(sh).all())

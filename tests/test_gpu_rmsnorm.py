"""GPU tests of the norms around a block, their codes and their gradient, against plain float64
forms under bounds that count the roundings."""
import math

import pytest
import torch

from fp8_block_scaled_scales_b200 import binding

import plain_step as plain
from plain_step import BF, U

pytestmark = pytest.mark.gpu
EPS = 1e-6
SIZES = [(1, 16), (1, 7168), (3, 144), (5, 128), (37, 1040), (300, 784), (2, 8192), (64, 4096), (3, 8208), (4, 16384),
         (700, 2048), (333, 4112), (1200, 256)]
FORMS = [(False, False, False), (True, False, False), (True, True, False), (True, False, True), (True, True, True)]


def inputs(T, H, seed, y, post, gate, vec=torch.float32):
    """Tensors on the GPU: x, y and the vectors, with outlier channels, a row of zeros and one of
    large values."""
    g = torch.Generator().manual_seed(seed)

    def make(std=1.0):
        v = torch.randn((T, H), generator=g) * std
        v[:, :: max(1, H // 3)] *= 30
        if T > 2:
            v[1] = 0
            v[2] *= 1e4
        return v.to(torch.bfloat16).cuda()

    def vector(mean):
        return (mean + 0.3 * torch.randn((H,), generator=g)).to(vec).cuda()

    return {"x": make(1.5), "y": make(0.7) if y else None, "weight": vector(1.0), "post_weight": vector(1.0) if post else None,
            "gate": vector(0.5) if gate else None}


def d(t):
    return None if t is None else t.double()


def forward64(v, alpha):
    return plain.norm_forward(d(v["x"]), d(v["y"]), d(v["weight"]), d(v["post_weight"]), d(v["gate"]), alpha, EPS)


def code_bound(n, en, s):
    """As code_error_bound of the block quantizer's tests, one scale per row and 128 columns."""
    w = s.double().t().repeat_interleave(128, 1)[:, :n.shape[1]]
    return torch.maximum(n.abs() * 2.0 ** -4, w * 2.0 ** -10) * (1 + 2.0 ** -19) + en * 1.125


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("y,post,gate", FORMS)
@pytest.mark.parametrize("vec", [torch.float32, torch.bfloat16])
def test_forward(T, H, y, post, gate, vec):
    v = inputs(T, H, T + H, y, post, gate, vec)
    alpha = 0.5 if y else 1.0
    (n64, r64, rstd64, rstdy64), en, er, rel = forward64(v, alpha)
    n, r, rstd, rstd_y = binding.rmsnorm_residual(**v, alpha=alpha, eps=EPS)
    if y:
        assert ((r.double() - r64).abs() <= er * (1 + BF) + BF * r64.abs()).all()
    else:
        assert r is v["x"] or r.data_ptr() == v["x"].data_ptr()
    assert ((n.double() - n64).abs() <= en * (1 + BF) + BF * n64.abs()).all()
    assert ((rstd.double() - rstd64).abs() <= rel * rstd64).all()
    assert (rstd_y is None) == (not post)
    if post:
        assert ((rstd_y.double() - rstdy64).abs() <= 40 * U * rstdy64).all()
    q, s, r2 = binding.rmsnorm_residual_quantize(**v, alpha=alpha, eps=EPS)
    assert torch.equal(r2, r) and s.shape == (-(-H // 128), T)
    value = q.view(torch.float8_e4m3fn).double() * s.double().t().repeat_interleave(128, 1)[:, :H]
    assert ((value - n64).abs() <= code_bound(n64, en, s)).all()
    # the scale is fl32(amax / 448) of values that are off by en
    pad = torch.nn.functional.pad(n64, (0, -H % 128)).view(T, -1, 128).abs()
    top = pad.amax(2).t()
    off = torch.nn.functional.pad(en, (0, -H % 128)).view(T, -1, 128).amax(2).t()
    want = torch.where(top == 0, torch.ones_like(top), top / 448)
    assert ((s.double() - want).abs() <= off / 448 + U * want).all()


@pytest.mark.parametrize("T,H", [(601, 4112), (640, 6000), (601, 8176), (620, 8208), (601, 12304), (601, 16368), (2001, 272), (3100, 272), (3001, 16), (3000, 1024),
                                 (1203, 3984)])
@pytest.mark.parametrize("y,post,gate", FORMS)
def test_many_rows_of_odd_widths(T, H, y, post, gate):
    """Rows that several CTAs share, and that end inside a group of 128 columns."""
    test_forward(T, H, y, post, gate, torch.float32)


def test_codes_are_those_of_the_quantizer():
    """With a weight of powers of two and rows whose norm is a power of two, n is a BF16 number:
    quantize_1x128 of it gives the same codes and scales, bit for bit."""
    T, H = 40, 1024
    g = torch.Generator().manual_seed(1)
    x = (torch.randint(0, 2, (T, H), generator=g) * 2 - 1).float()  # a mean square of 1
    x = (x * 2.0 ** torch.randint(-3, 4, (T, 1), generator=g)).to(torch.bfloat16).cuda()
    w = (2.0 ** torch.randint(-6, 7, (H,), generator=g)).cuda()
    n = binding.rmsnorm_residual(x, w, eps=0.0)[0]
    q, s, _ = binding.rmsnorm_residual_quantize(x, w, eps=0.0)
    wq, ws = binding.quantize_1x128(n)
    assert torch.equal(q, wq) and torch.equal(s, ws)


def test_in_place_and_preset_outputs():
    v = inputs(50, 512, 3, True, True, True)
    want = binding.rmsnorm_residual(**v)
    x = v.pop("x").clone()
    n = torch.empty_like(x)
    got = binding.rmsnorm_residual(x, **v, n=n, r=x)
    assert got[0] is n or got[0].data_ptr() == n.data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(x, want[1])


def test_values_that_are_not_finite_stay_in_their_row():
    v = inputs(8, 640, 4, True, True, True)
    v["x"][3, 7] = math.inf
    v["x"][5, 600] = math.nan
    v["y"][6, 1] = -math.inf
    n, r, rstd, rstd_y = binding.rmsnorm_residual(**v)
    bad = torch.tensor([3, 5, 6], device="cuda")
    keep = torch.tensor([0, 1, 2, 4, 7], device="cuda")
    assert torch.isfinite(n[keep].float()).all() and torch.isfinite(r[keep].float()).all()
    assert not torch.isfinite(r[bad].float()).all(1).any()
    assert math.isnan(float(rstd[5])) and float(rstd[3]) == 0.0
    q, s, _ = binding.rmsnorm_residual_quantize(**v)
    assert torch.isfinite(s[:, keep]).all() and torch.isnan(s[:, 5]).all()


def check_backward(T, H, y, post, gate, vec=torch.float32, dr=True, alpha=0.5, stream=None):
    v = inputs(T, H, T + H + 1, y, post, gate, vec)
    g = torch.Generator().manual_seed(T * 7 + H)
    grads = [(torch.randn((T, H), generator=g) * 1e-3).to(torch.bfloat16).cuda() for _ in range(2)]
    if T > 3:
        grads[0][3] = 0
    r, w = v.pop("x"), v.pop("weight")
    alpha = alpha if y else 1.0
    rstd = ((r.double() ** 2).mean(1) + EPS).pow(-0.5).float()
    rstd_y = ((v["y"].double() ** 2).mean(1) + EPS).pow(-0.5).float() if post else None
    torch.cuda.synchronize()
    got = binding.rmsnorm_residual_backward(grads[0], r, rstd, w, dr=grads[1] if dr else None, rstd_y=rstd_y, alpha=alpha,
                                            stream=stream, **v)
    torch.cuda.synchronize()
    want = plain.norm_backward(d(grads[0]), d(grads[1]) if dr else None, d(r), d(rstd), d(v["y"]), d(rstd_y), d(w),
                               d(v["post_weight"]), d(v["gate"]), alpha)
    for name, t in zip(("dx", "dy", "dweight", "dgate", "dpost_weight"), got):
        assert (t is not None) == (name in want), name
        if t is None:
            continue
        ref, bound = want[name]
        out = BF if t.dtype == torch.bfloat16 else U
        assert ((t.double() - ref).abs() <= bound * (1 + out) + out * ref.abs() + 2.0 ** -126).all(), name
    return got


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("y,post,gate", FORMS)
@pytest.mark.parametrize("dr", [True, False])
def test_backward(T, H, y, post, gate, dr):
    check_backward(T, H, y, post, gate, dr=dr, vec=torch.bfloat16 if dr else torch.float32)


@pytest.mark.parametrize("T,H", [(5000, 1024), (9001, 128), (1500, 8192), (700, 16384), (4001, 4096),
                                 (700, 6000), (500, 12304), (900, 4112)])
def test_backward_of_many_rows_repeats_bit_for_bit(T, H):
    a = check_backward(T, H, True, True, True)
    b = check_backward(T, H, True, True, True, stream=torch.cuda.Stream())
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_no_rows():
    x, w = torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda"), torch.ones(256, device="cuda")
    n, r, rstd, rstd_y = binding.rmsnorm_residual(x, w, y=x, gate=w, post_weight=w)
    assert n.shape == r.shape == (0, 256) and rstd.shape == rstd_y.shape == (0,)
    dx, dy, dw, dg, dp = binding.rmsnorm_residual_backward(x, x, rstd, w, y=x, rstd_y=rstd_y, gate=w, post_weight=w)
    assert dx.shape == (0, 256) and not dw.any() and not dg.any() and not dp.any()


def test_captured_and_replayed():
    v = inputs(200, 1024, 5, True, True, True)
    outs = binding.rmsnorm_residual(**v)
    dn = torch.randn((200, 1024), device="cuda").to(torch.bfloat16)
    back = dict(y=v["y"], gate=v["gate"], post_weight=v["post_weight"])
    grads = binding.rmsnorm_residual_backward(dn, outs[1], outs[2], v["weight"], rstd_y=outs[3], **back)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.rmsnorm_residual(**v, n=outs[0], r=outs[1], rstd=outs[2], rstd_y=outs[3])
        binding.rmsnorm_residual_backward(dn, outs[1], outs[2], v["weight"], rstd_y=outs[3], dx=grads[0], dy=grads[1],
                                          dweight=grads[2], dgate=grads[3], dpost_weight=grads[4], **back)
    for seed in (6, 7):
        w = inputs(200, 1024, seed, True, True, True)
        v["x"].copy_(w["x"])
        v["y"].copy_(w["y"])
        graph.replay()
        want = binding.rmsnorm_residual(**v)
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        for a, b in zip(grads, binding.rmsnorm_residual_backward(dn, want[1], want[2], v["weight"], rstd_y=want[3], **back)):
            assert torch.equal(a, b)

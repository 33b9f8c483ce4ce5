"""Refusals of the calls around the expert layer, decided on the host before any CUDA call, and
the plain forms' gradients against differences."""
import ctypes
import math

import pytest
import torch

from fp8_block_scaled_scales_b200 import binding
from fp8_block_scaled_scales_b200 import build as dgbuild

import plain_step as plain

NULL = ctypes.c_void_p(0)
P = ctypes.c_void_p(0x10000)   # never dereferenced: the refusal comes first
ODD = ctypes.c_void_p(0x10001)
OK, ARG, SHAPE, ALIGN = 0, 1, 2, 3


class RouteOptions(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int), ("renormalize", ctypes.c_int), ("scale", ctypes.c_float)]


class NormOptions(ctypes.Structure):
    _fields_ = [("alpha", ctypes.c_float), ("eps", ctypes.c_float), ("vectors_bf16", ctypes.c_int)]


def ref(s):
    return ctypes.cast(ctypes.pointer(s), ctypes.c_void_p)


@pytest.fixture(scope="module")
def lib():
    dgbuild.build()
    return binding.lib()


def test_route_refusals(lib):
    f, opt = lib.dg_moe_route, ref(RouteOptions(0, 1, 1.0))

    def call(z=P, bf16=0, o=opt, bias=NULL, mask=NULL, T=8, G=16, k=2, ids=P, w=P, c=NULL, loss=NULL, d=NULL, ws=NULL, n=0):
        return f(z, bf16, o, bias, mask, T, G, k, ids, w, c, loss, d, ws, n, NULL)

    for bad in (dict(T=-1), dict(G=0), dict(G=1025), dict(k=0), dict(k=17), dict(G=64, k=33), dict(T=1 << 30)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(z=NULL), dict(ids=NULL), dict(w=NULL), dict(o=NULL), dict(o=ref(RouteOptions(2, 1, 1.0))),
                dict(o=ref(RouteOptions(0, 1, math.inf))), dict(o=ref(RouteOptions(0, 1, math.nan))), dict(c=P),
                dict(loss=P), dict(d=P), dict(c=P, loss=P)):
        assert call(**bad) == ARG, bad
    # more tokens than one cluster takes: a workspace of the size that the library names
    need = lib.dg_moe_route_workspace(8000, 16)
    full = dict(T=8000, c=P, loss=P, d=P, ws=P, n=need)
    assert need > 0 and lib.dg_moe_route_workspace(8, 16) == 0
    assert call(**{**full, "n": need - 1}) == ARG and call(**{**full, "ws": NULL}) == ARG
    for bad in (dict(z=ODD), dict(z=ctypes.c_void_p(0x10002)), dict(bias=ODD), dict(ids=ODD), dict(w=ODD),
                dict(full, c=ODD), dict(full, loss=ODD), dict(full, d=ODD), dict(full, ws=ODD)):
        assert call(**bad) == ALIGN, bad
    assert call(z=ctypes.c_void_p(0x10002), bf16=1, ids=ODD) == ALIGN and call(T=0, z=NULL, ids=NULL, w=NULL) == OK
    assert lib.dg_moe_route_workspace(-1, 16) == lib.dg_moe_route_workspace(8000, 1025) == 0
    # the workspace never shrinks as the sizes grow
    assert all(lib.dg_moe_route_workspace(T, 64) <= lib.dg_moe_route_workspace(T + 1, 64) for T in range(0, 9000, 7))


def test_route_backward_refusals(lib):
    opt = ref(RouteOptions(1, 0, 1.0))

    def call(z=P, bf16=0, o=opt, ids=P, dw=P, d=NULL, loss=NULL, T=8, G=16, k=2, dz=P):
        return lib.dg_moe_route_backward(z, bf16, o, ids, dw, d, loss, T, G, k, dz, NULL)

    for bad in (dict(T=-1), dict(G=0), dict(k=17), dict(G=1025), dict(G=64, k=33)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(z=NULL), dict(ids=NULL), dict(dz=NULL), dict(d=P), dict(loss=P), dict(o=NULL)):
        assert call(**bad) == ARG, bad
    for bad in (dict(z=ODD), dict(dz=ODD), dict(ids=ODD), dict(dw=ODD), dict(d=ODD, loss=P), dict(d=P, loss=ODD)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, z=NULL, ids=NULL, dz=NULL) == OK


def test_norm_refusals(lib):
    opt = ref(NormOptions(1.0, 1e-6, 0))

    def call(x=P, y=NULL, w=P, post=NULL, gate=NULL, o=opt, T=8, H=64, n=P, r=NULL, rstd=P, ry=NULL):
        return lib.dg_rmsnorm_residual(x, y, w, post, gate, o, T, H, n, r, rstd, ry, NULL)

    def codes(x=P, y=NULL, w=P, post=NULL, gate=NULL, o=opt, T=8, H=64, q=P, s=P, r=NULL):
        return lib.dg_rmsnorm_residual_quantize(x, y, w, post, gate, o, T, H, q, s, r, NULL)

    for f in (call, codes):
        for bad in (dict(T=-1), dict(T=1 << 31), dict(H=-16), dict(H=24), dict(H=16400), dict(H=1 << 62)):
            assert f(**bad) == SHAPE, bad
        for bad in (dict(x=NULL), dict(w=NULL), dict(o=NULL), dict(y=P), dict(r=P), dict(post=P), dict(gate=P),
                    dict(o=ref(NormOptions(0.5, 1e-6, 0))), dict(o=ref(NormOptions(1.0, -1e-6, 0))),
                    dict(o=ref(NormOptions(1.0, math.nan, 0))), dict(o=ref(NormOptions(math.inf, 0.0, 0)), y=P, r=P)):
            assert f(**bad) == ARG, bad
        for bad in (dict(x=ODD), dict(w=ODD), dict(y=ODD, r=P), dict(y=P, r=ODD), dict(y=P, r=P, post=ODD),
                    dict(y=P, r=P, gate=ODD)):
            assert f(**bad) == ALIGN, bad
        assert f(T=0, x=NULL, w=NULL) == OK and f(H=0, x=NULL, w=NULL) == OK
    assert call(n=NULL) == ARG and call(ry=P) == ARG and call(n=ODD) == ALIGN and call(rstd=ODD) == ALIGN
    assert codes(q=NULL) == ARG and codes(s=NULL) == ARG and codes(q=ODD) == ALIGN and codes(s=ODD) == ALIGN


def test_norm_backward_refusals(lib):
    opt = ref(NormOptions(1.0, 0.0, 0))
    need = lib.dg_rmsnorm_residual_backward_workspace(8, 64, 1, 1)
    assert need >= 2 * 64 * 4

    def call(dn=P, dr=NULL, r=P, rstd=P, y=P, ry=P, w=P, post=P, gate=P, o=opt, T=8, H=64, dx=P, dy=P, dw=P, dp=P, dg=P,
             ws=P, n=need):
        return lib.dg_rmsnorm_residual_backward(dn, dr, r, rstd, y, ry, w, post, gate, o, T, H, dx, dy, dw, dp, dg, ws, n,
                                                NULL)

    for bad in (dict(T=-1), dict(T=1 << 31), dict(H=24), dict(H=16400)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(dn=NULL), dict(r=NULL), dict(rstd=NULL), dict(w=NULL), dict(dx=NULL), dict(dw=NULL), dict(dy=NULL),
                dict(y=NULL), dict(y=NULL, dy=NULL), dict(ry=NULL), dict(dp=NULL), dict(dg=NULL), dict(post=NULL),
                dict(gate=NULL), dict(ws=NULL), dict(n=need - 1), dict(o=NULL), dict(o=ref(NormOptions(math.nan, 0.0, 0)))):
        assert call(**bad) == ARG, bad
    for name in ("dn", "dr", "r", "rstd", "y", "ry", "w", "post", "gate", "dx", "dy", "dw", "dp", "dg", "ws"):
        assert call(**{name: ODD}) == ALIGN, name
    assert call(H=0, w=NULL) == OK
    assert lib.dg_rmsnorm_residual_backward_workspace(8, 24, 0, 0) == lib.dg_rmsnorm_residual_backward_workspace(-1, 64, 0, 0) == 0


def test_gradient_norm_refusals(lib):
    def arrays(addresses, sizes, types):
        n = len(addresses)
        return ((ctypes.c_void_p * n)(*addresses), (ctypes.c_int64 * n)(*sizes), (ctypes.c_uint8 * n)(*types), n)

    def vp(a):
        return ctypes.cast(a, ctypes.c_void_p)

    need = lib.dg_grad_norm_workspace(2)
    limit = ctypes.c_float(1.0)

    def both(addresses, sizes, types=(0, 1), out=None, norm=ctypes.c_void_p(0x90000), ws=P, n=need, m=limit):
        a, s, t, count = arrays(addresses, sizes, types)
        o = NULL if out is None else vp((ctypes.c_void_p * count)(*out))
        got = [lib.dg_grad_norm_clip(vp(a), vp(s), vp(t), count, vp(ctypes.pointer(m)), o, norm, ws, n, NULL),
               lib.dg_grad_clip(vp(a), vp(s), vp(t), count, norm, vp(ctypes.pointer(m)), o, NULL)]
        assert got[0] == got[1] or ws is not P or n != need
        return got[0]

    ok = [0x10000, 0x20000]
    assert both(ok, [4, -1]) == SHAPE and both(ok, [4, (1 << 42) + 1]) == SHAPE
    assert both([0, 0x20000], [4, 4]) == ARG and both(ok, [4, 4], norm=NULL) == ARG
    assert both(ok, [4, 4], out=[0x30000, 0]) == ARG
    for m in (-1.0, math.inf, math.nan):
        assert both(ok, [4, 4], m=ctypes.c_float(m)) == ARG
    assert both([0x10002, 0x20000], [4, 4]) == ALIGN and both([0x10000, 0x20001], [4, 4]) == ALIGN
    assert both(ok, [4, 4], out=[0x30002, 0x40000]) == ALIGN and both(ok, [4, 4], norm=ODD) == ALIGN
    assert both(ok, [4, 4], ws=NULL) == ARG and both(ok, [4, 4], n=need - 8) == ARG and both(ok, [4, 4], ws=ODD) == ALIGN
    # tensors that overlap: the same twice, one inside the other, outputs over inputs
    assert both([0x10000, 0x10000], [4, 4]) == ARG and both([0x10000, 0x1000E], [4, 4]) == ARG
    assert both([0x10000, 0x10008], [100, 2]) == ARG and both(ok, [4, 4], out=[0x20000, 0x30000]) == ARG
    assert both(ok, [4, 4], out=[0x10004, 0x30000]) == ARG and both(ok, [4, 4], out=[0x30000, 0x30000]) == ARG
    # a norm inside a tensor that is written, or, where it is written itself, that is read
    assert both(ok, [4, 4], norm=ctypes.c_void_p(0x1000C)) == ARG and both(ok, [4, 4], norm=ctypes.c_void_p(0x20004)) == ARG
    assert both(ok, [4, 4], out=[0x30000, 0x40000], norm=ctypes.c_void_p(0x30008)) == ARG
    a, s, t, count = arrays(ok, [4, 4], [0, 1])
    o = vp((ctypes.c_void_p * 2)(0x30000, 0x40000))
    assert lib.dg_grad_norm_clip(vp(a), vp(s), vp(t), 2, vp(ctypes.pointer(limit)), o, ctypes.c_void_p(0x10008), P, need,
                                 NULL) == ARG
    assert lib.dg_grad_norm(vp(a), vp(s), vp(t), -1, P, P, need, NULL) == SHAPE
    assert lib.dg_grad_norm(NULL, vp(s), vp(t), 2, P, P, need, NULL) == ARG
    assert lib.dg_grad_norm(vp(a), vp(s), vp(t), 2, P, NULL, need, NULL) == ARG
    assert lib.dg_grad_norm_workspace(-1) == 0 and lib.dg_grad_norm_workspace(5000) > need


def test_binding_refuses_host_tensors(lib):
    z, x, w = torch.zeros((4, 8)), torch.zeros((4, 16), dtype=torch.bfloat16), torch.ones(16)
    for call in (lambda: binding.moe_route(z, 2), lambda: binding.moe_route(z, 2, score="linear"),
                 lambda: binding.moe_route_backward(z, torch.zeros((4, 2), dtype=torch.int32)),
                 lambda: binding.rmsnorm_residual(x, w), lambda: binding.rmsnorm_residual_quantize(x, w),
                 lambda: binding.rmsnorm_residual_backward(x, x, torch.ones(4), w), lambda: binding.grad_norm([z]),
                 lambda: binding.clip_grad_norm([z, z], 1.0), lambda: binding.grad_clip([z], torch.ones(()), 1.0)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        binding.grad_norm(z)  # a tensor is not a sequence of gradients


# ------------------------------------------------------- the plain forms, against differences
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_plain_route_gradient_is_that_of_differences(score, renormalize):
    g = torch.Generator().manual_seed(3)
    z = torch.randn((5, 7), generator=g, dtype=torch.float64)
    ids = plain.choose(z, 3, score)
    ids[4] = -1
    dw = torch.randn((5, 3), generator=g, dtype=torch.float64)
    dprob, dloss = torch.rand(7, generator=g, dtype=torch.float64), torch.tensor(0.3, dtype=torch.float64)

    def total(z):
        p = plain.probabilities(z, score)[1] * (ids >= 0).any(1, keepdim=True)
        return (plain.weights(z, ids, score, renormalize, 1.5) * dw).sum() + dloss * (p * dprob).sum()

    got, _ = plain.route_backward(z, ids, dw, dprob, dloss, score, renormalize, 1.5)
    check_differences(total, z, got)


def check_differences(total, at, got, h=1e-5):
    """Central differences: off by h^2 of the third derivative and 2^-52 / h of the value."""
    flat = at.reshape(-1)
    for i in range(flat.numel()):
        a, b = flat.clone(), flat.clone()
        a[i] += h
        b[i] -= h
        diff = (total(a.view(at.shape)) - total(b.view(at.shape))) / (2 * h)
        assert abs(float(diff - got.reshape(-1)[i])) < 1e-7


def test_plain_norm_gradient_is_that_of_differences():
    g = torch.Generator().manual_seed(4)
    T, H, alpha, eps = 3, 6, 0.5, 1e-3

    def rand(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)

    v = {"x": rand(T, H), "y": rand(T, H), "weight": rand(H), "post": rand(H), "gate": rand(H)}
    dn, dr = rand(T, H), rand(T, H)
    for post in (True, False):
        for gate in (True, False):
            u = {**v, "post": v["post"] if post else None, "gate": v["gate"] if gate else None}

            def total(**change):
                n, r = plain.norm_forward(**{**u, **change}, alpha=alpha, eps=eps)[0][:2]
                return (n * dn).sum() + (r * dr).sum()

            (_, r, rstd, rstd_y), _, _, _ = plain.norm_forward(**u, alpha=alpha, eps=eps)
            got = plain.norm_backward(dn, dr, r, rstd, u["y"], rstd_y, u["weight"], u["post"], u["gate"], alpha)
            names = {"x": "dx", "y": "dy", "weight": "dweight", "post": "dpost_weight", "gate": "dgate"}
            for name, grad in names.items():
                if u[name] is not None:
                    check_differences(lambda t: total(**{name: t}), u[name], got[grad][0])

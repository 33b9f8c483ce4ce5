"""GPU tests of routing, its counts and balance loss, and their gradient, against plain float64
forms: ids and counts exactly, the rest under bounds that count its roundings."""
import math

import pytest
import torch

from fp8_block_scaled_scales_b200 import binding

import plain_step as plain
from plain_step import BF, U

pytestmark = pytest.mark.gpu
INF = math.inf


def logits(T, G, seed, dtype=torch.float32, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, G), generator=g) * std + torch.randn((G,), generator=g) * 0.5).to(dtype)


def check(z, k, score="softmax", bias=None, mask=None, renormalize=True, scale=1.0):
    """Both forms of the call against the plain form; returns the ids."""
    T, G = z.shape
    kw = dict(score=score, bias=None if bias is None else bias.cuda(), mask=None if mask is None else mask.cuda(),
              renormalize=renormalize, scale=scale)
    ids, w = binding.moe_route(z.cuda(), k, **kw)
    z64 = z.double()
    want = plain.choose(z64, k, score, bias, mask)
    assert torch.equal(ids.cpu().long(), want)
    ref = plain.weights(z64, want, score, renormalize, scale)
    # e^(z - top): the argument's rounding and two steps; a sum of 37 additions at most, one
    # quotient or two and the scale; numerator and denominator both
    rel = (2 * plain.spread(z64).clamp_max(104) + 64) * U
    assert ((w.cpu().double() - ref).abs() <= rel * ref.abs() + 2.0 ** -126).all()
    ids2, w2, counts, loss, dprob = binding.moe_route(z.cuda(), k, balance=True, **kw)
    assert torch.equal(ids2, ids) and torch.equal(w2, w)
    c64, l64, d64 = plain.balance(z64, want, score)
    assert torch.equal(counts.cpu().long(), c64)
    assert ((dprob.cpu().double() - d64).abs() <= 2 * U * d64).all()
    # every probability as above (the quotient two steps more), then sums of up to T / 16 + 32 positive terms
    top = float(plain.spread(z64).clamp_max(104).max()) if T else 0.0
    assert abs(float(loss) - float(l64)) <= (2 * top + 128 + T / 16) * U * float(l64)
    return ids


SIZES = [(1, 1, 1), (1, 256, 8), (5, 64, 6), (37, 8, 2), (130, 33, 5), (64, 128, 1), (77, 300, 8), (33, 1024, 32),
         (600, 96, 4), (3000, 16, 2), (40, 513, 9), (65, 32, 32), (50, 31, 31)]


@pytest.mark.parametrize("T,G,k", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route(T, G, k, score, dtype):
    z = logits(T, G, T + G + k, dtype)
    bias = (torch.rand((G,), generator=torch.Generator().manual_seed(G)) - 0.5) * 0.3
    mask = torch.arange(T) % 5 != 3
    check(z, k, score)
    check(z, k, score, bias=bias, renormalize=False, scale=2.5)
    check(z, k, score, mask=mask, renormalize=False)
    check(z, k, score, bias=bias, mask=mask.to(torch.uint8), scale=0.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G", [20, 64, 300])
def test_equal_scores_go_to_the_lowest_id(score, G):
    z = torch.randint(-2, 3, (200, G), generator=torch.Generator().manual_seed(G)).float()
    z[0] = 0.0
    z[1, ::2] = -0.0  # equal to +0
    z[1, 1::2] = 0.0
    ids = check(z, 6, score)
    assert ids[0].tolist() == list(range(6)) and ids[1].tolist() == list(range(6))
    check(z, 6, score, bias=torch.zeros(G))
    check(z, 6, score, bias=torch.randint(0, 2, (G,), generator=torch.Generator().manual_seed(1)).float() * 0.25)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G", [9, 64, 257])
def test_keys_that_float32_cannot_tell_apart(score, G):
    """Scores plus bias within a few float32 steps of each other: the order is that of the float64 keys."""
    z = logits(1, G, G + 3).repeat(50, 1)
    z += torch.randn((50, 1), generator=torch.Generator().manual_seed(2)) * 1e-4
    s = plain.probabilities(z[:1].double(), score)[0][0]
    check(z[:1].repeat(50, 1), min(G, 12), score, bias=(0.75 - s).float())
    check(z, min(G, 12), score, bias=(0.75 - s).float())
    # the same around sums far below the scores themselves
    check(z[:1].repeat(50, 1), min(G, 12), score, bias=(1e-3 - s).float())
    check(z, min(G, 12), score, bias=(1e-3 - s).float())


def test_experts_and_tokens_left_out():
    """-inf and NaN logits are not chosen; rows of nothing else reach no expert; a bias of -inf
    takes an expert out, one of +inf brings it first."""
    z = logits(40, 40, 7)
    z[:, 3] = -INF
    z[4, 5:] = -INF             # four experts are left
    z[5] = -INF                 # none
    z[6] = torch.finfo(torch.float32).min
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            ids = check(z, 6, score, renormalize=renormalize)
        assert ids[5].tolist() == [-1] * 6 and ids[4].tolist()[4:] == [-1, -1] and ids[6].tolist() == [0, 1, 2, 3, 4, 5]
        bias = torch.zeros(40)
        bias[7], bias[9], bias[11] = -INF, INF, math.nan
        ids, w = binding.moe_route(z.cuda(), 6, score=score, bias=bias.cuda())
        ids = ids.cpu()
        assert not ((ids == 7) | (ids == 11)).any() and not (ids[z[:, 3] == -INF] == 3).any()
        for t in range(40):
            assert (ids[t, 0] == 9) == bool(z[t, 9] > -INF), t
        nan = z.clone()
        nan[8, 2] = math.nan
        nan[9] = math.nan
        ids, w, counts, loss, _ = binding.moe_route(nan.cuda(), 6, score=score, balance=True)
        assert 2 not in ids[8].tolist() and ids[9].tolist() == [-1] * 6 and w[9].tolist() == [0.0] * 6
        keep = torch.arange(40) != 8
        assert not torch.isnan(w.cpu()[keep]).any() and math.isnan(float(loss))
        all_out, w, counts, loss, dprob = binding.moe_route(z.cuda(), 6, score=score, balance=True,
                                                            mask=torch.zeros(40, dtype=torch.bool, device="cuda"))
        assert bool((all_out == -1).all()) and bool((w == 0).all()) and bool((counts == 0).all())
        assert float(loss) == 0.0 and bool((dprob == 0).all())


def test_far_scores_neither_overflow_nor_vanish():
    z = logits(60, 30, 11)
    z[:20] -= 300.0   # every sigmoid is 0 in float32
    z[20:40] += 300.0
    z[40:] *= 40.0
    for score in ("softmax", "sigmoid"):
        check(z, 4, score)
        g = torch.randn((60, 4), generator=torch.Generator().manual_seed(1))
        check_backward(z, 4, score, True, g)


def check_backward(z, k, score, renormalize, dw, balance=True, mask=None, scale=1.5, ids=None):
    zc = z.cuda()
    if ids is None:
        ids = binding.moe_route(zc, k, score=score, mask=None if mask is None else mask.cuda())[0]
    dprob = torch.rand((z.shape[1],), generator=torch.Generator().manual_seed(5)) if balance else None
    dloss = torch.tensor(0.37) if balance else None
    got = binding.moe_route_backward(zc, ids, None if dw is None else dw.cuda(), None if dprob is None else dprob.cuda(),
                                     None if dloss is None else dloss.cuda(), score=score, renormalize=renormalize,
                                     scale=scale)
    assert got.dtype == z.dtype
    z64 = z.double()
    dw64 = torch.zeros(ids.shape, dtype=torch.float64) if dw is None else dw.double()
    want, mag = plain.route_backward(z64, ids.cpu().long(), dw64, None if dprob is None else dprob.double(),
                                     None if dloss is None else dloss.double(), score, renormalize, scale)
    # a probability's error as in the forward pass, sums of at most 37 and 32 terms of these
    # magnitudes, a few products; then the output's rounding
    rel = (4 * plain.spread(z64).clamp_max(104) + 192) * U
    out = {torch.float32: U, torch.bfloat16: BF}[z.dtype]
    bound = rel * mag * (1 + out) + out * want.abs() + 2.0 ** -126
    assert ((got.cpu().double() - want).abs() <= bound).all()
    return got


@pytest.mark.parametrize("T,G,k", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_backward(T, G, k, score, dtype):
    z = logits(T, G, T + G + k + 1, dtype)
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(T))
    mask = torch.arange(T) % 4 != 2
    for renormalize in (True, False):
        check_backward(z, k, score, renormalize, dw)
        check_backward(z, k, score, renormalize, dw, balance=False, mask=mask)
        check_backward(z, k, score, renormalize, None, mask=mask)


# several tokens a warp, whose slots are finished side by side
MANY = [(20011, 8, 2), (9001, 64, 1), (12000, 40, 3), (6007, 300, 8), (5003, 1000, 32), (11000, 33, 31), (10000, 128, 16)]


@pytest.mark.parametrize("T,G,k", MANY)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tokens(T, G, k, score):
    dtype = torch.bfloat16 if T % 2 else torch.float32
    z = logits(T, G, T + k, dtype)
    bias = (torch.rand((G,), generator=torch.Generator().manual_seed(G)) - 0.5) * 0.3
    mask = torch.arange(T) % 7 != 3
    check(z, k, score, bias=bias, mask=mask, renormalize=False, scale=2.5)
    ids = check(z, k, score)
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(T))
    for renormalize in (True, False):
        check_backward(z, k, score, renormalize, dw, ids=ids)
        check_backward(z, k, score, renormalize, dw, balance=False, mask=mask)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tokens_with_ids_named_twice(score):
    T, G = 15000, 50
    z = logits(T, G, 3)
    ids = torch.randint(-2, 53, (T, 5), generator=torch.Generator().manual_seed(4), dtype=torch.int32)
    ids[::50] = -1
    dw = torch.randn((T, 5), generator=torch.Generator().manual_seed(6))
    for renormalize in (True, False):
        for balance in (True, False):
            check_backward(z, 5, score, renormalize, dw, balance=balance, ids=ids.cuda())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_of_ids_named_twice_and_out_of_range(score):
    z = logits(300, 50, 3)
    ids = torch.randint(-2, 53, (300, 5), generator=torch.Generator().manual_seed(4), dtype=torch.int32)
    ids[0] = 7
    ids[1] = -1
    ids[2] = torch.tensor([50, 1 << 30, -(1 << 31), 2, 2])
    dw = torch.randn((300, 5), generator=torch.Generator().manual_seed(6))
    ok = (ids >= 0) & (ids < 50)
    for renormalize in (True, False):
        for balance in (True, False):
            got = check_backward(z, 5, score, renormalize, dw, balance=balance, ids=ids.cuda())
            assert not got.cpu()[~ok.any(1)].any()


def test_masked_experts_get_no_gradient():
    z = logits(20, 24, 9)
    z[:, 5] = -INF
    z[3] = -INF
    for score in ("softmax", "sigmoid"):
        got = check_backward(z, 3, score, True, torch.ones((20, 3)))
        assert not got[:, 5].any() and not got[3].any()


def test_many_tokens_repeat_bit_for_bit():
    """More tokens than a wave takes, one call after another on one stream and two at once."""
    z = logits(20011, 64, 21).cuda()
    bias = (torch.rand(64, device="cuda") - 0.5) * 0.1
    first = binding.moe_route(z, 6, score="sigmoid", bias=bias, balance=True)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a = binding.moe_route(z, 6, score="sigmoid", bias=bias, balance=True, stream=s1)
        b = binding.moe_route(z, 6, score="sigmoid", bias=bias, balance=True, stream=s2)
    torch.cuda.synchronize()
    for x, y, w in zip(first, a, b):
        assert torch.equal(x, y) and torch.equal(x, w)
    counts, loss, dprob = plain.balance(z.cpu().double(), first[0].cpu().long(), "sigmoid")
    assert torch.equal(first[2].cpu().long(), counts) and abs(float(first[3]) - float(loss)) < 1e-5 * float(loss)


def test_no_tokens():
    z = torch.zeros((0, 12), device="cuda")
    ids, w, counts, loss, dprob = binding.moe_route(z, 3, balance=True)
    assert ids.shape == (0, 3) and counts.tolist() == [0] * 12 and float(loss) == 0.0 and dprob.tolist() == [0.0] * 12
    assert binding.moe_route(z, 3)[0].shape == (0, 3)
    assert binding.moe_route_backward(z, ids, w).shape == (0, 12)


def test_captured_and_replayed():
    z, dw = logits(700, 40, 1).cuda(), torch.randn((700, 4), device="cuda")
    dloss = torch.tensor(0.01, device="cuda")
    outs = binding.moe_route(z, 4, balance=True)
    dz = binding.moe_route_backward(z, outs[0], dw, outs[4], dloss)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.moe_route(z, 4, balance=True, topk_ids=outs[0], weights=outs[1], counts=outs[2], loss=outs[3], dprob=outs[4])
        binding.moe_route_backward(z, outs[0], dw, outs[4], dloss, dlogits=dz)
    for seed in (2, 3):
        z.copy_(logits(700, 40, seed))
        graph.replay()
        want = binding.moe_route(z, 4, balance=True)
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        assert torch.equal(dz, binding.moe_route_backward(z, want[0], dw, want[4], dloss))

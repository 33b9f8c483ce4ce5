"""GPU tests of routing, the norms around a block and clipping where a call is allowed but unusual:
few experts beside other work, rows that reach no expert, extreme magnitudes, gradients given by
an iterator."""
import pytest
import torch

from fp8_block_scaled_scales_b200 import binding

import plain_step as plain
from plain_step import U

pytestmark = pytest.mark.gpu


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

"""GPU tests of the gradient products: every element against float64, integers bit for bit."""
import numpy as np
import pytest
import torch

from fp8_block_scaled_scales_b200 import binding

import plain_train as plain

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def quantized(R, C, seed, scale=1.0):
    x = torch.randn((R, C), generator=torch.Generator().manual_seed(seed)) * scale
    if R > 3:
        x[R // 3] *= 30
    q, s = binding.quantize_blockwise(x.to(BF16).cuda())
    return q, s


def check(got, ref, mag, blocks, dtype, what=""):
    err = (got.cpu().double() - ref).abs()
    bound = plain.product_bound(mag, blocks, ref, dtype)
    assert bool((err <= bound).all()), f"{what}: worst ratio {float((err / bound).max()):.4g}"


# one block and less, tails in every size, both tile widths, several rounds of tiles
DENSE = [(1, 16, 16), (5, 128, 128), (128, 128, 256), (200, 272, 144), (129, 400, 528), (1000, 528, 784),
         (384, 1280, 640), (2300, 1040, 2064), (5000, 272, 400)]  # the last: past the four-stage rule of wgrad


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dgrad_dense(M, N, K):
    dy, sdy = quantized(M, N, M + N, 1e-3)
    w, sw = quantized(N, K, N + K, 0.02)
    got = binding.dgrad_blockscaled(dy, sdy, w, sw)
    a, b = plain.decode(dy.cpu(), sdy.cpu()), plain.decode(w.cpu(), sw.cpu())
    check(got, a @ b, a.abs() @ b.abs(), -(-N // 128), BF16)
    assert binding.last_device_status() == 0


@pytest.mark.parametrize("M,N,K", DENSE)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_wgrad_dense(M, N, K, dtype):
    dy, sdy = quantized(M, N, M + N, 1e-3)
    x, sx = quantized(M, K, M + K)
    C = torch.full((N, K), float("nan"), dtype=dtype, device="cuda")
    binding.wgrad_blockscaled(dy, sdy, x, sx, C=C)
    a, b = plain.decode(dy.cpu(), sdy.cpu()).t(), plain.decode(x.cpu(), sx.cpu())
    check(C, a @ b, a.abs() @ b.abs(), -(-M // 128), dtype)
    assert binding.last_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(256, 128, 512), (300, 144, 400), (64, 512, 128)])
def test_products_of_small_integers_are_exact(M, N, K):
    """Codes of small integers and scales of powers of two: every sum is an FP32 integer multiple, so the
    FP32 result is the exact one and the BF16 result its rounding."""
    rng = np.random.default_rng(M)
    val = torch.tensor([-2.0, -1.0, 0.0, 1.0, 2.0])

    def codes(R, C):
        v = val[torch.from_numpy(rng.integers(0, 5, (R, C)))]
        s = torch.from_numpy(2.0 ** rng.integers(-2, 3, (-(-R // 128), -(-C // 128)))).float()
        return v.to(torch.float8_e4m3fn).cuda(), s.cuda()

    dy, sdy = codes(M, N)
    x, sx = codes(M, K)
    w, sw = codes(N, K)
    a = plain.decode(dy.cpu().view(torch.uint8), sdy.cpu())
    ref = a.t() @ plain.decode(x.cpu().view(torch.uint8), sx.cpu())
    got = binding.wgrad_blockscaled(dy, sdy, x, sx)
    assert torch.equal(got.cpu().double(), ref)
    binding.wgrad_blockscaled(dy, sdy, x, sx, C=got, accumulate=True)
    assert torch.equal(got.cpu().double(), 2 * ref)
    ref = (a @ plain.decode(w.cpu().view(torch.uint8), sw.cpu())).float().to(BF16)
    assert torch.equal(binding.dgrad_blockscaled(dy, sdy, w, sw).cpu(), ref)


# few tiles, long sums: cut into parts that are added up in order
LONG_WGRAD = [(1537, 48, 80), (2000, 528, 272), (8191, 16, 16), (4096, 256, 256), (3000, 1040, 528)]
LONG_DGRAD = [(1, 1552, 48), (37, 2000, 784), (130, 4096, 272), (300, 1536, 528)]


@pytest.mark.parametrize("M,N,K", LONG_WGRAD)
def test_wgrad_of_long_sums(M, N, K):
    """Both types, added to a gradient, twice the same bits, and no write outside the matrix."""
    assert binding.lib().dg_fp8_wgrad_workspace(M, N, K) > 0
    dy, sdy = quantized(M, N, M + N, 1e-3)
    x, sx = quantized(M, K, M + K)
    a, b = plain.decode(dy.cpu(), sdy.cpu()).t(), plain.decode(x.cpu(), sx.cpu())
    ref, mag = a @ b, a.abs() @ b.abs()
    for dtype in (F32, BF16):
        C = torch.full((N + 2, K), -3.0, dtype=dtype, device="cuda")
        binding.wgrad_blockscaled(dy, sdy, x, sx, C=C[1:-1])
        check(C[1:-1], ref, mag, -(-M // 128), dtype)
        assert bool((C[0] == -3.0).all()) and bool((C[-1] == -3.0).all())
        again = binding.wgrad_blockscaled(dy, sdy, x, sx, dtype=dtype)
        assert torch.equal(again, C[1:-1])
    base = torch.randn((N, K), generator=torch.Generator().manual_seed(1)).cuda()
    C = base.clone()
    binding.wgrad_blockscaled(dy, sdy, x, sx, C=C, accumulate=True)
    check(C, base.cpu().double() + ref, mag + base.cpu().double().abs(), -(-M // 128) + 1, F32)
    assert binding.last_device_status() == 0


@pytest.mark.parametrize("M,N,K", LONG_DGRAD)
def test_dgrad_of_long_sums(M, N, K):
    assert binding.lib().dg_fp8_dgrad_workspace(M, N, K) > 0
    dy, sdy = quantized(M, N, M + N, 1e-3)
    w, sw = quantized(N, K, N + K, 0.02)
    C = torch.full((M + 2, K), -3.0, dtype=BF16, device="cuda")
    binding.dgrad_blockscaled(dy, sdy, w, sw, C=C[1:-1])
    a, b = plain.decode(dy.cpu(), sdy.cpu()), plain.decode(w.cpu(), sw.cpu())
    check(C[1:-1], a @ b, a.abs() @ b.abs(), -(-N // 128), BF16)
    assert bool((C[0] == -3.0).all()) and bool((C[-1] == -3.0).all())
    assert torch.equal(binding.dgrad_blockscaled(dy, sdy, w, sw), C[1:-1])
    assert binding.last_device_status() == 0


def test_long_sums_at_once_and_captured():
    """Calls on two streams, each with parts of its own, and a captured one replayed on other codes."""
    M, N, K = 2500, 272, 400
    sets = [(*quantized(M, N, 10 + i, 1e-3), *quantized(M, K, 20 + i)) for i in range(3)]
    want = [binding.wgrad_blockscaled(*t) for t in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [binding.wgrad_blockscaled(*t, stream=st) for st, t in zip(streams, sets)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    live = [t.clone() for t in sets[0]]
    C = binding.wgrad_blockscaled(*live)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.wgrad_blockscaled(*live, C=C)
    for i in (1, 2):
        for dst, src in zip(live, sets[i]):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want[i])


COUNTS = [[128], [0, 0], [0, 384, 0, 128], [130, 0, 1, 700, 257], [1] * 9]


def grouped(counts, N, K, seed, extra=128):
    G = len(counts)
    off = np.concatenate([[0], np.cumsum((np.asarray(counts) + 127) // 128 * 128)])
    cap = int(off[-1]) + extra
    real = torch.zeros((cap, 1))
    for g, c in enumerate(counts):
        real[off[g]:off[g] + c] = 1
    gen = torch.Generator().manual_seed(seed)
    dy = binding.quantize_blockwise((torch.randn((cap, N), generator=gen) * real * 1e-3).to(BF16).cuda())
    x = binding.quantize_blockwise((torch.randn((cap, K), generator=gen) * real).to(BF16).cuda())
    w = binding.quantize_blockwise((torch.randn((G * N, K), generator=gen) * 0.02).to(BF16).cuda())
    w = (w[0].view(G, N, K), w[1].view(G, N // 128, -1))
    for t in (dy, x):  # rows past the last expert may hold anything
        t[0][int(off[-1]):] = 0x7F
        t[1][int(off[-1]) // 128:] = float("nan")
    return off, cap, dy, x, w, torch.from_numpy(off).int().cuda()


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", [(128, 128), (256, 528), (640, 400)])
def test_grouped_dgrad(counts, N, K):
    off, cap, dy, x, w, off_d = grouped(counts, N, K, N + K + len(counts))
    C = torch.full((cap, K), -3.0, dtype=BF16, device="cuda")
    binding.grouped_dgrad_contiguous(*dy, *w, off_d, C=C)
    assert binding.last_device_status() == 0
    for g in range(len(counts)):
        a, b = int(off[g]), int(off[g + 1])
        if b > a:
            p = plain.decode(dy[0][a:b].cpu(), dy[1][a // 128:b // 128].cpu())
            r = plain.decode(w[0][g].cpu(), w[1][g].cpu())
            check(C[a:b], p @ r, p.abs() @ r.abs(), N // 128, BF16, f"expert {g}")
    assert bool((C[int(off[-1]):] == -3).all()), "rows past the last expert were written"


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", [(128, 128), (256, 528), (640, 400)])
@pytest.mark.parametrize("dtype,accumulate", [(F32, False), (F32, True), (BF16, False)])
def test_grouped_wgrad(counts, N, K, dtype, accumulate):
    off, cap, dy, x, w, off_d = grouped(counts, N, K, N + K + len(counts))
    G = len(counts)
    C = torch.full((G, N, K), float("nan"), dtype=dtype, device="cuda")
    before = torch.zeros((G, N, K), dtype=torch.float64)
    if accumulate:
        before = torch.randn((G, N, K), generator=torch.Generator().manual_seed(1)) * 1e-2
        C.copy_(before)
        before = before.double()
    binding.grouped_wgrad_contiguous(*dy, *x, off_d, C=C, accumulate=accumulate)
    assert binding.last_device_status() == 0
    for g in range(G):
        a, b = int(off[g]), int(off[g + 1])
        if b == a:
            assert torch.equal(C[g].cpu().double(), before[g]), f"expert {g} without rows"
            continue
        p = plain.decode(dy[0][a:b].cpu(), dy[1][a // 128:b // 128].cpu()).t()
        r = plain.decode(x[0][a:b].cpu(), x[1][a // 128:b // 128].cpu())
        # the addition to C rounds once more
        check(C[g], p @ r + before[g], p.abs() @ r.abs() + before[g].abs(), (b - a) // 128, dtype, f"expert {g}")


def test_many_experts_and_two_calls_at_once():
    """More tiles than SMs, experts of very different length, on two streams; results do not change from run to run."""
    rng = np.random.default_rng(2)
    counts = [int(c) for c in rng.choice([0, 1, 128, 129, 900, 3000], size=24)]
    off, cap, dy, x, w, off_d = grouped(counts, 512, 768, 77)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    first = [binding.grouped_wgrad_contiguous(*dy, *x, off_d, stream=streams[0]),
             binding.grouped_dgrad_contiguous(*dy, *w, off_d, stream=streams[1])]
    again = [binding.grouped_wgrad_contiguous(*dy, *x, off_d, stream=streams[1]),
             binding.grouped_dgrad_contiguous(*dy, *w, off_d, stream=streams[0])]
    torch.cuda.synchronize()
    assert binding.last_device_status() == 0
    assert torch.equal(first[0], again[0]) and torch.equal(first[1][:int(off[-1])], again[1][:int(off[-1])])
    for g in np.argsort(counts)[-2:]:
        a, b = int(off[g]), int(off[g + 1])
        p = plain.decode(dy[0][a:b].cpu(), dy[1][a // 128:b // 128].cpu()).t()
        r = plain.decode(x[0][a:b].cpu(), x[1][a // 128:b // 128].cpu())
        check(first[0][g], p @ r, p.abs() @ r.abs(), (b - a) // 128, F32, f"expert {g}")


@pytest.mark.parametrize("bad", [[0, 100, 256], [128, 128, 256], [0, 256, 128], [0, 128, 1024]])
def test_malformed_offsets_compute_nothing(bad):
    off, cap, dy, x, w, off_d = grouped([128, 128], 256, 256, 3)
    bad_d = torch.tensor(bad, dtype=torch.int32, device="cuda")
    dw = torch.full((2, 256, 256), -3.0, device="cuda")
    dx = torch.full((cap, 256), -3.0, dtype=BF16, device="cuda")
    binding.grouped_wgrad_contiguous(*dy, *x, bad_d, C=dw)
    assert binding.last_device_status() == 7
    binding.grouped_dgrad_contiguous(*dy, *w, bad_d, C=dx)
    assert binding.last_device_status() == 7
    assert bool((dw == -3).all()) and bool((dx == -3).all())
    binding.grouped_dgrad_contiguous(*dy, *w, off_d, C=dx)
    assert binding.last_device_status() == 0 and not bool((dx[:256] == -3).any())


def test_outputs_past_32_bit_offsets():
    """More than 2^32 elements of dW and of dX: the last tiles are the ones looked at."""
    G, N, K = 33, 8192, 16384
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    off[G] = 256  # all rows belong to the last expert
    dy, sdy = quantized(256, N, 5)
    x, sx = quantized(256, K, 6)
    C = torch.empty((G, N, K), dtype=BF16, device="cuda")
    C[0, 0, :5] = 7
    binding.grouped_wgrad_contiguous(dy, sdy, x, sx, off, C=C)
    n, k = slice(N - 256, N), slice(K - 512, K)
    p = plain.decode(dy.cpu(), sdy.cpu())[:, n].t()
    r = plain.decode(x.cpu(), sx.cpu())[:, k]
    check(C[G - 1, n, k], p @ r, p.abs() @ r.abs(), 2, BF16)
    assert not bool(C[0, 0].any()) and not bool(C[G - 2, -1].any())
    del C
    M = 266_240  # x 16384 columns
    w, sw = quantized(128, K, 7)
    dy = torch.zeros((M, 128), dtype=torch.uint8, device="cuda")
    sdy = torch.ones((M // 128, 1), device="cuda")
    tail = quantized(128, 128, 8)
    dy[-128:], sdy[-1:] = tail
    dx = binding.dgrad_blockscaled(dy, sdy, w, sw)
    p, r = plain.decode(tail[0].cpu(), tail[1].cpu()), plain.decode(w.cpu(), sw.cpu())
    check(dx[-128:], p @ r, p.abs() @ r.abs(), 1, BF16)
    assert not bool(dx[M - 256:M - 128].any())
    assert binding.last_device_status() == 0


def test_no_rows():
    z = torch.empty((0, 128), dtype=torch.uint8, device="cuda")
    s = torch.empty((0, 1), device="cuda")
    C = torch.full((128, 128), 5.0, device="cuda")
    binding.wgrad_blockscaled(z, s, z, s, C=C, accumulate=True)
    assert bool((C == 5).all())
    assert not bool(binding.wgrad_blockscaled(z, s, z, s, C=C).any())
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert not bool(binding.grouped_wgrad_contiguous(z, s, z, s, off, dtype=BF16).any())
    assert binding.dgrad_blockscaled(z, s, torch.zeros((128, 16), dtype=torch.uint8, device="cuda"),
                                     torch.ones((1, 1), device="cuda")).shape == (0, 16)


def test_wgrad_against_differences():
    """d(sum of (X W^T) * dC) along a random direction of W; the product is linear in W."""
    M, N, K = 300, 144, 272
    dy, sdy = quantized(M, N, 1)
    x, sx = quantized(M, K, 2)
    d, X = plain.decode(dy.cpu(), sdy.cpu()), plain.decode(x.cpu(), sx.cpu())
    g = torch.Generator().manual_seed(0)
    W, D = torch.randn((N, K), generator=g).double(), torch.randn((N, K), generator=g).double()
    num = (((X @ (W + D).t()) * d).sum() - ((X @ (W - D).t()) * d).sum()) / 2
    got = binding.wgrad_blockscaled(dy, sdy, x, sx).cpu().double()
    bound = plain.product_bound(d.abs().t() @ X.abs(), 3, got, F32)
    assert abs(float((got * D).sum() - num)) <= float((bound * D.abs()).sum()) + 1e-9 * abs(float(num))


def test_bounded_wait_reports_timeout_and_context_survives():
    dy, sdy = quantized(256, 512, 1)
    x, sx = quantized(256, 384, 2)
    w, sw = quantized(512, 384, 3)
    want = binding.wgrad_blockscaled(dy, sdy, x, sx), binding.dgrad_blockscaled(dy, sdy, w, sw)
    assert binding.last_device_status() == 0
    for call in (lambda: binding.wgrad_blockscaled(dy, sdy, x, sx), lambda: binding.dgrad_blockscaled(dy, sdy, w, sw)):
        try:
            binding.set_kernel_control(timeout_ns=50_000_000, debug_flags=1)
            call()
            status = binding.last_device_status()
        finally:
            binding.set_kernel_control(0, 0)
        assert status == 6
    assert torch.equal(binding.wgrad_blockscaled(dy, sdy, x, sx), want[0])
    assert torch.equal(binding.dgrad_blockscaled(dy, sdy, w, sw), want[1])
    assert binding.last_device_status() == 0


# many rows and too many tiles to cut the sum into parts: whole sums of the four-stage form
WHOLE_LONG = [(3300, 1296, 1040), (3201, 2064, 784)]


@pytest.mark.parametrize("M,N,K", WHOLE_LONG)
@pytest.mark.parametrize("dtype,accumulate", [(F32, False), (F32, True), (BF16, False)])
def test_wgrad_of_long_sums_in_whole(M, N, K, dtype, accumulate):
    assert binding.lib().dg_fp8_wgrad_workspace(M, N, K) == 0 and M // 128 > 24
    dy, sdy = quantized(M, N, M + N, 1e-3)
    x, sx = quantized(M, K, M + K)
    a, b = plain.decode(dy.cpu(), sdy.cpu()).t(), plain.decode(x.cpu(), sx.cpu())
    base = torch.zeros((N, K))
    if accumulate:
        base = torch.randn((N, K), generator=torch.Generator().manual_seed(1)) * 1e-2
    C = torch.full((N + 2, K), -3.0, dtype=dtype, device="cuda")
    C[1:-1] = base.cuda() if accumulate else float("nan")
    binding.wgrad_blockscaled(dy, sdy, x, sx, C=C[1:-1], accumulate=accumulate)
    # the addition to C rounds once more
    check(C[1:-1], base.double() + a @ b, base.double().abs() + a.abs() @ b.abs(), -(-M // 128) + 1, dtype)
    assert bool((C[0] == -3.0).all()) and bool((C[-1] == -3.0).all())
    assert binding.last_device_status() == 0


@pytest.mark.parametrize("dtype,accumulate", [(F32, False), (F32, True), (BF16, False)])
def test_grouped_wgrad_of_long_sums(dtype, accumulate):
    """More than 24 row blocks an expert on average, one expert without rows and one with a few."""
    counts, N, K = [6500, 0, 130, 7000], 256, 528
    off, cap, dy, x, w, off_d = grouped(counts, N, K, 9)
    assert cap // 128 > 24 * len(counts)
    before = torch.randn((4, N, K), generator=torch.Generator().manual_seed(2)) * 1e-2 if accumulate else torch.zeros((4, N, K))
    C = before.to(dtype).cuda() if accumulate else torch.full((4, N, K), float("nan"), dtype=dtype, device="cuda")
    binding.grouped_wgrad_contiguous(*dy, *x, off_d, C=C, accumulate=accumulate)
    for g in range(4):
        a, b = int(off[g]), int(off[g + 1])
        if a == b:
            assert torch.equal(C[g].cpu(), before[g].to(dtype))
            continue
        p = plain.decode(dy[0][a:b].cpu(), dy[1][a // 128:b // 128].cpu()).t()
        r = plain.decode(x[0][a:b].cpu(), x[1][a // 128:b // 128].cpu())
        check(C[g], p @ r + before[g].double(), p.abs() @ r.abs() + before[g].double().abs(), (b - a) // 128 + 1, dtype, f"expert {g}")
    assert binding.last_device_status() == 0

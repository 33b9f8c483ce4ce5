"""GPU tests of the sort by expert, the quantizing gather and the combination with its
gradient, against plain float64 forms and (codes, integers) bit for bit."""
import numpy as np
import pytest
import torch

import oracle
from fp8_block_scaled_scales_b200 import binding, inputs

import plain_train as plain

pytestmark = pytest.mark.gpu


def route(T, k, G, seed, drop=0.0, dtype=torch.int64, skew=1.0):
    rng = np.random.default_rng(seed)
    p = np.arange(1, G + 1, dtype=np.float64) ** -skew
    ids = rng.choice(G, size=(T, k), p=p / p.sum())  # a token may name an expert twice
    if drop:
        bad = rng.random((T, k)) < drop
        ids[bad] = rng.choice([-1, -7, G, G + 5], size=int(bad.sum()))
    return torch.from_numpy(ids).to(dtype)


SORTS = [
    (1, 1, 1), (1, 8, 64), (3, 2, 5), (37, 2, 8), (0, 4, 16), (129, 1, 128), (5, 64, 1024),
    (256, 8, 1024), (257, 8, 1024),  # the most that one CTA takes, and just past it, with the most experts
    (512, 8, 1024), (1000, 6, 33), (513, 8, 256), (5000, 7, 257), (20000, 8, 64), (32768, 1, 2),
    (40000, 4, 3),                   # chunks of more than one step
]


@pytest.mark.parametrize("T,k,G", SORTS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_sort(T, k, G, dtype, drop):
    ids = route(T, k, G, seed=T + k + G, drop=drop, dtype=dtype)
    cap = binding.moe_capacity(T, k, G) + 256  # a caller's larger row map
    want = plain.sort_plain(ids.numpy(), G, cap)
    slot = torch.full((cap,), 7, dtype=torch.int32, device="cuda")
    got = binding.moe_sort(ids.cuda(), G, slot_of_row=slot)
    for a, b, what in zip(got, want, ("offsets", "row_of_slot", "slot_of_row")):
        assert np.array_equal(a.cpu().numpy(), b), what


@pytest.mark.parametrize("T,k,G", SORTS)
@pytest.mark.parametrize("m_max", [1, 100, 384])
def test_sort_masked(T, k, G, m_max):
    ids = route(T, k, G, seed=T + k + G + 1, drop=0.1, dtype=torch.int32)
    want = plain.sort_masked_plain(ids.numpy(), G, m_max)
    got = binding.moe_sort_masked(ids.cuda(), G, m_max)
    for a, b, what in zip(got, want, ("masked_m", "row_of_slot", "slot_of_row")):
        assert np.array_equal(a.cpu().numpy(), b), what


def test_sort_ids_past_32_bits_are_dropped():
    ids = torch.tensor([[0, 1 << 32], [(1 << 32) + 1, 1], [-(1 << 40), 1 << 62]], dtype=torch.int64)
    off, row, slot = binding.moe_sort(ids.cuda(), 2)
    assert off.tolist() == [0, 128, 256] and row.tolist() == [[0, -1], [-1, 128], [-1, -1]]


@pytest.mark.parametrize("m_max,G", [(0, 4)])
def test_sort_masked_without_rows_drops_everything(m_max, G):
    m, row, slot = binding.moe_sort_masked(route(9, 2, G, 1).cuda(), G, m_max)
    assert m.tolist() == [0] * G and bool((row == -1).all()) and slot.numel() == 0


def test_sort_two_streams_and_graph():
    """Two calls at once on their own streams, and a captured call replayed on new ids."""
    G, a, b = 64, route(20000, 8, 64, 5).cuda(), route(100, 8, 64, 6).cuda()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        r1 = binding.moe_sort(a, G, stream=s1)
        r2 = binding.moe_sort(b, G, stream=s2)
    torch.cuda.synchronize()
    for ids, got in ((a, r1), (b, r2)):
        for x, y in zip(got, plain.sort_plain(ids.cpu().numpy(), G, binding.moe_capacity(*ids.shape, G))):
            assert np.array_equal(x.cpu().numpy(), y)
    ids = a.clone()
    outs = binding.moe_sort(ids, G)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.moe_sort(ids, G, *outs)
    ids.copy_(route(20000, 8, 64, 7).cuda())
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(outs, plain.sort_plain(ids.cpu().numpy(), G, outs[2].numel())):
        assert np.array_equal(x.cpu().numpy(), y)


def tokens(T, H, seed, scale=1.0):
    x = torch.randn((T, H), generator=torch.Generator().manual_seed(seed)) * scale
    if T:
        x[:: max(1, T // 3)] *= 40
        x[T // 2] = 0
    return x.to(torch.bfloat16)


def gathered(x, slot, k, weights=None):
    """float32 rows of the sorted layout."""
    ok = torch.from_numpy(slot >= 0)
    s = torch.from_numpy(np.maximum(slot, 0))
    v = x.float()[s // k]
    if weights is not None:
        v = v * weights.reshape(-1)[s][:, None]
    return torch.where(ok[:, None], v, torch.zeros(()))


@pytest.mark.parametrize("T,k,G,H", [(1, 1, 1, 16), (1, 8, 16, 4096), (5, 2, 3, 144), (37, 2, 8, 528), (300, 4, 5, 1040),
                                     (257, 8, 64, 256)])
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_is_the_block_quantizer_on_the_gathered_rows(T, k, G, H, weighted):
    ids = route(T, k, G, seed=T * 7 + H, drop=0.2)
    cap = plain.cap_of(T, k, G) + 128
    off, row, slot = plain.sort_plain(ids.numpy(), G, cap)
    x = tokens(T, H, T + H, 3e-3 if weighted else 1.0)
    w = (torch.rand((T, k), generator=torch.Generator().manual_seed(3)) + 0.01) if weighted else None
    v = gathered(x, slot, k, w)
    used = int(off[-1])
    q = torch.full((cap, H), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((cap // 128, -(-H // 128)), -7.0, device="cuda")
    binding.moe_dispatch_quantize(x.cuda(), torch.from_numpy(slot).int().cuda(), torch.from_numpy(off).int().cuda(), k,
                                  weights=None if w is None else w.cuda(), q=q, s=s)
    q, s = q.cpu(), s.cpu()
    if used:
        wq, ws = plain.quantize_f32(v[:used])
        assert torch.equal(q[:used], wq)
        assert torch.equal(s[:used // 128].view(torch.int32), ws.view(torch.int32))
        if not weighted:  # and the CPU oracle's quantizer on the BF16 rows
            oq, os_ = oracle.quantize_blockwise(inputs.bf16_bits(v[:used].to(torch.bfloat16)))
            assert np.array_equal(q[:used].numpy(), oq) and np.array_equal(s[:used // 128].numpy(), os_)
    assert bool((q[used:] == 0xA5).all()) and bool((s[used // 128:] == -7).all()), "rows past the last expert"


@pytest.mark.parametrize("T,k,G,H,m_max", [(1, 8, 64, 4096, 128), (37, 2, 8, 144, 40), (600, 4, 3, 272, 500), (300, 1, 1, 128, 300)])
def test_dispatch_masked(T, k, G, H, m_max):
    ids = route(T, k, G, seed=T + H)
    m, row, slot = plain.sort_masked_plain(ids.numpy(), G, m_max)
    x = tokens(T, H, T)
    v = gathered(x, slot, k).view(G, m_max, H)
    q = torch.full((G, m_max, H), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((G, -(-m_max // 128), -(-H // 128)), -7.0, device="cuda")
    binding.moe_dispatch_quantize_masked(x.cuda(), torch.from_numpy(slot).int().cuda(),
                                         torch.from_numpy(m).int().cuda(), k, q=q, s=s)
    q, s = q.cpu(), s.cpu()
    for g in range(G):
        c = int(m[g])
        nb = -(-c // 128)
        if c:
            wq, ws = plain.quantize_f32(v[g, :c])
            assert torch.equal(q[g, :c], wq) and torch.equal(s[g, :nb], ws)
        assert bool((q[g, c:] == 0xA5).all()) and bool((s[g, nb:] == -7).all())


def test_dispatch_never_reads_tokens_without_a_slot():
    """Infinities and NaN in tokens that no row holds, and in weights of dropped slots, leave no trace;
    slots outside the table are rows without a slot."""
    T, k, G, H = 40, 2, 4, 256
    ids = route(T, k, G, 11)
    ids[::3] = -1
    cap = plain.cap_of(T, k, G)
    off, row, slot = plain.sort_plain(ids.numpy(), G, cap)
    x, w = tokens(T, H, 1), torch.rand((T, k))
    want = plain.quantize_f32(gathered(x, slot, k, w)[:int(off[-1])])
    x[::3], w[::3] = float("nan"), float("inf")
    slot[slot < 0] = np.resize([-1, T * k, 1 << 30, -(1 << 31)], (slot < 0).sum())
    q, s = binding.moe_dispatch_quantize(x.cuda(), torch.from_numpy(slot).int().cuda(),
                                         torch.from_numpy(off).int().cuda(), k, weights=w.cuda())
    assert torch.equal(q[:int(off[-1])].cpu(), want[0]) and torch.equal(s[:int(off[-1]) // 128].cpu(), want[1])


def test_dispatch_every_bf16_pattern_under_a_scale_sweep():
    """All finite BF16 values under block maxima over the whole range (subnormal to near the largest, powers of
    two, multiples of 7, arbitrary ones): the codes and scales of the block quantizer, bit for bit."""
    bits = torch.arange(65536, dtype=torch.int32)
    finite = bits[(bits & 0x7F80) != 0x7F80]
    tops = [0x0001, 0x0007, 0x0080, 0x0700, 0x1000, 0x123F, 0x2A5C, 0x3C00, 0x3F80, 0x3FE0, 0x4055, 0x43E0, 0x43E1,
            0x4B0E, 0x5A5A, 0x6C63, 0x7000, 0x7F7F]
    rows = []
    for top in tops:
        keep = finite[(finite & 0x7FFF) <= top]
        n = -(-keep.numel() // 16383) * 16383
        keep = torch.cat([keep, torch.full((n - keep.numel(),), top, dtype=torch.int32)])
        for block in keep.view(-1, 16383):  # every block holds the maximum
            rows.append(torch.cat([block, torch.tensor([top], dtype=torch.int32)]).view(128, 128))
    x = torch.cat(rows).to(torch.int16).view(torch.bfloat16).cuda()
    T = x.shape[0]
    off, row, slot = binding.moe_sort(torch.zeros((T, 1), dtype=torch.int32, device="cuda"), 1)
    q, s = binding.moe_dispatch_quantize(x, slot, off, 1)
    wq, ws = binding.quantize_blockwise(x)
    assert torch.equal(s[:T // 128].view(torch.int32), ws.view(torch.int32))
    assert torch.equal(q[:T], wq)


def dispatch_slot_by_slot(x, slot, off, k, weights=None):
    """The same gather with every slot a token of its own: k = 1, the form that reads rows once a slot."""
    w = None if weights is None else weights.reshape(-1, 1)
    return binding.moe_dispatch_quantize(x.repeat_interleave(k, 0), slot, off, 1, weights=w)


def assert_same_codes(got, want, off):
    used = int(off[-1])
    (q, s), (wq, ws) = got, want
    assert torch.equal(s[:used // 128].nan_to_num(nan=-1.0), ws[:used // 128].nan_to_num(nan=-1.0))
    assert torch.equal(q[:used], wq[:used])


# more than 2^26 codes and eight slots a token or more: gathered token by token
TOKEN_FORM = [(2100, 8, 64, 4112), (1030, 9, 5, 7440), (600, 20, 300, 8192), (65, 70, 128, 16400)]


@pytest.mark.parametrize("T,k,G,H", TOKEN_FORM)
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_token_by_token(T, k, G, H, weighted):
    """Odd columns, dropped slots, experts without tokens, more slots than the eight of one step; blocks of zeros,
    of very small and of very large values; rows past the last expert stay as they were."""
    assert binding.lib().dg_moe_dispatch_workspace(T, k, H, plain.cap_of(T, k, G)) > 0
    assert binding.lib().dg_moe_dispatch_workspace(T * k, 1, H, plain.cap_of(T, k, G)) == 0
    g = torch.Generator().manual_seed(T)
    ids = torch.stack([torch.randperm(G, generator=g)[:k] if k <= G else torch.randint(0, G, (k,), generator=g)
                       for _ in range(T)]).int()
    ids[::7, 1] = -1
    ids[ids == 3] = 4 % G  # expert 3 stays without tokens
    x = tokens(T, H, T + 1)
    x[:, 256:384] = 0
    x[:, 128:256] *= 1e-36
    x[: T // 2, 384:512] *= 1e36
    x = x.cuda()
    w = torch.randn((T, k), generator=g).cuda() if weighted else None
    if weighted:
        w[::5, 0], w[1::5, 1] = 0.0, 1e-30
    off, row, slot = binding.moe_sort(ids.cuda(), G)
    cap = slot.numel()
    assert int(off[-1]) < cap
    q = torch.full((cap, H), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((cap // 128, -(-H // 128)), -3.0, device="cuda")
    binding.moe_dispatch_quantize(x, slot, off, k, weights=w, q=q, s=s)
    assert_same_codes((q, s), dispatch_slot_by_slot(x, slot, off, k, w), off)
    used = int(off[-1])
    assert bool((q[used:] == 0xA5).all()) and bool((s[used // 128:] == -3.0).all())
    # against the definition, in a few row blocks
    slots = slot.cpu().numpy()
    for b in {0, used // 256, used // 128 - 1}:
        v = gathered(x.cpu(), slots[b * 128:(b + 1) * 128], k, None if w is None else w.cpu())
        wq, ws = plain.quantize_f32(v)
        assert torch.equal(s[b].cpu(), ws[0]) and torch.equal(q[b * 128:(b + 1) * 128].cpu(), wq)


@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_token_by_token_non_finite(weighted):
    """Blocks with NaN or infinite values or weights, the rows without a token in them included."""
    T, k, G, H = 1100, 8, 11, 7696
    x = tokens(T, H, 51).cuda()
    x[5, 10], x[200, 300], x[700, 7690] = float("nan"), float("inf"), -float("inf")
    w = torch.randn((T, k), generator=torch.Generator().manual_seed(52)).cuda() if weighted else None
    if weighted:
        w[3, 0], w[4, 1], w[20, 0] = float("inf"), -float("inf"), float("nan")
        x[3, 130:140], x[4, 256:384] = 0.0, 0.0
    off, row, slot = binding.moe_sort(route(T, k, G, 53).cuda(), G)
    got, want = binding.moe_dispatch_quantize(x, slot, off, k, weights=w), dispatch_slot_by_slot(x, slot, off, k, w)
    used = int(off[-1])
    bad = ~torch.isfinite(got[1][:used // 128])
    assert bool(bad.any()) and not bool(bad.all())
    assert_same_codes(got, want, off)


def test_dispatch_token_by_token_with_repeated_slots():
    """A row map of a caller's own, where slots stand in several rows, in none, or out of range."""
    T, k, H, cap = 1100, 8, 8208, 8960
    x = tokens(T, H, 61).cuda()
    g = torch.Generator().manual_seed(62)
    slot = torch.randint(-5, T * k + 5, (cap,), generator=g).int()
    slot[1000:1200] = 17
    slot[-128:] = -1
    slot, off = slot.cuda(), torch.tensor([0, 128, cap], dtype=torch.int32, device="cuda")
    w = torch.randn((T, k), generator=g).cuda()
    for weights in (None, w):
        assert_same_codes(binding.moe_dispatch_quantize(x, slot, off, k, weights=weights),
                          dispatch_slot_by_slot(x, slot, off, k, weights), off)


def test_dispatch_token_by_token_streams_and_graph():
    """Two calls at once on their own streams, and a captured call replayed on new tokens and routes."""
    T, k, G, H = 1100, 8, 16, 7696
    sets = []
    for i in range(3):
        x = tokens(T, H, 71 + i).cuda()
        sets.append((x, *binding.moe_sort(route(T, k, G, 81 + i).cuda(), G)))
    want = [dispatch_slot_by_slot(x, slot, off, k) for x, off, row, slot in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [binding.moe_dispatch_quantize(x, slot, off, k, stream=st) for st, (x, off, row, slot) in zip(streams, sets)]
    torch.cuda.synchronize()
    for a, b, (x, off, row, slot) in zip(got, want, sets):
        assert_same_codes(a, b, off)
    x, off, slot = (t.clone() for t in (sets[0][0], sets[0][1], sets[0][3]))
    q, s = binding.moe_dispatch_quantize(x, slot, off, k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.moe_dispatch_quantize(x, slot, off, k, q=q, s=s)
    for i in (2, 1):
        for dst, src in zip((x, off, slot), (sets[i][0], sets[i][1], sets[i][3])):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert_same_codes((q, s), want[i], off)


def test_dispatch_weights_of_both_signs_and_zero():
    """Negative and zero weights: magnitudes enter the scale, zeros keep the product's sign."""
    T, k, G, H = 50, 2, 3, 384
    ids = route(T, k, G, 21)
    cap = plain.cap_of(T, k, G)
    off, row, slot = plain.sort_plain(ids.numpy(), G, cap)
    x = tokens(T, H, 22)
    x[:, ::5] = 0
    w = torch.randn((T, k), generator=torch.Generator().manual_seed(23))
    w[::4, 0], w[1::4, 1] = 0.0, -0.0
    used = int(off[-1])
    q, s = binding.moe_dispatch_quantize(x.cuda(), torch.from_numpy(slot).int().cuda(),
                                         torch.from_numpy(off).int().cuda(), k, weights=w.cuda())
    wq, ws = plain.quantize_f32(gathered(x, slot, k, w)[:used])
    assert torch.equal(q[:used].cpu(), wq) and torch.equal(s[:used // 128].cpu(), ws)


def test_dispatch_non_finite_values_stay_in_their_block():
    """A NaN or an infinity in a used token makes its own block's scale non-finite, and no other."""
    T, H = 300, 384
    x = tokens(T, H, 31)
    clean = x.clone()
    x[5, 10], x[200, 300] = float("nan"), float("inf")
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    off, row, slot = binding.moe_sort(ids, 1)
    q, s = binding.moe_dispatch_quantize(x.cuda(), slot, off, 1)
    cq, cs = binding.moe_dispatch_quantize(clean.cuda(), slot, off, 1)
    bad = torch.zeros((3, 3), dtype=torch.bool)
    bad[0, 0] = bad[1, 2] = True
    assert torch.equal(~torch.isfinite(s[:3].cpu()), bad)
    assert torch.equal(s[:3].cpu()[~bad], cs[:3].cpu()[~bad])
    keep = ~bad.repeat_interleave(128, 0).repeat_interleave(128, 1)
    assert torch.equal(q[:384].cpu()[keep], cq[:384].cpu()[keep])


@pytest.mark.parametrize("T,k,H", [(40, 2, 400), (700, 8, 656)])
def test_dispatch_infinite_and_nan_weights(T, k, H):
    """Products with a weight that is not finite follow FP32: infinite (scale infinite, finite rows' codes 0) or,
    where the row has a zero in the block or the weight is NaN, NaN; other blocks stay as they are."""
    G = 3
    ids = route(T, k, G, 41)
    cap = plain.cap_of(T, k, G)
    off, row, slot = plain.sort_plain(ids.numpy(), G, cap)
    x = tokens(T, H, 42)
    x[x == 0] = 1.0
    x[3, 130:140] = 0.0  # zeros in one column block, next to values
    x[4, 256:384] = 0.0  # and a whole piece of them in another
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(43)) + 0.5
    w[3, 0], w[4, 1], w[20, 0] = float("inf"), -float("inf"), float("nan")
    used = int(off[-1])
    q, s = binding.moe_dispatch_quantize(x.cuda(), torch.from_numpy(slot).int().cuda(),
                                         torch.from_numpy(off).int().cuda(), k, weights=w.cuda())
    wq, ws = plain.quantize_f32(gathered(x, slot, k, w)[:used])
    assert bool(torch.isinf(ws).any()) and bool(torch.isnan(ws).any()) and bool(torch.isfinite(ws).any())
    assert torch.equal(s[:used // 128].cpu().nan_to_num(nan=-1.0), ws.nan_to_num(nan=-1.0))
    q, wq = q[:used].cpu(), wq.view(torch.uint8)
    nan = (wq & 0x7F) == 0x7F
    assert torch.equal((q & 0x7F) == 0x7F, nan) and torch.equal(q[~nan], wq[~nan])


@pytest.mark.parametrize("T,value", [(3, float("nan")), (20, float("inf")), (70, float("nan"))])
def test_dispatch_non_finite_values_in_blocks_of_few_rows(T, value):
    """The rows without a token take part: zero over a NaN scale is NaN, over an infinite one zero."""
    k, G, H = 2, 3, 272
    ids = route(T, k, G, T)
    cap = plain.cap_of(T, k, G)
    off, row, slot = plain.sort_plain(ids.numpy(), G, cap)
    x = tokens(T, H, T)
    x[1, 5] = value
    used = int(off[-1])
    q, s = binding.moe_dispatch_quantize(x.cuda(), torch.from_numpy(slot).int().cuda(),
                                         torch.from_numpy(off).int().cuda(), k)
    wq, ws = plain.quantize_f32(gathered(x, slot, k)[:used])
    assert torch.equal(s[:used // 128].cpu().nan_to_num(nan=-1.0), ws.nan_to_num(nan=-1.0))
    q, wq = q[:used].cpu(), wq.view(torch.uint8)
    nan = (wq & 0x7F) == 0x7F
    assert bool(nan.any()) and torch.equal((q & 0x7F) == 0x7F, nan) and torch.equal(q[~nan], wq[~nan])


def test_rows_past_32_bit_offsets():
    """Matrices of more than 2^32 elements: the last rows and tokens are the ones looked at."""
    H, rows = 16384, 270_080  # 4.4e9 elements
    T, k = 4, 2
    y = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
    r = torch.tensor([[0, rows - 1], [rows - 2, -1], [rows - 3, rows - 4], [131072, rows // 2]], dtype=torch.int32)
    for v in r.flatten().tolist():
        if v >= 0:
            y[v] = torch.randn(H, generator=torch.Generator().manual_seed(v)).to(torch.bfloat16)
    picked = torch.stack([torch.stack([y[v].cpu() if v >= 0 else torch.zeros(H, dtype=torch.bfloat16) for v in t]) for t in r.tolist()])
    ref = picked.double().sum(1)
    got = binding.moe_combine(y, r.cuda()).cpu().double()
    assert bool(((got - ref).abs() <= ref.abs() * 2.0 ** -8 + 2.0 ** -23 * picked.double().abs().sum(1)).all())
    dout = torch.randn((T, H), generator=torch.Generator().manual_seed(7)).to(torch.bfloat16)
    dw = binding.moe_combine_backward(dout.cuda(), y, r.cuda()).cpu().double()
    terms = picked.double() * dout.double()[:, None, :]
    assert bool(((dw - terms.sum(2)).abs() <= H * 2.0 ** -24 * terms.abs().sum(2)).all())
    # as tokens: the last ones gathered into the last rows of codes past 2^32 bytes
    cap = 270_080
    slot = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    slot[cap - 2], slot[cap - 1] = rows - 1, 0
    off = torch.tensor([0, cap], dtype=torch.int32, device="cuda")
    q = torch.empty((cap, H), dtype=torch.uint8, device="cuda")
    q, s = binding.moe_dispatch_quantize(y, slot, off, 1, q=q)
    block = torch.zeros((128, H))
    block[126], block[127] = y[rows - 1].cpu().float(), y[0].cpu().float()
    wq, ws = plain.quantize_f32(block)
    assert torch.equal(q[cap - 128:].cpu(), wq) and torch.equal(s[-1:].cpu(), ws)
    assert not bool(q[: cap - 128: 4096].any())


def test_dispatch_weights_so_small_that_the_scale_would_vanish():
    """amax / 448 rounds to zero in FP32: the scale is 1 and every code is a zero."""
    x = torch.full((1, 128), 2.0 ** -100, dtype=torch.bfloat16)
    q, s = binding.moe_dispatch_quantize(x.cuda(), torch.tensor([0] + [-1] * 127, dtype=torch.int32).cuda(),
                                         torch.tensor([0, 128], dtype=torch.int32).cuda(), 1,
                                         weights=torch.full((1, 1), 2.0 ** -46).cuda())
    assert s.item() == 1.0 and not bool((q & 0x7F).any())


COMBINES = [(1, 1, 16), (1, 8, 7168), (5, 8, 1040), (37, 2, 4096), (300, 6, 528), (64, 11, 144), (1030, 4, 2048)]


def combine_case(T, k, H, seed):
    G, g = 7, torch.Generator().manual_seed(seed)
    ids = route(T, k, G, seed, drop=0.25)
    ids[T // 2] = -1  # a token without any row
    cap = plain.cap_of(T, k, G)
    off, row, slot = plain.sort_plain(ids.numpy(), G, cap)
    y = torch.randn((cap, H), generator=g).to(torch.bfloat16)
    w = torch.randn((T, k), generator=g)
    return row, y, w, g


@pytest.mark.parametrize("T,k,H", COMBINES)
@pytest.mark.parametrize("weighted", [False, True])
def test_combine(T, k, H, weighted):
    row, y, w, _ = combine_case(T, k, H, T + k + H)
    r = torch.from_numpy(row)
    wt = torch.where(r >= 0, w.double() if weighted else torch.ones(T, k, dtype=torch.float64), torch.zeros((), dtype=torch.float64))
    terms = y.double()[r.clamp_min(0)] * wt[:, :, None]
    ref, mag = terms.sum(1), terms.abs().sum(1)
    y[torch.from_numpy(np.setdiff1d(np.arange(y.shape[0]), row))] = float("nan")  # rows no slot names
    got = binding.moe_combine(y.cuda(), r.int().cuda(), w.cuda() if weighted else None).cpu().double()
    # k FP32 multiply-adds, then one rounding to BF16
    assert bool(((got - ref).abs() <= k * 2.0 ** -24 * mag * (1 + 2.0 ** -8) + ref.abs() * 2.0 ** -8).all())
    assert bool((got[T // 2] == 0).all())


@pytest.mark.parametrize("T,k,H", COMBINES)
def test_combine_backward(T, k, H):
    row, y, w, g = combine_case(T, k, H, T + k + H + 1)
    dout = torch.randn((T, H), generator=g).to(torch.bfloat16)
    r = torch.from_numpy(row)
    terms = y.double()[r.clamp_min(0)] * dout.double()[:, None, :] * (r >= 0)[:, :, None]
    ref, mag = terms.sum(2), terms.abs().sum(2)
    y[torch.from_numpy(np.setdiff1d(np.arange(y.shape[0]), row))] = float("nan")
    got = binding.moe_combine_backward(dout.cuda(), y.cuda(), r.int().cuda()).cpu().double()
    # a chain of at most H FP32 multiply-adds, whatever its order
    assert bool(((got - ref).abs() <= H * 2.0 ** -24 * mag).all())
    assert bool((got[r < 0] == 0).all())


def test_combine_gradients_against_differences():
    """d(sum of out * dout) along a random direction of the weights, and of y, in float64."""
    T, k, H, G = 20, 3, 256, 4
    ids = route(T, k, G, 3, drop=0.2)
    cap = plain.cap_of(T, k, G)
    off, row, slot = plain.sort_plain(ids.numpy(), G, cap)
    g = torch.Generator().manual_seed(1)
    y = torch.randn((cap, H), generator=g).to(torch.bfloat16)
    w, dw_dir = torch.rand((T, k), generator=g), torch.randn((T, k), generator=g)
    dout = torch.randn((T, H), generator=g).to(torch.bfloat16)
    y_dir = torch.randn((cap, H), generator=g).double()
    r = torch.from_numpy(row)

    def loss(w, y):
        wt = torch.where(r >= 0, w.double(), torch.zeros((), dtype=torch.float64))
        return float(((y.double()[r.clamp_min(0)] * wt[:, :, None]).sum(1) * dout.double()).sum())

    e = 1e-3
    num_w = (loss(w + e * dw_dir.double(), y) - loss(w - e * dw_dir.double(), y)) / (2 * e)
    num_y = (loss(w, y.double() + e * y_dir) - loss(w, y.double() - e * y_dir)) / (2 * e)
    dw = binding.moe_combine_backward(dout.cuda(), y.cuda(), r.int().cuda()).cpu().double()
    # both are linear: the difference is exact up to float64; dw's own error as in the test above
    assert abs(float((dw * dw_dir).sum()) - num_w) <= 256 * 2.0 ** -24 * float((dw_dir.abs() * 256 * 8).sum()) + 1e-6
    q, s = binding.moe_dispatch_quantize(dout.cuda(), torch.from_numpy(slot).int().cuda(),
                                         torch.from_numpy(off).int().cuda(), k, weights=w.cuda())
    dy = plain.decode(q.cpu(), s.cpu())
    used = int(off[-1])
    step = plain.code_error_bound(gathered(dout, slot, k, w)[:used].double(), s[:used // 128].cpu(), 0.0)
    assert abs(float((dy[:used] * y_dir[:used]).sum()) - num_y) <= float((step * y_dir[:used].abs()).sum())


def test_combine_takes_the_masked_layout_and_no_rows():
    T, k, G, m_max, H = 30, 2, 5, 9, 144
    ids = route(T, k, G, 8)
    m, row, slot = plain.sort_masked_plain(ids.numpy(), G, m_max)  # some slots dropped
    assert (row < 0).any()
    y = torch.randn((G, m_max, H)).to(torch.bfloat16)
    r = torch.from_numpy(row)
    ref = (y.view(-1, H).double()[r.clamp_min(0)] * (r >= 0)[:, :, None]).sum(1)
    got = binding.moe_combine(y.cuda(), r.int().cuda()).cpu().double()
    assert bool(((got - ref).abs() <= 2.0 ** -22 * 10 + ref.abs() * 2.0 ** -8).all())
    none = binding.moe_combine(torch.empty((0, H), dtype=torch.bfloat16, device="cuda"), r.int().cuda())
    assert not bool(none.any())
    none = binding.moe_combine_backward(none, torch.empty((0, H), dtype=torch.bfloat16, device="cuda"), r.int().cuda())
    assert not bool(none.any())


def test_binding_refuses_wrong_types_shapes_and_strides():
    x = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    slot = torch.full((128,), -1, dtype=torch.int32, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    row = torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        binding.moe_dispatch_quantize(x.float(), slot, off, 2)
    with pytest.raises(ValueError):
        binding.moe_dispatch_quantize(x[:, ::2], slot, off, 2)
    with pytest.raises(ValueError):
        binding.moe_dispatch_quantize(x, slot.long(), off, 2)
    with pytest.raises(ValueError):
        binding.moe_dispatch_quantize(x, slot, off, 2, weights=torch.zeros((8, 3), device="cuda"))
    with pytest.raises(ValueError):
        binding.moe_combine(x, row, torch.zeros((8, 2), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        binding.moe_combine_backward(x, x[:, :32].contiguous(), row)
    with pytest.raises(ValueError):
        binding.moe_sort(row.float(), 4)
    with pytest.raises(binding.DGError):
        binding.moe_sort(row, 4, slot_of_row=slot)  # a row map too small for the worst case


@pytest.mark.parametrize("G,m_max", [(0, 1), (1025, 1), (2**31 - 1, 1), (1024, 2**21), (2**31 - 1, 2**31 - 1), (3, 2**31 - 1)])
def test_sorts_refuse_sizes_before_they_allocate(G, m_max):
    """G and M_max that the library refuses are refused as such, whatever their outputs would take."""
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    held = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    with pytest.raises(binding.DGError):
        binding.moe_sort_masked(ids, G, m_max)
    if not 1 <= G <= 1024:
        with pytest.raises(binding.DGError):
            binding.moe_sort(ids, G)
    assert torch.cuda.max_memory_allocated() == held


@pytest.mark.parametrize("T,k,G,m_max", [(0, 2, 8, 6912), (1, 8, 64, 4096), (128, 2, 8, 6912), (1024, 2, 8, 6912),
                                         (1025, 2, 8, 6912), (20000, 2, 8, 6912), (100, 8, 1024, 3001)])
def test_sort_masked_into_deep_slabs(T, k, G, m_max):
    """Slabs far deeper than an expert's tokens, by one CTA and in two launches; slabs that overflow."""
    ids = route(T, k, G, seed=T + G, drop=0.1, dtype=torch.int32)
    want = plain.sort_masked_plain(ids.numpy(), G, m_max)
    slot = torch.full((G * m_max,), 7, dtype=torch.int32, device="cuda")
    got = binding.moe_sort_masked(ids.cuda(), G, m_max, slot_of_row=slot)
    for a, b, what in zip(got, want, ("masked_m", "row_of_slot", "slot_of_row")):
        assert np.array_equal(a.cpu().numpy(), b), what


@pytest.mark.parametrize("T,k,H", [(300, 1, 400), (1100, 8, 7696)])
def test_dispatch_of_non_finite_tokens_is_the_block_quantizer(T, k, H):
    """Codes bit for bit (a NaN's too) and scales of dg_quantize_blockwise on the gathered rows, in both forms."""
    x = tokens(T, H, 91).cuda()
    x[5, 10], x[200, 300], x[7, 200], x[250, H - 1] = float("nan"), float("inf"), -float("inf"), -float("nan")
    x[:, 128:256] = -x[:, 128:256].abs()
    off, row, slot = binding.moe_sort(route(T, k, 5, 92).cuda(), 5)
    used, s_of_row = int(off[-1]), slot.clamp_min(0).long()
    rows = torch.where((slot >= 0)[:, None], x[s_of_row // k], torch.zeros((), dtype=x.dtype, device="cuda"))[:used]
    q, s = binding.moe_dispatch_quantize(x, slot, off, k)
    wq, ws = binding.quantize_blockwise(rows.contiguous())
    assert torch.equal(q[:used], wq)
    assert torch.equal(s[:used // 128].nan_to_num(nan=-1.0), ws.nan_to_num(nan=-1.0)) and not bool(torch.isfinite(ws).all())

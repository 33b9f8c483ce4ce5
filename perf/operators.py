"""Cases that measure the operators of a mixture-of-experts layer around the FP8 grouped
products: tokens sorted by expert, gathered and quantized; expert rows brought back with
their weights, and the gradient of that; SwiGLU with an 8-bit checkpoint of its input and
its backward pass; and the gradient products that read the 8-bit codes the forward pass
left.

Every case has a plain form in elementary torch operations (float32 sums), the call of
this repository's own kernels, and a float64 evaluation of the definition.

Layouts (those of the grouped products): an expert's rows start at a multiple of 128;
codes are E4M3 bytes with one float32 scale per 128 x 128 block, or per row and
128 columns (stored column-group first) for the checkpoint.
"""
import math

import torch

own = False

B = 128


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one generated token routed to its 8 of 64 experts: the smallest call of a decode step
        {"name": "sort_decode_1", "op": "sort_masked", "T": 1, "k": 8, "G": 64, "m_max": 128, "wide": True},
        # a large training batch, fine-grained experts
        {"name": "sort_train_16384x8", "op": "sort", "T": 16384, "k": 8, "G": 256, "wide": True, "drop": 0.0},
        # a decode batch into the masked slabs of 8 experts
        {"name": "dispatch_decode_37", "op": "dispatch_masked", "T": 37, "k": 2, "G": 8, "H": 4096, "m_max": 128},
        # the activations of the 64-expert workload (32768 slots, K = 7168), from its tokens
        {"name": "dispatch_g64", "op": "dispatch", "T": 4096, "k": 8, "G": 64, "H": 7168},
        # a decode batch brought back
        {"name": "combine_decode_5", "op": "combine", "T": 5, "k": 8, "G": 64, "H": 7168},
        # the 64-expert workload brought back
        {"name": "combine_g64", "op": "combine", "T": 4096, "k": 8, "G": 64, "H": 7168},
        # gradient of that for the 8-expert workload (16384 slots): weights' gradient, and
        # the rows' gradient as codes for the gradient products
        {"name": "combine_backward_g8", "op": "combine_backward", "T": 8191, "k": 2, "G": 8, "H": 4096},
        # SwiGLU between the two products of 8 experts, with the checkpoint for the backward pass
        {"name": "swiglu_g8", "op": "swiglu", "T": 8192, "k": 2, "G": 8, "F": 4096},
        # its backward pass on a ragged dense batch
        {"name": "swiglu_backward_1000", "op": "swiglu_backward", "M": 1000, "F": 2048},
        # input gradient of the 8-expert workload
        {"name": "dgrad_g8", "op": "grouped_dgrad", "T": 8192, "k": 2, "G": 8, "N": 4096, "K": 4096},
        # weight gradient of the 64-expert workload, float32 (the optimizer's type)
        {"name": "wgrad_g64", "op": "grouped_wgrad", "T": 4096, "k": 8, "G": 64, "N": 2048, "K": 7168, "bf16": False},
        # weight gradient of a small dense layer, ragged in every size
        {"name": "wgrad_dense_odd", "op": "wgrad", "M": 1000, "N": 528, "K": 784, "bf16": True},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(v / step) * step)


def draw(rng):
    op = rng.choice(["sort", "sort_masked", "dispatch", "dispatch_masked", "combine", "combine_backward",
                     "swiglu", "swiglu_backward", "dgrad", "wgrad", "grouped_dgrad", "grouped_wgrad"])
    k = rng.choice([1, 2, 4, 6, 8])
    G = max(k, _log(rng, 2, 256))
    T = _log(rng, 1, 32768 // k)
    H = _log(rng, 128, 8192, 16)
    if op == "sort":
        return {"op": op, "T": _log(rng, 1, 131072 // k), "k": k, "G": G, "wide": rng.random() < 0.5,
                "drop": rng.choice([0.0, 0.2])}
    if op == "sort_masked":
        T = min(T, 2048)
        return {"op": op, "T": T, "k": k, "G": G, "m_max": _log(rng, 16, 1024), "wide": rng.random() < 0.5}
    if op == "dispatch_masked":
        T = min(T, 512)
        return {"op": op, "T": T, "k": k, "G": min(G, 64), "H": H, "m_max": max(1, T)}
    if op in ("dispatch", "combine", "combine_backward"):
        return {"op": op, "T": T, "k": k, "G": G, "H": H}
    if op == "swiglu":
        return {"op": op, "T": T, "k": k, "G": min(G, 64), "F": _log(rng, 128, 4096, 128)}
    if op == "swiglu_backward":
        return {"op": op, "M": _log(rng, 1, 16384), "F": _log(rng, 128, 4096, 128)}
    if op == "dgrad":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 16, 4096, 16), "K": _log(rng, 16, 4096, 16)}
    if op == "wgrad":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 16, 4096, 16), "K": _log(rng, 16, 4096, 16),
                "bf16": rng.random() < 0.5}
    c = {"op": op, "T": T, "k": k, "G": min(G, 32), "N": _log(rng, 128, 4096, 128), "K": _log(rng, 128, 4096, 128)}
    c["k"] = min(k, c["G"])
    if op == "grouped_wgrad":
        c["bf16"] = rng.random() < 0.5
    return c


def _cap(c):
    s = c["T"] * c["k"]
    return (s + (B - 1) * min(c["G"], s)) // B * B


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _route(c, g):
    """Expert ids [T][k], distinct within a token, over skewed expert probabilities."""
    G = c["G"]
    p = torch.arange(1, G + 1, device="cuda", dtype=torch.float32).pow(-0.8)
    p = p[torch.randperm(G, generator=g, device="cuda")]
    u = torch.rand((c["T"], G), generator=g, device="cuda").clamp_min(1e-9)
    score = p.log() - (-u.log()).log()  # Gumbel draws: top k without replacement
    return score.topk(c["k"], dim=1)[1]


def _plain_sort(ids, G, cap):
    """(offsets [G+1], row_of_slot [T][k], slot_of_row [cap]), all int32."""
    flat = ids.reshape(-1).long()
    S, dev = flat.numel(), flat.device
    ok = (flat >= 0) & (flat < G)
    key = torch.where(ok, flat, torch.full_like(flat, G))
    counts = torch.zeros(G + 1, dtype=torch.int64, device=dev).index_add_(0, key, torch.ones_like(key))[:G]
    padded = (counts + B - 1) // B * B
    off = torch.zeros(G + 1, dtype=torch.int64, device=dev)
    off[1:] = padded.cumsum(0)
    first = torch.zeros(G + 1, dtype=torch.int64, device=dev)
    first[1:] = counts.cumsum(0)
    order = torch.sort(key, stable=True)[1]  # slots by expert, in their own order
    e = key[order]
    row = torch.where(e < G, off[e] + torch.arange(S, device=dev) - first[e], torch.full_like(e, -1))
    row_of_slot = torch.empty(S, dtype=torch.int32, device=dev)
    row_of_slot[order] = row.int()
    slot_of_row = torch.full((cap + 1,), -1, dtype=torch.int32, device=dev)
    slot_of_row[torch.where(row >= 0, row, torch.full_like(row, cap))] = order.int()
    slot_of_row[cap] = -1
    return off.int(), row_of_slot.view(ids.shape), slot_of_row[:cap]


def _plain_sort_masked(ids, G, m_max):
    """(masked_m [G], row_of_slot [T][k], slot_of_row [G * m_max]); slots past m_max are dropped."""
    flat = ids.reshape(-1).long()
    S, dev = flat.numel(), flat.device
    ok = (flat >= 0) & (flat < G)
    key = torch.where(ok, flat, torch.full_like(flat, G))
    counts = torch.zeros(G + 1, dtype=torch.int64, device=dev).index_add_(0, key, torch.ones_like(key))[:G]
    first = torch.zeros(G + 1, dtype=torch.int64, device=dev)
    first[1:] = counts.cumsum(0)
    order = torch.sort(key, stable=True)[1]
    e = key[order]
    rank = torch.arange(S, device=dev) - first[e]
    row = torch.where((e < G) & (rank < m_max), e * m_max + rank, torch.full_like(e, -1))
    row_of_slot = torch.empty(S, dtype=torch.int32, device=dev)
    row_of_slot[order] = row.int()
    slot_of_row = torch.full((G * m_max + 1,), -1, dtype=torch.int32, device=dev)
    slot_of_row[torch.where(row >= 0, row, torch.full_like(row, G * m_max))] = order.int()
    return counts.clamp_max(m_max).int(), row_of_slot.view(ids.shape), slot_of_row[:G * m_max]


def _blocks(v):
    """v [R][C] as [ceil(R/128)][128][ceil(C/128)][128], zeros past its edges."""
    R, C = v.shape
    rb, cb = -(-R // B), -(-C // B)
    if (rb * B, cb * B) != (R, C):
        w = v.new_zeros((rb * B, cb * B))
        w[:R, :C] = v
        v = w
    return v.view(rb, B, cb, B)


def _quantize(v):
    """float32 [R][C] -> E4M3 values [R][C] (float8) and scales [ceil(R/128)][ceil(C/128)].
    The divisor of amax is a tensor: a division by a Python number may be a product with its
    reciprocal, which rounds otherwise."""
    R, C = v.shape
    w = _blocks(v)
    amax = w.abs().amax(dim=(1, 3))
    s = torch.where(amax > 0, amax / amax.new_full((), 448.0), torch.ones_like(amax))
    q = (w / s[:, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.reshape(w.shape[0] * B, w.shape[2] * B)[:R, :C].contiguous(), s


def _quantize_rows(v):
    """float32 [R][C], C % 128 == 0 -> float8 [R][C] and scales [C/128][R]."""
    R, C = v.shape
    w = v.view(R, C // B, B)
    amax = w.abs().amax(dim=2)
    s = torch.where(amax > 0, amax / amax.new_full((), 448.0), torch.ones_like(amax))
    q = (w / s[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(R, C), s.t().contiguous()


def _decode(q, s):
    """float32 values of block-scaled codes."""
    R, C = q.shape
    w = s.repeat_interleave(B, 0)[:R].repeat_interleave(B, 1)[:, :C]
    return q.float() * w


def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _grouped_rows(c, g, cols, std, st):
    """Quantized rows [cap][cols] of sorted tokens: padding rows zero."""
    x = torch.randn((_cap(c), cols), generator=g, device="cuda").mul_(std)
    x.mul_((st["slot_of_row"] >= 0)[:, None])
    return _quantize(x)


def prepare(case, seed):
    c, g, st = case, _gen(seed), {"case": case}
    op = c["op"]
    if "T" in c:
        ids = _route(c, g)
        if c.get("drop"):
            ids[torch.rand(ids.shape, generator=g, device="cuda") < c["drop"]] = -1
        st["ids"] = ids if c.get("wide", True) else ids.int()
        if op in ("sort", "sort_masked"):
            return st
        w = torch.rand(ids.shape, generator=g, device="cuda") + 0.05
        st["weights"] = (w / w.sum(1, keepdim=True)).contiguous()
        if "m_max" in c:
            st["masked_m"], st["row_of_slot"], st["slot_of_row"] = _plain_sort_masked(ids, c["G"], c["m_max"])
        else:
            st["offsets"], st["row_of_slot"], st["slot_of_row"] = _plain_sort(ids, c["G"], _cap(c))
            st["spans"] = st["offsets"].tolist()
    if op in ("dispatch", "dispatch_masked"):
        st["x"] = _normal(g, (c["T"], c["H"]))
        hot = torch.randint(0, c["T"], (max(1, c["T"] // 100),), generator=g, device="cuda")
        st["x"][hot] *= 50  # a hundredth of the tokens are outliers
    elif op in ("combine", "combine_backward"):
        st["y"] = _normal(g, (_cap(c), c["H"]))
        st["dout"] = _normal(g, (c["T"], c["H"]), 1e-3) if op == "combine_backward" else None
    elif op == "swiglu":
        st["h"] = _normal(g, (_cap(c), 2 * c["F"]), 1.5)
        st["h"] *= (st["slot_of_row"] >= 0)[:, None]
    elif op == "swiglu_backward":
        st["h8"], st["sh"] = _quantize_rows(_normal(g, (c["M"], 2 * c["F"]), 1.5).float())
        st["da"] = _normal(g, (c["M"], c["F"]), 1e-3)
    elif op in ("dgrad", "wgrad"):
        st["dy"], st["sdy"] = _quantize(torch.randn((c["M"], c["N"]), generator=g, device="cuda") * 1e-3)
        if op == "dgrad":
            st["w"], st["sw"] = _quantize(torch.randn((c["N"], c["K"]), generator=g, device="cuda") * 0.02)
        else:
            st["x"], st["sx"] = _quantize(torch.randn((c["M"], c["K"]), generator=g, device="cuda"))
    elif op in ("grouped_dgrad", "grouped_wgrad"):
        st["dy"], st["sdy"] = _grouped_rows(c, g, c["N"], 1e-3, st)
        if op == "grouped_wgrad":
            st["x"], st["sx"] = _grouped_rows(c, g, c["K"], 1.0, st)
        else:
            G, N, K = c["G"], c["N"], c["K"]
            w, sw = _quantize(torch.randn((G * N, K), generator=g, device="cuda") * 0.02)
            st["w"], st["sw"] = w.view(G, N, K), sw.view(G, N // B, K // B)
    # the buffers that a program keeps: what lies past the last expert's rows stays as it is
    if op in ("dispatch", "combine_backward"):
        st["q"] = torch.zeros((_cap(c), c["H"]), dtype=torch.uint8, device="cuda")
        st["s"] = torch.zeros((_cap(c) // B, -(-c["H"] // B)), device="cuda")
    elif op == "dispatch_masked":
        st["q"] = torch.zeros((c["G"], c["m_max"], c["H"]), dtype=torch.uint8, device="cuda")
        st["s"] = torch.zeros((c["G"], -(-c["m_max"] // B), -(-c["H"] // B)), device="cuda")
    elif op == "swiglu":
        M, F = _cap(c), c["F"]
        st["q"] = torch.zeros((M, F), dtype=torch.uint8, device="cuda")
        st["s"] = torch.zeros((M // B, F // B), device="cuda")
        st["h8"] = torch.zeros((M, 2 * F), dtype=torch.uint8, device="cuda")
        st["sh"] = torch.zeros((2 * F // B, M), device="cuda")
    elif op == "grouped_dgrad":
        st["dx"] = torch.zeros((_cap(c), c["K"]), dtype=torch.bfloat16, device="cuda")
    return st


# --------------------------------------------------------------------------------- run
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from fp8_block_scaled_scales_b200 import binding as dg
    c = st["case"]
    op = c["op"]
    f8 = torch.float8_e4m3fn
    if op == "sort":
        return dg.moe_sort(st["ids"], c["G"])
    if op == "sort_masked":
        return dg.moe_sort_masked(st["ids"], c["G"], c["m_max"])
    if op == "dispatch":
        q, s = dg.moe_dispatch_quantize(st["x"], st["slot_of_row"], st["offsets"], c["k"], q=st["q"], s=st["s"])
        return q.view(f8), s
    if op == "dispatch_masked":
        q, s = dg.moe_dispatch_quantize_masked(st["x"], st["slot_of_row"], st["masked_m"], c["k"], q=st["q"], s=st["s"])
        return q.view(f8), s
    if op == "combine":
        return dg.moe_combine(st["y"], st["row_of_slot"], st["weights"])
    if op == "combine_backward":
        dw = dg.moe_combine_backward(st["dout"], st["y"], st["row_of_slot"])
        q, s = dg.moe_dispatch_quantize(st["dout"], st["slot_of_row"], st["offsets"], c["k"], weights=st["weights"],
                                        q=st["q"], s=st["s"])
        return dw, q.view(f8), s
    if op == "swiglu":
        q, s, h8, sh = dg.swiglu_quantize(st["h"], st["offsets"], checkpoint=True, q=st["q"], s=st["s"],
                                          h8=st["h8"], sh=st["sh"])
        return q.view(f8), s, h8.view(f8), sh
    if op == "swiglu_backward":
        q, s = dg.swiglu_quantize_backward(st["h8"], st["sh"], st["da"])
        return q.view(f8), s
    if op == "dgrad":
        return dg.dgrad_blockscaled(st["dy"], st["sdy"], st["w"], st["sw"])
    if op == "grouped_dgrad":
        return dg.grouped_dgrad_contiguous(st["dy"], st["sdy"], st["w"], st["sw"], st["offsets"], C=st["dx"])
    dtype = torch.bfloat16 if c["bf16"] else torch.float32
    if op == "wgrad":
        return dg.wgrad_blockscaled(st["dy"], st["sdy"], st["x"], st["sx"], dtype=dtype)
    return dg.grouped_wgrad_contiguous(st["dy"], st["sdy"], st["x"], st["sx"], st["offsets"], dtype=dtype)


def _gathered(x, slot_of_row, k, weights=None):
    """float32 rows x[slot // k] (times the slot's weight), zero where no slot is."""
    slot = slot_of_row.long()
    ok = slot >= 0
    slot = slot.clamp_min(0)
    v = x[slot // k].float()
    if weights is not None:
        v = v * weights.reshape(-1)[slot][:, None]
    return torch.where(ok[:, None], v, torch.zeros_like(v))


def _blank(q, s, used):
    """Codes and scales with the row blocks that hold nothing left at zero."""
    return torch.where(used.repeat_interleave(B)[:q.shape[0], None], q.view(torch.uint8), 0).view(q.dtype), \
        torch.where(used[:, None], s, 0.0)


def _swiglu(g, u):
    return g / (1.0 + torch.exp(-g)) * u


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op == "sort":
        return _plain_sort(st["ids"], c["G"], _cap(c))
    if op == "sort_masked":
        return _plain_sort_masked(st["ids"], c["G"], c["m_max"])
    if op in ("dispatch", "combine_backward"):
        src = st["x"] if op == "dispatch" else st["dout"]
        q, s = _quantize(_gathered(src, st["slot_of_row"], c["k"], None if op == "dispatch" else st["weights"]))
        q, s = _blank(q, s, torch.arange(s.shape[0], device=s.device) * B < st["offsets"][-1])
        if op == "dispatch":
            return q, s
        row = st["row_of_slot"].long()
        dot = (st["y"][row.clamp_min(0)].float() * st["dout"].float()[:, None, :]).sum(2)
        return torch.where(row >= 0, dot, torch.zeros_like(dot)), q, s
    if op == "dispatch_masked":
        G, m, H = c["G"], c["m_max"], c["H"]
        mp = -(-m // B) * B
        v = _gathered(st["x"], st["slot_of_row"], c["k"]).view(G, m, H)
        w = v.new_zeros((G, mp, H))
        w[:, :m] = v
        q, s = _quantize(w.view(G * mp, H))
        rows = torch.arange(mp // B, device=s.device)[None] * B < st["masked_m"][:, None]
        q, s = _blank(q, s, rows.reshape(-1))
        return q.view(G, mp, H)[:, :m].contiguous(), s.view(G, mp // B, -1)
    if op == "combine":
        row = st["row_of_slot"].long()
        w = torch.where(row >= 0, st["weights"], torch.zeros_like(st["weights"]))
        return (st["y"][row.clamp_min(0)].float() * w[:, :, None]).sum(1).to(torch.bfloat16)
    if op == "swiglu":
        F = c["F"]
        h = st["h"].float()
        q, s = _quantize(_swiglu(h[:, :F], h[:, F:]))
        h8, sh = _quantize_rows(h)
        used = torch.arange(s.shape[0], device=s.device) * B < st["offsets"][-1]
        q, s = _blank(q, s, used)
        rows = used.repeat_interleave(B)
        return q, s, torch.where(rows[:, None], h8.view(torch.uint8), 0).view(h8.dtype), torch.where(rows[None], sh, 0.0)
    if op == "swiglu_backward":
        F = c["F"]
        h = st["h8"].float() * st["sh"].t().repeat_interleave(B, 1)
        g, u, da = h[:, :F], h[:, F:], st["da"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        dg = da * u * sig * (1.0 + g * (1.0 - sig))
        return _quantize(torch.cat([dg, da * g * sig], 1))
    if op == "dgrad":
        return (_decode(st["dy"], st["sdy"]) @ _decode(st["w"], st["sw"])).to(torch.bfloat16)
    if op == "grouped_dgrad":
        dy, out = _decode(st["dy"], st["sdy"]), torch.zeros_like(st["dx"])
        for e, (a, b) in enumerate(zip(st["spans"], st["spans"][1:])):
            if b > a:
                out[a:b] = dy[a:b] @ _decode(st["w"][e], st["sw"][e])
        return out
    dtype = torch.bfloat16 if c["bf16"] else torch.float32
    dy, x = _decode(st["dy"], st["sdy"]), _decode(st["x"], st["sx"])
    if op == "wgrad":
        return (dy.t() @ x).to(dtype)
    out = torch.empty((c["G"], c["N"], c["K"]), dtype=dtype, device=dy.device)
    for e, (a, b) in enumerate(zip(st["spans"], st["spans"][1:])):
        out[e] = dy[a:b].t() @ x[a:b]
    return out


# ------------------------------------------------------------------------------- exact
def _exact_codes(v):
    """The block quantizer's definition on float64 values: (code values, scales), float64.
    The scale is rounded to float32 and the quotient to float32 before the E4M3 rounding."""
    R, C = v.shape
    w = _blocks(v).permute(0, 2, 1, 3).reshape(-1, B * B)
    top = w.abs().max(dim=1)[0].float().double()
    s = (top / 448.0).float().double()
    s[top == 0] = 1.0
    q = _e4m3((w / s[:, None]).float().double())
    rb, cb = -(-R // B), -(-C // B)
    return q.view(rb, cb, B, B).permute(0, 2, 1, 3).reshape(rb * B, cb * B)[:R, :C], s.view(rb, cb)


def _e4m3(t):
    """Nearest E4M3 value, ties to even, magnitudes above 448 to 448: 3 fraction bits above
    2^-6, multiples of 2^-9 below."""
    e = torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    r = torch.round(t / step) * step
    return r.clamp(-448.0, 448.0)


def exact(case, seed):
    c = case
    op = c["op"]
    if op in ("sort", "sort_masked"):
        return None  # whole numbers: there is one answer, and the plain form has it
    st = prepare(case, seed)
    if op in ("dispatch", "dispatch_masked", "combine_backward"):
        k = c["k"]
        src = (st["dout"] if op == "combine_backward" else st["x"]).double()
        H = src.shape[1]
        rows = st["slot_of_row"].shape[0] if op != "dispatch_masked" else c["G"] * (-(-c["m_max"] // B) * B)
        v = torch.zeros((rows, H), dtype=torch.float64, device="cuda")
        # scattered from the tokens' side
        row = st["row_of_slot"].long()
        if op == "dispatch_masked":
            mp = -(-c["m_max"] // B) * B
            row = torch.where(row >= 0, row // c["m_max"] * mp + row % c["m_max"], row)
        for j in range(k):
            t = torch.nonzero(row[:, j] >= 0)[:, 0]
            u = src[t]
            if op == "combine_backward":
                u = (u * st["weights"][t, j].double()[:, None]).float().double()  # the product is a float32
            v[row[t, j]] = u
        q, s = _exact_codes(v)
        if op == "dispatch_masked":
            nb = s.shape[0] // c["G"]
            s = s.view(c["G"], nb, -1)
            for e, m in enumerate(st["masked_m"].tolist()):
                s[e, -(-m // B):] = 0
            return q.view(c["G"], nb * B, H)[:, :c["m_max"]], s
        last = st["spans"][-1]
        s[last // B:] = 0
        if op == "dispatch":
            return q, s
        dw = torch.zeros((c["T"], k), dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(st["row_of_slot"][:, j] >= 0)[:, 0]
            dw[t, j] = torch.einsum("th,th->t", src[t], st["y"][st["row_of_slot"][t, j].long()].double())
        return dw, q, s
    if op == "combine":
        out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            t = torch.nonzero(st["row_of_slot"][:, j] >= 0)[:, 0]
            out[t] += st["weights"][t, j].double()[:, None] * st["y"][st["row_of_slot"][t, j].long()].double()
        return out
    if op == "swiglu":
        F, last = c["F"], st["spans"][-1]
        h = st["h"].double()
        q, s = _exact_codes(h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:])
        s[last // B:] = 0
        w = h.view(h.shape[0], -1, B)
        top = w.abs().max(dim=2)[0]
        sh = (top / 448.0).float().double()
        sh[top == 0] = 1.0
        h8 = _e4m3((w / sh[:, :, None]).float().double()).view(h.shape)
        sh = sh.t().contiguous()
        sh[:, last:] = 0
        return q, s, h8, sh
    if op == "swiglu_backward":
        F = c["F"]
        h = st["h8"].double().view(c["M"], -1, B) * st["sh"].double().t()[:, :, None]
        h = h.reshape(c["M"], 2 * F)
        with torch.enable_grad():  # by differentiation
            h.requires_grad_(True)
            a = h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:]
            d = torch.autograd.grad(a, h, st["da"].double())[0]
        return _exact_codes(d)
    # the products, one 128-deep block of the contraction at a time: codes first, scales after
    dy, sdy = st["dy"].double(), st["sdy"].double()
    if op in ("dgrad", "grouped_dgrad"):
        w = st["w"].double().view(-1, c["N"], c["K"])
        sw = st["sw"].double().view(w.shape[0], -1, -(-c["K"] // B))
        out = torch.zeros((dy.shape[0], c["K"]), dtype=torch.float64, device="cuda")
        spans = st.get("spans", [0, dy.shape[0]])
        for e, (a, b) in enumerate(zip(spans, spans[1:])):
            rows = torch.arange(a, b, device="cuda") // B
            for n in range(-(-c["N"] // B)):
                part = dy[a:b, n * B:(n + 1) * B] @ w[e, n * B:(n + 1) * B]
                out[a:b] += part * sdy[rows, n][:, None] * sw[e, n].repeat_interleave(B)[None, :c["K"]]
        return out
    x, sx = st["x"].double(), st["sx"].double()
    spans = st.get("spans", [0, dy.shape[0]])
    out = torch.zeros((len(spans) - 1, c["N"], c["K"]), dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(zip(spans, spans[1:])):
        for m in range(a, b, B):
            part = dy[m:min(b, m + B)].t() @ x[m:min(b, m + B)]
            part *= sdy[m // B].repeat_interleave(B)[:c["N"], None]
            part *= sx[m // B].repeat_interleave(B)[None, :c["K"]]
            out[e] += part
    return out if op == "grouped_wgrad" else out[0]


# -------------------------------------------------------------------------------- work
def work(case):
    """Bytes read and written once and operations; expert rows without their padding."""
    c = case
    op = c["op"]
    S = c["T"] * c["k"] if "T" in c else 0
    if op in ("sort", "sort_masked"):
        rows = _cap(c) if op == "sort" else c["G"] * c["m_max"]
        return {"bytes": S * (8 if c["wide"] else 4) + 4 * S + 4 * rows + 4 * (c["G"] + 1), "flops": S}
    if op in ("dispatch", "dispatch_masked"):
        return {"bytes": 2 * c["T"] * c["H"] + S * (c["H"] + 4), "flops": 2 * S * c["H"]}
    if op == "combine":
        return {"bytes": 2 * S * c["H"] + 8 * S + 2 * c["T"] * c["H"], "flops": 2 * S * c["H"]}
    if op == "combine_backward":
        return {"bytes": 2 * c["T"] * c["H"] + S * (3 * c["H"] + 16), "flops": 5 * S * c["H"]}
    if op == "swiglu":
        return {"bytes": S * c["F"] * 7, "flops": 10 * S * c["F"]}
    if op == "swiglu_backward":
        return {"bytes": c["M"] * c["F"] * 6, "flops": 16 * c["M"] * c["F"]}
    M = S if op.startswith("grouped") else c["M"]
    G, N, K = c.get("G", 1), c["N"], c["K"]
    flops = 2 * M * N * K
    if op.endswith("dgrad"):
        return {"bytes": M * N + G * N * K + 2 * M * K, "flops": flops}
    return {"bytes": M * (N + K) + G * N * K * (2 if c["bf16"] else 4), "flops": flops}

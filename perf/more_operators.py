"""Cases that measure what a training or decode step needs around the expert layer: routing
(scores to expert ids and weights, with the balance loss and per-expert counts) and its
gradient; the RMS norms before and after a block, fused with its gate and the scaled
residual, and their gradient; and the global norm of a step's gradients with clipping.

Every case has a plain form in elementary torch operations (float32, float64 where a
selection or a long sum needs it), the call of this repository's own kernels, and a
float64 evaluation of the definition.
"""
import math

import torch

own = False

B = 128
EPS = 1e-6


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # five generated tokens routed to 8 of 256 experts by sigmoid scores and a selection
        # bias: a decode step, the smallest call
        {"name": "route_decode_5", "op": "route", "T": 5, "G": 256, "k": 8, "score": "sigmoid", "bias": True,
         "bf16": False, "balance": False, "pad": 0.0, "renormalize": True, "scale": 2.5},
        # a large training batch over fine-grained experts, with counts and the balance loss
        {"name": "route_train_16384x8", "op": "route", "T": 16384, "G": 256, "k": 8, "score": "sigmoid", "bias": True,
         "bf16": False, "balance": True, "pad": 0.0, "renormalize": True, "scale": 2.5},
        # a padded batch of BF16 scores, softmax, 2 of 64 experts
        {"name": "route_padded_1000", "op": "route", "T": 1000, "G": 64, "k": 2, "score": "softmax", "bias": False,
         "bf16": True, "balance": True, "pad": 0.1, "renormalize": True, "scale": 1.0},
        # gradient of the large training batch
        {"name": "route_backward_16384x8", "op": "route_backward", "T": 16384, "G": 256, "k": 8, "score": "sigmoid",
         "bf16": False, "balance": True, "pad": 0.0, "renormalize": True, "scale": 2.5},
        # gradient of the 8-expert workload's routing: few experts, an odd batch with padding
        {"name": "route_backward_8191x2", "op": "route_backward", "T": 8191, "G": 8, "k": 2, "score": "softmax",
         "bf16": True, "balance": True, "pad": 0.1, "renormalize": False, "scale": 1.0},
        # one generated token: residual, norm and codes for the next product in a single pass
        {"name": "norm_decode_1", "op": "norm_codes", "T": 1, "H": 7168, "post": True, "gate": False,
         "bf16": False, "alpha": 1.0},
        # a ragged serving batch
        {"name": "norm_codes_1000", "op": "norm_codes", "T": 1000, "H": 2048, "post": False, "gate": False,
         "bf16": True, "alpha": 1.0},
        # training: norm after the block, learned gate, scaled residual, norm before the next one
        {"name": "norm_train_16384", "op": "norm", "T": 16384, "H": 4096, "post": True, "gate": True,
         "bf16": False, "alpha": 0.5},
        # its gradient
        {"name": "norm_backward_16384", "op": "norm_backward", "T": 16384, "H": 4096, "post": True, "gate": True,
         "bf16": False, "alpha": 0.5},
        # gradient for a small ragged batch of a narrow model, no norm after the block
        {"name": "norm_backward_333", "op": "norm_backward", "T": 333, "H": 784, "post": False, "gate": True,
         "bf16": True, "alpha": 1.0},
        # the gradients of a small dense model: many tensors, ragged sizes, two types
        {"name": "clip_many_300", "op": "clip", "tensors": 300, "largest": 200000, "mixed": True, "ratio": 0.25},
        # weight gradients (float32) of the 8-expert workload: two products per expert
        {"name": "clip_g8", "op": "clip_experts", "G": 8, "F": 4096, "H": 4096, "ratio": 0.25},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(v / step) * step)


def draw(rng):
    op = rng.choice(["route", "route_backward", "norm", "norm_codes", "norm_backward", "clip", "clip_experts"])
    if op in ("route", "route_backward"):
        G = _log(rng, 2, 512)
        k = min(G, rng.choice([1, 2, 4, 6, 8]))
        c = {"op": op, "T": _log(rng, 1, 16384), "G": G, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
             "bf16": rng.random() < 0.5, "balance": rng.random() < 0.6, "pad": rng.choice([0.0, 0.2]),
             "renormalize": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5])}
        if op == "route":
            c["bias"] = rng.random() < 0.5
        return c
    if op in ("norm", "norm_codes", "norm_backward"):
        return {"op": op, "T": _log(rng, 1, 16384), "H": _log(rng, 128, 8192, 16), "post": rng.random() < 0.5,
                "gate": rng.random() < 0.5, "bf16": rng.random() < 0.5, "alpha": rng.choice([1.0, 0.5])}
    ratio = rng.choice([0.25, 2.0])  # of the limit to the norm: clipped, or left as they are
    if op == "clip":
        return {"op": op, "tensors": _log(rng, 1, 600), "largest": _log(rng, 1, 1000000), "mixed": rng.random() < 0.5,
                "ratio": ratio}
    return {"op": op, "G": _log(rng, 1, 8), "F": _log(rng, 128, 4096, 128), "H": _log(rng, 128, 4096, 16),
            "ratio": ratio}


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _clip_shapes(c):
    """(elements, bf16) of every gradient."""
    if c["op"] == "clip_experts":
        G, F, H = c["G"], c["F"], c["H"]
        return [(G * 2 * F * H, False), (G * F * H, False), (G * H, False), (H, False), (H, False)]
    # sizes spread over their logarithm from 1 to the largest, by a fixed low-discrepancy sequence
    n, top = c["tensors"], c["largest"]
    return [(max(1, int(top ** ((0.618034 * i + 1.0) % 1.0))) if i else top, c["mixed"] and i % 3 == 1)
            for i in range(n)]


def prepare(case, seed):
    c, g, st = case, _gen(seed), {"case": case}
    op = c["op"]
    if op in ("route", "route_backward"):
        T, G = c["T"], c["G"]
        skew = torch.randn((G,), generator=g, device="cuda") * 0.5  # some experts are liked by all tokens
        z = torch.randn((T, G), generator=g, device="cuda") + skew
        st["logits"] = z.to(torch.bfloat16) if c["bf16"] else z
        st["bias"] = (torch.rand((G,), generator=g, device="cuda") - 0.5) * 0.2 if c.get("bias") else None
        st["mask"] = None
        if c["pad"]:  # a batch is padded at its end
            st["mask"] = torch.arange(T, device="cuda") < T - int(T * c["pad"])
        if op == "route_backward":
            st["topk_ids"], _, _, _, dprob = _plain_route(st)
            st["dprob"] = dprob if c["balance"] else None
            st["dweights"] = torch.randn((T, c["k"]), generator=g, device="cuda") * 1e-3
            # gradient of the balance loss: its coefficient in the total loss
            st["dloss"] = torch.full((), 0.01, device="cuda") if c["balance"] else None
        return st
    if op in ("norm", "norm_codes", "norm_backward"):
        T, H = c["T"], c["H"]
        vec = torch.bfloat16 if c["bf16"] else torch.float32
        st["weight"] = (1.0 + 0.1 * torch.randn((H,), generator=g, device="cuda")).to(vec)
        st["post"] = (1.0 + 0.1 * torch.randn((H,), generator=g, device="cuda")).to(vec) if c["post"] else None
        st["gate"] = (torch.rand((H,), generator=g, device="cuda")).to(vec) if c["gate"] else None
        st["y"] = _randn(g, (T, H), 0.7)
        st["x"] = _randn(g, (T, H), 1.5)
        hot = torch.randint(0, H, (max(1, H // 200),), generator=g, device="cuda")
        st["x"][:, hot] *= 20  # outlier channels of the residual stream
        if op == "norm_backward":
            st["r"] = st.pop("x")
            st["rstd"] = _rstd(st["r"])
            st["rstd_y"] = _rstd(st["y"]) if c["post"] else None
            st["dn"] = _randn(g, (T, H), 1e-3)
            st["dr"] = _randn(g, (T, H), 1e-3)
        return st
    shapes = _clip_shapes(c)
    st["grads"] = [_randn(g, (n,), 1e-3, torch.bfloat16 if b else torch.float32) for n, b in shapes]
    # where the clipped gradients go: one buffer per type, as an optimizer keeps them, each
    # tensor at a multiple of 16 bytes
    at, place = {True: 0, False: 0}, []
    for n, b in shapes:
        place.append((b, at[b], n))
        at[b] += -(-n // 8) * 8
    st["flat"] = {b: torch.zeros(size, dtype=torch.bfloat16 if b else torch.float32, device="cuda")
                  for b, size in at.items() if size}
    st["out"] = [st["flat"][b][i:i + n] for b, i, n in place]
    # the limit follows the expected norm, so that a case clips or does not, whatever the seed
    st["max_norm"] = c["ratio"] * 1e-3 * math.sqrt(sum(n for n, _ in shapes))
    return st


# --------------------------------------------------------------------------------- run
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from fp8_block_scaled_scales_b200 import binding as dg
    c = st["case"]
    op = c["op"]
    if op == "route":
        return dg.moe_route(st["logits"], c["k"], score=c["score"], bias=st["bias"], mask=st["mask"],
                            renormalize=c["renormalize"], scale=c["scale"], balance=c["balance"])
    if op == "route_backward":
        return dg.moe_route_backward(st["logits"], st["topk_ids"], dweights=st["dweights"], dprob=st["dprob"],
                                     dloss=st["dloss"], score=c["score"], renormalize=c["renormalize"],
                                     scale=c["scale"])
    if op == "norm":
        out = dg.rmsnorm_residual(st["x"], st["weight"], y=st["y"], gate=st["gate"], post_weight=st["post"],
                                  alpha=c["alpha"], eps=EPS)
        return [t for t in out if t is not None]
    if op == "norm_codes":
        q, s, r = dg.rmsnorm_residual_quantize(st["x"], st["weight"], y=st["y"], gate=st["gate"],
                                               post_weight=st["post"], alpha=c["alpha"], eps=EPS)
        return q.view(torch.float8_e4m3fn), s, r
    if op == "norm_backward":
        out = dg.rmsnorm_residual_backward(st["dn"], st["r"], st["rstd"], st["weight"], dr=st["dr"], y=st["y"],
                                           rstd_y=st["rstd_y"], gate=st["gate"], post_weight=st["post"],
                                           alpha=c["alpha"])
        return [t for t in out if t is not None]
    norm = dg.clip_grad_norm(st["grads"], st["max_norm"], out=st["out"])
    return [norm, *st["flat"].values()]


def _plain_scores(z, score):
    """Scores and the probabilities of the balance loss, in z's precision; a row without a
    score above -inf has zeros."""
    if score == "softmax":
        top = z.amax(1, keepdim=True)
        e = torch.exp(z - torch.where(top > -math.inf, top, torch.zeros_like(top)))
        s = e / e.sum(1, keepdim=True).clamp_min(1e-30)
        return s, s
    s = 1.0 / (1.0 + torch.exp(-z))
    return s, s / s.sum(1, keepdim=True).clamp_min(1e-30)


def _plain_route(st):
    """(ids, weights, counts, loss, dprob)."""
    c = st["case"]
    k, G = c["k"], c["G"]
    z = st["logits"].float()
    s, p = _plain_scores(z, c["score"])
    key = z  # both scores grow with the logit: without a bias the order is the logits' own
    if st.get("bias") is not None:
        key = _plain_scores(z.double(), c["score"])[0] + st["bias"].double()
    allowed = z > -math.inf
    key = torch.where(allowed, key, torch.full_like(key, -math.inf))
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
    ok = torch.gather(allowed, 1, ids)
    if st.get("mask") is not None:
        ok = ok & st["mask"][:, None]
    chosen = torch.where(ok, torch.gather(s, 1, ids), torch.zeros((), device=z.device))
    w = chosen * c["scale"]
    if c["renormalize"]:
        w = w / chosen.sum(1, keepdim=True).clamp_min(1e-30)
    ids = torch.where(ok, ids, torch.full_like(ids, -1))
    routed = ok.any(1)
    n = routed.sum()
    counts = torch.zeros(G + 1, dtype=torch.int32, device=z.device)
    counts.index_add_(0, ids.reshape(-1) % (G + 1), torch.ones(ids.numel(), dtype=torch.int32, device=z.device))
    counts = counts[:G]
    sums = torch.where(routed[:, None], p, torch.zeros_like(p)).double().sum(0)
    nd = n.double().clamp_min(1.0)
    dprob = counts.double() * G / (k * nd * nd)
    return ids.int(), w, counts, (dprob * sums).sum().float(), dprob.float()


def _plain_route_backward(st):
    c = st["case"]
    z, ids = st["logits"].float(), st["topk_ids"].long()
    ok = ids >= 0
    ids = ids.clamp_min(0)
    s, p = _plain_scores(z, c["score"])
    si = torch.where(ok, torch.gather(s, 1, ids), torch.zeros_like(st["dweights"]))
    gw = torch.where(ok, st["dweights"], torch.zeros_like(st["dweights"])) * c["scale"]
    if c["renormalize"]:
        S = si.sum(1, keepdim=True).clamp_min(1e-30)
        gw = (gw - (gw * si).sum(1, keepdim=True) / S) / S
    ds = torch.zeros_like(z).scatter_add_(1, ids, torch.where(ok, gw, torch.zeros_like(gw)))
    dp = torch.zeros_like(z)
    if st["dprob"] is not None:
        dp = dp + st["dprob"] * st["dloss"]
    if c["score"] == "softmax":
        ds = ds + dp
        dz = s * (ds - (ds * s).sum(1, keepdim=True))
    else:
        not_s = 1.0 / (1.0 + torch.exp(z))
        dz = not_s * (s * ds + p * (dp - (dp * p).sum(1, keepdim=True)))
    return torch.where(ok.any(1)[:, None], dz, torch.zeros_like(dz)).to(st["logits"].dtype)


def _rstd(v):
    return (1.0 / torch.sqrt((v.double() ** 2).mean(1) + EPS)).float()


def _quantize_rows(v):
    """float32 [R][C] -> float8 codes and scales [ceil(C/128)][R], one per row and 128 columns."""
    R, C = v.shape
    nb = -(-C // B)
    w = v.new_zeros((R, nb * B))
    w[:, :C] = v
    w = w.view(R, nb, B)
    amax = w.abs().amax(dim=2)
    s = torch.where(amax > 0, amax / amax.new_full((), 448.0), torch.ones_like(amax))
    q = (w / s[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(R, nb * B)[:, :C].contiguous(), s.t().contiguous()


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op == "route":
        ids, w, counts, loss, dprob = _plain_route(st)
        return (ids, w, counts, loss, dprob) if c["balance"] else (ids, w)
    if op == "route_backward":
        return _plain_route_backward(st)
    if op in ("norm", "norm_codes"):
        x, u = st["x"].float(), st["y"].float()
        rstd_y = None
        if st["post"] is not None:
            rstd_y = 1.0 / torch.sqrt((u * u).mean(1) + EPS)
            u = u * rstd_y[:, None] * st["post"].float()
        if st["gate"] is not None:
            u = u * st["gate"].float()
        r = c["alpha"] * x + u
        rstd = 1.0 / torch.sqrt((r * r).mean(1) + EPS)
        n = r * rstd[:, None] * st["weight"].float()
        if op == "norm_codes":
            return (*_quantize_rows(n), r.to(torch.bfloat16))
        out = [n.to(torch.bfloat16), r.to(torch.bfloat16), rstd]
        return out if rstd_y is None else out + [rstd_y]
    if op == "norm_backward":
        dn, y = st["dn"].float(), st["y"].float()
        rhat = st["r"].float() * st["rstd"][:, None]
        gw = dn * st["weight"].float()
        dR = st["dr"].float() + st["rstd"][:, None] * (gw - rhat * (gw * rhat).mean(1, keepdim=True))
        out = {"dx": (c["alpha"] * dR).to(torch.bfloat16), "dweight": (dn * rhat).double().sum(0).float()}
        u, du = y, dR
        if st["post"] is not None:
            yhat = y * st["rstd_y"][:, None]
            u = yhat * st["post"].float()
        if st["gate"] is not None:
            out["dgate"] = (dR * u).double().sum(0).float()
            du = dR * st["gate"].float()
        if st["post"] is not None:
            out["dpost"] = (du * yhat).double().sum(0).float()
            gp = du * st["post"].float()
            du = st["rstd_y"][:, None] * (gp - yhat * (gp * yhat).mean(1, keepdim=True))
        out["dy"] = du.to(torch.bfloat16)
        return [out[n] for n in ("dx", "dy", "dweight", "dgate", "dpost") if n in out]
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for t in st["grads"]:
        total = total + (t.float() * t.float()).sum(dtype=torch.float64)
    norm = torch.sqrt(total).float()
    coef = torch.where(norm > st["max_norm"], st["max_norm"] / norm, torch.ones_like(norm))
    for t, o in zip(st["grads"], st["out"]):
        o.copy_(t.float() * coef)
    return [norm, *st["flat"].values()]


# ------------------------------------------------------------------------------- exact
def _exact_p(z, score):
    """Scores and balance probabilities by log-sums, float64."""
    if score == "softmax":
        s = torch.exp(torch.log_softmax(z, 1))
        return s, s
    ls = torch.nn.functional.logsigmoid(z)
    return torch.exp(ls), torch.exp(ls - torch.logsumexp(ls, 1, keepdim=True))


def _exact_weights(z, onehots, c):
    """Weights of the chosen experts from their indicators [T][k][G]."""
    s, p = _exact_p(z, c["score"])
    chosen = torch.einsum("tkg,tg->tk", onehots, s)
    w = chosen / chosen.sum(1, keepdim=True).clamp_min(1e-300) if c["renormalize"] else chosen
    return w * c["scale"], p


def _exact_e4m3(t):
    """Nearest E4M3 value, ties to even, magnitudes above 448 to 448: 3 fraction bits above
    2^-6, multiples of 2^-9 below."""
    e = torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(t / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    c = case
    op = c["op"]
    st = prepare(case, seed)
    if op in ("route", "route_backward"):
        T, G, k = c["T"], c["G"], c["k"]
        z = st["logits"].double()
        alive = st["mask"] if st["mask"] is not None else torch.ones(T, dtype=torch.bool, device="cuda")
        if op == "route":
            # the largest of what is left, k times; the lowest index among equals
            key = z.clone()
            if st["bias"] is not None:
                key = _exact_p(z, c["score"])[0] + st["bias"].double()
            index = torch.arange(G, device="cuda")
            hots = []
            for _ in range(k):
                best = key == key.amax(1, keepdim=True)
                first = torch.where(best, index, torch.full_like(index, G)).amin(1)
                hots.append((index == first[:, None]) & alive[:, None])
                key = key.masked_fill(index == first[:, None], -math.inf)
            hots = torch.stack(hots, 1).double()
            w, p = _exact_weights(z, hots, c)
            if not c["balance"]:
                return None, w
            n = max(1, int(alive.sum()))
            f = hots.sum((0, 1)) / (n * k)
            P = p[alive].sum(0) / n
            return None, w, None, G * (f * P).sum(), G * f / n
        ids = st["topk_ids"].long()
        hots = (ids[:, :, None] == torch.arange(G, device="cuda")).double()
        with torch.enable_grad():  # by differentiation
            z.requires_grad_(True)
            w, p = _exact_weights(z, hots, c)
            total = (w * st["dweights"].double() * (ids >= 0)).sum()
            if st["dprob"] is not None:
                total = total + st["dloss"].double() * (p * st["dprob"].double() * alive[:, None]).sum()
            return torch.autograd.grad(total, z)[0]
    if op in ("norm", "norm_codes", "norm_backward"):
        H = c["H"]
        d = {n: st[n].double() for n in ("weight", "post", "gate", "y") if st[n] is not None}

        def normed(v):
            ms = torch.einsum("th,th->t", v, v) / H + EPS
            return v * ms.pow(-0.5)[:, None], ms.pow(-0.5)

        def branch(y, post, gate):
            u = y
            if post is not None:
                u = normed(y)[0] * post
            return u if gate is None else u * gate

        if op == "norm_backward":
            # n = norm(r) * weight and r = alpha x + branch(y), differentiated; x enters only
            # through r, so the point is r itself
            leaves = [d["y"], d["weight"]] + [d[n] for n in ("gate", "post") if n in d]
            with torch.enable_grad():
                for t in leaves:
                    t.requires_grad_(True)
                b = branch(d["y"], d.get("post"), d.get("gate"))
                x = ((st["r"].double() - b.detach()) / c["alpha"]).requires_grad_(True)
                r = c["alpha"] * x + b
                n = normed(r)[0] * d["weight"]
                total = (n * st["dn"].double()).sum() + (r * st["dr"].double()).sum()
                return list(torch.autograd.grad(total, [x] + leaves))
        r = c["alpha"] * st["x"].double() + branch(d["y"], d.get("post"), d.get("gate"))
        n, rstd = normed(r)
        n = n * d["weight"]
        if op == "norm":
            out = [n, r, rstd]
            return out + [normed(d["y"])[1]] if c["post"] else out
        nb = -(-H // B)
        w = torch.nn.functional.pad(n.float().double(), (0, nb * B - H)).view(c["T"], nb, B)
        top = w.abs().amax(2)
        s = torch.where(top > 0, (top / 448.0).float().double(), torch.ones_like(top))
        q = _exact_e4m3((w / s[:, :, None]).float().double()).view(c["T"], nb * B)[:, :H]
        return q, s.t(), r
    norm = math.sqrt(sum(float(torch.dot(t.double(), t.double())) for t in st["grads"]))
    coef = min(1.0, st["max_norm"] / norm) if norm > 0 else 1.0
    out = [torch.tensor(norm, dtype=torch.float64, device="cuda")]
    for b, flat in st["flat"].items():
        v = torch.zeros(flat.shape, dtype=torch.float64, device="cuda")
        at = 0
        for t in st["grads"]:
            if (t.dtype == torch.bfloat16) == b:
                v[at:at + t.numel()] = t.double() * coef
                at += (t.numel() + 7) // 8 * 8
        out.append(v)
    return out


# -------------------------------------------------------------------------------- work
def work(case):
    """Bytes read and written once and operations."""
    c = case
    op = c["op"]
    if op in ("route", "route_backward"):
        T, G, k = c["T"], c["G"], c["k"]
        e = 2 if c["bf16"] else 4
        pad = T if c["pad"] else 0
        if op == "route":
            vectors = 12 * G + 4 if c["balance"] else 0
            return {"bytes": T * (G * e + 8 * k) + pad + vectors + (4 * G if c["bias"] else 0), "flops": T * G * (5 + k)}
        return {"bytes": T * (2 * G * e + 8 * k) + (4 * G if c["balance"] else 0), "flops": T * G * 8}
    if op in ("norm", "norm_codes", "norm_backward"):
        T, H = c["T"], c["H"]
        vectors = (2 if c["bf16"] else 4) * H * (1 + c["post"] + c["gate"])
        if op == "norm":
            return {"bytes": 8 * T * H + 4 * T * (1 + c["post"]) + vectors, "flops": 8 * T * H}
        if op == "norm_codes":
            return {"bytes": 7 * T * H + 4 * T * -(-H // B) + vectors, "flops": 10 * T * H}
        grads = 4 * H * (1 + c["post"] + c["gate"])
        return {"bytes": 12 * T * H + 4 * T * (1 + c["post"]) + vectors + grads, "flops": 20 * T * H}
    bytes_ = sum(n * (2 if b else 4) for n, b in _clip_shapes(c))
    return {"bytes": 2 * bytes_ + 4, "flops": 3 * sum(n for n, _ in _clip_shapes(c))}

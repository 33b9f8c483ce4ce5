"""Plain float64 / numpy forms of the expert-layer operators and gradient products, written
from their definitions, for the tests to compare with."""
from __future__ import annotations

import numpy as np
import torch

B = 128
U8, F8 = torch.uint8, torch.float8_e4m3fn


def cap_of(T, k, G):
    S = T * k
    return (S + 127 * min(G, S)) // 128 * 128


def sort_plain(ids, G, cap):
    """(offsets, row_of_slot, slot_of_row) by walking the slots in order."""
    flat = np.asarray(ids).reshape(-1)
    counts = np.zeros(G, np.int64)
    for e in flat:
        if 0 <= e < G:
            counts[e] += 1
    off = np.zeros(G + 1, np.int64)
    off[1:] = np.cumsum((counts + 127) // 128 * 128)
    row = np.full(flat.size, -1, np.int64)
    slot = np.full(cap, -1, np.int64)
    seen = np.zeros(G, np.int64)
    for s, e in enumerate(flat):
        if 0 <= e < G:
            row[s] = off[e] + seen[e]
            slot[row[s]] = s
            seen[e] += 1
    return off, row.reshape(np.asarray(ids).shape), slot


def sort_masked_plain(ids, G, m_max):
    flat = np.asarray(ids).reshape(-1)
    row = np.full(flat.size, -1, np.int64)
    slot = np.full(G * m_max, -1, np.int64)
    seen = np.zeros(G, np.int64)
    for s, e in enumerate(flat):
        if 0 <= e < G:
            if seen[e] < m_max:
                row[s] = e * m_max + seen[e]
                slot[row[s]] = s
            seen[e] += 1
    return np.minimum(seen, m_max), row.reshape(np.asarray(ids).shape), slot


def quantize_f32(v: torch.Tensor):
    """The block quantizer's definition on CPU float32 [R][C]: (codes uint8, scales)."""
    R, C = v.shape
    q = torch.zeros((R, C), dtype=U8)
    s = torch.ones((-(-R // B), -(-C // B)), dtype=torch.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            b = v[i * B:(i + 1) * B, j * B:(j + 1) * B]
            t = b.abs().max() / torch.tensor(448.0)
            if t != 0:  # a NaN too
                s[i, j] = t
            q[i * B:(i + 1) * B, j * B:(j + 1) * B] = (b / s[i, j]).clamp(-448, 448).to(F8).view(U8)
    return q, s


def decode(q: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    """float64 values of 128x128-block-scaled codes (CPU)."""
    R, C = q.shape
    w = s.double().repeat_interleave(B, 0)[:R].repeat_interleave(B, 1)[:, :C]
    return q.view(F8).double() * w


def decode_rows(q: torch.Tensor, s_t: torch.Tensor) -> torch.Tensor:
    """float64 values of codes with one scale per row and 128 columns, s_t [C/128][R] (CPU)."""
    return q.view(F8).double() * s_t.double().t().repeat_interleave(B, 1)[:, :q.shape[1]]


def code_error_bound(value: torch.Tensor, s: torch.Tensor, noise) -> torch.Tensor:
    """How far scale * code may be from a float64 value: half an E4M3 step (2^-4 of the value,
    or 2^-10 of the scale below the normal range; the quotient's own FP32 rounding and the
    scale's widen it by less than 2^-19) plus the kernel's absolute error `noise` of the value
    itself before rounding (times 1 + 2^-3, since the rounding can carry it one more step)."""
    R, C = value.shape
    w = s.double().repeat_interleave(B, 0)[:R].repeat_interleave(B, 1)[:, :C]
    return torch.maximum(value.abs() * 2.0 ** -4, w * 2.0 ** -10) * (1 + 2.0 ** -19) + noise * 1.125


def sigma_error(g: torch.Tensor) -> torch.Tensor:
    """Relative error bound of the hardware sigmoid times a few products: the exponential's
    documented bound is 2 + 1.173 |x| units of 2^-23, the reciprocal's 2, and up to eight more
    FP32 roundings follow (half a unit each)."""
    return (2 + 1.2 * g.abs() + 2 + 4 + 1) * 2.0 ** -23


def swiglu64(h: torch.Tensor):
    F = h.shape[1] // 2
    g, u = h[:, :F].double(), h[:, F:].double()
    return g * torch.sigmoid(g) * u


def product_bound(abs_sum: torch.Tensor, blocks: int, ref: torch.Tensor, dtype) -> torch.Tensor:
    """|kernel - float64| for a block-scaled product: at most 128 FP32 additions inside a block
    and `blocks` scaled ones after it, each off by at most 2^-23 of the sum of magnitudes, the
    scales' product and the FMA's rounding alike, and the output's rounding."""
    out = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}[dtype]
    return (128 + blocks + 4) * 2.0 ** -23 * abs_sum * (1 + out) + out * ref.abs() + 1e-300

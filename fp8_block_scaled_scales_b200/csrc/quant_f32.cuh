// FP32 -> E4M3 for values that a kernel computes itself (a weighted row, an activation, a
// gradient), and E4M3 -> FP32.  Same definition as the BF16 quantizer:
//   s = fl32(amax / 448), 1 if that is 0;  q = E4M3_rn_satfinite(fl32(x / s)).
// amax is an FP32 maximum here, so s may be any FP32; with amax below 448 times the least
// subnormal the quotient amax / 448 rounds to 0 and s = 1 (every code is then 0).
#pragma once

#include <cuda_fp16.h>

#include "quant_e4m3.cuh"

namespace dg {

// Eight BF16 of a 16-byte group as FP32.
__device__ __forceinline__ void bf16x8_to_f32(uint4 v, float2 (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        x[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
}

__device__ __forceinline__ BlockScale block_scale_f32(float amax) {
    BlockScale b;
    const float q = __fdiv_rn(amax, 448.0f);
    b.s = (q == 0.0f) ? 1.0f : q;
    const float r = __frcp_rn(b.s);
    b.fast_ok = isfinite(r);
    const float rlo = __fmul_rn(r, 1.0f - 0x1p-21f), rhi = __fmul_rn(r, 1.0f + 0x1p-21f);
    b.rlo2 = make_float2(rlo, rlo);
    b.rhi2 = make_float2(rhi, rhi);
    return b;
}

// quantize8 (quant_e4m3.cuh) for eight FP32 values: the bracket's proof takes any FP32 x.
__device__ __forceinline__ uint2 quantize8_f32(const float2 (&x)[4], const BlockScale &b) {
    float2 lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        lo[j] = __fmul2_rn(x[j], b.rlo2);
        hi[j] = __fmul2_rn(x[j], b.rhi2);
    }
    uint2 out;
    out.x = e4m3x4(hi[0].x, hi[0].y, hi[1].x, hi[1].y);
    out.y = e4m3x4(hi[2].x, hi[2].y, hi[3].x, hi[3].y);
    const uint32_t lx = e4m3x4(lo[0].x, lo[0].y, lo[1].x, lo[1].y);
    const uint32_t ly = e4m3x4(lo[2].x, lo[2].y, lo[3].x, lo[3].y);
    if (__builtin_expect(((out.x ^ lx) | (out.y ^ ly)) != 0u || !b.fast_ok, 0)) {
        float2 y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = make_float2(__fdiv_rn(x[j].x, b.s), __fdiv_rn(x[j].y, b.s));
        out.x = e4m3x4(y[0].x, y[0].y, y[1].x, y[1].y);
        out.y = e4m3x4(y[2].x, y[2].y, y[3].x, y[3].y);
    }
    return out;
}

// Scale of a block of such values and its reciprocal.
struct NearScale {
    float s, r;
    bool fast_ok;
};

__device__ __forceinline__ NearScale near_scale(uint32_t amax_bits) {
    NearScale b;
    const float q = __fdiv_rn(__uint_as_float(amax_bits), 448.0f);
    b.s = (q == 0.0f) ? 1.0f : q;
    b.r = __frcp_rn(b.s);
    b.fast_ok = isfinite(b.r);
    return b;
}

// Eight FP32 values that are themselves rounded results (an activation, a gradient): x / s as
// the product with the rounded reciprocal, off by two roundings of 2^-24 where the quotient
// is off by one.  The values carry larger errors already, so the exact quotient that
// quantize8 pays for would decide nothing.
__device__ __forceinline__ uint2 quantize8_near(const float2 (&x)[4], const NearScale &b) {
    float2 y[4];
    if (__builtin_expect(b.fast_ok, 1)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = __fmul2_rn(x[j], make_float2(b.r, b.r));
    } else {  // 1/s is not finite
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = make_float2(__fdiv_rn(x[j].x, b.s), __fdiv_rn(x[j].y, b.s));
    }
    return make_uint2(e4m3x4(y[0].x, y[0].y, y[1].x, y[1].y), e4m3x4(y[2].x, y[2].y, y[3].x, y[3].y));
}

// Eight BF16 -> eight E4M3 codes of fl32(x / s), given s and r = fl32(1/s): a quotient
// corrected by its remainder (P. W. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", IBM J. Res. Dev. 34, 1990, on division with a fused
// multiply-add): z = x (-r), e = z s + x exactly rounded, -x/s = e (-r) + z.  Signs are
// arranged so that a zero keeps its sign, hence the flip of all eight at the end.  Three
// multiply-adds a pair and one conversion, with no second path for values near a rounding
// boundary, which a row whose amax is a multiple of 7 meets often.  For every BF16 x and
// amax with 2^-100 <= s <= 2^100 the code is that of the IEEE quotient (checked
// exhaustively on the CPU); outside that range the caller divides (in_window).
__device__ __forceinline__ bool in_window(float s) { return s >= 0x1p-100f && s <= 0x1p100f; }

__device__ __forceinline__ uint2 quantize8_corrected(uint4 v, float s, float r) {
    float2 x[4], q[4];
    bf16x8_to_f32(v, x);
    if (__builtin_expect(in_window(s), 1)) {
        const float2 s2 = make_float2(s, s), nr = make_float2(-r, -r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 z = __fmul2_rn(x[j], nr);
            q[j] = __ffma2_rn(__ffma2_rn(z, s2, x[j]), nr, z);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = make_float2(-__fdiv_rn(x[j].x, s), -__fdiv_rn(x[j].y, s));
    }
    return make_uint2(e4m3x4(q[0].x, q[0].y, q[1].x, q[1].y) ^ 0x80808080u,
                      e4m3x4(q[2].x, q[2].y, q[3].x, q[3].y) ^ 0x80808080u);
}

// The largest |x| of eight BF16 as two magnitudes side by side, a NaN above infinity.
__device__ __forceinline__ uint32_t amax_pair8(uint4 v) {
    uint32_t a, b;
    asm("{\n\t.reg .b32 x, y;\n\t"
        "abs.bf16x2 x, %1;\n\tabs.bf16x2 y, %2;\n\tmax.NaN.bf16x2 %0, x, y;\n\t}"
        : "=r"(a)
        : "r"(v.x), "r"(v.y));
    asm("{\n\t.reg .b32 x, y;\n\t"
        "abs.bf16x2 x, %1;\n\tabs.bf16x2 y, %2;\n\tmax.NaN.bf16x2 %0, x, y;\n\t}"
        : "=r"(b)
        : "r"(v.z), "r"(v.w));
    return __vmaxu2(a, b);
}

// Four E4M3 codes (lowest byte first) as FP32, exact: every E4M3 value is an FP16 value.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t q, float2 &lo, float2 &hi) {
    uint32_t a, b;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(q));
    lo = __half22float2(*reinterpret_cast<__half2 *>(&a));
    hi = __half22float2(*reinterpret_cast<__half2 *>(&b));
}

// |x| folded into an FP32 magnitude kept as bits: the order of non-negative FP32 is that of
// their bits, and a NaN is above infinity, so a NaN in a block reaches its scale.
__device__ __forceinline__ uint32_t amax_fold_f32(uint32_t m, float2 x) {
    return max(m, max(__float_as_uint(x.x) & 0x7FFFFFFFu, __float_as_uint(x.y) & 0x7FFFFFFFu));
}

// max(m, |x.x|, |x.y|), a NaN winning, in one instruction; m >= 0.
__device__ __forceinline__ float amax3(float m, float2 x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(x.x)), "f"(fabsf(x.y)));
    return r;
}

// The maximum of `v` over the CTA's warps.  red: one word per warp, not in use by an
// earlier call that some thread may still read.
template <int WARPS>
__device__ __forceinline__ uint32_t cta_max(uint32_t v, uint32_t *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if ((threadIdx.x & 31u) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t m = red[0];
#pragma unroll
    for (int i = 1; i < WARPS; ++i) m = max(m, red[i]);
    return m;
}

}  // namespace dg

// FP32 -> E4M3 for values that a kernel computes itself (a weighted row, an activation, a
// gradient), and E4M3 -> FP32.  Same definition as the BF16 quantizer:
//   s = fl32(amax / 448), 1 if that is 0;  q = E4M3_rn_satfinite(fl32(x / s)).
// amax is an FP32 maximum here, so s may be any FP32; with amax below 448 times the least
// subnormal the quotient amax / 448 rounds to 0 and s = 1 (every code is then 0).
#pragma once

#include <cuda_fp16.h>

#include "quant_e4m3.cuh"

namespace dg {

// Eight BF16 of a 16-byte group as FP32: x + (-0) by the mixed-precision addition, which keeps
// every value and the sign of zero.  Its pipe has room where the shifts and masks of the
// integer form share theirs with the conversions to E4M3 that bound these kernels.
__device__ __forceinline__ void bf16x8_to_f32(uint4 v, float2 (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        asm("{\n\t.reg .b16 l, h;\n\t"
            "mov.b32 {l, h}, %2;\n\t"
            "add.f32.bf16 %0, l, %3;\n\t"
            "add.f32.bf16 %1, h, %3;\n\t}"
            : "=f"(x[j].x), "=f"(x[j].y)
            : "r"(w[j]), "f"(-0.0f));
}

// A block's scale and its reciprocal in two parts.  Inside the window s is a quotient corrected
// by its remainder, two multiply-adds after the product with 1/448 (P. W. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34, 1990, on division with a fused multiply-add): equal to fl32(amax / 448) for every
// FP32 amax there.  r is the hardware's approximation (within 1 unit of 1/s) lowered by
// 2^-21, so that it lies below 1/s; r_lo > 0 is the rest: with e = 1 - s r, exact but for
// its rounding, 1/s = r / (1 - e) = r + r (e + e^2 + ...), together good to 2^-43.
// Outside the window (NaN included) s comes from the division, and values are divided by it.
// The IEEE division and reciprocal cost every thread some 60 instructions a block, against
// 80 for converting one of its rows.
struct FastScale {
    float s, r, r_lo;
    bool fast;

    // For values that come with their sign flipped.
    __device__ __forceinline__ FastScale negated() const { return FastScale{-s, -r, -r_lo, fast}; }
};

__device__ __forceinline__ bool scale_is_fast(float amax) {
    return (amax >= 0x1p-90f && amax <= 0x1p100f) || amax == 0.0f;
}

__device__ __forceinline__ void split_reciprocal(FastScale &b) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b.s));
    b.r = __fmul_rn(r, 1.0f - 0x1p-21f);
    const float e = __fmaf_rn(-b.s, b.r, 1.0f);
    b.r_lo = __fmul_rn(__fmaf_rn(e, e, e), b.r);
}

// FAST: scale_is_fast(amax).
template <bool FAST>
__device__ __forceinline__ FastScale scale_of(float amax) {
    FastScale b;
    b.fast = FAST;
    if (FAST) {
        constexpr float c = 1.0f / 448.0f;
        const float q = __fmul_rn(amax, c);
        b.s = amax == 0.0f ? 1.0f : __fmaf_rn(__fmaf_rn(-q, 448.0f, amax), c, q);  // 1 for a block of zeros
    } else {
        const float q = __fdiv_rn(amax, 448.0f);
        b.s = (q == 0.0f) ? 1.0f : q;
    }
    split_reciprocal(b);
    return b;
}

__device__ __forceinline__ FastScale fast_scale(float amax) {
    return __builtin_expect(scale_is_fast(amax), 1) ? scale_of<true>(amax) : scale_of<false>(amax);
}

// Four pairs -> codes of fl32(x / s), as the rounding of x r + fl32(x r_lo): two operations a
// pair and one conversion, with no second path for values near a rounding boundary, which a
// block whose amax is a multiple of 7 meets often.  r_lo > 0 keeps the sign of a zero.
//   x BF16: for every x and amax in the window, and any approximation within 2 units of 1/s,
//     the code is that of the IEEE quotient (checked exhaustively on the CPU).
//   x any FP32: the quotient is the rounding of a value within 2^-43 of x/s, so the code can
//     differ only where x/s lies that close to the middle between an E4M3 rounding boundary
//     and the next FP32 number.
// (The product with the reciprocal corrected by its remainder, three operations, was as exact;
// FP32 products bound the gather's conversion.)
// FAST: b.fast, which the caller tests once for all its rows (a branch a row cost a tenth of
// the instructions and kept the rows' arithmetic apart).
template <bool FAST>
__device__ __forceinline__ uint2 quantize8_f32(const float2 (&x)[4], const FastScale &b) {
    float2 q[4];
    if (FAST) {
        const float2 r = make_float2(b.r, b.r), r_lo = make_float2(b.r_lo, b.r_lo);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = __ffma2_rn(x[j], r, __fmul2_rn(x[j], r_lo));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = make_float2(__fdiv_rn(x[j].x, b.s), __fdiv_rn(x[j].y, b.s));
    }
    return make_uint2(e4m3x4(q[0].x, q[0].y, q[1].x, q[1].y), e4m3x4(q[2].x, q[2].y, q[3].x, q[3].y));
}

// Eight BF16 -> codes of fl32(x / s), exactly.
template <bool FAST>
__device__ __forceinline__ uint2 quantize8_bf16(uint4 v, const FastScale &b) {
    float2 x[4];
    bf16x8_to_f32(v, x);
    return quantize8_f32<FAST>(x, b);
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

// Whether one of eight BF16 is a zero.
__device__ __forceinline__ bool has_zero8(uint4 v) {
    return (__vcmpeq2(v.x & 0x7FFF7FFFu, 0u) | __vcmpeq2(v.y & 0x7FFF7FFFu, 0u) | __vcmpeq2(v.z & 0x7FFF7FFFu, 0u) |
            __vcmpeq2(v.w & 0x7FFF7FFFu, 0u)) != 0u;
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

// max(m, |x.x|, |x.y|), a NaN winning, in one instruction; m >= 0.
__device__ __forceinline__ float amax3(float m, float2 x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(x.x)), "f"(fabsf(x.y)));
    return r;
}

// The maximum of `v` over the CTA's warps.  red: one word per warp, 16-byte aligned, not in
// use by an earlier call that some thread may still read.
template <int WARPS>
__device__ __forceinline__ uint32_t cta_max(uint32_t v, uint32_t *red) {
    static_assert(WARPS % 4 == 0, "read four words at a time");
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if ((threadIdx.x & 31u) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < WARPS / 4; ++i) {
        const uint4 w = reinterpret_cast<const uint4 *>(red)[i];
        m = max(m, max(max(w.x, w.y), max(w.z, w.w)));
    }
    return m;
}

}  // namespace dg

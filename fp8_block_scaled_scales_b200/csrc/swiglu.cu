// SwiGLU between the two products of an expert, with its output quantized for the second one
// and its input kept in 8 bits for the backward pass.
//
//   forward:  a = g * sigma(g) * u in FP32 from the BF16 row h = [g | u] (F columns each);
//             Q, S = the block quantizer's definition on a (FP32 values, no BF16 between);
//             H8, sH = the codes and per-row scales of dg_quantize_1x128 on h, bit for bit:
//             the checkpoint, half the bytes of h.
//   backward: from the checkpoint (g, u the decoded values) and dA (BF16):
//             dg = dA * u * sigma(g) * (1 + g * (1 - sigma(g))),   du = dA * g * sigma(g);
//             Q, S = the block quantizer's definition on [dg | du], ready for both gradient
//             products.
// sigma uses the hardware exponential and reciprocal (relative error of a few 2^-23 where
// the result is not negligible), far below the E4M3 rounding that follows.
#include <cuda_bf16.h>

#include "dg_device.cuh"
#include "quant_f32.cuh"
#include "train_internal.h"

namespace dg {

constexpr int kGluThreads = 512;  // 16 lanes a row, 32 rows at a time, 4 times
constexpr int kGluPer = 4;
constexpr int64_t kGluMaskedRowCtas = 16;

__device__ __forceinline__ float sigmoid_f32(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// Rows row0 .. row0 + rows - 1 (at most 128) of h [.][2F], column block bc of both halves.
// M: rows of the checkpoint's scale array.
template <bool CKPT>
__device__ __forceinline__ void glu_block(const uint16_t *__restrict__ Hin, int64_t F, int64_t M, int64_t row0,
                                          int rows, int64_t bc, uint8_t *__restrict__ Q, float *__restrict__ Sp,
                                          uint8_t *__restrict__ H8, float *__restrict__ sH, uint32_t *red) {
    const int tid = static_cast<int>(threadIdx.x);
    const int64_t col = bc * 128 + (tid & 15) * 8;
    const int sub = tid >> 4;
    uint4 vg[kGluPer], vu[kGluPer];
#pragma unroll
    for (int i = 0; i < kGluPer; ++i) {
        const int r = sub + 32 * i;
        const uint16_t *p = Hin + (row0 + r) * 2 * F + col;
        vg[i] = r < rows ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0, 0, 0, 0);
        vu[i] = r < rows ? __ldg(reinterpret_cast<const uint4 *>(p + F)) : make_uint4(0, 0, 0, 0);
    }
    float2 a[kGluPer][4];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kGluPer; ++i) {
        float2 g[4], u[4];
        bf16x8_to_f32(vg[i], g);
        bf16x8_to_f32(vu[i], u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[i][j].x = g[j].x * sigmoid_f32(g[j].x) * u[j].x;
            a[i][j].y = g[j].y * sigmoid_f32(g[j].y) * u[j].y;
            m = amax_fold_f32(m, a[i][j]);
        }
    }
    if (CKPT) {
#pragma unroll
        for (int i = 0; i < kGluPer; ++i) {
            const int64_t row = row0 + sub + 32 * i;
            const bool ok = sub + 32 * i < rows;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint4 v = half ? vu[i] : vg[i];
                uint32_t bits = amax_bits_of(amax_fold8(0u, v));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, o));
                const BlockScale bs = block_scale(bits);
                if (ok) {
                    *reinterpret_cast<uint2 *>(H8 + row * 2 * F + half * F + col) = quantize8(v, bs);
                    if ((tid & 15) == 0) sH[(half * (F / 128) + bc) * M + row] = bs.s;
                }
            }
        }
    }
    const BlockScale bs = block_scale_f32(__uint_as_float(cta_max<kGluThreads / 32>(m, red)));
    if (tid == 0) *Sp = bs.s;
#pragma unroll
    for (int i = 0; i < kGluPer; ++i) {
        const int r = sub + 32 * i;
        if (r < rows) *reinterpret_cast<uint2 *>(Q + (row0 + r) * F + col) = quantize8_f32(a[i], bs);
    }
}

// rows of the layout that hold something: all M, or up to the last expert's end
__device__ __forceinline__ int64_t used_rows(const int32_t *offsets, int G, int64_t M) {
    return offsets ? min(max(static_cast<int64_t>(__ldg(offsets + G)), int64_t(0)), M) : M;
}

template <bool CKPT>
__global__ void __launch_bounds__(kGluThreads, 2)
    swiglu_kernel(const uint16_t *__restrict__ Hin, const int32_t *__restrict__ offsets, int G, int64_t M, int64_t F,
                  uint8_t *__restrict__ Q, float *__restrict__ S, uint8_t *__restrict__ H8, float *__restrict__ sH) {
    __shared__ uint32_t red[kGluThreads / 32];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int64_t Fb = F / 128, blk = blockIdx.x;
    const int64_t lb = blk / Fb, bc = blk - lb * Fb;
    const int64_t left = used_rows(offsets, G, M) - lb * 128;
    if (left <= 0) return;
    glu_block<CKPT>(Hin, F, M, lb * 128, static_cast<int>(min(left, int64_t(128))), bc, Q, S + blk, H8, sH, red);
}

__global__ void __launch_bounds__(kGluThreads, 2)
    swiglu_masked_kernel(const uint16_t *__restrict__ Hin, const int32_t *__restrict__ masked_m, int64_t M, int64_t F,
                         int64_t Rb, int64_t Ry, uint8_t *__restrict__ Q, float *__restrict__ S) {
    __shared__ uint32_t red[2][kGluThreads / 32];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int64_t Fb = F / 128, blk = blockIdx.x;
    const int64_t gy = blk / Fb, bc = blk - gy * Fb;
    const int64_t g = gy / Ry, y = gy - g * Ry;
    const int64_t rows = min(max(static_cast<int64_t>(__ldg(masked_m + g)), int64_t(0)), M);
    int par = 0;
    for (int64_t lb = y; lb * 128 < rows; lb += Ry) {
        glu_block<false>(Hin, F, M, g * M + lb * 128, static_cast<int>(min(rows - lb * 128, int64_t(128))), bc, Q,
                         S + (g * Rb + lb) * Fb + bc, nullptr, nullptr, red[par]);
        par ^= 1;
    }
}

__global__ void __launch_bounds__(kGluThreads)
    swiglu_backward_kernel(const uint8_t *__restrict__ H8, const float *__restrict__ sH,
                           const uint16_t *__restrict__ dA, const int32_t *__restrict__ offsets, int G, int64_t M,
                           int64_t F, uint8_t *__restrict__ Q, float *__restrict__ S) {
    __shared__ uint32_t red[2][kGluThreads / 32];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int tid = static_cast<int>(threadIdx.x);
    const int64_t Fb = F / 128, blk = blockIdx.x;
    const int64_t lb = blk / Fb, bc = blk - lb * Fb;
    const int64_t left = used_rows(offsets, G, M) - lb * 128;
    if (left <= 0) return;
    const int rows = static_cast<int>(min(left, int64_t(128)));
    const int64_t col = bc * 128 + (tid & 15) * 8;
    const int sub = tid >> 4;
    uint2 cg[kGluPer], cu[kGluPer];
    uint4 va[kGluPer];
    float sg[kGluPer], su[kGluPer];
#pragma unroll
    for (int i = 0; i < kGluPer; ++i) {
        const int r = sub + 32 * i;
        const int64_t row = lb * 128 + r;
        const bool ok = r < rows;
        const uint8_t *p = H8 + row * 2 * F + col;
        cg[i] = ok ? __ldg(reinterpret_cast<const uint2 *>(p)) : make_uint2(0, 0);
        cu[i] = ok ? __ldg(reinterpret_cast<const uint2 *>(p + F)) : make_uint2(0, 0);
        va[i] = ok ? __ldg(reinterpret_cast<const uint4 *>(dA + row * F + col)) : make_uint4(0, 0, 0, 0);
        sg[i] = ok ? __ldg(sH + bc * M + row) : 0.0f;
        su[i] = ok ? __ldg(sH + (Fb + bc) * M + row) : 0.0f;
    }
    float2 dg[kGluPer][4], du[kGluPer][4];
    uint32_t mg = 0, mu = 0;
#pragma unroll
    for (int i = 0; i < kGluPer; ++i) {
        float2 g[4], u[4], d[4];
        e4m3x4_to_f32(cg[i].x, g[0], g[1]);
        e4m3x4_to_f32(cg[i].y, g[2], g[3]);
        e4m3x4_to_f32(cu[i].x, u[0], u[1]);
        e4m3x4_to_f32(cu[i].y, u[2], u[3]);
        bf16x8_to_f32(va[i], d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float gx = g[j].x * sg[i], gy = g[j].y * sg[i];
            const float ux = u[j].x * su[i], uy = u[j].y * su[i];
            const float px = sigmoid_f32(gx), py = sigmoid_f32(gy);
            dg[i][j] = make_float2(d[j].x * ux * px * (1.0f + gx * (1.0f - px)),
                                   d[j].y * uy * py * (1.0f + gy * (1.0f - py)));
            du[i][j] = make_float2(d[j].x * gx * px, d[j].y * gy * py);
            mg = amax_fold_f32(mg, dg[i][j]);
            mu = amax_fold_f32(mu, du[i][j]);
        }
    }
    const BlockScale bg = block_scale_f32(__uint_as_float(cta_max<kGluThreads / 32>(mg, red[0])));
    const BlockScale bu = block_scale_f32(__uint_as_float(cta_max<kGluThreads / 32>(mu, red[1])));
    if (tid == 0) {
        S[lb * 2 * Fb + bc] = bg.s;
        S[lb * 2 * Fb + Fb + bc] = bu.s;
    }
#pragma unroll
    for (int i = 0; i < kGluPer; ++i) {
        const int r = sub + 32 * i;
        if (r < rows) {
            uint8_t *q = Q + (lb * 128 + r) * 2 * F + col;
            *reinterpret_cast<uint2 *>(q) = quantize8_f32(dg[i], bg);
            *reinterpret_cast<uint2 *>(q + F) = quantize8_f32(du[i], bu);
        }
    }
}

dg_status_t launch_swiglu(const void *H, const int32_t *offsets, const int32_t *masked_m, int G, int64_t M,
                          int64_t F, uint8_t *Q, float *S, uint8_t *H8, float *sH, cudaStream_t stream) {
    const int64_t Rb = (M + 127) / 128, Fb = F / 128;
    const uint16_t *h = static_cast<const uint16_t *>(H);
    if (masked_m) {
        const int64_t Ry = Rb < kGluMaskedRowCtas ? Rb : kGluMaskedRowCtas;
        if (G * Ry * Fb > 0x7FFFFFFFLL) return DG_ERR_SHAPE;
        return launch_pdl(swiglu_masked_kernel, static_cast<int>(G * Ry * Fb), kGluThreads, 0, stream, h, masked_m, M,
                          F, Rb, Ry, Q, S);
    }
    if (Rb * Fb > 0x7FFFFFFFLL) return DG_ERR_SHAPE;
    const int n = static_cast<int>(Rb * Fb);
    if (H8) return launch_pdl(swiglu_kernel<true>, n, kGluThreads, 0, stream, h, offsets, G, M, F, Q, S, H8, sH);
    return launch_pdl(swiglu_kernel<false>, n, kGluThreads, 0, stream, h, offsets, G, M, F, Q, S, H8, sH);
}

dg_status_t launch_swiglu_backward(const uint8_t *H8, const float *sH, const void *dA, const int32_t *offsets,
                                   int G, int64_t M, int64_t F, uint8_t *Q, float *S, cudaStream_t stream) {
    const int64_t n = (M + 127) / 128 * (F / 128);
    if (n > 0x7FFFFFFFLL) return DG_ERR_SHAPE;
    return launch_pdl(swiglu_backward_kernel, static_cast<int>(n), kGluThreads, 0, stream, H8, sH,
                      static_cast<const uint16_t *>(dA), offsets, G, M, F, Q, S);
}

}  // namespace dg

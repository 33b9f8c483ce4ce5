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
// the result is not negligible), far below the E4M3 rounding that follows; for the same
// reason a / s is a product with the rounded 1/s (quantize8_near).
#include <cuda_bf16.h>

#include "dg_device.cuh"
#include "quant_f32.cuh"
#include "train_internal.h"

namespace dg {

constexpr int kGluThreads = 512;  // 16 lanes a row, 32 rows at a time, 4 times
constexpr int kGluPer = 4;
constexpr int64_t kGluMaskedRowCtas = 16;

// sigma of two values; exp overflows to infinity for x < -88, whose reciprocal is 0
__device__ __forceinline__ float2 sigmoid2(float2 x) {
    const float2 e = make_float2(__expf(-x.x), __expf(-x.y));
    return make_float2(__fdividef(1.0f, 1.0f + e.x), __fdividef(1.0f, 1.0f + e.y));
}

// One row group of 128 columns (16 lanes, 8 values each) as a 1 x 128 block: codes to *q, the
// scale to *s by the first lane.  All lanes of the warp call it.
__device__ __forceinline__ void checkpoint_row(uint4 v, bool ok, bool first, uint8_t *q, float *s) {
    uint32_t bits = amax_bits_of(amax_fold8(0u, v));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, o));
    const BlockScale bs = block_scale(bits);
    if (ok) {
        *reinterpret_cast<uint2 *>(q) = quantize8(v, bs);
        if (first) *s = bs.s;
    }
}

// Rows row0 .. row0 + rows - 1 (at most 128) of h [.][2F], column block bc of both halves.
// M: rows of the checkpoint's scale array.  Rows are taken two at a time: with all four
// loaded first the 64 registers that let two CTAs share an SM spill (386 us against
// 0.07 ms of traffic on 16384 x 4096), and two rows of both CTAs keep 64 KB in flight.
template <bool CKPT>
__device__ __forceinline__ void glu_block(const uint16_t *__restrict__ Hin, int64_t F, int64_t M, int64_t row0,
                                          int rows, int64_t bc, uint8_t *__restrict__ Q, float *__restrict__ Sp,
                                          uint8_t *__restrict__ H8, float *__restrict__ sH, uint32_t *red) {
    const int tid = static_cast<int>(threadIdx.x);
    const int64_t col = bc * 128 + (tid & 15) * 8;
    const int sub = tid >> 4;
    const bool first = (tid & 15) == 0;
    const int64_t at = (row0 + sub) * 2 * F + col, step = 64 * F;  // 32 rows of h
    const uint16_t *p = Hin + at;
    uint8_t *p8 = CKPT ? H8 + at : nullptr;
    float *ps = CKPT ? sH + bc * M + row0 + sub : nullptr;
    float2 a[kGluPer][4];
    uint32_t m = 0;
#pragma unroll
    for (int i0 = 0; i0 < kGluPer; i0 += 2) {
        uint4 vg[2], vu[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool ok = sub + 32 * (i0 + i) < rows;
            vg[i] = ok ? __ldg(reinterpret_cast<const uint4 *>(p + (i0 + i) * step)) : make_uint4(0, 0, 0, 0);
            vu[i] = ok ? __ldg(reinterpret_cast<const uint4 *>(p + (i0 + i) * step + F)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float2 g[4], u[4];
            bf16x8_to_f32(vg[i], g);
            bf16x8_to_f32(vu[i], u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = __fmul2_rn(__fmul2_rn(g[j], sigmoid2(g[j])), u[j]);
                m = amax_fold_f32(m, x);
                a[i0 + i][j] = x;
            }
            if (CKPT) {
                const bool ok = sub + 32 * (i0 + i) < rows;
                uint8_t *q = p8 + (i0 + i) * step;
                float *sp = ps + 32 * (i0 + i);
                checkpoint_row(vg[i], ok, first, q, sp);
                checkpoint_row(vu[i], ok, first, q + F, sp + (F / 128) * M);
            }
        }
    }
    const NearScale bs = near_scale(cta_max<kGluThreads / 32>(m, red));
    if (tid == 0) *Sp = bs.s;
    uint8_t *q = Q + (row0 + sub) * F + col;
#pragma unroll
    for (int i = 0; i < kGluPer; ++i)
        if (sub + 32 * i < rows) *reinterpret_cast<uint2 *>(q + i * (step >> 1)) = quantize8_near(a[i], bs);
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

// Backward: one persistent CTA per SM.  A block's [dg | du] in FP32 is half the register
// file, so no second CTA fits beside it; instead every thread copies its own piece of the
// next block into shared memory (cp.async) before it computes the current one, so loads
// run under the arithmetic.
struct GluBackSmem {
    uint2 cg[kGluPer][kGluThreads];
    uint2 cu[kGluPer][kGluThreads];
    uint4 da[kGluPer][kGluThreads];
    float scale[2][128];  // the block's row scales, gate then up
};

__device__ __forceinline__ void cp_async(void *dst, const void *src, int bytes_8_or_16) {
    if (bytes_8_or_16 == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

__global__ void __launch_bounds__(kGluThreads, 1)
    swiglu_backward_kernel(const uint8_t *__restrict__ H8, const float *__restrict__ sH,
                           const uint16_t *__restrict__ dA, const int32_t *__restrict__ offsets, int G, int64_t M,
                           int64_t F, uint8_t *__restrict__ Q, float *__restrict__ S) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    GluBackSmem *stage = reinterpret_cast<GluBackSmem *>(smem_raw);
    __shared__ uint32_t red[2][2][kGluThreads / 32];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int tid = static_cast<int>(threadIdx.x);
    const int lane16 = tid & 15, sub = tid >> 4;
    const int64_t Fb = F / 128;
    const int64_t used = used_rows(offsets, G, M);
    const int64_t blocks = (used + 127) / 128 * Fb;

    auto prefetch = [&](int64_t blk, GluBackSmem &st) {
        if (blk < blocks) {
            const int64_t lb = blk / Fb, bc = blk - lb * Fb;
            const int rows = static_cast<int>(min(used - lb * 128, int64_t(128)));
            const int64_t row = lb * 128 + sub, col = bc * 128 + lane16 * 8;
            const uint8_t *p = H8 + row * 2 * F + col;
            const uint16_t *pa = dA + row * F + col;
#pragma unroll
            for (int i = 0; i < kGluPer; ++i) {
                if (sub + 32 * i < rows) {
                    cp_async(&st.cg[i][tid], p + i * 64 * F, 8);
                    cp_async(&st.cu[i][tid], p + i * 64 * F + F, 8);
                    cp_async(&st.da[i][tid], pa + i * 32 * F, 16);
                }
            }
            if (tid < 256) {
                const int r = tid & 127, half = tid >> 7;
                if (r < rows) cp_async4(&st.scale[half][r], sH + (half * Fb + bc) * M + lb * 128 + r);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    int par = 0;
    prefetch(blockIdx.x, stage[0]);
    for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x, par ^= 1) {
        prefetch(blk + gridDim.x, stage[par ^ 1]);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();  // the scales come from other threads' copies
        const GluBackSmem &st = stage[par];
        const int64_t lb = blk / Fb, bc = blk - lb * Fb;
        const int rows = static_cast<int>(min(used - lb * 128, int64_t(128)));
        float2 dg[kGluPer][4], du[kGluPer][4];
        uint32_t mg = 0, mu = 0;
#pragma unroll
        for (int i = 0; i < kGluPer; ++i) {
            const int r = sub + 32 * i;
            const bool ok = r < rows;
            const uint2 cg = ok ? st.cg[i][tid] : make_uint2(0, 0), cu = ok ? st.cu[i][tid] : make_uint2(0, 0);
            const uint4 va = ok ? st.da[i][tid] : make_uint4(0, 0, 0, 0);
            const float sg = ok ? st.scale[0][r] : 0.0f, su = ok ? st.scale[1][r] : 0.0f;
            float2 g[4], u[4], d[4];
            e4m3x4_to_f32(cg.x, g[0], g[1]);
            e4m3x4_to_f32(cg.y, g[2], g[3]);
            e4m3x4_to_f32(cu.x, u[0], u[1]);
            e4m3x4_to_f32(cu.y, u[2], u[3]);
            bf16x8_to_f32(va, d);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 gs = __fmul2_rn(g[j], make_float2(sg, sg)), us = __fmul2_rn(u[j], make_float2(su, su));
                const float2 p = sigmoid2(gs);
                const float2 t = __fmul2_rn(d[j], p);
                const float2 np = make_float2(1.0f - p.x, 1.0f - p.y);
                du[i][j] = __fmul2_rn(t, gs);
                dg[i][j] = __fmul2_rn(__fmul2_rn(t, us), __ffma2_rn(gs, np, make_float2(1.0f, 1.0f)));
                mg = amax_fold_f32(mg, dg[i][j]);
                mu = amax_fold_f32(mu, du[i][j]);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            mg = max(mg, __shfl_xor_sync(0xFFFFFFFFu, mg, o));
            mu = max(mu, __shfl_xor_sync(0xFFFFFFFFu, mu, o));
        }
        if ((tid & 31) == 0) {
            red[par][0][tid >> 5] = mg;
            red[par][1][tid >> 5] = mu;
        }
        __syncthreads();
        mg = red[par][0][lane16];
        mu = red[par][1][lane16];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            mg = max(mg, __shfl_xor_sync(0xFFFFFFFFu, mg, o));
            mu = max(mu, __shfl_xor_sync(0xFFFFFFFFu, mu, o));
        }
        const NearScale bg = near_scale(mg), bu = near_scale(mu);
        if (tid == 0) {
            S[lb * 2 * Fb + bc] = bg.s;
            S[lb * 2 * Fb + Fb + bc] = bu.s;
        }
        uint8_t *q = Q + (lb * 128 + sub) * 2 * F + bc * 128 + lane16 * 8;
#pragma unroll
        for (int i = 0; i < kGluPer; ++i) {
            if (sub + 32 * i < rows) {
                *reinterpret_cast<uint2 *>(q + i * 64 * F) = quantize8_near(dg[i], bg);
                *reinterpret_cast<uint2 *>(q + i * 64 * F + F) = quantize8_near(du[i], bu);
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}
static_assert(kGluThreads / 32 == 16, "the reduction over warps uses 16 lanes");

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
                                   int G, int64_t M, int64_t F, uint8_t *Q, float *S, const DeviceInfo &dev,
                                   cudaStream_t stream) {
    const int64_t blocks = (M + 127) / 128 * (F / 128);
    const size_t smem = 2 * sizeof(GluBackSmem);
    static thread_local int configured_device = -1;
    int device = 0;
    cudaGetDevice(&device);
    if (configured_device != device) {
        if (cudaFuncSetAttribute(swiglu_backward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem)) != cudaSuccess)
            return DG_ERR_CUDA;
        configured_device = device;
    }
    const int n = static_cast<int>(blocks < dev.num_sms ? blocks : dev.num_sms);
    return launch_pdl(swiglu_backward_kernel, n, kGluThreads, smem, stream, H8, sH,
                      static_cast<const uint16_t *>(dA), offsets, G, M, F, Q, S);
}

}  // namespace dg

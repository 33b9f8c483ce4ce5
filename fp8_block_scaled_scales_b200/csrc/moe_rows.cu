// Rows between tokens and experts: tokens gathered by expert and quantized in one pass, and
// expert rows brought back to their tokens with weights, with the weights' gradient.
//
// dispatch_quantize:  v[r] = x[slot / k] (times weights[slot] as an FP32 product), zero for a
//   row without a slot; then the block quantizer's definition on v:
//   s = fl32(amax / 448) per 128x128 block (1 if 0), q = E4M3_rn_satfinite(fl32(v / s)).
//   Without weights the codes and scales are those of the block quantizer on the gathered
//   matrix, bit for bit.  With weights it is the gradient of the combination with respect to
//   the expert rows.
// combine:            out[t] = bf16(sum_j weights[t][j] * y[row(t, j)]), FP32, ascending j;
//   without weights it is the gradient of the dispatch.
// combine_backward:   dweights[t][j] = sum_h dout[t][h] * y[row(t, j)][h], FP32.
#include <cuda_bf16.h>

#include "dg_device.cuh"
#include "quant_f32.cuh"
#include "train_internal.h"

namespace dg {

constexpr int kRowThreads = 256;
constexpr int64_t kDispatchMaskedRowCtas = 16;  // CTAs per slab and column block, as in the masked quantizer

// One 128x128 block: rows row0 .. of the sorted layout (`rows` of them in the block, at most
// 128), column block bc.  tok / wgt: the block's tokens (-1: no slot) and weights.
template <bool WEIGHTS>
__device__ __forceinline__ void dispatch_block(const uint16_t *__restrict__ X, const float *__restrict__ weights,
                                               const int32_t *__restrict__ slot_of_row, int slots, int k, int64_t H,
                                               int64_t row0, int rows, int64_t bc, uint8_t *__restrict__ Q,
                                               float *__restrict__ Sp, int *tok, float *wgt, uint32_t *red) {
    const int tid = static_cast<int>(threadIdx.x);
    if (tid < 128) {
        const int slot = tid < rows ? __ldg(slot_of_row + row0 + tid) : -1;
        const bool ok = slot >= 0 && slot < slots;  // anything else is a row without a slot
        tok[tid] = ok ? slot / k : -1;
        if (WEIGHTS) wgt[tid] = ok ? __ldg(weights + slot) : 0.0f;
    }
    __syncthreads();
    const int chunk = tid & 15, sub = tid >> 4;
    const int64_t col = bc * 128 + chunk * 8;
    const bool col_ok = col < H;  // H % 16 == 0: an 8-column piece is whole or absent
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int t = tok[sub + 16 * i];
        v[i] = (t >= 0 && col_ok) ? __ldg(reinterpret_cast<const uint4 *>(X + static_cast<int64_t>(t) * H + col))
                                  : make_uint4(0, 0, 0, 0);
    }
    float w[8];
    uint32_t m = 0;
    if (WEIGHTS) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = wgt[sub + 16 * i];
            float2 x[4];
            bf16x8_to_f32(v[i], x);
#pragma unroll
            for (int j = 0; j < 4; ++j) m = amax_fold_f32(m, __fmul2_rn(x[j], make_float2(w[i], w[i])));
        }
    } else {
        uint32_t m2 = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m2 = amax_fold8(m2, v[i]);
        m = amax_bits_of(m2);
    }
    m = cta_max<kRowThreads / 32>(m, red);
    const BlockScale bs = WEIGHTS ? block_scale_f32(__uint_as_float(m)) : block_scale(m);
    if (tid == 0) *Sp = bs.s;
    uint8_t *qp = Q + (row0 + sub) * H + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (!col_ok || sub + 16 * i >= rows) break;
        uint2 q;
        if (WEIGHTS) {
            float2 x[4];
            bf16x8_to_f32(v[i], x);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = __fmul2_rn(x[j], make_float2(w[i], w[i]));
            q = quantize8_f32(x, bs);
        } else {
            q = quantize8(v[i], bs);
        }
        *reinterpret_cast<uint2 *>(qp + static_cast<int64_t>(16 * i) * H) = q;
    }
}

// Contiguous layout: one CTA per block of the row capacity; those past the last expert's
// rows leave at once and write nothing.
template <bool WEIGHTS>
__global__ void __launch_bounds__(kRowThreads, 4)
    dispatch_kernel(const uint16_t *__restrict__ X, const float *__restrict__ weights,
                    const int32_t *__restrict__ slot_of_row, const int32_t *__restrict__ offsets, int G, int slots,
                    int k, int64_t H, int64_t Cb, uint8_t *__restrict__ Q, float *__restrict__ S) {
    __shared__ int tok[128];
    __shared__ float wgt[128];
    __shared__ uint32_t red[kRowThreads / 32];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int64_t blk = blockIdx.x;
    const int64_t lb = blk / Cb, bc = blk - lb * Cb;
    if (lb * 128 >= __ldg(offsets + G)) return;
    dispatch_block<WEIGHTS>(X, weights, slot_of_row, slots, k, H, lb * 128, 128, bc, Q, S + blk, tok, wgt, red);
}

// Masked layout: CTA (g, y, bc) takes the slab's row blocks y, y + Ry, ... that hold tokens;
// rows past the count are neither read nor written.
__global__ void __launch_bounds__(kRowThreads, 4)
    dispatch_masked_kernel(const uint16_t *__restrict__ X, const int32_t *__restrict__ slot_of_row,
                           const int32_t *__restrict__ masked_m, int slots, int k, int64_t H, int64_t Cb,
                           int64_t m_max, int64_t Rb, int64_t Ry, uint8_t *__restrict__ Q, float *__restrict__ S) {
    __shared__ int tok[128];
    __shared__ uint32_t red[kRowThreads / 32];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int64_t blk = blockIdx.x;
    const int64_t gy = blk / Cb, bc = blk - gy * Cb;
    const int64_t g = gy / Ry, y = gy - g * Ry;
    const int64_t rows = min(max(static_cast<int64_t>(__ldg(masked_m + g)), int64_t(0)), m_max);
    for (int64_t lb = y; lb * 128 < rows; lb += Ry) {
        if (lb != y) __syncthreads();  // tok and red of the previous block are no longer read
        dispatch_block<false>(X, nullptr, slot_of_row, slots, k, H, g * m_max + lb * 128,
                              static_cast<int>(min(rows - lb * 128, int64_t(128))), bc, Q, S + (g * Rb + lb) * Cb + bc,
                              tok, nullptr, red);
    }
}

// One CTA per token and 1024 columns, eight columns a thread; the rows of up to four slots
// are in flight at a time.
constexpr int kCombineThreads = 128;
constexpr int kCombineCols = kCombineThreads * 8;

template <bool WEIGHTS>
__global__ void __launch_bounds__(kCombineThreads)
    combine_kernel(const uint16_t *__restrict__ Y, const float *__restrict__ weights,
                   const int32_t *__restrict__ row_of_slot, int k, int64_t H, int rows, int chunks,
                   uint16_t *__restrict__ out) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int64_t t = blockIdx.x / chunks;
    const int64_t col = static_cast<int64_t>(blockIdx.x - t * chunks) * kCombineCols + threadIdx.x * 8;
    if (col >= H) return;
    float2 acc[4] = {};
    for (int j0 = 0; j0 < k; j0 += 4) {
        uint4 v[4];
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t slot = t * k + j0 + j;
            const int row = j0 + j < k ? __ldg(row_of_slot + slot) : -1;
            const bool ok = row >= 0 && row < rows;
            w[j] = WEIGHTS ? (ok ? __ldg(weights + slot) : 0.0f) : 1.0f;
            v[j] = ok ? __ldg(reinterpret_cast<const uint4 *>(Y + static_cast<int64_t>(row) * H + col))
                      : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 x[4];
            bf16x8_to_f32(v[j], x);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = __ffma2_rn(x[i], make_float2(w[j], w[j]), acc[i]);
        }
    }
    *reinterpret_cast<uint4 *>(out + t * H + col) =
        make_uint4(pack_bf16x2(acc[0].x, acc[0].y), pack_bf16x2(acc[1].x, acc[1].y),
                   pack_bf16x2(acc[2].x, acc[2].y), pack_bf16x2(acc[3].x, acc[3].y));
}

// One warp per slot: each lane adds the products of every 32nd group of eight columns, then
// the lanes are added in a fixed tree.  The slots of a token are neighbours, so its row of
// dout comes from the cache.
__global__ void __launch_bounds__(kRowThreads)
    combine_backward_kernel(const uint16_t *__restrict__ dout, const uint16_t *__restrict__ Y,
                            const int32_t *__restrict__ row_of_slot, int64_t slots, int k, int64_t H, int rows,
                            float *__restrict__ dweights) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (slot >= slots) return;
    const int lane = lane_id();
    const int row = __ldg(row_of_slot + slot);
    float sum = 0.0f;
    if (row >= 0 && row < rows) {
        const uint4 *a = reinterpret_cast<const uint4 *>(dout + slot / k * H);
        const uint4 *b = reinterpret_cast<const uint4 *>(Y + static_cast<int64_t>(row) * H);
        const int n = static_cast<int>(H / 8);
        float2 acc = make_float2(0.0f, 0.0f);
        for (int i0 = lane; i0 < n; i0 += 128) {
            uint4 p[4], q[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u * 32;
                p[u] = i < n ? __ldg(a + i) : make_uint4(0, 0, 0, 0);
                q[u] = i < n ? __ldg(b + i) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float2 x[4], y[4];
                bf16x8_to_f32(p[u], x);
                bf16x8_to_f32(q[u], y);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc = __ffma2_rn(x[i], y[i], acc);
            }
        }
        sum = acc.x + acc.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
    if (lane == 0) dweights[slot] = sum;
}

dg_status_t launch_dispatch_quantize(const void *X, const float *weights, const int32_t *slot_of_row,
                                     const int32_t *offsets, int64_t slots, int k, int64_t H, int64_t rows, int G,
                                     uint8_t *Q, float *S, cudaStream_t stream) {
    const int64_t Cb = (H + 127) / 128, blocks = rows / 128 * Cb;
    if (blocks > 0x7FFFFFFFLL) return DG_ERR_SHAPE;
    const uint16_t *x = static_cast<const uint16_t *>(X);
    const int n = static_cast<int>(blocks), s = static_cast<int>(slots);
    if (weights)
        return launch_pdl(dispatch_kernel<true>, n, kRowThreads, 0, stream, x, weights, slot_of_row, offsets, G, s, k,
                          H, Cb, Q, S);
    return launch_pdl(dispatch_kernel<false>, n, kRowThreads, 0, stream, x, weights, slot_of_row, offsets, G, s, k, H,
                      Cb, Q, S);
}

dg_status_t launch_dispatch_quantize_masked(const void *X, const int32_t *slot_of_row, const int32_t *masked_m,
                                            int64_t slots, int k, int64_t H, int G, int64_t m_max, uint8_t *Q,
                                            float *S, cudaStream_t stream) {
    const int64_t Rb = (m_max + 127) / 128, Cb = (H + 127) / 128;
    const int64_t Ry = Rb < kDispatchMaskedRowCtas ? Rb : kDispatchMaskedRowCtas;
    if (G * Ry * Cb > 0x7FFFFFFFLL) return DG_ERR_SHAPE;
    return launch_pdl(dispatch_masked_kernel, static_cast<int>(G * Ry * Cb), kRowThreads, 0, stream,
                      static_cast<const uint16_t *>(X), slot_of_row, masked_m, static_cast<int>(slots), k, H, Cb, m_max,
                      Rb, Ry, Q, S);
}

dg_status_t launch_combine(const void *Y, const float *weights, const int32_t *row_of_slot, int64_t T, int k,
                           int64_t H, int64_t rows, void *out, cudaStream_t stream) {
    const int64_t chunks = (H + kCombineCols - 1) / kCombineCols;
    if (T * chunks > 0x7FFFFFFFLL) return DG_ERR_SHAPE;
    const int n = static_cast<int>(T * chunks);
    if (weights)
        return launch_pdl(combine_kernel<true>, n, kCombineThreads, 0, stream, static_cast<const uint16_t *>(Y),
                          weights, row_of_slot, k, H, static_cast<int>(rows), static_cast<int>(chunks),
                          static_cast<uint16_t *>(out));
    return launch_pdl(combine_kernel<false>, n, kCombineThreads, 0, stream, static_cast<const uint16_t *>(Y), weights,
                      row_of_slot, k, H, static_cast<int>(rows), static_cast<int>(chunks),
                      static_cast<uint16_t *>(out));
}

dg_status_t launch_combine_backward(const void *dout, const void *Y, const int32_t *row_of_slot, int64_t T, int k,
                                    int64_t H, int64_t rows, float *dweights, cudaStream_t stream) {
    const int64_t slots = T * k;
    const int64_t n = (slots + kRowThreads / 32 - 1) / (kRowThreads / 32);
    return launch_pdl(combine_backward_kernel, static_cast<int>(n), kRowThreads, 0, stream,
                      static_cast<const uint16_t *>(dout), static_cast<const uint16_t *>(Y), row_of_slot, slots, k, H,
                      static_cast<int>(rows), dweights);
}

}  // namespace dg

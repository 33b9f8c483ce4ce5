// Rows between tokens and experts: tokens gathered by expert and quantized in one pass, and
// expert rows brought back to their tokens with weights, with the weights' gradient.
//
// dispatch_quantize:  v[r] = x[slot / k] (times weights[slot] as an FP32 product), zero for a
//   row without a slot; then the block quantizer's definition on v:
//   s = fl32(amax / 448) per 128x128 block (1 if 0), q = E4M3_rn_satfinite(fl32(v / s)).
//   Without weights the codes and scales are those of the block quantizer on the gathered
//   matrix, bit for bit.  With weights it is the gradient of the combination with respect to
//   the expert rows (quantize8_f32 says where a code may differ from the definition's).
// combine:            out[t] = bf16(sum_j weights[t][j] * y[row(t, j)]), FP32, ascending j;
//   without weights it is the gradient of the dispatch.
// combine_backward:   dweights[t][j] = sum_h dout[t][h] * y[row(t, j)][h], FP32.
#include <cuda_bf16.h>

#include <type_traits>

#include "dg_device.cuh"
#include "quant_f32.cuh"
#include "train_internal.h"

namespace dg {

constexpr int kRowThreads = 256;

// A CTA's share of the gather: one row block of 128 rows (masked: of a slab, every Ry-th) and
// a run of column blocks.  The tokens are looked up once; then, column block by column block,
// a thread reads its eight 16-byte pieces from shared memory, asks for the next column
// block's (cp.async), and reduces and converts the current ones, so that the gather runs under
// the conversion.  All CTAs walk the columns at the same pace, so the k copies of a token's
// piece are read close together: once from memory (ncu: 64 MB of 59), then from L2.  32768
// slots x 7168: 92 us, 730 MB through L2; without the conversion, the moves and the block
// maximum alone take 78 us, without the maximum 85.  (A CTA per block, rows first: 137 us with
// 28 % L2 hits.)  With weights 96 us.  256 threads of eight rows: 512 of four 116 us, 128 of
// sixteen 99.
struct DispatchSmem {
    uint4 piece[8][kRowThreads];
    int tok[128];
    float wgt[128];
    alignas(16) uint32_t red[2][kRowThreads / 32];
};

template <bool WEIGHTS>
__device__ __forceinline__ void dispatch_rows(const uint16_t *__restrict__ X, const float *__restrict__ weights,
                                              const int32_t *__restrict__ slot_of_row, int slots, int k, int64_t H,
                                              int64_t row0, int rows, int bc0, int bc1, uint8_t *__restrict__ Q,
                                              float *__restrict__ S, DispatchSmem &sm) {
    const int tid = static_cast<int>(threadIdx.x);
    const int sub = tid >> 4, lane_col = (tid & 15) * 8;
    const int Hi = static_cast<int>(H);  // a 32 x 32 bit product for each address
    __syncthreads();  // an earlier row block's tokens are no longer read
    bool infinite = false;
    if (tid < 128) {
        const int slot = tid < rows ? __ldg(slot_of_row + row0 + tid) : -1;
        const bool ok = slot >= 0 && slot < slots;  // anything else is a row without a slot
        sm.tok[tid] = ok ? slot / k : -1;
        if (WEIGHTS) {
            const float w = ok ? __ldg(weights + slot) : 0.0f;
            sm.wgt[tid] = w;
            infinite = isinf(w);
        }
    }
    infinite = __syncthreads_or(infinite);  // some row's weight is
    // a row without a token: its pieces stay zero
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (sm.tok[sub + 16 * i] < 0) sm.piece[i][tid] = make_uint4(0, 0, 0, 0);

    auto ask = [&](int bc) {
        const int64_t col = static_cast<int64_t>(bc) * 128 + lane_col;
        if (col < H) {  // H % 16 == 0: an 8-column piece is whole or absent
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = sm.tok[sub + 16 * i];
                if (t >= 0) {
                    const uint16_t *p = X + static_cast<int64_t>(t) * Hi + col;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&sm.piece[i][tid])), "l"(p)
                                 : "memory");
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) sm.piece[i][tid] = make_uint4(0, 0, 0, 0);
        }
    };

    ask(bc0);
    uint8_t *qp = Q + (row0 + sub) * H + static_cast<int64_t>(bc0) * 128 + lane_col;
    const int64_t step = 16 * H;
    for (int bc = bc0; bc < bc1; ++bc, qp += 128) {
        const bool col_ok = static_cast<int64_t>(bc) * 128 + lane_col < H;
        asm volatile("cp.async.wait_all;" ::: "memory");
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = sm.piece[i][tid];
        if (bc + 1 < bc1) ask(bc + 1);
        uint32_t m;
        if (WEIGHTS) {
            // the largest |fl32(w x)| of a row's piece is that of its largest |x|
            float f = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float a = __uint_as_float(amax_bits_of(amax_pair8(v[i])) << 16);
                const float b = __uint_as_float(amax_bits_of(amax_pair8(v[i + 1])) << 16);
                f = amax3(f, make_float2(a * sm.wgt[sub + 16 * i], b * sm.wgt[sub + 16 * (i + 1)]));
            }
            if (__builtin_expect(infinite, 0)) {  // then a zero among the row's columns is a NaN
                f = col_ok ? f : 0.0f;            // and there is none past the last column
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (col_ok && isinf(sm.wgt[sub + 16 * i]) && has_zero8(v[i])) f = __int_as_float(0x7FFFFFFF);
            }
            m = __float_as_uint(f);
        } else {
            uint32_t m2 = amax_pair8(v[0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) m2 = __vmaxu2(m2, amax_pair8(v[i]));
            m = amax_bits_of(m2) << 16;  // the maximum's FP32 bits
        }
        m = cta_max<kRowThreads / 32>(m, sm.red[bc & 1]);
        const FastScale bs = fast_scale(__uint_as_float(m));
        if (tid == 0) S[bc] = bs.s;
        auto convert = [&](auto fast) {
            constexpr bool kFast = decltype(fast)::value;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint2 q;
                if (WEIGHTS) {
                    const float w = sm.wgt[sub + 16 * i];
                    float2 x[4];
                    bf16x8_to_f32(v[i], x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = __fmul2_rn(x[j], make_float2(w, w));
                    q = quantize8_f32<kFast>(x, bs);
                } else {
                    q = quantize8_bf16<kFast>(v[i], bs);
                }
                if (sub + 16 * i < rows) *reinterpret_cast<uint2 *>(qp + i * step) = q;
            }
        };
        if (col_ok) {
            if (__builtin_expect(bs.fast, 1))
                convert(std::true_type{});
            else
                convert(std::false_type{});
        }
    }
}

// How the column blocks are cut: CTA (chunk, row block), row block fastest, takes column
// blocks [chunk * cols, ...).
template <bool WEIGHTS>
__global__ void __launch_bounds__(kRowThreads, 4)
    dispatch_kernel(const uint16_t *__restrict__ X, const float *__restrict__ weights,
                    const int32_t *__restrict__ slot_of_row, const int32_t *__restrict__ offsets, int G, int slots,
                    int k, int64_t H, int Cb, int cols, int Rb, uint8_t *__restrict__ Q, float *__restrict__ S) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    DispatchSmem &sm = *reinterpret_cast<DispatchSmem *>(smem_raw);
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int chunk = static_cast<int>(blockIdx.x) / Rb, lb = static_cast<int>(blockIdx.x) - chunk * Rb;
    if (static_cast<int64_t>(lb) * 128 >= __ldg(offsets + G)) return;  // past the last expert's rows
    const int bc0 = chunk * cols;
    dispatch_rows<WEIGHTS>(X, weights, slot_of_row, slots, k, H, static_cast<int64_t>(lb) * 128, 128, bc0,
                           min(bc0 + cols, Cb), Q, S + static_cast<int64_t>(lb) * Cb, sm);
}

// Masked layout: CTA (chunk, g, y) takes the slab's row blocks y, y + Ry, ... that hold
// tokens; rows past the count are neither read nor written.
__global__ void __launch_bounds__(kRowThreads, 4)
    dispatch_masked_kernel(const uint16_t *__restrict__ X, const int32_t *__restrict__ slot_of_row,
                           const int32_t *__restrict__ masked_m, int slots, int k, int64_t H, int Cb, int cols, int G,
                           int m_max, int Rb, int Ry, uint8_t *__restrict__ Q, float *__restrict__ S) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    DispatchSmem &sm = *reinterpret_cast<DispatchSmem *>(smem_raw);
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int chunk = static_cast<int>(blockIdx.x) / (G * Ry), gy = static_cast<int>(blockIdx.x) - chunk * (G * Ry);
    const int g = gy / Ry, y = gy - g * Ry;
    const int rows = min(max(__ldg(masked_m + g), 0), m_max);
    const int bc0 = chunk * cols;
    for (int lb = y, blocks = (rows >> 7) + ((rows & 127) != 0); lb < blocks; lb += Ry)
        dispatch_rows<false>(X, nullptr, slot_of_row, slots, k, H, static_cast<int64_t>(g) * m_max + lb * 128,
                             min(rows - lb * 128, 128), bc0, min(bc0 + cols, Cb), Q,
                             S + (static_cast<int64_t>(g) * Rb + lb) * Cb, sm);
}

// One CTA per token and 1024 columns, eight columns a thread; the rows of up to four slots
// are in flight at a time.  Bound by memory: 32768 slots x 7168 take 84 us, 6.2 TB/s; 16384
// slots x 4096 with k = 2 40 us, 5.1 TB/s (two pieces a thread: 39).
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
// dout comes from the cache.  Bound by memory: 16382 slots x 4096 take 34 us in a graph, 201
// MB, 5.9 TB/s.
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

// Column blocks per CTA: runs as long as possible (the token lookup and the first, uncovered
// gather are paid once a run) that still give the SMs about kDispatchWaves CTAs for each of
// their four places.
constexpr int64_t kDispatchWaves = 2;
static int dispatch_cols(int64_t row_ctas, int64_t Cb, int num_sms) {
    const int64_t want = (kDispatchWaves * 4 * num_sms + row_ctas - 1) / row_ctas;  // runs per row block
    const int64_t runs = want < 1 ? 1 : (want > Cb ? Cb : want);
    return static_cast<int>((Cb + runs - 1) / runs);
}

template <bool WEIGHTS>
static dg_status_t launch_dispatch_impl(const void *X, const float *weights, const int32_t *slot_of_row,
                                        const int32_t *offsets, int64_t slots, int k, int64_t H, int64_t rows, int G,
                                        uint8_t *Q, float *S, const DeviceInfo &dev, cudaStream_t stream) {
    static thread_local int configured_device = -1;
    const dg_status_t st = allow_smem(dispatch_kernel<WEIGHTS>, sizeof(DispatchSmem), configured_device);
    if (st != DG_OK) return st;
    const int64_t Cb = (H + 127) / 128, Rb = rows / 128;
    const int cols = dispatch_cols(Rb, Cb, dev.num_sms);
    const int64_t n = (Cb + cols - 1) / cols * Rb;
    if (n > 0x7FFFFFFFLL) return DG_ERR_SHAPE;
    return launch_pdl(dispatch_kernel<WEIGHTS>, static_cast<int>(n), kRowThreads, sizeof(DispatchSmem), stream,
                      static_cast<const uint16_t *>(X), weights, slot_of_row, offsets, G, static_cast<int>(slots), k, H,
                      static_cast<int>(Cb), cols, static_cast<int>(Rb), Q, S);
}

dg_status_t launch_dispatch_quantize(const void *X, const float *weights, const int32_t *slot_of_row,
                                     const int32_t *offsets, int64_t slots, int k, int64_t H, int64_t rows, int G,
                                     uint8_t *Q, float *S, const DeviceInfo &dev, cudaStream_t stream) {
    return weights ? launch_dispatch_impl<true>(X, weights, slot_of_row, offsets, slots, k, H, rows, G, Q, S, dev, stream)
                   : launch_dispatch_impl<false>(X, weights, slot_of_row, offsets, slots, k, H, rows, G, Q, S, dev,
                                                 stream);
}

// Row blocks of a slab taken by different CTAs, as in the masked quantizer.
constexpr int64_t kDispatchMaskedRowCtas = 16;

dg_status_t launch_dispatch_quantize_masked(const void *X, const int32_t *slot_of_row, const int32_t *masked_m,
                                            int64_t slots, int k, int64_t H, int G, int64_t m_max, uint8_t *Q,
                                            float *S, const DeviceInfo &dev, cudaStream_t stream) {
    static thread_local int configured_device = -1;
    const dg_status_t st = allow_smem(dispatch_masked_kernel, sizeof(DispatchSmem), configured_device);
    if (st != DG_OK) return st;
    const int64_t Rb = (m_max + 127) / 128, Cb = (H + 127) / 128;
    const int64_t Ry = Rb < kDispatchMaskedRowCtas ? Rb : kDispatchMaskedRowCtas;
    const int cols = dispatch_cols(G * Ry, Cb, dev.num_sms);
    const int64_t n = (Cb + cols - 1) / cols * G * Ry;
    if (n > 0x7FFFFFFFLL) return DG_ERR_SHAPE;
    return launch_pdl(dispatch_masked_kernel, static_cast<int>(n), kRowThreads, sizeof(DispatchSmem), stream,
                      static_cast<const uint16_t *>(X), slot_of_row, masked_m, static_cast<int>(slots), k, H,
                      static_cast<int>(Cb), cols, G, static_cast<int>(m_max), static_cast<int>(Rb),
                      static_cast<int>(Ry), Q, S);
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

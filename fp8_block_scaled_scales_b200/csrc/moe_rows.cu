// Rows between tokens and experts: tokens gathered by expert and quantized in one call, and
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
    int groups[4];  // per 32 rows: groups of 16 rows, counted from row 0, up to the last with a token
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
        const uint32_t used = __ballot_sync(0xFFFFFFFFu, ok);
        if ((tid & 31) == 0) sm.groups[tid >> 5] = used ? (tid + 31 - __clz(used)) / 16 + 1 : 0;
    }
    infinite = __syncthreads_or(infinite);  // some row's weight is
    const int groups = max(max(sm.groups[0], sm.groups[1]), max(sm.groups[2], sm.groups[3]));
    uint8_t *const q0 = Q + (row0 + sub) * H + lane_col;
    const int64_t step = 16 * H;

    // ALL: every group of rows has a token.  Otherwise the groups past the last one are
    // neither read nor converted: a decode step's blocks are mostly empty (64 tokens x 8 in
    // 64 slabs, 7168 columns: 19 us without the distinction, 13 with it; contiguous 22 and 16).
    auto walk = [&](auto all) {
        constexpr bool kAll = decltype(all)::value;
        // a row without a token: its pieces stay zero
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (sm.tok[sub + 16 * i] < 0) sm.piece[i][tid] = make_uint4(0, 0, 0, 0);

        auto ask = [&](int bc) {
            const int64_t col = static_cast<int64_t>(bc) * 128 + lane_col;
            if (col < H) {  // H % 16 == 0: an 8-column piece is whole or absent
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (!kAll && i >= groups) break;
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
        uint8_t *qp = q0 + static_cast<int64_t>(bc0) * 128;
        for (int bc = bc0; bc < bc1; ++bc, qp += 128) {
            const bool col_ok = static_cast<int64_t>(bc) * 128 + lane_col < H;
            asm volatile("cp.async.wait_all;" ::: "memory");
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = kAll || i < groups ? sm.piece[i][tid] : make_uint4(0, 0, 0, 0);
            if (bc + 1 < bc1) ask(bc + 1);
            uint32_t m;
            if (WEIGHTS) {
                // the largest |fl32(w x)| of a row's piece is that of its largest |x|
                float f = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    if (!kAll && i >= groups) break;
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
                for (int i = 1; i < 8; ++i) {
                    if (!kAll && i >= groups) break;
                    m2 = __vmaxu2(m2, amax_pair8(v[i]));
                }
                m = amax_bits_of(m2) << 16;  // the maximum's FP32 bits
            }
            m = cta_max<kRowThreads / 32>(m, sm.red[bc & 1]);
            const FastScale bs = fast_scale(__uint_as_float(m));
            if (tid == 0) S[bc] = bs.s;
            const uint32_t none = isnan(bs.s) ? 0x7F7F7F7Fu : 0u;  // four codes of a row without a token
            auto convert = [&](auto fast) {
                constexpr bool kFast = decltype(fast)::value;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint2 q = make_uint2(none, none);
                    if (kAll || i < groups) {
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
    };
    if (groups == 8)
        walk(std::true_type{});
    else
        walk(std::false_type{});
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

// The gather token by token, for tokens of several slots: a token's columns are read and
// unpacked once and converted k times, where the form above reads them from L2 once a slot.
// The scales must be known first, so it takes three launches:
//   tops:   the largest magnitude of every token and column block (T x H read once), and no
//           row for any slot yet;
//   scales: per row block the maximum of its tokens' tops, the scale; rows without a token
//           are written; each other row goes to the head of its slot's list (one row, unless
//           slot_of_row names the slot again);
//   rows:   a warp per token and 1024 columns writes the token's rows, 512 bytes at a time.
// Codes and scales are those of the form above.  HBM bounds it: 32768 slots x 7168, k = 8,
// 77 us against 88 above, 11 of them for the first launch and about 8 for the second; 131072
// slots 256 us against 362, 1.44 GB, 5.6 TB/s (without the conversions 256).  One segment a
// warp 82 and 277 us, four 80 and 267; persistent warps that looked two items ahead 81 and 268.
constexpr int kTokCols = 512;  // a segment: columns of a warp, 16 a lane
constexpr int kTokRun = 2;     // segments of a warp in the last launch, the second one's loads under the first
constexpr int kTokWarps = kRowThreads / 32;
constexpr int kTopsAhead = 8;  // column blocks of a scales CTA: one 16-byte load of tops

struct TokenGather {
    const uint16_t *X;
    const float *weights;
    const int32_t *slot_of_row, *offsets;
    int G, k;
    int64_t T, H;
    int segs, parts;  // 512-column segments of a token, and its warps in the last launch
    int Cb, Cb8;           // 128-column blocks, and that rounded up to 8
    int32_t *head;      // [T][k] first row of a slot, -1: none
    int32_t *next;      // [rows] the slot's next row
    int32_t *repeated;  // whether a slot has one
    uint16_t *tops;     // [T][Cb8] BF16 magnitude bits; with weights bit 15: a zero among them
    uint8_t *Q;
    float *S;
};

template <bool WEIGHTS>
__global__ void __launch_bounds__(kRowThreads) dispatch_tops_kernel(const TokenGather p) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
    for (int64_t i = first; i < p.T * p.k; i += static_cast<int64_t>(gridDim.x) * kRowThreads) p.head[i] = -1;
    if (first == 0) *p.repeated = 0;
    const int64_t w = first >> 5, t = w / p.segs;
    if (t >= p.T) return;
    const int lane = lane_id(), col = static_cast<int>(w - t * p.segs) * kTokCols + lane * 16;
    uint32_t m = 0;
    bool zero = false;
    if (col < p.H) {
        const uint4 *x = reinterpret_cast<const uint4 *>(p.X + t * p.H + col);
        const uint4 a = __ldg(x), b = __ldg(x + 1);
        m = amax_bits_of(__vmaxu2(amax_pair8(a), amax_pair8(b)));
        if (WEIGHTS) zero = has_zero8(a) || has_zero8(b);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (WEIGHTS) {
        const uint32_t zeros = __ballot_sync(0xFFFFFFFFu, zero);
        if ((zeros >> (lane & ~7)) & 0xFFu) m |= 0x8000u;
    }
    if ((lane & 7) == 0 && col < p.H) p.tops[t * p.Cb8 + col / 128] = static_cast<uint16_t>(m);
}

template <bool WEIGHTS>
__global__ void __launch_bounds__(128) dispatch_scales_kernel(const TokenGather p) {
    __shared__ uint32_t red[4][kTopsAhead];
    __shared__ uint32_t empty[kTopsAhead];  // the code of a row without a token, four times
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int chunks = p.Cb8 / kTopsAhead;
    const int lb = static_cast<int>(blockIdx.x) / chunks, chunk = static_cast<int>(blockIdx.x) - lb * chunks;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int row = lb * 128 + tid;
    if (lb * 128 >= __ldg(p.offsets + p.G)) return;
    const int slot = __ldg(p.slot_of_row + row);
    const bool ok = slot >= 0 && slot < p.T * p.k;
    uint4 v = make_uint4(0, 0, 0, 0);
    float w = 0.0f;
    if (ok) {
        v = *reinterpret_cast<const uint4 *>(p.tops + static_cast<int64_t>(slot / p.k) * p.Cb8 + chunk * kTopsAhead);
        if (WEIGHTS) w = __ldg(p.weights + slot);
        if (chunk == 0) {
            const int before = atomicExch(p.head + slot, row);  // a list's order changes nothing
            p.next[row] = before;
            if (before >= 0) *p.repeated = 1;
        }
    }
    const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < kTopsAhead; ++i) {
        const uint32_t bits = (i & 1) ? words[i / 2] & 0xFFFF0000u : words[i / 2] << 16;
        uint32_t m = bits;
        if (WEIGHTS) {
            float f = fabsf(__uint_as_float(bits & 0x7FFFFFFFu) * w);
            if (isinf(w) && (bits >> 31)) f = __int_as_float(0x7FFFFFFF);  // infinity times a zero
            m = __float_as_uint(f);
        }
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (lane == 0) red[warp][i] = m;
    }
    __syncthreads();
    const int bc = chunk * kTopsAhead + tid;
    if (tid < kTopsAhead && bc < p.Cb) {
        const float s = fast_scale(__uint_as_float(max(max(red[0][tid], red[1][tid]), max(red[2][tid], red[3][tid])))).s;
        p.S[static_cast<int64_t>(lb) * p.Cb + bc] = s;
        empty[tid] = isnan(s) ? 0x7F7F7F7Fu : 0u;
    }
    __syncthreads();
    for (uint32_t rest = __ballot_sync(0xFFFFFFFFu, !ok); rest; rest &= rest - 1) {
        const int r = __ffs(rest) - 1;
        uint8_t *q = p.Q + static_cast<int64_t>(row - lane + r) * p.H;
#pragma unroll
        for (int i = 0; i < kTopsAhead / 4; ++i) {
            const int64_t col = static_cast<int64_t>(chunk) * kTopsAhead * 128 + i * 512 + lane * 16;
            if (col < p.H) {
                const uint32_t c = empty[i * 4 + lane / 8];
                *reinterpret_cast<uint4 *>(q + col) = make_uint4(c, c, c, c);
            }
        }
    }
}

template <bool WEIGHTS>
__global__ void __launch_bounds__(kRowThreads, 3) dispatch_rows_kernel(const TokenGather p) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x) >> 5, t = w / p.parts;
    if (t >= p.T) return;
    const int seg0 = static_cast<int>(w - t * p.parts) * kTokRun, seg1 = min(seg0 + kTokRun, p.segs);
    const int lane = lane_id();
    const uint16_t *x = p.X + t * p.H;
    auto load = [&](int seg, uint4 (&v)[2]) {
        const int64_t col = static_cast<int64_t>(seg) * kTokCols + lane * 16;
        v[0] = v[1] = make_uint4(0, 0, 0, 0);
        if (seg < seg1 && col < p.H) {
            const uint4 *src = reinterpret_cast<const uint4 *>(x + col);
            v[0] = __ldg(src), v[1] = __ldg(src + 1);
        }
    };
    // Eight slots at a time; lane 4 i + b looks up slot i's row and its scale of column block b.
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        const int j = j0 + (lane >> 2);
        const int64_t slot = t * p.k + j;
        int row = j < p.k ? __ldg(p.head + slot) : -1;
        const float wgt = WEIGHTS && row >= 0 ? __ldg(p.weights + slot) : 0.0f;
        const bool again = __ldg(p.repeated) != 0;
        do {
            uint4 v[2];
            load(seg0, v);
            const float *scales = p.S + static_cast<int64_t>(row >> 7) * p.Cb;
            auto scale = [&](int seg) {
                const int bc = seg * 4 + (lane & 3);
                return row >= 0 && seg < seg1 && bc < p.Cb ? __ldg(scales + bc) : 1.0f;
            };
            float s = scale(seg0);
            int r[8];
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                r[i] = __shfl_sync(0xFFFFFFFFu, row, 4 * i);
                if (WEIGHTS) f[i] = __shfl_sync(0xFFFFFFFFu, wgt, 4 * i);
            }
            for (int seg = seg0; seg < seg1; ++seg) {
                float2 n[2][4];
                bf16x8_to_f32(v[0], n[0]), bf16x8_to_f32(v[1], n[1]);
                FastScale mine;
                mine.s = s;
                split_reciprocal(mine);
                const bool fast = s >= 0x1p-90f / 448.0f && s <= 0x1p100f / 448.0f;  // scale_is_fast of its maximum
                load(seg + 1, v);
                s = scale(seg + 1);
                const int64_t col = static_cast<int64_t>(seg) * kTokCols + lane * 16;
                uint8_t *q = p.Q + col;
                auto convert = [&](auto fast) {
                    constexpr bool kFast = decltype(fast)::value;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (r[i] < 0) continue;  // the same for the whole warp
                        FastScale bs;
                        if (kFast) {
                            bs.r = __shfl_sync(0xFFFFFFFFu, mine.r, 4 * i + lane / 8);
                            bs.r_lo = __shfl_sync(0xFFFFFFFFu, mine.r_lo, 4 * i + lane / 8);
                        } else {
                            bs.s = __shfl_sync(0xFFFFFFFFu, mine.s, 4 * i + lane / 8);
                        }
                        uint2 c[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (WEIGHTS) {
                                float2 y[4];
#pragma unroll
                                for (int d = 0; d < 4; ++d) y[d] = __fmul2_rn(n[h][d], make_float2(f[i], f[i]));
                                c[h] = quantize8_f32<kFast>(y, bs);
                            } else {
                                c[h] = quantize8_f32<kFast>(n[h], bs);
                            }
                        }
                        if (col < p.H)
                            *reinterpret_cast<uint4 *>(q + static_cast<int64_t>(r[i]) * p.H) =
                                make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
                    }
                };
                if (__all_sync(0xFFFFFFFFu, fast))
                    convert(std::true_type{});
                else
                    convert(std::false_type{});
            }
            if (!again) break;
            row = row >= 0 ? __ldg(p.next + row) : -1;
        } while (__any_sync(0xFFFFFFFFu, row >= 0));
    }
}

// One CTA per token and 1024 columns, eight columns a thread; the rows of up to four slots
// are in flight at a time.  Bound by memory: in a graph 32768 slots x 7168 take 79 us, 6.7
// TB/s; 16384 slots x 4096 with k = 2 37 us, 5.4 TB/s.  Sixteen CTAs an SM: with the 34 registers
// that they would otherwise take, 84 and 40 us.  Streaming loads and stores, two pieces a
// thread: within 2 %.
constexpr int kCombineThreads = 128;
constexpr int kCombineCols = kCombineThreads * 8;

template <bool WEIGHTS>
__global__ void __launch_bounds__(kCombineThreads, 16)
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
// their four places; masked twice as many, since the CTAs of a slab's empty row blocks leave
// at once (2048 tokens x 2 in 8 slabs of 2048 rows: 14.8 us with two waves, 12.3 with four; 256
// x 8 in 64 slabs of 1024: 37 and 27; 64 x 8 in 64 slabs of 128: 13.2 and 14.4).
constexpr int64_t kDispatchWaves = 2;
constexpr int64_t kDispatchMaskedWaves = 4;

static int dispatch_cols(int64_t row_ctas, int64_t Cb, int num_sms, int64_t waves) {
    const int64_t want = (waves * 4 * num_sms + row_ctas - 1) / row_ctas;  // runs per row block
    const int64_t runs = want < 1 ? 1 : (want > Cb ? Cb : want);
    return static_cast<int>((Cb + runs - 1) / runs);
}

// Bytes of the token form's workspace, 0 where the other form is used: few slots per token
// (it reads the tokens twice more, the other one k times from L2), or so little work that its
// two further launches cost more than they save.  Measured, this form against the other: k = 8,
// H = 7168: 16384 tokens 256 and 362 us, 4096 77 and 88, 1024 32 and 36, 64 29 and 23; H = 2048:
// 4096 tokens 28 and 28, 1024 19 and 13.  4096 tokens of 7168, k = 4: 62 and 54.  The bound on the
// codes lies just above the tie, and gives away the 4 us of 1024 tokens of 7168, which have fewer;
// k of 5 to 7 and weights were not measured on both sides.
constexpr int kTokenFormSlots = 8;
constexpr int64_t kTokenFormWork = (1LL << 26) + 1;  // codes
int64_t dispatch_workspace(int64_t T, int k, int64_t H, int64_t rows) {
    const int64_t segs = (H + kTokCols - 1) / kTokCols, Cb8 = (H + 1023) / 1024 * 8;
    if (k < kTokenFormSlots || T * k * H < kTokenFormWork) return 0;
    if (T * segs > 0x7FFFFFFFLL || rows / 128 * Cb8 > 0x7FFFFFFFLL) return 0;  // grids
    return (T * k * 4 + 15) / 16 * 16 + rows * 4 + 16 + T * Cb8 * 2;
}

template <bool WEIGHTS>
static dg_status_t launch_token_form(const TokenGather &p, int64_t rows, cudaStream_t stream) {
    const int n = static_cast<int>((p.T * p.segs + kTokWarps - 1) / kTokWarps);
    dg_status_t st = launch_pdl(dispatch_tops_kernel<WEIGHTS>, n, kRowThreads, 0, stream, p);
    if (st != DG_OK) return st;
    st = launch_pdl(dispatch_scales_kernel<WEIGHTS>, static_cast<int>(rows / 128 * (p.Cb8 / kTopsAhead)), 128, 0, stream, p);
    if (st != DG_OK) return st;
    const int m = static_cast<int>((p.T * p.parts + kTokWarps - 1) / kTokWarps);
    return launch_pdl(dispatch_rows_kernel<WEIGHTS>, m, kRowThreads, 0, stream, p);
}

template <bool WEIGHTS>
static dg_status_t launch_dispatch_impl(const void *X, const float *weights, const int32_t *slot_of_row,
                                        const int32_t *offsets, int64_t slots, int k, int64_t H, int64_t rows, int G,
                                        uint8_t *Q, float *S, const DeviceInfo &dev, cudaStream_t stream) {
    static thread_local int configured_device = -1;
    const dg_status_t st = allow_smem(dispatch_kernel<WEIGHTS>, sizeof(DispatchSmem), configured_device);
    if (st != DG_OK) return st;
    const int64_t Cb = (H + 127) / 128, Rb = rows / 128;
    const int cols = dispatch_cols(Rb, Cb, dev.num_sms, kDispatchWaves);
    const int64_t n = (Cb + cols - 1) / cols * Rb;
    if (n > 0x7FFFFFFFLL) return DG_ERR_SHAPE;
    return launch_pdl(dispatch_kernel<WEIGHTS>, static_cast<int>(n), kRowThreads, sizeof(DispatchSmem), stream,
                      static_cast<const uint16_t *>(X), weights, slot_of_row, offsets, G, static_cast<int>(slots), k, H,
                      static_cast<int>(Cb), cols, static_cast<int>(Rb), Q, S);
}

dg_status_t launch_dispatch_quantize(const void *X, const float *weights, const int32_t *slot_of_row,
                                     const int32_t *offsets, int64_t slots, int k, int64_t H, int64_t rows, int G,
                                     uint8_t *Q, float *S, void *workspace, const DeviceInfo &dev, cudaStream_t stream) {
    const int64_t T = slots / k;
    if (dispatch_workspace(T, k, H, rows) > 0) {
        const int64_t Cb8 = (H + 1023) / 1024 * 8;
        const int segs = static_cast<int>((H + kTokCols - 1) / kTokCols);
        int32_t *head = static_cast<int32_t *>(workspace), *next = head + (slots + 3) / 4 * 4;
        const TokenGather p = {static_cast<const uint16_t *>(X), weights, slot_of_row, offsets, G, k, T, H,
                               segs, (segs + kTokRun - 1) / kTokRun, static_cast<int>((H + 127) / 128),
                               static_cast<int>(Cb8), head, next, next + rows, reinterpret_cast<uint16_t *>(next + rows + 4), Q, S};
        return weights ? launch_token_form<true>(p, rows, stream)
                       : launch_token_form<false>(p, rows, stream);
    }
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
    const int cols = dispatch_cols(G * Ry, Cb, dev.num_sms, kDispatchMaskedWaves);
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

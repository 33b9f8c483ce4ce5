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
// Every step rounds about once in FP32, but the exponential's argument is one rounded product:
// exp(-g) may be off by 2 + 1.2 |g| units of 2^-23, and sigma with it by that times 1 - sigma, so
// for negative gates in full.  A code differs from the exact value's only next to a rounding
// boundary, and each wrong ulp would show there for a whole block through its scale.
#include <cuda_bf16.h>

#include <type_traits>

#include "dg_device.cuh"
#include "quant_f32.cuh"
#include "train_internal.h"

namespace dg {

constexpr int kGluThreads = 512;      // forward: 16 lanes a row, 32 rows at a time, 4 times
constexpr int kGluPer = 4;
constexpr int kGluBackThreads = 512;   // backward: 32 rows at a time, four times
constexpr int kGluBackPer = 4;

// d = 1 + exp(-x) and an approximation r of -1/d, one exponential and one reciprocal
// instruction a value.  x below -88.5 is taken as that: exp(-x) is still finite there and r
// flushed to 0, so no infinity meets a zero.  (Putting the rounding of exp2's argument
// back into the result cost 4 % and left the codes' error where it was.)
__device__ __forceinline__ void one_plus_exp(float2 x, float2 &d, float2 &r) {
    const float2 t = __fmul2_rn(make_float2(fmaxf(x.x, -88.5f), fmaxf(x.y, -88.5f)),
                                make_float2(-1.44269504f, -1.44269504f));  // -log2 e
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    d = __fadd2_rn(e, make_float2(1.0f, 1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(-d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(-d.y));
}

// -n / d from r = -1/d: the product corrected by its remainder (Markstein, as in
// quant_f32.cuh).  With the approximate reciprocal alone, and a / s as a product with one, the kernels
// were a tenth faster and a third of the inputs tried had half as much error again in the
// codes as a plain FP32 evaluation; as it stands they have the same on the inputs tried.  An
// infinite n gives NaN.
__device__ __forceinline__ float2 negated_quotient(float2 n, float2 d, float2 r) {
    const float2 z = __fmul2_rn(n, r);
    return __ffma2_rn(__ffma2_rn(z, d, n), r, z);
}

// Two rows of h, 128 columns of the gate and of the up half each, as four 1 x 128 blocks
// (16 lanes a row, 8 values each); the maxima of gate and up are found together, packed in one
// word.  All lanes of the warp call it; ok[i]: row i exists.  q + in_q, s + in_s: the first
// row's gate codes and scale; the up half lies q_up codes and s_up scales on, the second
// row q_row codes and 32 scales on.
__device__ __forceinline__ void checkpoint_rows(const uint4 (&vg)[2], const uint4 (&vu)[2], const bool (&ok)[2],
                                                uint8_t *q, uint32_t in_q, int64_t q_up, int64_t q_row, float *s,
                                                int in_s, int64_t s_up) {
    uint32_t pk[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        pk[i] = amax_bits_of(amax_pair8(vg[i])) | amax_bits_of(amax_pair8(vu[i])) << 16;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) pk[i] = __vmaxu2(pk[i], __shfl_xor_sync(0xFFFFFFFFu, pk[i], o));
    }
    float amax[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        amax[i][0] = __uint_as_float(pk[i] << 16);
        amax[i][1] = __uint_as_float(pk[i] & 0xFFFF0000u);
    }
    auto write = [&](auto fast) {
        constexpr bool kFast = decltype(fast)::value;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const FastScale g = scale_of<kFast>(amax[i][0]), u = scale_of<kFast>(amax[i][1]);
            const uint2 qg = quantize8_bf16<kFast>(vg[i], g), qu = quantize8_bf16<kFast>(vu[i], u);
            if (ok[i]) {
                *reinterpret_cast<uint2 *>(q + i * q_row + in_q) = qg;
                *reinterpret_cast<uint2 *>(q + i * q_row + q_up + in_q) = qu;
                if ((threadIdx.x & 15u) == 0) {
                    s[in_s + i * 32] = g.s;
                    s[in_s + i * 32 + s_up] = u.s;
                }
            }
        }
    };
    if (__builtin_expect(scale_is_fast(amax[0][0]) && scale_is_fast(amax[0][1]) && scale_is_fast(amax[1][0]) &&
                             scale_is_fast(amax[1][1]),
                         1))
        write(std::true_type{});
    else
        write(std::false_type{});
}

// 16- and 8-byte copies to shared memory that the thread waits for later.
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The row blocks of a layout: G slabs of M rows (dense and contiguous: one), of which the
// first ones hold something: all M, or up to the last expert's end, or the slab's count.
struct GluRows {
    const int32_t *offsets, *masked_m;  // at most one
    int G, M;                           // G * M < 2^31
    int Rb, Fb;                         // 128-row blocks of a slab, 128-column blocks
};

// A CTA's walk over the blocks (row block rb of all slabs, column block bc), every gridDim-th
// one, without a division per step.
struct GluWalk {
    int rb, bc, step_rb, step_bc, end_rb;
    int used;  // dense and contiguous: rows that hold something

    __device__ __forceinline__ void start(const GluRows &l) {
        const int grid = static_cast<int>(gridDim.x), first = static_cast<int>(blockIdx.x);
        rb = first / l.Fb;
        bc = first - rb * l.Fb;
        step_rb = grid / l.Fb;
        step_bc = grid - step_rb * l.Fb;
        used = l.offsets ? min(max(__ldg(l.offsets + l.G), 0), l.M) : l.M;
        end_rb = l.masked_m ? l.G * l.Rb : (used >> 7) + ((used & 127) != 0);
    }
    __device__ __forceinline__ void advance(const GluRows &l) {
        rb += step_rb;
        bc += step_bc;
        if (bc >= l.Fb) {
            bc -= l.Fb;
            ++rb;
        }
    }
    // First row of block rb in the whole matrix, and its rows that hold something (0: none).
    __device__ __forceinline__ int rows(const GluRows &l, int &row0) const {
        if (!l.masked_m) {
            row0 = rb * 128;
            return min(used - row0, 128);
        }
        const int g = rb / l.Rb, at = (rb - g * l.Rb) * 128;
        row0 = g * l.M + at;
        return min(max(min(__ldg(l.masked_m + g), l.M) - at, 0), 128);
    }
    // To the next block, this one included, that holds something; false: there is none.
    __device__ __forceinline__ bool find(const GluRows &l, int &row0, int &n) {
        for (; rb < end_rb; advance(l)) {
            n = rows(l, row0);
            if (n > 0) return true;
        }
        return false;
    }
};

// Forward, persistent: two CTAs per SM walk over the blocks.  A thread keeps its 16-byte
// pieces of a block in shared memory and asks for the same pieces of the next block as soon
// as it has read them, so loads run under the arithmetic, the block maximum and the stores
// without costing registers.  16384 x 4096 in a graph, without checkpoint: 57 us, 336 MB, 5.8
// TB/s; with checkpoint 99 us, 470 MB, 4.8 TB/s, bound by instruction issue (74 % of the slots;
// the conversions of three values for each output).  A CTA per block that loaded into registers
// took 124 us, and 386 us while it held all four rows at once and spilled.
struct GluSmem {
    uint4 g[kGluPer][kGluThreads];
    uint4 u[kGluPer][kGluThreads];
};

// FEW (the masked layout): a block's rows past its last one are left out in steps of 32, since a
// decode step's slabs hold a few.  In a graph of ten calls on the same input (which stays in L2): 64
// slabs of 8 rows, F = 2048, 14.7 us without, 9.8 with it; 8 full slabs of 512, F = 4096, 16.1 and
// 17.2, as the steps keep the rows' arithmetic apart.  (Both ways in one kernel spilled.)
template <bool CKPT, bool FEW>
__global__ void __launch_bounds__(kGluThreads, 2)
    swiglu_kernel(const uint16_t *__restrict__ Hin, const GluRows layout, uint8_t *__restrict__ Q,
                  float *__restrict__ S, uint8_t *__restrict__ H8, float *__restrict__ sH) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    GluSmem &st = *reinterpret_cast<GluSmem *>(smem_raw);
    __shared__ __align__(16) uint32_t red[2][kGluThreads / 32];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int tid = static_cast<int>(threadIdx.x);
    const int sub = tid >> 4;
    const int64_t F = static_cast<int64_t>(layout.Fb) * 128;
    const int64_t step = 64 * F;  // 32 rows of h
    // this thread's place in a block of h and of Q; the block's own address is the same for all
    const uint32_t in_h = sub * 2 * static_cast<uint32_t>(F) + (tid & 15) * 8;
    const uint32_t in_q = sub * static_cast<uint32_t>(F) + (tid & 15) * 8;

    auto ask = [&](int i, int row0, int rows, int bc) {
        if (sub + 32 * i < rows) {
            const uint16_t *p = Hin + static_cast<int64_t>(row0) * 2 * F + bc * 128 + i * step;
            cp_async16(&st.g[i][tid], p + in_h);
            cp_async16(&st.u[i][tid], p + F + in_h);
        }
    };

    GluWalk walk;
    walk.start(layout);
    int row0 = 0, rows = 0;
    bool have = walk.find(layout, row0, rows);
    if (have) {
#pragma unroll
        for (int i = 0; i < kGluPer; ++i) ask(i, row0, rows, walk.bc);
    }
    int par = 0;
    while (have) {
        const int rb = walk.rb, bc = walk.bc;
        int next_row0 = 0, next_rows = 0;
        walk.advance(layout);
        const bool more = walk.find(layout, next_row0, next_rows);
        if (!more) next_rows = 0;
        float2 a[kGluPer][4];  // negated, as negated_quotient leaves them
        float m = 0.0f;
        cp_async_wait();
#pragma unroll
        for (int i0 = 0; i0 < kGluPer; i0 += 2) {
            uint4 vg[2], vu[2];
            const bool ok[2] = {sub + 32 * i0 < rows, sub + 32 * (i0 + 1) < rows};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                vg[i] = ok[i] ? st.g[i0 + i][tid] : make_uint4(0, 0, 0, 0);
                vu[i] = ok[i] ? st.u[i0 + i][tid] : make_uint4(0, 0, 0, 0);
            }
            if (CKPT)
                checkpoint_rows(vg, vu, ok, H8 + static_cast<int64_t>(row0) * 2 * F + bc * 128 + i0 * step, in_h, F,
                                step, sH + static_cast<int64_t>(bc) * layout.M + row0 + 32 * i0, sub,
                                static_cast<int64_t>(layout.Fb) * layout.M);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!FEW || 32 * (i0 + i) < rows) {
                    float2 g[4], u[4];
                    bf16x8_to_f32(vg[i], g);
                    bf16x8_to_f32(vu[i], u);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float2 d, r;
                        one_plus_exp(g[j], d, r);
                        const float2 x = __fmul2_rn(negated_quotient(g[j], d, r), u[j]);  // -(g / d) u
                        m = amax3(m, x);
                        a[i0 + i][j] = x;
                    }
                }
                ask(i0 + i, next_row0, next_rows, walk.bc);
            }
        }
        uint32_t top = cta_max<kGluThreads / 32>(__float_as_uint(m), red[par]);
        if (__builtin_expect(top > 0x7F800000u, 0)) {
            // A NaN, perhaps an infinite gate's: that counts as the gate itself times u (and keeps the
            // code of a NaN, which is infinity over infinity).  The block is read once more, so that
            // blocks of numbers do without the test, and in a loop, whose code they do not load.
            const uint16_t *p = Hin + static_cast<int64_t>(row0) * 2 * F + bc * 128 + in_h;
            m = 0.0f;
#pragma unroll 1
            for (int r = sub; r < rows; r += 32, p += step) {
                float2 g[4], u[4];
                bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(p)), g);
                bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(p + F)), u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 d, n;
                    one_plus_exp(g[j], d, n);
                    n = negated_quotient(g[j], d, n);
                    n = make_float2(g[j].x == INFINITY ? g[j].x : n.x, g[j].y == INFINITY ? g[j].y : n.y);
                    m = amax3(m, __fmul2_rn(n, u[j]));
                }
            }
            __syncthreads();  // red[par] has been read
            top = cta_max<kGluThreads / 32>(__float_as_uint(m), red[par]);
        }
        const FastScale bs = fast_scale(__uint_as_float(top));
        if (tid == 0) S[static_cast<int64_t>(rb) * layout.Fb + bc] = bs.s;
        const FastScale nb = bs.negated();
        uint8_t *q = Q + static_cast<int64_t>(row0) * F + bc * 128;
        auto convert = [&](auto fast) {
#pragma unroll
            for (int i = 0; i < kGluPer; ++i) {
                if (FEW && 32 * i >= rows) break;
                const uint2 c = quantize8_f32<decltype(fast)::value>(a[i], nb);
                if (sub + 32 * i < rows) *reinterpret_cast<uint2 *>(q + i * (step >> 1) + in_q) = c;
            }
        };
        if (__builtin_expect(bs.fast, 1))
            convert(std::true_type{});
        else
            convert(std::false_type{});
        have = more;
        row0 = next_row0;
        rows = next_rows;
        par ^= 1;
    }
}

// Backward, persistent, one CTA per SM: a block's [dg | du] in FP32 is half the register
// file.  16384 x 4096: 87 us in a graph, 403 MB, 4.6 TB/s, issue-bound with 16 warps (a CTA
// per block 168 us; 1024 threads of two rows each 112 against 98 then).  Pieces of the next
// block are asked for as in the forward kernel; the row scales, which other threads copy,
// alternate between two buffers.
struct GluBackSmem {
    uint4 da[kGluBackPer][kGluBackThreads];
    uint2 cg[kGluBackPer][kGluBackThreads];
    uint2 cu[kGluBackPer][kGluBackThreads];
    float scale[2][2][128];  // [buffer][gate, up][row]
};

__global__ void __launch_bounds__(kGluBackThreads, 1)
    swiglu_backward_kernel(const uint8_t *__restrict__ H8, const float *__restrict__ sH,
                           const uint16_t *__restrict__ dA, const GluRows layout, uint8_t *__restrict__ Q,
                           float *__restrict__ S) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    GluBackSmem &st = *reinterpret_cast<GluBackSmem *>(smem_raw);
    __shared__ uint32_t red[2][2][kGluBackThreads / 32];
    grid_dep_launch_dependents();
    grid_dep_wait();
    constexpr int kRows = kGluBackThreads / 16;  // rows at a time
    const int tid = static_cast<int>(threadIdx.x);
    const int sub = tid >> 4, lane_col = (tid & 15) * 8;
    const int64_t F = static_cast<int64_t>(layout.Fb) * 128;

    const uint32_t in_h = sub * 2 * static_cast<uint32_t>(F) + lane_col;  // this thread's place in a block
    const uint32_t in_a = sub * static_cast<uint32_t>(F) + lane_col;

    // one row piece and, with the first, this thread's share of the block's scales
    auto ask = [&](int i, int row0, int rows, int bc, int buffer) {
        if (sub + kRows * i < rows) {
            const int64_t row = row0 + kRows * i;
            const uint8_t *p = H8 + row * 2 * F + bc * 128;
            cp_async8(&st.cg[i][tid], p + in_h);
            cp_async8(&st.cu[i][tid], p + F + in_h);
            cp_async16(&st.da[i][tid], dA + row * F + bc * 128 + in_a);
        }
        if (i == 0 && tid < 256) {
            const int r = tid & 127, half = tid >> 7;
            if (r < rows)
                cp_async4(&st.scale[buffer][half][r],
                          sH + static_cast<int64_t>(half * layout.Fb + bc) * layout.M + row0 + r);
        }
    };

    GluWalk walk;
    walk.start(layout);
    int row0 = 0, rows = 0;
    bool have = walk.find(layout, row0, rows);
    if (have) {
#pragma unroll
        for (int i = 0; i < kGluBackPer; ++i) ask(i, row0, rows, walk.bc, 0);
    }
    int par = 0;
    while (have) {
        const int rb = walk.rb, bc = walk.bc;
        int next_row0 = 0, next_rows = 0;
        walk.advance(layout);
        const bool more = walk.find(layout, next_row0, next_rows);
        if (!more) next_rows = 0;
        cp_async_wait();
        __syncthreads();  // the scales come from other threads' copies
        float2 dg[kGluBackPer][4], du[kGluBackPer][4];
        float ag = 0.0f, au = 0.0f;
#pragma unroll
        for (int i = 0; i < kGluBackPer; ++i) {
            const int r = sub + kRows * i;
            const bool ok = r < rows;
            const uint2 cg = ok ? st.cg[i][tid] : make_uint2(0, 0), cu = ok ? st.cu[i][tid] : make_uint2(0, 0);
            const uint4 va = ok ? st.da[i][tid] : make_uint4(0, 0, 0, 0);
            const float sg = ok ? st.scale[par][0][r] : 0.0f, su = ok ? st.scale[par][1][r] : 0.0f;
            float2 g[4], u[4], d[4];
            e4m3x4_to_f32(cg.x, g[0], g[1]);
            e4m3x4_to_f32(cg.y, g[2], g[3]);
            e4m3x4_to_f32(cu.x, u[0], u[1]);
            e4m3x4_to_f32(cu.y, u[2], u[3]);
            bf16x8_to_f32(va, d);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 gs = __fmul2_rn(g[j], make_float2(sg, sg)), us = __fmul2_rn(u[j], make_float2(su, su));
                float2 e, r;
                one_plus_exp(gs, e, r);
                const float2 ns = __ffma2_rn(__ffma2_rn(r, e, make_float2(1.0f, 1.0f)), r, r);  // -sigma
                const float2 t = __fmul2_rn(d[j], ns);
                const float2 w = __ffma2_rn(gs, __fadd2_rn(ns, make_float2(1.0f, 1.0f)), make_float2(1.0f, 1.0f));
                du[i][j] = __fmul2_rn(t, gs);  // both negated
                dg[i][j] = __fmul2_rn(__fmul2_rn(t, us), w);
                ag = amax3(ag, dg[i][j]);
                au = amax3(au, du[i][j]);
            }
            ask(i, next_row0, next_rows, walk.bc, par ^ 1);
        }
        uint32_t mg = __float_as_uint(ag), mu = __float_as_uint(au);  // NaN above infinity
        mg = __reduce_max_sync(0xFFFFFFFFu, mg);
        mu = __reduce_max_sync(0xFFFFFFFFu, mu);
        if ((tid & 31) == 0) {
            red[par][0][tid >> 5] = mg;
            red[par][1][tid >> 5] = mu;
        }
        __syncthreads();
        constexpr int kWarps = kGluBackThreads / 32;
        mg = red[par][0][tid & (kWarps - 1)];
        mu = red[par][1][tid & (kWarps - 1)];
        mg = __reduce_max_sync(0xFFFFFFFFu, mg);
        mu = __reduce_max_sync(0xFFFFFFFFu, mu);
        const FastScale bg = fast_scale(__uint_as_float(mg)), bu = fast_scale(__uint_as_float(mu));
        if (tid == 0) {
            float *sp = S + static_cast<int64_t>(rb) * 2 * layout.Fb + bc;
            sp[0] = bg.s;
            sp[layout.Fb] = bu.s;
        }
        const FastScale ng = bg.negated(), nu = bu.negated();
        uint8_t *q = Q + static_cast<int64_t>(row0) * 2 * F + bc * 128;
        auto convert = [&](auto fast) {
            constexpr bool kFast = decltype(fast)::value;
#pragma unroll
            for (int i = 0; i < kGluBackPer; ++i) {
                const uint2 cg = quantize8_f32<kFast>(dg[i], ng), cu = quantize8_f32<kFast>(du[i], nu);
                if (sub + kRows * i < rows) {
                    *reinterpret_cast<uint2 *>(q + i * kRows * 2 * F + in_h) = cg;
                    *reinterpret_cast<uint2 *>(q + i * kRows * 2 * F + F + in_h) = cu;
                }
            }
        };
        if (__builtin_expect(bg.fast && bu.fast, 1))
            convert(std::true_type{});
        else
            convert(std::false_type{});
        have = more;
        row0 = next_row0;
        rows = next_rows;
        par ^= 1;
    }
}
static_assert(kGluBackThreads == 512 || kGluBackThreads == 1024, "the reduction over warps uses 16 or 32 lanes");

template <bool CKPT, bool FEW>
static dg_status_t launch_swiglu_impl(const uint16_t *h, const GluRows &layout, int64_t blocks, uint8_t *Q, float *S,
                                      uint8_t *H8, float *sH, const DeviceInfo &dev, cudaStream_t stream) {
    static thread_local int configured_device = -1;
    const dg_status_t st = allow_smem(swiglu_kernel<CKPT, FEW>, sizeof(GluSmem), configured_device);
    if (st != DG_OK) return st;
    const int grid = static_cast<int>(blocks < 2 * dev.num_sms ? blocks : 2 * dev.num_sms);
    return launch_pdl(swiglu_kernel<CKPT, FEW>, grid, kGluThreads, sizeof(GluSmem), stream, h, layout, Q, S, H8, sH);
}

dg_status_t launch_swiglu(const void *H, const int32_t *offsets, const int32_t *masked_m, int G, int64_t M,
                          int64_t F, uint8_t *Q, float *S, uint8_t *H8, float *sH, const DeviceInfo &dev,
                          cudaStream_t stream) {
    const int64_t Rb = (M + 127) / 128, Fb = F / 128, blocks = (masked_m ? G : 1) * Rb * Fb;
    if (blocks > 0x3FFFFFFFLL) return DG_ERR_SHAPE;
    const GluRows layout = {offsets, masked_m, G, static_cast<int>(M), static_cast<int>(Rb), static_cast<int>(Fb)};
    const uint16_t *h = static_cast<const uint16_t *>(H);
    if (masked_m) return launch_swiglu_impl<false, true>(h, layout, blocks, Q, S, H8, sH, dev, stream);
    return H8 ? launch_swiglu_impl<true, false>(h, layout, blocks, Q, S, H8, sH, dev, stream)
              : launch_swiglu_impl<false, false>(h, layout, blocks, Q, S, H8, sH, dev, stream);
}

dg_status_t launch_swiglu_backward(const uint8_t *H8, const float *sH, const void *dA, const int32_t *offsets,
                                   int G, int64_t M, int64_t F, uint8_t *Q, float *S, const DeviceInfo &dev,
                                   cudaStream_t stream) {
    const int64_t Rb = (M + 127) / 128, Fb = F / 128, blocks = Rb * Fb;
    if (blocks > 0x3FFFFFFFLL) return DG_ERR_SHAPE;
    const GluRows layout = {offsets, nullptr, G, static_cast<int>(M), static_cast<int>(Rb), static_cast<int>(Fb)};
    static thread_local int configured_device = -1;
    const dg_status_t st = allow_smem(swiglu_backward_kernel, sizeof(GluBackSmem), configured_device);
    if (st != DG_OK) return st;
    const int grid = static_cast<int>(blocks < dev.num_sms ? blocks : dev.num_sms);
    return launch_pdl(swiglu_backward_kernel, grid, kGluBackThreads, sizeof(GluBackSmem), stream, H8, sH,
                      static_cast<const uint16_t *>(dA), layout, Q, S);
}

}  // namespace dg

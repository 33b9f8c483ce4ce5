// The norms before and after a block, fused with its gate and the scaled residual, and their
// gradient.
//
// forward:   u = y * rstd_y * post (or y);  r = alpha x + gate * u;  n = r * rstd * weight,
//   rstd = 1 / sqrt(mean r^2 + eps) over a row, rstd_y likewise over y; FP32 throughout, n from
//   r before r is rounded to BF16.  n as BF16, or as E4M3 codes with one scale per row and 128
//   columns (s = fl32(amax / 448) of the FP32 values, 1 if 0).
// backward, with rh = r rstd, yh = y rstd_y:
//   dR = dr + rstd (dn w - rh c1),      c1 = mean(dn w rh)
//   dx = alpha dR,   dw = sum_t dn rh,   dgate = sum_t dR u,   dpost = sum_t dR gate yh
//   dy = rstd_y (dR gate post - yh c2), c2 = mean(dR gate post yh);  without post: dy = dR gate
//   c2's sum needs c1's; written out with g = dn w and q = gate post y,
//     c1 = rstd mean(g r),  c2 = rstd_y (mean(dr q) + rstd mean(g q) - rstd^2 c1 mean(r q)),
//   all four sums come out of one reduction.  dgate and dpost have one sum in common:
//     E = sum_t dR yh,  dgate = post E,  dpost = gate E   (yh = y without post).
// The two forward kernels round alike in kind but not in order: a CTA a row multiplies u by post and gate one after the
// other and divides by H, walking CTAs hold gate * post and 1 / H, and their sums run over other threads' shares.
#include <cuda_bf16.h>

#include "dg_device.cuh"
#include "quant_f32.cuh"
#include "train_internal.h"

namespace dg {

constexpr int kVec = 8;  // columns of a 16-byte piece

struct NormParams {
    const uint4 *x, *y;
    const void *weight, *post, *gate;
    bool vec_bf16;
    float alpha, eps;
    int64_t T;
    int H;
    uint4 *n, *r;
    uint8_t *q;
    float *s_t;
    float *rstd, *rstd_y;
};

// Eight elements of a per-column vector as FP32.
__device__ __forceinline__ void load_vec8(const void *v, bool bf16, int col, float2 (&out)[4]) {
    if (bf16) {
        bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(v) + col)), out);
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(v) + col);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        out[0] = make_float2(a.x, a.y);
        out[1] = make_float2(a.z, a.w);
        out[2] = make_float2(b.x, b.y);
        out[3] = make_float2(b.z, b.w);
    }
}

__device__ __forceinline__ uint4 pack8(const float2 (&v)[4]) {
    return make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                      pack_bf16x2(v[3].x, v[3].y));
}

// The sum over a CTA; red: 32 words of its own for this call.
__device__ __forceinline__ float cta_sum(float v, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane_id() == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane_id() < static_cast<int>(blockDim.x >> 5) ? red[lane_id()] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// A thread's eight columns as codes; 16 threads hold a group of 128 columns and share its scale.
// All lanes call it; those without columns (in == false) bring zeros.
__device__ __forceinline__ void store_codes(const float2 (&n)[4], uint2 *q, float *scale, bool in) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = amax3(m, n[j]);
    uint32_t bits = __float_as_uint(m);  // a NaN above infinity
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, o));
    const FastScale s = fast_scale(__uint_as_float(bits));
    if (in) {
        *q = s.fast ? quantize8_f32<true>(n, s) : quantize8_f32<false>(n, s);
        if ((lane_id() & 15) == 0) *scale = s.s;
    }
}

// Few rows: a CTA per row, NV pieces of eight columns a thread.
template <int NV, bool CODES>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormParams p) {
    __shared__ float red[2][32];
    const int64_t t = blockIdx.x;
    const int tid = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x);
    const int64_t row = t * (p.H / kVec);
    grid_dep_wait();
    grid_dep_launch_dependents();

    uint4 xv[NV], yv[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = tid + v * threads;
        xv[v] = yv[v] = make_uint4(0, 0, 0, 0);
        if (i * kVec < p.H) {
            xv[v] = __ldcs(p.x + row + i);
            if (p.y) yv[v] = __ldcs(p.y + row + i);
        }
    }
    float rstd_y = 1.0f;
    if (p.post) {
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float2 y[4];
            bf16x8_to_f32(yv[v], y);
#pragma unroll
            for (int j = 0; j < 4; ++j) ss += y[j].x * y[j].x + y[j].y * y[j].y;
        }
        rstd_y = __frsqrt_rn(cta_sum(ss, red[0]) / static_cast<float>(p.H) + p.eps);
        if (tid == 0 && p.rstd_y) p.rstd_y[t] = rstd_y;
    }
    float2 r[NV][4];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = tid + v * threads;
        bf16x8_to_f32(xv[v], r[v]);
        if (p.y && i * kVec < p.H) {
            float2 u[4], w[4];
            bf16x8_to_f32(yv[v], u);
            if (p.post) {
                load_vec8(p.post, p.vec_bf16, i * kVec, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = make_float2(u[j].x * rstd_y * w[j].x, u[j].y * rstd_y * w[j].y);
            }
            if (p.gate) {
                load_vec8(p.gate, p.vec_bf16, i * kVec, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = make_float2(u[j].x * w[j].x, u[j].y * w[j].y);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r[v][j] = make_float2(fmaf(p.alpha, r[v][j].x, u[j].x), fmaf(p.alpha, r[v][j].y, u[j].y));
            p.r[row + i] = pack8(r[v]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) ss += r[v][j].x * r[v][j].x + r[v][j].y * r[v][j].y;
    }
    const float rstd = __frsqrt_rn(cta_sum(ss, red[1]) / static_cast<float>(p.H) + p.eps);
    if (tid == 0 && p.rstd) p.rstd[t] = rstd;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = tid + v * threads;
        const bool in = i * kVec < p.H;
        float2 w[4];
        if (in) {
            load_vec8(p.weight, p.vec_bf16, i * kVec, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = make_float2(r[v][j].x * rstd * w[j].x, r[v][j].y * rstd * w[j].y);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = make_float2(0.0f, 0.0f);
        }
        if (!CODES) {
            if (in) p.n[row + i] = pack8(w);
        } else {
            store_codes(w, reinterpret_cast<uint2 *>(p.q) + row + i, p.s_t + static_cast<int64_t>(i >> 4) * p.T + t, in);
        }
    }
}

// ------------------------------------------------------------------- walking over rows
constexpr int kWalkThreads = 512;                      // eight columns a thread: 4096 columns a CTA
constexpr int kWalkCols = kWalkThreads * kVec;
constexpr int kWalkMaxStages = 6;
constexpr int kWalkHeader = 3072;  // barriers and flag, then the warps' sums, then the ring of rows
constexpr int kWalkSums = 128;     // [2][4][16 warps x 4 CTAs] floats
constexpr int kSmemLimit = 232448;
constexpr int kSms = 148;  // of a B200: the workspace is sized without asking a device

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// One float to the same place in CTA `rank` of the cluster, counted by that CTA's barrier `bar`.
__device__ __forceinline__ void store_share(float *word, float v, uint64_t *bar, uint32_t rank) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                     mapa_shared(smem_u32(word), rank)),
                 "r"(__float_as_uint(v)), "r"(mapa_shared(smem_u32(bar), rank))
                 : "memory");
}

struct WalkShape {
    int ctas, threads, cols, stages, grid;
    size_t smem;
};

// For rows of H columns in `arrays` arrays: CTAs that walk a row together, threads of each, and
// as many walkers as run at once with `warps` warps an SM.
static WalkShape walk_shape(int64_t T, int64_t H, int arrays, int threads_per_sm, int most_stages) {
    WalkShape s;
    s.ctas = H <= kWalkCols ? 1 : H <= 2 * kWalkCols ? 2 : 4;
    s.cols = s.ctas == 1 ? static_cast<int>(H) : static_cast<int>((H / s.ctas + 127) / 128 * 128);  // whole groups
    s.threads = (s.cols / kVec + 31) / 32 * 32;
    const int per_sm = threads_per_sm / s.threads;
    const int stage = arrays * s.cols * 2;
    s.stages = (kSmemLimit / per_sm - 1024 - kWalkHeader) / stage;
    if (s.stages > most_stages) s.stages = most_stages;
    s.smem = static_cast<size_t>(kWalkHeader) + static_cast<size_t>(s.stages) * stage;
    // clusters of four lie within a GPC: 33 of them run at once on 148 SMs, not 37 (the gradient of 4000 x 16384
    // with 37: 332 us, in two rounds; with 32 198)
    int64_t walkers = (s.ctas == 4 ? 32 : static_cast<int64_t>(kSms / s.ctas)) * per_sm;
    // two rows each at least, once every SM has a walker: fewer sums to add up (the gradient of 333 x 784: 6.9 -> 6.7 us)
    const int64_t one_round = kSms / s.ctas;
    if (walkers > one_round && walkers > T / 2) walkers = T / 2 > one_round ? T / 2 : one_round;
    if (walkers > T) walkers = T;
    s.grid = static_cast<int>(walkers) * s.ctas;
    return s;
}

template <typename Kernel, typename Params>
static dg_status_t launch_walk(Kernel kernel, const Params &p, const WalkShape &s, int &configured_device, cudaStream_t stream) {
    const dg_status_t st = allow_smem(kernel, kSmemLimit, configured_device);
    if (st != DG_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(s.grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(s.threads), 1, 1);
    cfg.dynamicSmemBytes = s.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(s.ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = s.ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

struct NormWalkParams {
    NormParams n;
    int cols, stages;
    uint64_t timeout_ns;
    int *status;
};

// Many rows: CTAS CTAs (a cluster) walk rows together, each over up to 4096 columns.  The vectors
// stay in registers, rows come through a ring of bulk copies.  An iteration finishes row k, forms r
// of row k + 1 and squares y of row k + 2, so that a row's two sums take one barrier an
// iteration and their latency passes under the other rows' arithmetic.  In a cluster the warps'
// shares go to every CTA as in the gradient's kernel below.  VECTOR: y has a post or a gate.
template <int CTAS, bool Y, bool POST, bool VECTOR, bool CODES>
__global__ void __launch_bounds__(kWalkThreads, 2) rmsnorm_walk_kernel(const NormWalkParams wp) {
    extern __shared__ __align__(128) uint8_t smem[];
    const NormParams &p = wp.n;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem);
    uint64_t *shared_sums = full + kWalkMaxStages;  // [2], in a cluster: an iteration's shares have come
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + 64);
    constexpr int kWords = 16 * CTAS;
    float *red = reinterpret_cast<float *>(smem + kWalkSums);  // [2][2][kWords]: y^2 of row k + 2, r^2 of row k + 1
    uint8_t *ring = smem + kWalkHeader;
    const uint32_t row_bytes = static_cast<uint32_t>(wp.cols) * 2, stage_bytes = row_bytes * (1 + Y);

    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = lane_id();
    const int rank = CTAS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int first = static_cast<int>(blockIdx.x) / CTAS, step = static_cast<int>(gridDim.x) / CTAS;
    const int col0 = rank * wp.cols;
    const int cols = min(wp.cols, p.H - col0);
    const uint32_t load_bytes = static_cast<uint32_t>(cols) * 2;
    const bool mine = tid * kVec < cols;
    const int rows = static_cast<int>((p.T - first + step - 1) / step);  // the grid has no more walkers than rows

    if (tid == 0) {
        for (int s = 0; s < kWalkMaxStages + 2; ++s) mbar_init(&full[s], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    for (int i = tid; i < 2 * 2 * kWords; i += static_cast<int>(blockDim.x)) red[i] = 0.0f;  // absent warps add nothing
    grid_dep_wait();
    grid_dep_launch_dependents();
    const float2 zero = make_float2(0.0f, 0.0f);
    float2 w[4], gp[4], r[4];  // weight, gate * post
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = gp[j] = r[j] = zero;
    if (mine) {
        load_vec8(p.weight, p.vec_bf16, col0 + tid * kVec, w);
        if (VECTOR) load_vec8(POST ? p.post : p.gate, p.vec_bf16, col0 + tid * kVec, gp);
        if (POST && p.gate) {
            load_vec8(p.gate, p.vec_bf16, col0 + tid * kVec, r);
#pragma unroll
            for (int j = 0; j < 4; ++j) gp[j] = __fmul2_rn(gp[j], r[j]);
        }
    }
    if (CTAS > 1)
        cluster_sync();  // every CTA's barriers are there
    else
        __syncthreads();
    const uint32_t share_bytes = static_cast<uint32_t>(blockDim.x >> 5) * 8 * CTAS;

    auto row_of = [&](int i) { return first + static_cast<int64_t>(i) * step; };
    auto ask = [&](int i, int s) {  // one thread
        uint8_t *dst = ring + s * stage_bytes;
        const int64_t at = (row_of(i) * p.H + col0) * 2;
        mbar_arrive_expect_tx(&full[s], load_bytes * (1 + Y));
        bulk_load(dst, reinterpret_cast<const uint8_t *>(p.x) + at, load_bytes, &full[s]);
        if (Y) bulk_load(dst + row_bytes, reinterpret_cast<const uint8_t *>(p.y) + at, load_bytes, &full[s]);
    };
    int asked = 0;
    if (tid == 0)
        for (; asked < wp.stages && asked < rows; ++asked) ask(asked, asked);
    auto piece = [&](int s, int array, float2(&out)[4]) {
        bf16x8_to_f32(reinterpret_cast<const uint4 *>(ring + s * stage_bytes + array * row_bytes)[tid], out);
    };
    const float inv_h = 1.0f / static_cast<float>(p.H);
    const float2 alpha2 = make_float2(p.alpha, p.alpha);
    constexpr int kAhead = POST ? 2 : 1;  // rows that come in before row k is finished
    float rstd = 0.0f, rstd_y = 1.0f;     // of rows k and k + 1
    // the thread's piece in row k + 1, and its group's scale in row k (a 64-bit product a row saved)
    const int64_t row_pieces = static_cast<int64_t>(step) * (p.H / kVec);
    int64_t at = (row_of(0) * p.H + col0) / kVec + tid;
    const int col = col0 + tid * kVec;
    float *scale_at = CODES && mine ? p.s_t + static_cast<int64_t>(col >> 7) * p.T + first : nullptr;
    int s_in = 0, s_r = 0;                // stages of rows k + kAhead and k + 1
    uint32_t parity = 0u;                 // of the first

    for (int k = -kAhead; k < rows; ++k) {
        const int it = k + kAhead;
        float yy = 0.0f, rr = 0.0f;
        if (it < rows) {
            if (!mbar_wait(&full[s_in], parity, abort_flag, wp.timeout_ns)) {
                // no row is asked for any more, and every later wait ends at once
                record_failure(wp.status, kStatusTimeout, 22, it);
                *abort_flag = 1;
            }
            if (POST && mine) {
                float2 y[4], sum = zero;
                piece(s_in, 1, y);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = __ffma2_rn(y[j], y[j], sum);
                yy = sum.x + sum.y;
            }
        }
        if (k >= 0) {  // n of row k
            if (tid == 0 && rank == 0 && p.rstd) p.rstd[row_of(k)] = rstd;
            const float2 rs = make_float2(rstd, rstd);
            float2 n[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) n[j] = __fmul2_rn(__fmul2_rn(r[j], rs), w[j]);
            if (!CODES) {
                if (mine) p.n[at - row_pieces] = pack8(n);
            } else {
                store_codes(n, reinterpret_cast<uint2 *>(p.q) + (at - row_pieces), scale_at, mine);
                scale_at += step;
            }
        }
        if (k + 1 >= 0 && k + 1 < rows) {  // r of row k + 1
            if (POST && tid == 0 && rank == 0 && p.rstd_y) p.rstd_y[row_of(k + 1)] = rstd_y;
            if (mine) {
                piece(s_r, 0, r);
                if (Y) {
                    const float2 ry = make_float2(rstd_y, rstd_y);
                    float2 u[4];
                    piece(s_r, 1, u);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (POST) u[j] = __fmul2_rn(u[j], ry);
                        if (VECTOR) u[j] = __fmul2_rn(u[j], gp[j]);
                        r[j] = __ffma2_rn(alpha2, r[j], u[j]);
                    }
                    p.r[at] = pack8(r);
                }
                float2 sum = zero;
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = __ffma2_rn(r[j], r[j], sum);
                rr = sum.x + sum.y;
            }
        }
        {  // lanes 0 to 15 sum y^2, the others r^2
            const bool high = lane & 16;
            float v = (high ? rr : yy) + __shfl_xor_sync(0xFFFFFFFFu, high ? yy : rr, 16);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            float *word = red + ((it & 1) * 2 + (lane >> 4)) * kWords + rank * 16 + warp;
            if (CTAS == 1) {
                if ((lane & 15) == 0) *word = v;
            } else {
                if (tid == 0) mbar_arrive_expect_tx(&shared_sums[it & 1], share_bytes);
                if ((lane & 15) < CTAS) store_share(word, v, &shared_sums[it & 1], lane & 15);
            }
        }
        __syncthreads();  // row k + 1's stage has been read, and the CTA's sums are there
        if (tid == 0 && k + 1 >= 0 && k + 1 + wp.stages < rows && !*abort_flag) {
            ask(k + 1 + wp.stages, s_r);
            ++asked;
        }
        if (CTAS > 1 && !mbar_wait(&shared_sums[it & 1], static_cast<uint32_t>(it >> 1) & 1u, abort_flag, wp.timeout_ns)) {
            record_failure(wp.status, kStatusTimeout, 23, it);
            *abort_flag = 1;
        }
        float v = 0.0f;
#pragma unroll
        for (int c = 0; c < CTAS; ++c) v += red[((it & 1) * 2 + (lane >> 4)) * kWords + c * 16 + (lane & 15)];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = __frsqrt_rn(fmaf(v, inv_h, p.eps));
        if (POST) rstd_y = __shfl_sync(0xFFFFFFFFu, v, 0);
        rstd = __shfl_sync(0xFFFFFFFFu, v, 16);
        if (k + 1 >= 0) {
            s_r = s_r + 1 == wp.stages ? 0 : s_r + 1;
            at += row_pieces;
        }
        if (++s_in == wp.stages) {
            s_in = 0;
            parity ^= 1u;
        }
    }
    if (tid == 0 && *abort_flag) {  // every copy must land before the CTA may exit
        const int never = 0;
        for (int i = asked > wp.stages ? asked - wp.stages : 0; i < asked; ++i)
            if (!mbar_wait(&full[i % wp.stages], static_cast<uint32_t>(i / wp.stages) & 1u, &never, wp.timeout_ns))
                record_failure(wp.status, kStatusTimeout, 22, -1);
    }
    if (CTAS > 1) cluster_sync();  // after a failure a CTA could leave while shares are on their way to it
}

template <bool Y, bool POST, bool VECTOR, bool CODES>
static dg_status_t launch_walk_forward(const NormWalkParams &p, const WalkShape &s, cudaStream_t stream) {
    static thread_local int one = -1, two = -1, four = -1;
    if (s.ctas == 1) return launch_walk(rmsnorm_walk_kernel<1, Y, POST, VECTOR, CODES>, p, s, one, stream);
    if (s.ctas == 2) return launch_walk(rmsnorm_walk_kernel<2, Y, POST, VECTOR, CODES>, p, s, two, stream);
    return launch_walk(rmsnorm_walk_kernel<4, Y, POST, VECTOR, CODES>, p, s, four, stream);
}

template <bool CODES>
static dg_status_t launch_walk_form(const NormWalkParams &p, const WalkShape &s, cudaStream_t stream) {
    if (!p.n.y) return launch_walk_forward<false, false, false, CODES>(p, s, stream);
    if (p.n.post) return launch_walk_forward<true, true, true, CODES>(p, s, stream);
    if (p.n.gate) return launch_walk_forward<true, false, true, CODES>(p, s, stream);
    return launch_walk_forward<true, false, false, CODES>(p, s, stream);
}

// Above this many rows they are walked over.  A CTA a row has no ring to fill first: 1500 x 1024 with post and gate
// as codes 5.3 us against 6.9 walked over, 700 x 256 3.1 against 4.5, about the same from 3000 rows on.  Of wider
// rows fewer run at once, and the forms cross earlier, between 160 and 300 rows with post and gate: 601 x 7168 as codes 17 us
// against 13 walked over, 300 x 7168 9.8 and 8.4, 300 x 4096 7.3 and 6.7, 160 x 4096 4.0 and 5.1; without them 300 x 4096
// 5.2 and 4.8, 500 x 7168 8.2 and 9.5, 500 x 16384 16.2 and 18.2.  The bound is the row count from which the walk
// is no slower in any of them but wide rows without vectors; a finer one would have to follow the form too.
static int64_t walk_rows(int64_t H) { return H <= 1024 ? 3000 : 600; }

dg_status_t launch_rmsnorm(const NormArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    NormParams p;
    p.x = static_cast<const uint4 *>(a.x);
    p.y = static_cast<const uint4 *>(a.y);
    p.weight = a.weight;
    p.post = a.post;
    p.gate = a.gate;
    p.vec_bf16 = a.vec_bf16;
    p.alpha = a.alpha;
    p.eps = a.eps;
    p.T = a.T;
    p.H = static_cast<int>(a.H);
    p.n = static_cast<uint4 *>(a.n);
    p.r = static_cast<uint4 *>(a.r);
    p.q = a.q;
    p.s_t = a.s_t;
    p.rstd = a.rstd;
    p.rstd_y = a.rstd_y;
    const bool codes = a.q != nullptr;
    if (a.T > walk_rows(a.H)) {
        // Reads far ahead of the writes cost bandwidth: 16384 x 4096 with a post and a gate, two CTAs an SM, takes
        // 87 us with three rows in the ring, 94 with four, 101 with six (one CTA: 104).  With less arithmetic one
        // CTA and four rows keep up: 86 us without post, against 107 with two CTAs and three rows; in clusters two
        // CTAs and two rows do (16384 x 8192 164 us, with three rows 193, one CTA and four rows 188; 4000 x 16384
        // 93, 94 and 146).
        const bool heavy = codes || a.post, two = heavy || a.H > kWalkCols;
        const WalkShape s = walk_shape(a.T, a.H, 1 + (a.y != nullptr), two ? 2 * kWalkThreads : kWalkThreads, heavy ? 3 : two ? 2 : 4);
        const KernelControl ctl = kernel_control();
        const NormWalkParams wp = {p, s.cols, s.stages, ctl.timeout_ns, ctl.status};
        return codes ? launch_walk_form<true>(wp, s, stream) : launch_walk_form<false>(wp, s, stream);
    }
    const int pieces = p.H / kVec;
    auto threads_for = [&](int nv) { return (((pieces + nv - 1) / nv) + 31) / 32 * 32; };
    const int grid = static_cast<int>(a.T);
    const bool few = a.T <= 2 * dev.num_sms;  // rows that do not fill the GPU: short rather than many
    if (pieces <= 1024 && (few || pieces <= 128))
        return codes ? launch_pdl(rmsnorm_kernel<1, true>, grid, threads_for(1), 0, stream, p)
                     : launch_pdl(rmsnorm_kernel<1, false>, grid, threads_for(1), 0, stream, p);
    return codes ? launch_pdl(rmsnorm_kernel<4, true>, grid, threads_for(4), 0, stream, p)
                 : launch_pdl(rmsnorm_kernel<4, false>, grid, threads_for(4), 0, stream, p);
}

// ----------------------------------------------------------------------------- backward
struct NormBackwardParams {
    const uint8_t *dn, *dr, *r, *y;  // rows of 2 H bytes
    const void *weight, *post, *gate;
    const float *rstd, *rstd_y;
    bool vec_bf16;
    float alpha;
    int64_t T;
    int H;
    int cols;    // columns of a CTA: H, or a share of it
    int stages;
    uint4 *dx, *dy;
    float *part;  // [grid / CTAS][sums][H] per-column sums of a CTA's rows
    uint64_t timeout_ns;
    int *status;
};

// Four values summed over a warp's lanes: lane l holds the sum of value (l / 8) % 4.  Two exchanges
// halve what each lane carries, so this takes six shuffles instead of twenty.
__device__ __forceinline__ float warp_sum4(float a, float b, float c, float d) {
    const int lane = lane_id();
    const bool high = lane & 16, odd = lane & 8;
    const float keep0 = high ? c : a, keep1 = high ? d : b, give0 = high ? a : c, give1 = high ? b : d;
    const float x = keep0 + __shfl_xor_sync(0xFFFFFFFFu, give0, 16), y = keep1 + __shfl_xor_sync(0xFFFFFFFFu, give1, 16);
    float v = (odd ? y : x) + __shfl_xor_sync(0xFFFFFFFFu, odd ? x : y, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// CTAS CTAs (a cluster) walk rows together, each over up to 4096 columns, eight a thread.  The
// vectors and the per-column sums stay in registers; rows come through a ring of bulk copies.
// The loop takes a row's sums one iteration before it uses them, so that one barrier a row
// publishes the next row's sums and frees a stage.  A row's pieces stay in registers from its sums to its outputs,
// and the next row's are read behind these (16384 x 4096: 133 us, 8192 x 8192 150; a second read of the ring cost 9 us of
// either); clusters of four take the next row's sums first and read the row at hand from the ring once more, so that the shares' way
// passes under its arithmetic (4000 x 16384: 201 us as in smaller clusters, 190 so).  In a cluster each warp
// stores its share into every CTA asynchronously, counted by that CTA's barrier of the row's parity: the
// cluster's own barrier would wait for the row's stores to global memory (8192 x 8192: 232 us with it).  A share of row
// i + 2 cannot overtake a reader of row i: it is sent after all shares of row i + 1 have come, and a warp
// sends its share of row i + 1 after it has read row i.
// VECTOR: y has a post or a gate (POST implies it).
template <int CTAS, bool Y, bool POST, bool VECTOR>
__global__ void __launch_bounds__(kWalkThreads, 1) rmsnorm_backward_kernel(const NormBackwardParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem);
    uint64_t *shared_sums = full + kWalkMaxStages;  // [2], in a cluster: a row's shares have come
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + 64);
    constexpr int kWords = 16 * CTAS;  // warps of the cluster
    constexpr bool kAhead = CTAS == 4;
    float *red = reinterpret_cast<float *>(smem + kWalkSums);  // [2][4][kWords]
    uint8_t *ring = smem + kWalkHeader;
    constexpr int kSumsKept = 1 + VECTOR;
    const int arrays = 2 + (p.dr != nullptr) + Y;
    const uint32_t row_bytes = static_cast<uint32_t>(p.cols) * 2;
    const uint32_t stage_bytes = row_bytes * arrays;

    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = lane_id();
    const int rank = CTAS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int first = static_cast<int>(blockIdx.x) / CTAS, step = static_cast<int>(gridDim.x) / CTAS;
    const int col0 = rank * p.cols;
    const int cols = min(p.cols, p.H - col0);
    const uint32_t load_bytes = static_cast<uint32_t>(cols) * 2;
    const bool mine = tid * kVec < cols;  // this thread has columns

    if (tid == 0) {
        for (int s = 0; s < kWalkMaxStages + 2; ++s) mbar_init(&full[s], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    for (int i = tid; i < 2 * 4 * kWords; i += static_cast<int>(blockDim.x)) red[i] = 0.0f;  // absent warps add nothing
    grid_dep_wait();
    grid_dep_launch_dependents();
    const float2 zero = make_float2(0.0f, 0.0f);
    float2 w[4], gp[4], acc_w[4], acc_e[4];  // weight, gate * post
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = gp[j] = acc_w[j] = acc_e[j] = zero;
    if (mine) {
        load_vec8(p.weight, p.vec_bf16, col0 + tid * kVec, w);
        if (VECTOR) load_vec8(POST ? p.post : p.gate, p.vec_bf16, col0 + tid * kVec, gp);
        if (POST && p.gate) {
            float2 gate[4];
            load_vec8(p.gate, p.vec_bf16, col0 + tid * kVec, gate);
#pragma unroll
            for (int j = 0; j < 4; ++j) gp[j] = __fmul2_rn(gp[j], gate[j]);
        }
    }
    if (CTAS > 1)
        cluster_sync();  // every CTA's barriers are there
    else
        __syncthreads();
    const uint32_t share_bytes = static_cast<uint32_t>(blockDim.x >> 5) * 16 * CTAS;

    auto ask = [&](int64_t t, int s) {  // one thread
        uint8_t *dst = ring + s * stage_bytes;
        const int64_t at = (t * p.H + col0) * 2;
        mbar_arrive_expect_tx(&full[s], load_bytes * arrays);
        bulk_load(dst, p.dn + at, load_bytes, &full[s]);
        bulk_load(dst + row_bytes, p.r + at, load_bytes, &full[s]);
        if (Y) bulk_load(dst + 2 * row_bytes, p.y + at, load_bytes, &full[s]);
        if (p.dr) bulk_load(dst + (2 + Y) * row_bytes, p.dr + at, load_bytes, &full[s]);
    };
    int asked = 0;  // rows that thread 0 asked for
    if (tid == 0)
        for (; asked < p.stages && first + static_cast<int64_t>(asked) * step < p.T; ++asked)
            ask(first + static_cast<int64_t>(asked) * step, asked);

    uint4 held[4];     // the thread's pieces of the row whose sums were taken last: dn, r, y, dr
    float2 held_g[4];  // and dn w
    auto take = [&](int s, int array) { return reinterpret_cast<const uint4 *>(ring + s * stage_bytes + array * row_bytes)[tid]; };
    // the warp's share of a row's sums (g r, dr q, g q, r q), to every CTA of the cluster
    auto sum_row = [&](int it, int s, uint32_t parity) {
        if (!mbar_wait(&full[s], parity, abort_flag, p.timeout_ns)) {
            // no row is asked for any more, and every later wait ends at once
            record_failure(p.status, kStatusTimeout, 20, it);
            *abort_flag = 1;
        }
        float2 gr = zero, dq = zero, gq = zero, rq = zero;
        if (mine) {
            held[0] = take(s, 0);
            held[1] = take(s, 1);
            if (Y) held[2] = take(s, 2);
            if (p.dr) held[3] = take(s, 2 + Y);
            float2 r[4], (&g)[4] = held_g;
            bf16x8_to_f32(held[0], g);
            bf16x8_to_f32(held[1], r);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                g[j] = __fmul2_rn(g[j], w[j]);
                gr = __ffma2_rn(g[j], r[j], gr);
            }
            if (POST) {
                float2 q[4];
                bf16x8_to_f32(held[2], q);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    q[j] = __fmul2_rn(q[j], gp[j]);
                    gq = __ffma2_rn(g[j], q[j], gq);
                    rq = __ffma2_rn(r[j], q[j], rq);
                }
                if (p.dr) {
                    bf16x8_to_f32(held[3], r);
#pragma unroll
                    for (int j = 0; j < 4; ++j) dq = __ffma2_rn(r[j], q[j], dq);
                }
            }
        }
        const float v = warp_sum4(gr.x + gr.y, dq.x + dq.y, gq.x + gq.y, rq.x + rq.y);
        float *word = red + ((it & 1) * 4 + (lane >> 3)) * kWords + rank * 16 + warp;
        if (CTAS == 1) {
            if ((lane & 7) == 0) *word = v;
        } else {
            if (tid == 0) mbar_arrive_expect_tx(&shared_sums[it & 1], share_bytes);
            if ((lane & 7) < CTAS)  // one lane for each value and CTA
                store_share(word, v, &shared_sums[it & 1], lane & 7);
        }
    };
    // -c1 and -c2 of the row.  They and the normed rows rh and yh are of the size of what they are made from.  rstd^2 c1
    // in their place saves a product an element and sum (16384 x 4096 131.6 us against 132.7, 8192 x 8192 147 against
    // 149), but it leaves FP32 in rows whose mean square FP32 holds (from an RMS of 1e13 on, and below 1e-13).
    float back = 0.0f, back_y = 0.0f;
    const float inv_h = 1.0f / static_cast<float>(p.H);
    auto read_sums = [&](int it, float rstd, float rstd_y) {  // in the same order in every warp and CTA
        if (CTAS > 1 && !mbar_wait(&shared_sums[it & 1], static_cast<uint32_t>(it >> 1) & 1u, abort_flag, p.timeout_ns)) {
            record_failure(p.status, kStatusTimeout, 21, it);
            *abort_flag = 1;
        }
        const float *words = red + ((it & 1) * 4 + (lane >> 3)) * kWords + (lane & 7) * 2;
        float v = 0.0f;
#pragma unroll
        for (int c = 0; c < CTAS; ++c) {
            const float2 two = *reinterpret_cast<const float2 *>(words + 16 * c);
            v += two.x + two.y;
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v *= inv_h;
        back = -rstd * __shfl_sync(0xFFFFFFFFu, v, 0);
        if (POST) {
            const float dq = __shfl_sync(0xFFFFFFFFu, v, 8), gq = __shfl_sync(0xFFFFFFFFu, v, 16), rq = __shfl_sync(0xFFFFFFFFu, v, 24);
            back_y = -rstd_y * fmaf(rstd, fmaf(back, rstd * rq, gq), dq);
        }
    };
    auto scale_of_row = [&](const float *v, int64_t t) { return t < p.T ? __ldg(v + t) : 0.0f; };

    int64_t t = first;
    float rstd = scale_of_row(p.rstd, t), rstd_y = POST ? scale_of_row(p.rstd_y, t) : 1.0f;
    if (t < p.T) sum_row(0, 0, 0u);
    __syncthreads();
    auto refill = [&](int64_t row, int s) {  // the stage that it was read from
        const int64_t later = row + static_cast<int64_t>(p.stages) * step;
        if (tid == 0 && later < p.T && !*abort_flag) {
            ask(later, s);
            ++asked;
        }
    };
    if (!kAhead) refill(t, 0);
    if (t < p.T) read_sums(0, rstd, rstd_y);
    int s = 0, next_s = 1;  // at least two stages
    uint32_t next_parity = 0u;
    float next_rstd = scale_of_row(p.rstd, t + step), next_rstd_y = POST ? scale_of_row(p.rstd_y, t + step) : 1.0f;
    const int64_t row_pieces = static_cast<int64_t>(step) * (p.H / kVec);
    int64_t out = (t * p.H + col0) / kVec + tid;  // the thread's piece in row t
    for (int it = 0; t < p.T; t += step, out += row_pieces, ++it) {
        const int64_t next = t + step;
        const float later_rstd = scale_of_row(p.rstd, next + step);
        const float later_rstd_y = POST ? scale_of_row(p.rstd_y, next + step) : 1.0f;
        if (kAhead && next < p.T) sum_row(it + 1, next_s, next_parity);
        if (mine) {
            auto piece = [&](int i, int array, float2(&v)[4]) { bf16x8_to_f32(kAhead ? take(s, array) : held[i], v); };
            const float2 rs = make_float2(rstd, rstd), ry = make_float2(rstd_y, rstd_y), alpha2 = make_float2(p.alpha, p.alpha);
            const float2 back2 = make_float2(back, back), back_y2 = make_float2(back_y, back_y);
            float2 m[4], r[4], d[4];
            piece(0, 0, m);
            piece(1, 1, r);
            if (p.dr) {
                piece(3, 2 + Y, d);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = zero;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r[j] = __fmul2_rn(r[j], rs);  // rh
                acc_w[j] = __ffma2_rn(m[j], r[j], acc_w[j]);
                m[j] = __ffma2_rn(r[j], back2, kAhead ? __fmul2_rn(m[j], w[j]) : held_g[j]);
                d[j] = __ffma2_rn(m[j], rs, d[j]);  // dR
                m[j] = __fmul2_rn(d[j], alpha2);
            }
            p.dx[out] = pack8(m);
            if (Y) {
                if (VECTOR) {
                    piece(2, 2, r);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (POST) r[j] = __fmul2_rn(r[j], ry);  // yh
                        acc_e[j] = __ffma2_rn(d[j], r[j], acc_e[j]);
                        d[j] = __fmul2_rn(d[j], gp[j]);
                        if (POST) d[j] = __fmul2_rn(__ffma2_rn(r[j], back_y2, d[j]), ry);
                    }
                }
                p.dy[out] = pack8(d);
            }
        }
        if (!kAhead && next < p.T) sum_row(it + 1, next_s, next_parity);
        __syncthreads();  // a stage has been read by all, and the next row's sums are there
        refill(kAhead ? t : next, kAhead ? s : next_s);
        rstd = next_rstd;
        rstd_y = next_rstd_y;
        next_rstd = later_rstd;
        next_rstd_y = later_rstd_y;
        if (next < p.T) read_sums(it + 1, rstd, rstd_y);
        s = next_s;
        if (++next_s == p.stages) {
            next_s = 0;
            next_parity ^= 1u;
        }
    }
    if (tid == 0 && *abort_flag) {  // every copy must land before the CTA may exit
        const int never = 0;
        for (int i = asked > p.stages ? asked - p.stages : 0; i < asked; ++i)
            if (!mbar_wait(&full[i % p.stages], static_cast<uint32_t>(i / p.stages) & 1u, &never, p.timeout_ns))
                record_failure(p.status, kStatusTimeout, 20, -1);
    }
    if (CTAS > 1) cluster_sync();  // after a failure a CTA could leave while shares are on their way to it
    if (mine) {
        auto put = [&](int which, const float2(&a)[4]) {
            float4 *dst = reinterpret_cast<float4 *>(p.part + (static_cast<int64_t>(first) * kSumsKept + which) * p.H + col0) + 2 * tid;
            dst[0] = make_float4(a[0].x, a[0].y, a[1].x, a[1].y);
            dst[1] = make_float4(a[2].x, a[2].y, a[3].x, a[3].y);
        };
        put(0, acc_w);
        if (VECTOR) put(1, acc_e);
    }
}

// Columns of [parts][sums][H] added up in order: 32 columns a CTA, sixteen threads a column.  The
// second sum is E, of which dgate and dpost are multiples.
__global__ void __launch_bounds__(512) rmsnorm_columns_kernel(const float *__restrict__ part, int parts, int H, int sums,
                                                              const void *post, const void *gate, bool vec_bf16,
                                                              float *__restrict__ dweight, float *__restrict__ dpost,
                                                              float *__restrict__ dgate) {
    __shared__ float shares[16][33];
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int lane = lane_id(), w = static_cast<int>(threadIdx.x) >> 5;
    const int64_t width = static_cast<int64_t>(sums) * H, c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < width) {
        constexpr int kDeep = 10;  // loads in flight: 148 parts over 16 warps
        for (int i0 = w; i0 < parts; i0 += kDeep * 16) {
            float v[kDeep];
#pragma unroll
            for (int j = 0; j < kDeep; ++j) v[j] = i0 + 16 * j < parts ? __ldg(part + (i0 + 16 * j) * width + c) : 0.0f;
#pragma unroll
            for (int j = 0; j < kDeep; ++j) s += v[j];
        }
    }
    shares[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < width) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += shares[i][lane];
        if (c < H) {
            dweight[c] = s;
        } else {
            const int64_t h = c - H;
            auto times = [&](const void *v) {  // one element of a vector, or 1; no rows: the sum is 0 whatever that holds
                if (!v || parts == 0) return 1.0f;
                return vec_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(v)[h]) : static_cast<const float *>(v)[h];
            };
            if (dgate) dgate[h] = s * times(post);
            if (dpost) dpost[h] = s * times(gate);
        }
    }
}

template <bool Y, bool POST, bool VECTOR>
static dg_status_t launch_backward_form(const NormBackwardParams &p, const WalkShape &s, cudaStream_t stream) {
    static thread_local int one = -1, two = -1, four = -1;
    if (s.ctas == 1) return launch_walk(rmsnorm_backward_kernel<1, Y, POST, VECTOR>, p, s, one, stream);
    if (s.ctas == 2) return launch_walk(rmsnorm_backward_kernel<2, Y, POST, VECTOR>, p, s, two, stream);
    return launch_walk(rmsnorm_backward_kernel<4, Y, POST, VECTOR>, p, s, four, stream);
}

int64_t rmsnorm_backward_workspace(int64_t T, int64_t H, bool post, bool gate) {
    const WalkShape s = walk_shape(T, H, 2, kWalkThreads, 4);
    return static_cast<int64_t>(s.grid / s.ctas) * (1 + (post || gate)) * H * 4;
}

dg_status_t launch_rmsnorm_backward(const NormBackwardArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    (void)dev;
    const bool y = a.y != nullptr, post = a.post != nullptr, gate = a.gate != nullptr;
    // four rows in the ring: 16384 x 4096 with all vectors 131.5 us, with three 131.1, with six 133; 4000 x 16384 194, 195, 197
    // (measured with rstd^2 c1 and rstd_y^2 c2 in place of c1 and c2)
    const WalkShape s = walk_shape(a.T, a.H, 2 + y + (a.dr != nullptr), kWalkThreads, 4);
    const KernelControl ctl = kernel_control();
    NormBackwardParams p;
    p.dn = static_cast<const uint8_t *>(a.dn);
    p.dr = static_cast<const uint8_t *>(a.dr);
    p.r = static_cast<const uint8_t *>(a.r);
    p.y = static_cast<const uint8_t *>(a.y);
    p.weight = a.weight;
    p.post = a.post;
    p.gate = a.gate;
    p.rstd = a.rstd;
    p.rstd_y = a.rstd_y;
    p.vec_bf16 = a.vec_bf16;
    p.alpha = a.alpha;
    p.T = a.T;
    p.H = static_cast<int>(a.H);
    p.cols = s.cols;
    p.stages = s.stages;
    p.dx = static_cast<uint4 *>(a.dx);
    p.dy = static_cast<uint4 *>(a.dy);
    p.part = static_cast<float *>(a.workspace);
    p.timeout_ns = ctl.timeout_ns;
    p.status = ctl.status;
    if (a.T > 0) {
        dg_status_t st;
        if (!y) st = launch_backward_form<false, false, false>(p, s, stream);
        else if (post) st = launch_backward_form<true, true, true>(p, s, stream);
        else if (gate) st = launch_backward_form<true, false, true>(p, s, stream);
        else st = launch_backward_form<true, false, false>(p, s, stream);
        if (st != DG_OK) return st;
    }
    const int sums = 1 + (post || gate);
    return launch_pdl(rmsnorm_columns_kernel, static_cast<int>((sums * a.H + 31) / 32), 512, 0, stream,
                      static_cast<const float *>(p.part), s.grid / s.ctas, p.H, sums, a.post, a.gate, a.vec_bf16, a.dweight,
                      a.dpost, a.dgate);
}

}  // namespace dg

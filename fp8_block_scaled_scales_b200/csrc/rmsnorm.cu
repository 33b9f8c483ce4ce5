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
//   c2's sum needs c1's; written out, mean((dr + rstd dn w) q) - rstd c1 mean(rh q) with
//   q = gate post yh, all three sums come out of one reduction.
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

// A CTA per row, NV pieces of eight columns a thread.
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
            // 16 threads hold a group of 128 columns
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) m = amax3(m, w[j]);
            uint32_t bits = __float_as_uint(m);  // a NaN above infinity
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, o));
            const FastScale s = fast_scale(__uint_as_float(bits));
            if (in) {
                const uint2 c = s.fast ? quantize8_f32<true>(w, s) : quantize8_f32<false>(w, s);
                *reinterpret_cast<uint2 *>(p.q + t * p.H + i * kVec) = c;
                if ((tid & 15) == 0) p.s_t[static_cast<int64_t>(i >> 4) * p.T + t] = s.s;
            }
        }
    }
}

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
    const int pieces = p.H / kVec;
    auto threads_for = [&](int nv) { return (((pieces + nv - 1) / nv) + 31) / 32 * 32; };
    const int grid = static_cast<int>(a.T);
    const bool codes = a.q != nullptr;
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
    int cols;    // columns of a CTA: H, or half of it
    int stages;
    uint4 *dx, *dy;
    float *part;  // [grid / CTAS][sums][H] per-column sums of a CTA's rows
    uint64_t timeout_ns;
    int *status;
};

// Shared memory of the backward kernel: barriers, the reduction's words, the vectors in FP32
// and a ring of rows (dn, r, dr, y).
constexpr int kNormHeader = 1024;
constexpr int kNormMaxStages = 4;

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// CTAS CTAs (a cluster) walk rows together, each over its columns, NV pieces a thread.  The
// per-column sums stay in registers until the last row.
template <int NV, int CTAS, bool Y, bool POST, bool GATE>
__global__ void __launch_bounds__(512) rmsnorm_backward_kernel(const NormBackwardParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + 64);
    float *exchange = reinterpret_cast<float *>(smem + 80);                // [2][3]: the CTA's sums, per row parity
    float4 *red = reinterpret_cast<float4 *>(smem + 128);                  // [2][16] per row parity and warp
    float *vec = reinterpret_cast<float *>(smem + kNormHeader);            // weight, post, gate: [cols] each
    constexpr int kVectors = 1 + POST + GATE;
    uint8_t *ring = smem + kNormHeader + kVectors * p.cols * 4;
    const int arrays = 2 + (p.dr != nullptr) + Y;
    const uint32_t row_bytes = static_cast<uint32_t>(p.cols) * 2;
    const uint32_t stage_bytes = row_bytes * arrays;

    const int tid = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x);
    const int warp = tid >> 5, warps = threads >> 5, lane = lane_id();
    const int rank = CTAS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int first = static_cast<int>(blockIdx.x) / CTAS, step = static_cast<int>(gridDim.x) / CTAS;
    const int col0 = rank * p.cols;
    const int cols = min(p.cols, p.H - col0);
    const uint32_t load_bytes = static_cast<uint32_t>(cols) * 2;

    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    grid_dep_wait();
    grid_dep_launch_dependents();
    for (int c = tid; c < cols; c += threads) {
        auto one = [&](const void *v) {
            return p.vec_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(v)[col0 + c])
                              : static_cast<const float *>(v)[col0 + c];
        };
        vec[c] = one(p.weight);
        if (POST) vec[p.cols + c] = one(p.post);
        if (GATE) vec[(1 + POST) * p.cols + c] = one(p.gate);
    }
    __syncthreads();

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

    float2 acc_w[NV][4], acc_g[GATE ? NV : 1][4], acc_p[POST ? NV : 1][4];
    const float2 zero = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc_w[v][j] = zero;
            if (GATE) acc_g[v][j] = zero;
            if (POST) acc_p[v][j] = zero;
        }
    const float inv_h = 1.0f / static_cast<float>(p.H);

    int it = 0;
    for (int64_t t = first; t < p.T; t += step, ++it) {
        const int s = it % p.stages;
        const uint8_t *src = ring + s * stage_bytes;
        const float rstd = __ldg(p.rstd + t), rstd_y = POST ? __ldg(p.rstd_y + t) : 1.0f;
        if (!mbar_wait(&full[s], static_cast<uint32_t>(it / p.stages) & 1u, abort_flag, p.timeout_ns)) {
            // no row is asked for any more, and every later wait ends at once
            record_failure(p.status, kStatusTimeout, 20, it);
            *abort_flag = 1;
        }
        const float2 rstd2 = make_float2(rstd, rstd), rstd_y2 = make_float2(rstd_y, rstd_y);
        float2 s1 = zero, s2 = zero, s3 = zero;
        auto load = [&](int array, int i, float2(&out)[4]) {
            bf16x8_to_f32(reinterpret_cast<const uint4 *>(src + array * row_bytes)[i], out);
        };
        auto vec8 = [&](int which, int i, float2(&out)[4]) {
            const float4 *q = reinterpret_cast<const float4 *>(vec + which * p.cols) + 2 * i;
            const float4 a = q[0], b = q[1];
            out[0] = make_float2(a.x, a.y);
            out[1] = make_float2(a.z, a.w);
            out[2] = make_float2(b.x, b.y);
            out[3] = make_float2(b.z, b.w);
        };
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = tid + v * threads;
            if (i * kVec >= cols) break;
            float2 dn[4], rh[4], w[4];
            load(0, i, dn);
            load(1, i, rh);
            vec8(0, i, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                rh[j] = __fmul2_rn(rh[j], rstd2);
                dn[j] = __fmul2_rn(dn[j], w[j]);
                s1 = __ffma2_rn(dn[j], rh[j], s1);
            }
            if (POST) {
                float2 q[4], d[4];
                load(2, i, q);
                vec8(1, i, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = __fmul2_rn(__fmul2_rn(q[j], rstd_y2), w[j]);
                if (GATE) {
                    vec8(1 + POST, i, w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) q[j] = __fmul2_rn(q[j], w[j]);
                }
                if (p.dr) {
                    load(2 + Y, i, d);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) d[j] = zero;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s2 = __ffma2_rn(__ffma2_rn(dn[j], rstd2, d[j]), q[j], s2);
                    s3 = __ffma2_rn(rh[j], q[j], s3);
                }
            }
        }
        float a = s1.x + s1.y, b = s2.x + s2.y, c = s3.x + s3.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            if (POST) {
                b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
                c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
            }
        }
        float4 *words = red + (it & 1) * 16;  // the other row's may still be read
        if (lane == 0) words[warp] = make_float4(a, b, c, 0.0f);
        __syncthreads();
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i = 0; i < warps; ++i) {
            const float4 w = words[i];
            sum.x += w.x;
            sum.y += w.y;
            sum.z += w.z;
        }
        if (CTAS > 1) {
            float *mine = exchange + (it & 1) * 3;
            if (tid == 0) mine[0] = sum.x, mine[1] = sum.y, mine[2] = sum.z;
            cluster_sync();
            const uint32_t at = smem_u32(mine);
            sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int q = 0; q < CTAS; ++q) {  // the same order in every CTA
                const uint32_t far = mapa_shared(at, q);
                sum.x += ld_cluster_f32(far);
                sum.y += ld_cluster_f32(far + 4);
                sum.z += ld_cluster_f32(far + 8);
            }
        }
        const float c1 = sum.x * inv_h;
        const float c2 = (sum.y - rstd * c1 * sum.z) * inv_h;
        const float2 back = make_float2(-rstd * c1, -rstd * c1), alpha2 = make_float2(p.alpha, p.alpha);
        const float2 c2n = make_float2(-c2, -c2);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = tid + v * threads;
            if (i * kVec >= cols) break;
            float2 dn[4], rh[4], w[4], d[4];
            load(0, i, dn);
            load(1, i, rh);
            vec8(0, i, w);
            if (p.dr) {
                load(2 + Y, i, d);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = zero;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                rh[j] = __fmul2_rn(rh[j], rstd2);
                acc_w[v][j] = __ffma2_rn(dn[j], rh[j], acc_w[v][j]);
                d[j] = __ffma2_rn(__fmul2_rn(dn[j], w[j]), rstd2, d[j]);
                d[j] = __ffma2_rn(back, rh[j], d[j]);  // dR
                w[j] = __fmul2_rn(d[j], alpha2);
            }
            const int64_t out = (t * p.H + col0) / kVec + i;
            p.dx[out] = pack8(w);
            if (Y) {
                float2 u[4], g[4], yh[4];
                load(2, i, u);
                if (POST) {
                    vec8(1, i, w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        yh[j] = __fmul2_rn(u[j], rstd_y2);
                        u[j] = __fmul2_rn(yh[j], w[j]);
                    }
                }
                if (GATE) {
                    vec8(1 + POST, i, g);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc_g[v][j] = __ffma2_rn(d[j], u[j], acc_g[v][j]);
                        d[j] = __fmul2_rn(d[j], g[j]);
                    }
                }
                if (POST) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc_p[v][j] = __ffma2_rn(d[j], yh[j], acc_p[v][j]);
                        d[j] = __fmul2_rn(__ffma2_rn(c2n, yh[j], __fmul2_rn(d[j], w[j])), rstd_y2);
                    }
                }
                p.dy[out] = pack8(d);
            }
        }
        __syncthreads();  // the stage has been read
        const int64_t next = t + static_cast<int64_t>(p.stages) * step;
        if (tid == 0 && next < p.T && !*abort_flag) {
            ask(next, s);
            ++asked;
        }
    }
    if (tid == 0 && *abort_flag) {  // every copy must land before the CTA may exit
        const int never = 0;
        for (int i = asked > p.stages ? asked - p.stages : 0; i < asked; ++i)
            if (!mbar_wait(&full[i % p.stages], static_cast<uint32_t>(i / p.stages) & 1u, &never, p.timeout_ns))
                record_failure(p.status, kStatusTimeout, 20, -1);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = tid + v * threads;
        if (i * kVec >= cols) break;
        auto put = [&](int which, const float2(&a)[4]) {
            float4 *dst = reinterpret_cast<float4 *>(p.part + (static_cast<int64_t>(first) * kVectors + which) * p.H + col0) + 2 * i;
            dst[0] = make_float4(a[0].x, a[0].y, a[1].x, a[1].y);
            dst[1] = make_float4(a[2].x, a[2].y, a[3].x, a[3].y);
        };
        put(0, acc_w[v]);
        if (POST) put(1, acc_p[v]);
        if (GATE) put(1 + POST, acc_g[v]);
    }
    if (CTAS > 1) cluster_sync();  // no CTA leaves while the other reads its sums
}

// Columns of [parts][columns] added up in order: 32 columns a CTA, eight threads a column.
__global__ void __launch_bounds__(256) rmsnorm_columns_kernel(const float *__restrict__ part, int parts, int H, int vectors,
                                                              float *__restrict__ out0, float *__restrict__ out1,
                                                              float *__restrict__ out2) {
    __shared__ float sums[8][33];
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int lane = lane_id(), w = static_cast<int>(threadIdx.x) >> 5;
    const int64_t width = static_cast<int64_t>(vectors) * H, c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < width) {
#pragma unroll 4
        for (int i = w; i < parts; i += 8) s += __ldg(part + i * width + c);
    }
    sums[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < width) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sums[i][lane];
        const int which = static_cast<int>(c / H);
        (which == 0 ? out0 : which == 1 ? out1 : out2)[c - static_cast<int64_t>(which) * H] = s;
    }
}

namespace {

struct NormShape {
    int nv, ctas, threads, cols, stages, grid;
    size_t smem;
};

constexpr int kSmemLimit = 232448;
constexpr int kSms = 148;  // of a B200: the workspace is sized without asking a device

NormShape norm_shape(int64_t T, int64_t H, bool y, bool post, bool gate, bool dr) {
    NormShape s;
    s.ctas = H > 8192 ? 2 : 1;
    s.cols = s.ctas == 1 ? static_cast<int>(H) : static_cast<int>((H / 2 + 15) / 16 * 16);
    const int pieces = s.cols / kVec;
    s.nv = pieces <= 512 ? 1 : 2;
    s.threads = ((pieces + s.nv - 1) / s.nv + 31) / 32 * 32;
    const int fixed = kNormHeader + (1 + post + gate) * s.cols * 4, stage = (2 + y + dr) * s.cols * 2;
    s.stages = (kSmemLimit - fixed) / stage;
    if (s.stages > kNormMaxStages) s.stages = kNormMaxStages;
    s.smem = static_cast<size_t>(fixed) + static_cast<size_t>(s.stages) * stage;
    int per_sm = 512 / s.threads;
    const int fit = kSmemLimit / static_cast<int>(s.smem + 1024);
    if (per_sm > fit) per_sm = fit;
    if (per_sm < 1) per_sm = 1;
    int64_t walkers = static_cast<int64_t>(kSms / s.ctas) * per_sm;
    if (walkers > T) walkers = T;
    s.grid = static_cast<int>(walkers) * s.ctas;
    return s;
}

template <int NV, int CTAS, bool Y, bool POST, bool GATE>
dg_status_t launch_backward_impl(const NormBackwardParams &p, const NormShape &s, cudaStream_t stream) {
    auto kernel = rmsnorm_backward_kernel<NV, CTAS, Y, POST, GATE>;
    static thread_local int configured_device = -1;
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
    attr[1].val.clusterDim.x = CTAS;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

template <bool Y, bool POST, bool GATE>
dg_status_t launch_backward_shape(const NormBackwardParams &p, const NormShape &s, cudaStream_t stream) {
    if (s.ctas == 2) return launch_backward_impl<2, 2, Y, POST, GATE>(p, s, stream);
    return s.nv == 1 ? launch_backward_impl<1, 1, Y, POST, GATE>(p, s, stream)
                     : launch_backward_impl<2, 1, Y, POST, GATE>(p, s, stream);
}

}  // namespace

int64_t rmsnorm_backward_workspace(int64_t T, int64_t H, bool post, bool gate) {
    // the shape with the most walkers is the one with the smallest stages
    const NormShape s = norm_shape(T, H, false, post, gate, false);
    return static_cast<int64_t>(s.grid / s.ctas) * (1 + post + gate) * H * 4;
}

dg_status_t launch_rmsnorm_backward(const NormBackwardArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    (void)dev;
    const bool y = a.y != nullptr, post = a.post != nullptr, gate = a.gate != nullptr;
    const NormShape s = norm_shape(a.T, a.H, y, post, gate, a.dr != nullptr);
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
        if (!y) st = launch_backward_shape<false, false, false>(p, s, stream);
        else if (post) st = gate ? launch_backward_shape<true, true, true>(p, s, stream)
                                 : launch_backward_shape<true, true, false>(p, s, stream);
        else st = gate ? launch_backward_shape<true, false, true>(p, s, stream)
                       : launch_backward_shape<true, false, false>(p, s, stream);
        if (st != DG_OK) return st;
    }
    const int vectors = 1 + post + gate;
    float *second = post ? a.dpost : a.dgate;
    const int64_t width = vectors * a.H;
    return launch_pdl(rmsnorm_columns_kernel, static_cast<int>((width + 31) / 32), 256, 0, stream,
                      static_cast<const float *>(p.part), s.grid / s.ctas, p.H, vectors, a.dweight, second, a.dgate);
}

}  // namespace dg

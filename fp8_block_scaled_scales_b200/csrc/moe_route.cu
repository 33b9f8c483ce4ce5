// Routing: a token's scores over the experts to the ids and weights of its k experts, with
// per-expert counts and the balance loss, and the gradient of both.
//
// route:   s = softmax(z) or sigmoid(z) per token; key = z, or s + bias; the k largest keys,
//   the lowest index among equals, keys of -inf or NaN never; w_j = scale s_j, divided by the
//   sum of the chosen s when renormalized.  p = s (softmax) or s / sum(s) (sigmoid):
//   dprob_e = G counts_e / (k n^2),  loss = sum_e dprob_e sum_t p_te  for the n tokens that
//   reach an expert (that is G sum_e f_e P_e with f the share of the slots and P the mean p).
// route_backward, for A_j = s_j dL/ds_j of slot j:
//   softmax: dz_e = sum_{j: e_j = e} A_j + s_e (dp_e - sum_j A_j - sum_i dp_i s_i)
//   sigmoid: dz_e = (1 - s_e) (sum_{j: e_j = e} A_j + p_e (dp_e - sum_i dp_i p_i))
//   A_j = scale dw_j s_j, or, renormalized, scale v_j (dw_j - sum_i dw_i v_i), v_j = s_j / sum_i s_i,
//   whose sum is zero;  dp = dloss dprob.
//
// A warp takes a token; lane l holds experts l, l + 32, ...
#include <cuda_bf16.h>
#include <math_constants.h>

#include "dg_device.cuh"
#include "train_internal.h"

namespace dg {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr uint32_t kNoKey = 0x007FFFFFu;  // ordered(-inf): a key at or below it is not chosen
constexpr int kRouteThreads = 512;        // with the balance loss; 128 without
constexpr int kFinishCtas = 8;
constexpr int kFinishThreads = 512;

struct RouteParams {
    const void *logits;
    const float *bias;
    const uint8_t *mask;
    int64_t T;
    int G, k;
    bool bf16, sigmoid, renormalize;
    float scale;
    int32_t *ids;
    float *weights;
    // partial sums of a CTA: [grid][G] of p, [grid][G] slots, [grid] tokens
    float *part_p;
    int32_t *part_count, *part_tokens;
};

// Floats as integers of the same order; -0 must have been made +0.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}

__device__ __forceinline__ float load_score(const void *logits, bool bf16, int64_t at) {
    if (bf16) return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t *>(logits) + at)) << 16);
    return __ldg(static_cast<const float *>(logits) + at);
}

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {  // a NaN loses
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// Rows whose largest score is below this: 1 / (1 + e^-z) is e^z to far below an FP32 rounding,
// and ratios of sigmoids are those of exponentials, which do not vanish together.
constexpr float kFarBelow = -60.0f;

__device__ __forceinline__ float sigmoid_of(float z) {
    const float e = expf(-fabsf(z));
    return __fdividef(z >= 0.0f ? 1.0f : e, 1.0f + e);
}

// What p is proportional to, for a row whose largest score is `top`.
__device__ __forceinline__ float unnormalized(float z, float top, bool exponential) {
    return exponential ? expf(z - top) : sigmoid_of(z);
}

// Lane j's share of the chosen scores' sum, in FP32 without common under- or overflow; lanes
// with ok == false hold no slot.
__device__ __forceinline__ float share_of_chosen(float z, bool ok, bool sigmoid) {
    const float m = warp_max(ok ? z : -CUDART_INF_F);
    float s = 0.0f;
    if (ok) {
        if (!sigmoid || m < kFarBelow) {
            s = expf(z - m);
        } else {
            const float e = expf(-fabsf(z));
            s = (z >= 0.0f ? 1.0f : e) / (1.0f + e);
        }
    }
    return s / warp_sum(s);  // 0 / 0 where no lane holds a slot: the caller's ok is false then
}

// Among the experts whose keys lie within the FP32 error of the largest one, `near` (bit i: the
// lane's i-th expert), the one whose key is largest in FP64, the lowest index among equals.
// Two keys s + b in FP32 come that close for about one token in a hundred.
__device__ __noinline__ int choose_in_fp64(const void *logits, const float *bias, int64_t row, int G, bool bf16, bool sigmoid,
                                           uint32_t near, float top) {
    const int lane = lane_id();
    double sum = 1.0;
    if (!sigmoid) {
        sum = 0.0;
        for (int e = lane; e < G; e += 32) sum += exp(static_cast<double>(load_score(logits, bf16, row + e)) - top);
        sum = warp_sum(sum);
    }
    uint64_t best = 0;
    int at = 0x7FFFFFFF;
    while (near) {
        const int e = lane + 32 * (__ffs(near) - 1);
        near &= near - 1;
        const double z = load_score(logits, bf16, row + e);
        const double s = sigmoid ? 1.0 / (1.0 + exp(-z)) : exp(z - top) / sum;
        const double key = s + __ldg(bias + e) + 0.0;
        const uint64_t u = static_cast<uint64_t>(__double_as_longlong(key));
        const uint64_t o = (u >> 63) ? ~u : u | 0x8000000000000000ull;
        if (o > best) best = o, at = e;  // ascending e: the lowest index stays
    }
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(best >> 32));
    bool in = static_cast<uint32_t>(best >> 32) == hi && at != 0x7FFFFFFF;
    const uint32_t lo = __reduce_max_sync(kAll, in ? static_cast<uint32_t>(best) : 0u);
    in = in && static_cast<uint32_t>(best) == lo;
    return __reduce_min_sync(kAll, in ? at : 0x7FFFFFFF);
}

template <int PER, bool BIAS, bool BALANCE>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
    extern __shared__ float sums[];  // BALANCE: [warps][G] of p, then [G] counts, then the tokens
    const int lane = lane_id();
    const int warps = static_cast<int>(blockDim.x) >> 5, warp = static_cast<int>(threadIdx.x) >> 5;
    int *counts = reinterpret_cast<int *>(sums + warps * p.G);
    if (BALANCE) {
        for (int e = static_cast<int>(threadIdx.x); e <= p.G; e += static_cast<int>(blockDim.x)) counts[e] = 0;
        __syncthreads();
    }
    float psum[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) psum[i] = 0.0f;
    int tokens = 0;
    grid_dep_wait();
    grid_dep_launch_dependents();

    const int64_t stride = static_cast<int64_t>(gridDim.x) * warps;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * warps + warp; t < p.T; t += stride) {
        const bool live = !p.mask || __ldg(p.mask + t) != 0;
        int id = -1;       // lane j: slot j
        float z_id = 0.0f;
        float top = -CUDART_INF_F, sum = 1.0f;
        if (live) {
            float z[PER];
            uint32_t key[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i)
                z[i] = lane + 32 * i < p.G ? load_score(p.logits, p.bf16, t * p.G + lane + 32 * i) : -CUDART_INF_F;
#pragma unroll
            for (int i = 0; i < PER; ++i) top = fmaxf(top, z[i]);
            top = warp_max(top);
            if (top > -CUDART_INF_F) {
                if (BALANCE || BIAS || (!p.renormalize && !p.sigmoid)) {
                    const bool exponential = !p.sigmoid || (BALANCE && top < kFarBelow);
                    float q[PER];
                    sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        q[i] = unnormalized(z[i], top, exponential);
                        if (lane + 32 * i >= p.G) q[i] = 0.0f;
                        sum += q[i];
                    }
                    sum = warp_sum(sum);
                    const float r = 1.0f / sum;
                    if (BALANCE) {
#pragma unroll
                        for (int i = 0; i < PER; ++i) psum[i] += q[i] * r;
                    }
                    if (BIAS) {
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            const float s = p.sigmoid ? (exponential ? sigmoid_of(z[i]) : q[i]) : q[i] * r;
                            const float c = lane + 32 * i < p.G ? s + __ldg(p.bias + lane + 32 * i) + 0.0f : 0.0f;
                            key[i] = c == c && z[i] > -CUDART_INF_F ? ordered(c) : 0u;
                        }
                    }
                }
                if (!BIAS) {
#pragma unroll
                    for (int i = 0; i < PER; ++i) key[i] = z[i] == z[i] ? ordered(z[i] + 0.0f) : 0u;
                }
                for (int j = 0; j < p.k; ++j) {
                    uint32_t most = key[0];
#pragma unroll
                    for (int i = 1; i < PER; ++i) most = max(most, key[i]);
                    most = __reduce_max_sync(kAll, most);
                    if (most <= kNoKey) break;
                    int at = 0x7FFFFFFF;
                    if (BIAS) {
                        const float f = from_ordered(most);
                        // keys are off by less than 2^-18 max(1, |key|): 2^-22 in s (37 additions
                        // of softmax's sum among them) and a rounding of s + b
                        const float least = f - 0x1p-17f * fminf(fmaxf(1.0f, fabsf(f)), 0x1p126f);
                        const uint32_t u = max(ordered(least + 0.0f), kNoKey + 1u);
                        uint32_t near = 0;
#pragma unroll
                        for (int i = 0; i < PER; ++i) near |= key[i] >= u ? 1u << i : 0u;
                        const uint32_t lanes = __ballot_sync(kAll, near != 0);
                        const bool several = (lanes & (lanes - 1)) != 0 || __any_sync(kAll, (near & (near - 1)) != 0);
                        if (several)
                            at = choose_in_fp64(p.logits, p.bias, t * p.G, p.G, p.bf16, p.sigmoid, near, top);
                        else
                            at = __shfl_sync(kAll, lane + 32 * (__ffs(near) - 1), __ffs(lanes) - 1);
                    } else {
#pragma unroll
                        for (int i = PER - 1; i >= 0; --i)
                            if (key[i] == most) at = lane + 32 * i;
                        at = __reduce_min_sync(kAll, at);
                    }
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        if (lane + 32 * i == at) key[i] = 0u;
                    if (lane == j) id = at;
                }
            }
        }
        const bool ok = id >= 0;
        if (ok) z_id = load_score(p.logits, p.bf16, t * p.G + id);
        const bool routed = __any_sync(kAll, ok);
        float w = 0.0f;
        if (routed) {
            if (p.renormalize) {
                w = share_of_chosen(z_id, ok, p.sigmoid);
            } else if (p.sigmoid) {
                const float e = expf(-fabsf(z_id));
                w = (z_id >= 0.0f ? 1.0f : e) / (1.0f + e);
            } else {
                w = expf(z_id - top) / sum;
            }
        }
        if (lane < p.k) {
            p.ids[t * p.k + lane] = id;
            p.weights[t * p.k + lane] = ok ? w * p.scale : 0.0f;
        }
        if (BALANCE) {
            if (ok) atomicAdd(&counts[id], 1);
            tokens += routed ? 1 : 0;
        }
    }
    if (BALANCE) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 32 * i < p.G) sums[warp * p.G + lane + 32 * i] = psum[i];
        if (lane == 0) atomicAdd(&counts[p.G], tokens);
        __syncthreads();
        const int64_t at = static_cast<int64_t>(blockIdx.x) * p.G;
        for (int e = static_cast<int>(threadIdx.x); e < p.G; e += static_cast<int>(blockDim.x)) {
            float s = 0.0f;
            for (int w = 0; w < warps; ++w) s += sums[w * p.G + e];
            p.part_p[at + e] = s;
            p.part_count[at + e] = counts[e];
        }
        if (threadIdx.x == 0) p.part_tokens[blockIdx.x] = counts[p.G];
    }
}

// The CTAs' sums to counts, dprob and the loss: one cluster, each CTA a share of the experts,
// 16 threads an expert (parts in turn), FP64 sums in a fixed order.
__global__ void __cluster_dims__(kFinishCtas, 1, 1) __launch_bounds__(kFinishThreads)
    route_finish_kernel(const float *__restrict__ part_p, const int32_t *__restrict__ part_count,
                        const int32_t *__restrict__ part_tokens, int parts, int G, int k,
                        int32_t *__restrict__ counts, float *__restrict__ loss, float *__restrict__ dprob) {
    __shared__ double warp_loss[kFinishThreads / 32], cta_loss;
    __shared__ int warp_tokens[kFinishThreads / 32];
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int tid = static_cast<int>(threadIdx.x), lane = lane_id(), warp = tid >> 5;
    int n = 0;
    for (int i = tid; i < parts; i += kFinishThreads) n += __ldg(part_tokens + i);
    n = warp_sum(n);
    if (lane == 0) warp_tokens[warp] = n;
    __syncthreads();
    n = 0;
    for (int i = 0; i < kFinishThreads / 32; ++i) n += warp_tokens[i];
    const double nd = n > 0 ? static_cast<double>(n) : 1.0;
    const double unit = static_cast<double>(G) / (static_cast<double>(k) * nd * nd);

    // lane: expert lane % 8 of the warp's eight, parts lane / 8, + 4, ...
    double mine = 0.0;
    const int rank = static_cast<int>(cluster_ctarank());
    for (int e0 = (rank * (kFinishThreads / 32) + warp) * 8; e0 < G; e0 += kFinishCtas * (kFinishThreads / 32) * 8) {
        const int e = e0 + (lane & 7);
        double s = 0.0;
        int c = 0;
        if (e < G) {
#pragma unroll 4
            for (int i = lane >> 3; i < parts; i += 4) {
                s += static_cast<double>(__ldg(part_p + static_cast<int64_t>(i) * G + e));
                c += __ldg(part_count + static_cast<int64_t>(i) * G + e);
            }
        }
        s += __shfl_xor_sync(kAll, s, 8);
        s += __shfl_xor_sync(kAll, s, 16);
        c += __shfl_xor_sync(kAll, c, 8);
        c += __shfl_xor_sync(kAll, c, 16);
        if (e < G && lane < 8) {
            const double d = unit * c;
            counts[e] = c;
            dprob[e] = static_cast<float>(d);
            mine += d * s;
        }
    }
    mine = warp_sum(mine);
    if (lane == 0) warp_loss[warp] = mine;
    __syncthreads();
    if (tid == 0) {
        double s = 0.0;
        for (int i = 0; i < kFinishThreads / 32; ++i) s += warp_loss[i];
        cta_loss = s;
    }
    cluster_sync();
    if (rank == 0 && tid == 0) {
        double s = 0.0;
        for (int r = 0; r < kFinishCtas; ++r) {
            double v;
            asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(mapa_shared(smem_u32(&cta_loss), r)) : "memory");
            s += v;
        }
        *loss = static_cast<float>(s);
    }
    cluster_sync();  // no CTA leaves while rank 0 reads its sum
}

struct RouteBackwardParams {
    const void *logits;
    const int32_t *ids;
    const float *dweights, *dprob, *dloss;
    int64_t T;
    int G, k;
    bool bf16, sigmoid, renormalize;
    float scale;
    void *dlogits;
};

__device__ __forceinline__ void store_score(void *out, bool bf16, int64_t at, float v) {
    if (bf16)
        static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16(v);
    else
        static_cast<float *>(out)[at] = v;
}

// ROWS: every expert's score matters (the balance loss, or softmax without renormalization);
// otherwise only the chosen experts have a gradient, and only their scores are read.
template <int PER, bool ROWS>
__global__ void __launch_bounds__(256) route_backward_kernel(const RouteBackwardParams p) {
    const int lane = lane_id();
    const int warps = static_cast<int>(blockDim.x) >> 5, warp = static_cast<int>(threadIdx.x) >> 5;
    grid_dep_wait();
    grid_dep_launch_dependents();
    float dp[PER];
    const float dloss = p.dprob ? __ldg(p.dloss) : 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) dp[i] = p.dprob && lane + 32 * i < p.G ? __ldg(p.dprob + lane + 32 * i) * dloss : 0.0f;

    const int64_t stride = static_cast<int64_t>(gridDim.x) * warps;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * warps + warp; t < p.T; t += stride) {
        const int64_t row = t * p.G;
        const int id = lane < p.k ? __ldg(p.ids + t * p.k + lane) : -1;
        const bool ok = id >= 0 && id < p.G;
        const bool routed = __any_sync(kAll, ok);
        float z[PER];
        if (ROWS) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                z[i] = lane + 32 * i < p.G ? load_score(p.logits, p.bf16, row + lane + 32 * i) : -CUDART_INF_F;
        }
        const float z_id = ok ? load_score(p.logits, p.bf16, row + id) : 0.0f;
        const float dw = ok && p.dweights ? __ldg(p.dweights + t * p.k + lane) : 0.0f;
        float top = -CUDART_INF_F, r = 0.0f, base = 0.0f;
        bool exponential = !p.sigmoid;
        float q[PER];
        if (ROWS && routed) {
#pragma unroll
            for (int i = 0; i < PER; ++i) top = fmaxf(top, z[i]);
            top = warp_max(top);
            exponential = exponential || top < kFarBelow;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                q[i] = unnormalized(z[i], top, exponential);
                if (lane + 32 * i >= p.G) q[i] = 0.0f;
                sum += q[i];
            }
            r = 1.0f / warp_sum(sum);
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) dot += dp[i] * (q[i] * r);
            base = warp_sum(dot);
        }
        float a = 0.0f;  // lane j: A_j
        if (routed) {
            if (p.renormalize) {
                const float v = share_of_chosen(z_id, ok, p.sigmoid);
                const float mean = warp_sum(ok ? dw * v : 0.0f);
                a = ok ? p.scale * v * (dw - mean) : 0.0f;
            } else {
                float s;
                if (p.sigmoid) {
                    const float e = expf(-fabsf(z_id));
                    s = (z_id >= 0.0f ? 1.0f : e) / (1.0f + e);
                } else {
                    s = expf(z_id - top) * r;
                }
                a = ok ? p.scale * dw * s : 0.0f;
                if (!p.sigmoid) base += warp_sum(a);
            }
        }
        // every expert's part, then the chosen ones' whole gradient over it
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            float v = 0.0f;
            if (ROWS && routed) {
                v = q[i] * r * (dp[i] - base);
                if (p.sigmoid) v *= sigmoid_of(-z[i]);
            }
            if (lane + 32 * i < p.G) store_score(p.dlogits, p.bf16, row + lane + 32 * i, v);
        }
        if (routed) {
            // an expert that a token names twice gets both slots' parts
            const uint32_t same = __match_any_sync(kAll, ok ? id : -1 - lane);
            if (__any_sync(kAll, (same & (same - 1)) != 0)) {
                float both = 0.0f;
                for (int j = 0; j < 32; ++j) {
                    const float other = __shfl_sync(kAll, a, j);
                    if ((same >> j) & 1u) both += other;
                }
                a = both;
            }
            float v = a;
            if (ROWS && ok) {
                const float d = p.dprob ? __ldg(p.dprob + id) * dloss : 0.0f;
                v += unnormalized(z_id, top, exponential) * r * (d - base);
            }
            if (p.sigmoid) v *= sigmoid_of(-z_id);
            __syncwarp();  // the row's stores come first
            if (ok) store_score(p.dlogits, p.bf16, row + id, v);
        }
    }
}

// --------------------------------------------------------------------------- launchers
static int route_grid(int64_t T, const DeviceInfo &dev) {
    const int64_t want = (T + kRouteThreads / 32 - 1) / (kRouteThreads / 32), most = 2 * dev.num_sms;
    return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

// The partial sums of at most two CTAs per SM; SMs of a B200, since no device is asked here.
int64_t route_workspace(int64_t T, int G) {
    DeviceInfo dev = {};
    dev.num_sms = 148;
    return static_cast<int64_t>(route_grid(T, dev)) * (G * 8 + 4);
}

template <int PER, bool BIAS, bool BALANCE>
static dg_status_t launch_route_impl(const RouteParams &p, int grid, int threads, cudaStream_t stream) {
    auto kernel = route_kernel<PER, BIAS, BALANCE>;
    const size_t smem = BALANCE ? (static_cast<size_t>(threads / 32) * p.G + p.G + 1) * 4 : 0;
    if (smem > 48 * 1024) {
        static thread_local int configured_device = -1;
        const dg_status_t st = allow_smem(kernel, (static_cast<size_t>(kRouteThreads / 32) * 1024 + 1025) * 4, configured_device);
        if (st != DG_OK) return st;
    }
    return launch_pdl(kernel, grid, threads, smem, stream, p);
}

template <int PER>
static dg_status_t launch_route_per(const RouteParams &p, bool balance, int grid, int threads, cudaStream_t stream) {
    if (p.bias)
        return balance ? launch_route_impl<PER, true, true>(p, grid, threads, stream)
                       : launch_route_impl<PER, true, false>(p, grid, threads, stream);
    return balance ? launch_route_impl<PER, false, true>(p, grid, threads, stream)
                   : launch_route_impl<PER, false, false>(p, grid, threads, stream);
}

dg_status_t launch_route(const RouteArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    const bool balance = a.counts != nullptr;
    RouteParams p = {};
    p.logits = a.logits;
    p.bias = a.bias;
    p.mask = a.mask;
    p.T = a.T;
    p.G = a.G;
    p.k = a.k;
    p.bf16 = a.bf16;
    p.sigmoid = a.sigmoid;
    p.renormalize = a.renormalize;
    p.scale = a.scale;
    p.ids = a.ids;
    p.weights = a.weights;
    int grid, threads;
    if (balance) {
        DeviceInfo sized = dev;
        sized.num_sms = 148;  // as route_workspace counts
        grid = route_grid(a.T, sized);
        threads = kRouteThreads;
        p.part_p = static_cast<float *>(a.workspace);
        p.part_count = reinterpret_cast<int32_t *>(p.part_p + static_cast<int64_t>(grid) * a.G);
        p.part_tokens = p.part_count + static_cast<int64_t>(grid) * a.G;
    } else {
        threads = 128;
        const int64_t want = (a.T + 3) / 4, most = 16 * static_cast<int64_t>(dev.num_sms);
        grid = static_cast<int>(want < most ? want : most);
    }
    dg_status_t st;
    if (a.G <= 32) st = launch_route_per<1>(p, balance, grid, threads, stream);
    else if (a.G <= 64) st = launch_route_per<2>(p, balance, grid, threads, stream);
    else if (a.G <= 128) st = launch_route_per<4>(p, balance, grid, threads, stream);
    else if (a.G <= 256) st = launch_route_per<8>(p, balance, grid, threads, stream);
    else if (a.G <= 512) st = launch_route_per<16>(p, balance, grid, threads, stream);
    else st = launch_route_per<32>(p, balance, grid, threads, stream);
    if (st != DG_OK || !balance) return st;
    return launch_pdl(route_finish_kernel, kFinishCtas, kFinishThreads, 0, stream, static_cast<const float *>(p.part_p),
                      static_cast<const int32_t *>(p.part_count), static_cast<const int32_t *>(p.part_tokens), grid, a.G,
                      a.k, a.counts, a.loss, a.dprob);
}

template <int PER>
static dg_status_t launch_route_backward_per(const RouteBackwardParams &p, int grid, cudaStream_t stream) {
    if (p.dprob || (!p.sigmoid && !p.renormalize))
        return launch_pdl(route_backward_kernel<PER, true>, grid, 256, 0, stream, p);
    return launch_pdl(route_backward_kernel<PER, false>, grid, 256, 0, stream, p);
}

dg_status_t launch_route_backward(const RouteBackwardArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    RouteBackwardParams p = {a.logits, a.ids, a.dweights, a.dprob, a.dloss, a.T, a.G, a.k,
                             a.bf16, a.sigmoid, a.renormalize, a.scale, a.dlogits};
    const int64_t want = (a.T + 7) / 8, most = 8 * static_cast<int64_t>(dev.num_sms);
    const int grid = static_cast<int>(want < most ? want : most);
    if (a.G <= 32) return launch_route_backward_per<1>(p, grid, stream);
    if (a.G <= 64) return launch_route_backward_per<2>(p, grid, stream);
    if (a.G <= 128) return launch_route_backward_per<4>(p, grid, stream);
    if (a.G <= 256) return launch_route_backward_per<8>(p, grid, stream);
    if (a.G <= 512) return launch_route_backward_per<16>(p, grid, stream);
    return launch_route_backward_per<32>(p, grid, stream);
}

}  // namespace dg

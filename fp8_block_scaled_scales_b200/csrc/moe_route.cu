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

__device__ __forceinline__ float warp_max(float v) {  // a NaN loses against anything, alone it is -inf
    return from_ordered(__reduce_max_sync(kAll, ordered(fmaxf(v, -CUDART_INF_F) + 0.0f)));
}

__device__ __forceinline__ float reciprocal(float x) {  // within one unit; 0 for 2^126 and more
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Rows whose largest score is below this: 1 / (1 + e^-z) is e^z to far below an FP32 rounding,
// and ratios of sigmoids are those of exponentials, which do not vanish together.
constexpr float kFarBelow = -60.0f;

// e^x, for sums over a row and for keys: the argument's product and the hardware's approximation are
// off by 2 + 1.2 |x| units of the last place; 0 below 2^-126.
__device__ __forceinline__ float exp_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504f));  // log2(e)
    return r;
}

__device__ __forceinline__ float sigmoid_fast(float z) { return reciprocal(1.0f + exp_fast(-z)); }

// What p is proportional to, for a row whose largest score is `top`.
__device__ __forceinline__ float unnormalized(float z, float top, bool exponential) {
    return exponential ? exp_fast(z - top) : sigmoid_fast(z);
}

__device__ __forceinline__ float sigmoid_of(float z) {
    const float e = expf(-fabsf(z));
    return (z >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// Lane j's share of the chosen scores' sum, in FP32 without common under- or overflow; lanes
// with ok == false hold no slot.
__device__ __forceinline__ float share_of_chosen(float z, bool ok, bool sigmoid) {
    const float m = warp_max(ok ? z : -CUDART_INF_F);
    float s = 0.0f;
    if (ok) s = !sigmoid || m < kFarBelow ? expf(z - m) : sigmoid_of(z);
    return s / warp_sum(s);  // 0 / 0 where no lane holds a slot: the caller's ok is false then
}

// A key in FP64: z itself without a bias (top and sum: of a row's exponentials).
template <bool BIAS>
__device__ __forceinline__ double exact_key(float z, const float *bias, int e, bool sigmoid, double top, double sum) {
    double key = z;
    if (BIAS) key = (sigmoid ? 1.0 / (1.0 + exp(-key)) : exp(key - top) / sum) + __ldg(bias + e);
    return key + 0.0;  // -0 is +0
}

__device__ __forceinline__ void exact_sum(const void *logits, int64_t row, int G, bool bf16, double &top, double &sum) {
    float m = -CUDART_INF_F;
    for (int e = lane_id(); e < G; e += 32) m = fmaxf(m, load_score(logits, bf16, row + e));
    top = warp_max(m);
    sum = 0.0;
    for (int e = lane_id(); e < G; e += 32) sum += exp(load_score(logits, bf16, row + e) - top);
    sum = warp_sum(sum);
}

// Lanes below n hold the candidates, no other expert comes before any of them: their order by FP64
// keys, the lowest id among equals.
template <bool BIAS>
__device__ __noinline__ int order_exactly(const void *logits, const float *bias, int64_t row, int G, bool bf16, bool sigmoid,
                                          int id, int n) {
    const int lane = lane_id();
    double top = 0.0, sum = 1.0;
    if (BIAS && !sigmoid) exact_sum(logits, row, G, bf16, top, sum);
    double key = 0.0;
    if (lane < n) key = exact_key<BIAS>(load_score(logits, bf16, row + id), bias, id, sigmoid, top, sum);
    int rank = 0;
    for (int i = 0; i < n; ++i) {
        const double other = __shfl_sync(kAll, key, i);
        const int e = __shfl_sync(kAll, id, i);
        rank += other > key || (other == key && e < id) ? 1 : 0;
    }
    int sorted = -1;
    for (int i = 0; i < n; ++i) {
        const int r = __shfl_sync(kAll, rank, i), e = __shfl_sync(kAll, id, i);
        if (r == lane) sorted = e;
    }
    return sorted;
}

// The choice among all experts by FP64 keys, for rows with more near keys than a warp has lanes:
// lane j returns slot j's expert or -1.
template <int PER, bool BIAS>
__device__ __noinline__ int choose_exactly(const void *logits, const float *bias, int64_t row, int G, int k, bool bf16,
                                           bool sigmoid) {
    const int lane = lane_id();
    double top = 0.0, sum = 1.0;
    if (BIAS && !sigmoid) exact_sum(logits, row, G, bf16, top, sum);
    uint64_t keys[PER];
#pragma unroll 1
    for (int i = 0; i < PER; ++i) {
        keys[i] = 0;
        const int e = lane + 32 * i;
        if (e >= G) continue;
        const float z = load_score(logits, bf16, row + e);
        const double key = exact_key<BIAS>(z, bias, e, sigmoid, top, sum);
        const uint64_t u = static_cast<uint64_t>(__double_as_longlong(key));
        if (z > -CUDART_INF_F && key > -CUDART_INF) keys[i] = (u >> 63) ? ~u : u | 0x8000000000000000ull;
    }
    int id = -1;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
        uint64_t best = 0;
        int at = 0x7FFFFFFF;
#pragma unroll 1
        for (int i = 0; i < PER; ++i)
            if (keys[i] > best) best = keys[i], at = i;  // ascending: the lowest id stays
        const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(best >> 32));
        if (hi == 0) break;
        bool in = static_cast<uint32_t>(best >> 32) == hi;
        const uint32_t lo = __reduce_max_sync(kAll, in ? static_cast<uint32_t>(best) : 0u);
        in = in && static_cast<uint32_t>(best) == lo;
        const int e = __reduce_min_sync(kAll, in ? lane + 32 * at : 0x7FFFFFFF);
        if (in && lane + 32 * at == e) keys[at] = 0;
        if (lane == j) id = e;
    }
    return id;
}

// Descending order of a lane's keys (odd-even merge sort, K. E. Batcher, "Sorting networks and
// their applications", 1968): a minimum and a maximum per comparator.
template <int N>
__device__ __forceinline__ void sort_descending(uint32_t (&v)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t a = v[i + j], b = v[i + j + q];
                        v[i + j] = max(a, b);
                        v[i + j + q] = min(a, b);
                    }
}

// A warp chooses by 32-bit keys whose low bits are the expert's id, inverted: one maximum over the
// warp gives key and id, the lowest id among equals, and no two keys are the same.  The id takes the place of
// the key's last 5 to 10 bits, so the choice is settled only where neighbours in the order differ
// by more than those (and, with a bias, by more than the key's own FP32 error); otherwise (a token
// in thirty) the candidates are put in order by FP64 keys.  BF16 logits without a bias have the bits to spare.
// 16384 tokens x 256 experts, k = 8, with bias and balance loss: see launch_route.
constexpr int route_max_threads(int per) { return per <= 8 ? 1024 : 512; }

template <int PER, bool BIAS, bool BALANCE>
__global__ void __launch_bounds__(route_max_threads(PER)) route_kernel(const RouteParams p) {
    extern __shared__ float sums[];  // BALANCE: [warps][G] of p, then [G] counts, then the tokens
    constexpr uint32_t kIdBits = 32 * PER - 1;
    const int lane = lane_id();
    const int warps = static_cast<int>(blockDim.x) >> 5, warp = static_cast<int>(threadIdx.x) >> 5;
    int *counts = reinterpret_cast<int *>(sums + warps * p.G);
    if (BALANCE) {
        for (int e = static_cast<int>(threadIdx.x); e <= p.G; e += static_cast<int>(blockDim.x)) counts[e] = 0;
        __syncthreads();
    }
    grid_dep_wait();
    grid_dep_launch_dependents();
    float psum[PER], b[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        psum[i] = 0.0f;
        b[i] = (BIAS && lane + 32 * i < p.G ? __ldg(p.bias + lane + 32 * i) : 0.0f) + 0.0f;
    }
    const bool exact_keys = !BIAS && p.bf16;
    const int rounds = exact_keys || p.k == p.G ? p.k : p.k + 1;  // the next one too: is the last one settled?
    int tokens = 0;

    const int64_t stride = static_cast<int64_t>(gridDim.x) * warps;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * warps + warp; t < p.T; t += stride) {
        const int64_t row = t * p.G;
        int id = -1;  // lane j: slot j
        float top = 0.0f, sum = 1.0f;
        if (!p.mask || __ldg(p.mask + t) != 0) {
            float z[PER];
            uint32_t key[PER];
            if (p.bf16) {
                const uint16_t *at = static_cast<const uint16_t *>(p.logits) + row + lane;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    z[i] = lane + 32 * i < p.G ? __uint_as_float(static_cast<uint32_t>(__ldg(at + 32 * i)) << 16) : -CUDART_INF_F;
            } else {
                const float *at = static_cast<const float *>(p.logits) + row + lane;
#pragma unroll
                for (int i = 0; i < PER; ++i) z[i] = lane + 32 * i < p.G ? __ldg(at + 32 * i) : -CUDART_INF_F;
            }
            // the id goes under the key's high bits; 0 for an expert that is not chosen
            auto keyed = [&](float c, bool able, int i) {
                const uint32_t id_bits = kIdBits - static_cast<uint32_t>(lane + 32 * i);
                return able ? (ordered(c) & ~kIdBits) | id_bits : 0u;
            };
            if (BALANCE || BIAS || (!p.renormalize && !p.sigmoid)) {
                float q[PER];
                auto exponentials = [&] {
                    top = -CUDART_INF_F;
#pragma unroll
                    for (int i = 0; i < PER; ++i) top = fmaxf(top, z[i]);
                    top = warp_max(top);
                    sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        q[i] = exp_fast(z[i] - top);  // 0 past the last expert; NaN in a row without a score
                        sum += q[i];
                    }
                    sum = warp_sum(sum);
                };
                if (p.sigmoid) {
                    sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        q[i] = sigmoid_fast(z[i]);
                        sum += q[i];
                    }
                    if (BIAS) {
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            const float c = q[i] + b[i];  // never -0: b is not
                            key[i] = keyed(c, z[i] > -CUDART_INF_F && c > -CUDART_INF_F, i);
                        }
                    }
                    if (BALANCE) {
                        sum = warp_sum(sum);
                        if (sum < 0x1p-80f) exponentials();  // all far below 0: ratios of exponentials
                    }
                } else {
                    exponentials();
                    if (BIAS) {
                        const float r = reciprocal(sum);
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            const float c = fmaf(q[i], r, b[i]);
                            key[i] = keyed(c, z[i] > -CUDART_INF_F && c > -CUDART_INF_F, i);
                        }
                    }
                }
                if (BALANCE) {
                    const float r = reciprocal(sum);
                    if (top > -CUDART_INF_F) {  // for sigmoids 0, unless no expert has a score
#pragma unroll
                        for (int i = 0; i < PER; ++i) psum[i] = fmaf(q[i], r, psum[i]);
                    }
                }
            }
            if (!BIAS) {
#pragma unroll
                for (int i = 0; i < PER; ++i) key[i] = keyed(z[i] + 0.0f, z[i] > -CUDART_INF_F, i);
            }
            sort_descending(key);
            uint32_t mine = 0u, prev = 0u, last = 0u;  // lane j: the j-th largest; the last two of them
            int found = 0;
            auto next = [&] {
                prev = last;
                last = __reduce_max_sync(kAll, key[0]);
                if (lane == found) mine = last;
                ++found;
                if (key[0] == last) {
#pragma unroll
                    for (int i = 0; i + 1 < PER; ++i) key[i] = key[i + 1];
                    key[PER - 1] = 0u;
                }
            };
            // whether b may come before a, its predecessor in the order of the 32-bit keys
            auto unsettled = [&](uint32_t a, uint32_t b) {
                if (b == 0u) return false;
                if (!BIAS) return (a ^ b) <= kIdBits;
                // keys are off by less than 2^-18 max(1, |key|): 2^-21 in s (37 additions of softmax's
                // sum among them) and a rounding of s + b
                const float x = from_ordered(a & ~kIdBits), y = from_ordered(b | kIdBits);
                return !(x - y > 0x1p-17f * fmaxf(1.0f, fabsf(x)));  // infinite keys too
            };
            while (found < rounds) next();
            if (!exact_keys) {
                uint32_t below = __shfl_down_sync(kAll, mine, 1);
                if (lane == p.k - 1) below = p.k == p.G ? 0u : last;
                if (__any_sync(kAll, lane < p.k && unsettled(mine, below))) {
                    // more candidates, until the next one certainly comes after them
                    while (p.k < p.G && found < 32 && unsettled(prev, last)) next();
                    const int n = p.k == p.G ? p.k : found - 1;
                    const uint32_t held = __ballot_sync(kAll, lane < n && mine != 0u);
                    id = static_cast<int>(kIdBits - (mine & kIdBits));
                    if (p.k == p.G || !unsettled(prev, last))
                        id = order_exactly<BIAS>(p.logits, p.bias, row, p.G, p.bf16, p.sigmoid, id, __popc(held));
                    else
                        id = choose_exactly<PER, BIAS>(p.logits, p.bias, row, p.G, p.k, p.bf16, p.sigmoid);
                    if (lane >= p.k) id = -1;
                } else if (lane < p.k && mine != 0u) {
                    id = static_cast<int>(kIdBits - (mine & kIdBits));
                }
            } else if (lane < p.k && mine != 0u) {
                id = static_cast<int>(kIdBits - (mine & kIdBits));
            }
        }
        const bool ok = id >= 0;
        const bool routed = __any_sync(kAll, ok);
        float w = 0.0f;
        if (routed) {
            const float z = ok ? load_score(p.logits, p.bf16, row + id) : 0.0f;
            if (p.renormalize)
                w = share_of_chosen(z, ok, p.sigmoid);
            else
                w = p.sigmoid ? sigmoid_of(z) : expf(z - top) / sum;
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

// The CTAs' sums to counts, dprob and the loss: one cluster; a CTA takes 32 experts at a time, a lane
// each, and its warps share the parts.  FP64 sums in a fixed order.
__global__ void __cluster_dims__(kFinishCtas, 1, 1) __launch_bounds__(kFinishThreads)
    route_finish_kernel(const float *__restrict__ part_p, const int32_t *__restrict__ part_count,
                        const int32_t *__restrict__ part_tokens, int parts, int G, int k,
                        int32_t *__restrict__ counts, float *__restrict__ loss, float *__restrict__ dprob) {
    constexpr int kWarps = kFinishThreads / 32;
    __shared__ double warp_p[kWarps][32], cta_loss;
    __shared__ int warp_count[kWarps][32], warp_tokens[kWarps];
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int tid = static_cast<int>(threadIdx.x), lane = lane_id(), warp = tid >> 5;
    const int rank = static_cast<int>(cluster_ctarank());
    int n = 0;
    for (int i = tid; i < parts; i += kFinishThreads) n += __ldg(part_tokens + i);
    n = warp_sum(n);
    if (lane == 0) warp_tokens[warp] = n;

    double mine = 0.0, unit = 0.0;
    for (int e0 = rank * 32; e0 < G; e0 += kFinishCtas * 32) {
        const int e = e0 + lane;
        double s = 0.0;
        int c = 0;
        if (e < G) {
            constexpr int kDeep = 10;  // loads in flight: 148 parts over 16 warps
            for (int i0 = warp; i0 < parts; i0 += kDeep * kWarps) {
                float v[kDeep];
                int w[kDeep];
#pragma unroll
                for (int j = 0; j < kDeep; ++j) {
                    const int i = i0 + j * kWarps;
                    v[j] = i < parts ? __ldg(part_p + static_cast<int64_t>(i) * G + e) : 0.0f;
                    w[j] = i < parts ? __ldg(part_count + static_cast<int64_t>(i) * G + e) : 0;
                }
#pragma unroll
                for (int j = 0; j < kDeep; ++j) {
                    s += static_cast<double>(v[j]);
                    c += w[j];
                }
            }
        }
        warp_p[warp][lane] = s;
        warp_count[warp][lane] = c;
        __syncthreads();
        if (warp == 0) {
            n = 0;
            s = 0.0;
            c = 0;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                n += warp_tokens[i];
                s += warp_p[i][lane];
                c += warp_count[i][lane];
            }
            const double nd = n > 0 ? static_cast<double>(n) : 1.0;
            unit = static_cast<double>(G) / (static_cast<double>(k) * nd * nd);
            if (e < G) {
                const double d = unit * c;
                counts[e] = c;
                dprob[e] = static_cast<float>(d);
                mine += d * s;
            }
        }
        __syncthreads();
    }
    if (warp == 0) {
        mine = warp_sum(mine);
        if (lane == 0) cta_loss = mine;
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
__global__ void __launch_bounds__(256, PER <= 8 ? 4 : 1) route_backward_kernel(const RouteBackwardParams p) {
    const int lane = lane_id();
    const int warps = static_cast<int>(blockDim.x) >> 5, warp = static_cast<int>(threadIdx.x) >> 5;
    grid_dep_wait();
    grid_dep_launch_dependents();
    float dp[PER];
    const float dloss = ROWS && p.dprob ? __ldg(p.dloss) : 0.0f;
    if (ROWS) {
#pragma unroll
        for (int i = 0; i < PER; ++i) dp[i] = p.dprob && lane + 32 * i < p.G ? __ldg(p.dprob + lane + 32 * i) * dloss : 0.0f;
    }

    const int64_t stride = static_cast<int64_t>(gridDim.x) * warps;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * warps + warp; t < p.T; t += stride) {
        const int64_t row = t * p.G;
        const int id = lane < p.k ? __ldg(p.ids + t * p.k + lane) : -1;
        const float given = lane < p.k && p.dweights ? __ldg(p.dweights + t * p.k + lane) : 0.0f;
        float q[PER], ns[PER];  // what p is proportional to, and 1 - sigmoid
        if (ROWS) {
            if (p.bf16) {
                const uint16_t *at = static_cast<const uint16_t *>(p.logits) + row + lane;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    q[i] = lane + 32 * i < p.G ? __uint_as_float(static_cast<uint32_t>(__ldg(at + 32 * i)) << 16) : -CUDART_INF_F;
            } else {
                const float *at = static_cast<const float *>(p.logits) + row + lane;
#pragma unroll
                for (int i = 0; i < PER; ++i) q[i] = lane + 32 * i < p.G ? __ldg(at + 32 * i) : -CUDART_INF_F;
            }
        }
        const bool ok = id >= 0 && id < p.G;
        const float z_id = ok ? load_score(p.logits, p.bf16, row + id) : 0.0f;
        const bool routed = __any_sync(kAll, ok);
        const float dw = ok ? given : 0.0f;
        float top = -CUDART_INF_F, r = 0.0f, base = 0.0f;
        bool exponential = !p.sigmoid;
        if (ROWS && routed) {
            float sum = 0.0f, dot = 0.0f;
            if (!exponential) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const float z = q[i], e = fminf(exp_fast(-z), 0x1p125f);  // the bound: e times its reciprocal is 1
                    q[i] = reciprocal(1.0f + e);
                    ns[i] = e * q[i];
                    if (z == -CUDART_INF_F) q[i] = 0.0f;  // an expert that is left out, or none
                    sum += q[i];
                    dot = fmaf(dp[i], q[i], dot);
                    top = fmaxf(top, z);
                }
                sum = warp_sum(sum);
                exponential = sum < 0x1p-80f;
                if (exponential) {  // all far below 0: ratios of exponentials
                    sum = dot = 0.0f;
                    top = warp_max(top);
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const float z = lane + 32 * i < p.G ? load_score(p.logits, p.bf16, row + lane + 32 * i) : -CUDART_INF_F;
                        q[i] = exp_fast(z - top);
                        sum += q[i];
                        dot = fmaf(dp[i], q[i], dot);
                    }
                    sum = warp_sum(sum);
                }
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i) top = fmaxf(top, q[i]);
                top = warp_max(top);
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    q[i] = exp_fast(q[i] - top);
                    sum += q[i];
                    dot = fmaf(dp[i], q[i], dot);
                }
                sum = warp_sum(sum);
            }
            r = 1.0f / sum;
            if (p.dprob) base = warp_sum(dot) * r;
        }
        float a = 0.0f;  // lane j: A_j
        if (routed) {
            if (p.renormalize) {
                const float v = share_of_chosen(z_id, ok, p.sigmoid);
                const float mean = warp_sum(ok ? dw * v : 0.0f);
                a = ok ? p.scale * v * (dw - mean) : 0.0f;
            } else {
                const float s = p.sigmoid ? sigmoid_of(z_id) : expf(z_id - top) * r;
                a = ok ? p.scale * dw * s : 0.0f;
                if (!p.sigmoid) base += warp_sum(a);
            }
        }
        // every expert's part, then the chosen ones' whole gradient over it
        float v[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            v[i] = 0.0f;
            if (ROWS && routed) {
                v[i] = q[i] * r * (dp[i] - base);
                if (p.sigmoid) v[i] *= ns[i];
            }
        }
        if (p.bf16) {
            __nv_bfloat16 *at = static_cast<__nv_bfloat16 *>(p.dlogits) + row + lane;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 32 * i < p.G) at[32 * i] = __float2bfloat16(v[i]);
        } else {
            float *at = static_cast<float *>(p.dlogits) + row + lane;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 32 * i < p.G) at[32 * i] = v[i];
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
            float g = a;
            if (ROWS && ok) {
                const float d = p.dprob ? __ldg(p.dprob + id) * dloss : 0.0f;
                g += unnormalized(z_id, top, exponential) * r * (d - base);
            }
            if (p.sigmoid) {
                const float e = fminf(exp_fast(-z_id), 0x1p125f);
                g *= e * reciprocal(1.0f + e);
            }
            __syncwarp();  // the row's stores come first
            if (ok) store_score(p.dlogits, p.bf16, row + id, g);
        }
    }
}

// --------------------------------------------------------------------------- launchers
namespace {

constexpr int kSms = 148;  // of a B200: the workspace is sized without asking a device

int per_lane(int G) {
    int per = 1;
    while (32 * per < G) per *= 2;
    return per;
}

struct RouteShape {
    int threads, grid;
};

// A CTA per SM with as many warps as there are tokens for, up to 32: fewer parts to add up.
RouteShape balance_shape(int64_t T, int G) {
    const int64_t most = route_max_threads(per_lane(G)) / 32;
    int64_t warps = (T + kSms - 1) / kSms;
    warps = warps < 4 ? 4 : warps > most ? most : warps;
    const int64_t grid = (T + warps - 1) / warps, limit = kSms * (32 / most);
    return {static_cast<int>(warps) * 32, static_cast<int>(grid < 1 ? 1 : grid > limit ? limit : grid)};
}

}  // namespace

// As many parts as any T up to this one gives: a workspace for the largest batch serves smaller ones.
int64_t route_workspace(int64_t T, int G) {
    const int64_t most = T < 4 ? 1 : (T + 3) / 4, limit = kSms * (32 * 32 / route_max_threads(per_lane(G)));
    return (most < limit ? most : limit) * (G * 8 + 4);
}

template <int PER, bool BIAS, bool BALANCE>
static dg_status_t launch_route_impl(const RouteParams &p, const RouteShape &s, cudaStream_t stream) {
    auto kernel = route_kernel<PER, BIAS, BALANCE>;
    const size_t smem = BALANCE ? (static_cast<size_t>(s.threads / 32) * p.G + p.G + 1) * 4 : 0;
    if (smem > 48 * 1024) {
        static thread_local int configured_device = -1;
        const dg_status_t st = allow_smem(kernel, (static_cast<size_t>(route_max_threads(PER) / 32 + 1) * 32 * PER + 1) * 4,
                                          configured_device);
        if (st != DG_OK) return st;
    }
    return launch_pdl(kernel, s.grid, s.threads, smem, stream, p);
}

template <int PER>
static dg_status_t launch_route_per(const RouteParams &p, bool balance, const RouteShape &s, cudaStream_t stream) {
    if (p.bias)
        return balance ? launch_route_impl<PER, true, true>(p, s, stream) : launch_route_impl<PER, true, false>(p, s, stream);
    return balance ? launch_route_impl<PER, false, true>(p, s, stream) : launch_route_impl<PER, false, false>(p, s, stream);
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
    RouteShape s;
    if (balance) {
        s = balance_shape(a.T, a.G);
        p.part_p = static_cast<float *>(a.workspace);
        p.part_count = reinterpret_cast<int32_t *>(p.part_p + static_cast<int64_t>(s.grid) * a.G);
        p.part_tokens = p.part_count + static_cast<int64_t>(s.grid) * a.G;
    } else {
        const int64_t want = (a.T + 3) / 4, most = 16 * static_cast<int64_t>(dev.num_sms);
        s = {128, static_cast<int>(want < most ? want : most)};
    }
    dg_status_t st;
    switch (per_lane(a.G)) {
    case 1: st = launch_route_per<1>(p, balance, s, stream); break;
    case 2: st = launch_route_per<2>(p, balance, s, stream); break;
    case 4: st = launch_route_per<4>(p, balance, s, stream); break;
    case 8: st = launch_route_per<8>(p, balance, s, stream); break;
    case 16: st = launch_route_per<16>(p, balance, s, stream); break;
    default: st = launch_route_per<32>(p, balance, s, stream); break;
    }
    if (st != DG_OK || !balance) return st;
    return launch_pdl(route_finish_kernel, kFinishCtas, kFinishThreads, 0, stream, static_cast<const float *>(p.part_p),
                      static_cast<const int32_t *>(p.part_count), static_cast<const int32_t *>(p.part_tokens), s.grid, a.G,
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
    const int64_t want = (a.T + 7) / 8, most = 4 * static_cast<int64_t>(dev.num_sms);
    const int grid = static_cast<int>(want < most ? want : most);
    switch (per_lane(a.G)) {
    case 1: return launch_route_backward_per<1>(p, grid, stream);
    case 2: return launch_route_backward_per<2>(p, grid, stream);
    case 4: return launch_route_backward_per<4>(p, grid, stream);
    case 8: return launch_route_backward_per<8>(p, grid, stream);
    case 16: return launch_route_backward_per<16>(p, grid, stream);
    default: return launch_route_backward_per<32>(p, grid, stream);
    }
}

}  // namespace dg

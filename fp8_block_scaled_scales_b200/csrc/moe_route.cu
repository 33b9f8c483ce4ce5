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

#include <type_traits>

#include "dg_device.cuh"
#include "train_internal.h"

namespace dg {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kFinishCtas = 8;
constexpr int kClusterCtas = 16;  // of the cluster that takes few tokens alone
constexpr int kFinishThreads = 512;

// How the tokens are shared out: `per` to each warp, one more to the first `extra`; and lanes for
// a token's slots when they are finished side by side, 2^shift of them.
struct WarpShare {
    int64_t per;
    int extra, shift;

    __device__ __forceinline__ int64_t first(int warp) const { return warp * per + (warp < extra ? warp : extra); }
    __device__ __forceinline__ int64_t count(int warp) const { return per + (warp < extra ? 1 : 0); }
};

struct RouteParams {
    const void *logits;
    const float *bias;
    const uint8_t *mask;
    int64_t T;
    int G, k;
    WarpShare share;
    bool bf16, sigmoid, renormalize;
    float scale;
    int32_t *ids;
    float *weights;
    // partial sums of a CTA: [grid][G] of p, [grid][G] slots, [grid] tokens
    float *part_p;
    int32_t *part_count, *part_tokens;
    // part_p null: the grid is one cluster, which writes the results itself
    int32_t *counts;
    float *loss, *dprob;
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

// A warp's lanes as segments of `width` (a power of two), one token's slots in each.
__device__ __forceinline__ float segment_sum(float v, int width) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < width) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float segment_max(float v, int width) {  // a NaN loses
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < width) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// A slot's share of its token's chosen scores, in FP32 without common under- or overflow; lanes
// with ok == false hold no slot.  m: the segment's largest chosen score.
__device__ __forceinline__ float share_of_chosen(float z, bool ok, bool sigmoid, float m, int width) {
    const float s = ok ? (!sigmoid || m < kFarBelow ? expf(z - m) : sigmoid_of(z)) : 0.0f;
    return s / segment_sum(s, width);  // 0 / 0 where the segment holds no slot: ok is false then
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

template <typename T>
__device__ __forceinline__ T from_cta(const T *shared, uint32_t rank) {
    T v;
    const uint32_t at = mapa_shared(smem_u32(shared), rank);
    if constexpr (sizeof(T) == 8)
        asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(at) : "memory");
    else if constexpr (std::is_same<T, float>::value)
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    else
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// The cluster's barrier in two parts, where the other CTAs only have to have started: nothing written before the first
// part is visible after the second.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }

__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The loss from what the threads of a cluster of CTAS hold of it, in FP64 and a fixed order; called by
// all of them, after every CTA has met the others once: the shared memory of a CTA that may not have started yet
// must not be written.  The CTAs' shares go to the first one, so nobody reads another CTA's memory at the end.
template <int CTAS>
__device__ __forceinline__ void loss_of_cluster(double mine, double *warp_loss, double *cta_loss, float *loss) {
    const int warps = static_cast<int>(blockDim.x) >> 5, lane = lane_id();
    mine = warp_sum(mine);
    if (lane == 0) warp_loss[threadIdx.x >> 5] = mine;
    __syncthreads();
    if (threadIdx.x < 32) {
        mine = warp_sum(lane < warps ? warp_loss[lane] : 0.0);
        if (lane == 0)
            asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(mapa_shared(smem_u32(cta_loss + cluster_ctarank()), 0)), "d"(mine)
                         : "memory");
    }
    cluster_sync();
    if (cluster_ctarank() == 0 && threadIdx.x < 32) {
        mine = warp_sum(lane < CTAS ? cta_loss[lane] : 0.0);
        if (lane == 0) *loss = static_cast<float>(mine);
    }
}

// counts, dprob and the loss from the CTAs' shared memory: sums [G] of p, counts [G] and the tokens.
// A lane for each CTA of the cluster, half a warp an expert.
__device__ __forceinline__ void finish_in_cluster(const RouteParams &p, const float *sums, const int *counts) {
    static_assert(kClusterCtas == 16, "half a warp");
    __shared__ double warp_loss[32], cta_loss[kClusterCtas];
    cluster_sync();
    const int half = static_cast<int>(threadIdx.x) >> 4, halves = static_cast<int>(blockDim.x) >> 4;
    const uint32_t r = threadIdx.x & 15u;
    const int share = (p.G + kClusterCtas - 1) / kClusterCtas, e0 = static_cast<int>(cluster_ctarank()) * share;
    const int end = e0 + share < p.G ? e0 + share : p.G;
    int n = from_cta(counts + p.G, r);
    double unit = 0.0, mine = 0.0;
    for (int base = e0; base < end || base == e0; base += halves) {  // the same for the whole CTA
        const int e = base + half;
        float part = 0.0f;
        int c = 0;
        if (e < end) {
            part = from_cta(sums + e, r);
            c = from_cta(counts + e, r);
        }
        if (base == e0) {  // under the loads
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) n += __shfl_xor_sync(kAll, n, o);
            const double nd = n > 0 ? static_cast<double>(n) : 1.0;
            unit = static_cast<double>(p.G) / (static_cast<double>(p.k) * nd * nd);
        }
        double s = static_cast<double>(part);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            s += __shfl_xor_sync(kAll, s, o);
            c += __shfl_xor_sync(kAll, c, o);
        }
        if (e < end && r == 0) {
            const double d = unit * c;
            p.counts[e] = c;
            p.dprob[e] = static_cast<float>(d);
            mine += d * s;
        }
    }
    loss_of_cluster<kClusterCtas>(mine, warp_loss, cta_loss, p.loss);
}

// A warp chooses by 32-bit keys whose low bits are the expert's id, inverted: one maximum over the
// warp gives key and id, the lowest id among equals, and no two keys are the same.  The id takes the place of
// the key's last 5 to 10 bits, so the choice is settled only where neighbours in the order differ
// by more than those (and, with a bias, by more than the key's own FP32 error); otherwise (a token
// in thirty) the candidates are put in order by FP64 keys.  BF16 logits without a bias have the bits to spare.
// Bound by instruction issue, most of it the sort and the k + 1 rounds: 16384 tokens x 256 experts, k = 8,
// FP32 sigmoid scores 11.0 us, with balance loss 15.8, with bias too 19.0 (the logits alone: 2.6); over 512 experts 32, 42 and 51, over 1024 98, 116 and 159.
// The last of these forms spills 92 and 116 bytes at 256 experts (the loss's sums live beside the keys); past 512 every form spills.
constexpr int route_max_threads(int per) { return per <= 8 ? 1024 : 512; }

template <int PER, bool BIAS, bool BALANCE, bool CLUSTER>
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
    // sums of p: in registers, or, where those run out, in the warp's shared memory
    constexpr bool kSumsInRegisters = PER <= 8;
    float psum[kSumsInRegisters ? PER : 1];
    if (BALANCE) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if constexpr (kSumsInRegisters)
                psum[i] = 0.0f;
            else if (lane + 32 * i < p.G)
                sums[warp * p.G + lane + 32 * i] = 0.0f;
        }
    }
    auto bias = [&](int i) { return lane + 32 * i < p.G ? __ldg(p.bias + lane + 32 * i) + 0.0f : 0.0f; };  // from L1; never -0
    const bool exact_keys = !BIAS && p.bf16;
    const int rounds = exact_keys || p.k == p.G ? p.k : p.k + 1;  // the next one too: is the last one settled?
    int tokens = 0;

    // the warp's tokens, 32 / width at a time: each is chosen for by the whole warp, their slots are
    // finished side by side
    const int me = static_cast<int>(blockIdx.x) * warps + warp, width = 1 << p.share.shift;
    const int segment = lane >> p.share.shift, slot = lane & (width - 1);
    int64_t t = p.share.first(me);
    const int64_t end = t + p.share.count(me);
    int my_id = -1;  // slot `slot` of the batch's token `segment`
    float my_top = 0.0f, my_sum = 1.0f;
    int held = 0;
    for (; t < end; ++t) {
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
                            const float c = q[i] + bias(i);
                            key[i] = keyed(c, z[i] > -CUDART_INF_F && c > -CUDART_INF_F, i);
                        }
                    }
                    if (BALANCE) {
                        sum = warp_sum(sum);
                        // all far below 0: ratios of exponentials; with a NaN, for `top`
                        if (!(sum >= 0x1p-80f)) exponentials();
                    }
                } else {
                    exponentials();
                    if (BIAS) {
                        const float r = reciprocal(sum);
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            const float c = fmaf(q[i], r, bias(i));
                            key[i] = keyed(c, z[i] > -CUDART_INF_F && c > -CUDART_INF_F, i);
                        }
                    }
                }
                if (BALANCE) {
                    const float r = reciprocal(sum);
                    // a token that reaches no expert has no part in the loss: without a score above -inf (for
                    // sigmoids whose sum is a number, and not 0, `top` is 0), or where the bias leaves no key
                    bool routed = top > -CUDART_INF_F;
                    if (BIAS) {
                        uint32_t keys = 0u;
#pragma unroll
                        for (int i = 0; i < PER; ++i) keys |= key[i];
                        routed = __any_sync(kAll, keys != 0u);
                    }
                    if (routed) {
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            if constexpr (kSumsInRegisters)
                                psum[i] = fmaf(q[i], r, psum[i]);
                            else if (lane + 32 * i < p.G)
                                sums[warp * p.G + lane + 32 * i] += q[i] * r;
                        }
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
                // s: the row's largest score (1 for sigmoids).  Two keys' difference is off by less than 2^-17.8 of s:
                // - softmax's sum and its reciprocal move both scores alike, so that the difference of the scores takes
                //   their error: 37 additions and a unit, 2^-18.7, and the exponentials', 2 + 1.7 |x| units with the rounding
                //   of x = z - top, averaged over the sum, where |x| is 4.5 at most (1024 experts): 2^-19.7;
                // - each score alone is off by 2 units of s (an exponential falls faster than its error grows; for
                //   sigmoids (2 + 1.2 |z|) s (1 - s) units, a sum and a reciprocal), 2^-21 for both keys;
                // and by a rounding of each s + b, 2^-23 of the larger key for both
                const float x = from_ordered(a & ~kIdBits), y = from_ordered(b | kIdBits);
                const float s = p.sigmoid ? 1.0f : reciprocal(sum);
                return !(x - y > 0x1p-17f * fmaxf(s, fabsf(x)));  // infinite keys too
            };
            while (found < rounds) next();
            if (!exact_keys) {
                uint32_t below = __shfl_down_sync(kAll, mine, 1);
                if (lane == p.k - 1) below = p.k == p.G ? 0u : last;
                if (__any_sync(kAll, lane < p.k && unsettled(mine, below))) {
                    // more candidates, until the next one certainly comes after them
                    while (p.k < p.G && found < 32 && unsettled(prev, last)) next();
                    const int n = p.k == p.G ? p.k : found - 1;
                    const uint32_t candidates = __ballot_sync(kAll, lane < n && mine != 0u);
                    id = static_cast<int>(kIdBits - (mine & kIdBits));
                    if (p.k == p.G || !unsettled(prev, last))
                        id = order_exactly<BIAS>(p.logits, p.bias, row, p.G, p.bf16, p.sigmoid, id, __popc(candidates));
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
        if (BALANCE) tokens += __any_sync(kAll, id >= 0) ? 1 : 0;
        const int moved = __shfl_sync(kAll, id, slot);
        if (segment == held) {
            my_id = moved;
            my_top = top;
            my_sum = sum;
        }
        if (++held < (32 >> p.share.shift) && t + 1 < end) continue;
        // the batch's slots
        const int64_t first = t + 1 - held;
        const bool ok = segment < held && my_id >= 0;
        const float z = ok ? load_score(p.logits, p.bf16, (first + segment) * p.G + my_id) : 0.0f;
        float w;
        if (p.renormalize)
            w = share_of_chosen(z, ok, p.sigmoid, segment_max(ok ? z : -CUDART_INF_F, width), width);
        else
            w = p.sigmoid ? sigmoid_of(z) : expf(z - my_top) / my_sum;
        if (segment < held && slot < p.k) {
            const int64_t at = (first + segment) * p.k + slot;
            p.ids[at] = ok ? my_id : -1;
            p.weights[at] = ok ? w * p.scale : 0.0f;
        }
        if (BALANCE && ok) atomicAdd(&counts[my_id], 1);
        held = 0;
    }
    if (BALANCE) {
        if constexpr (kSumsInRegisters) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 32 * i < p.G) sums[warp * p.G + lane + 32 * i] = psum[i];
        }
        if (lane == 0) atomicAdd(&counts[p.G], tokens);
        __syncthreads();
        const int64_t at = static_cast<int64_t>(blockIdx.x) * p.G;
        for (int e = static_cast<int>(threadIdx.x); e < p.G; e += static_cast<int>(blockDim.x)) {
            float s = 0.0f;
#pragma unroll 8
            for (int w = 0; w < warps; ++w) s += sums[w * p.G + e];
            if constexpr (!CLUSTER) {
                p.part_p[at + e] = s;
                p.part_count[at + e] = counts[e];
            } else {
                sums[e] = s;  // read by no other thread until the cluster has met
            }
        }
        if constexpr (!CLUSTER) {
            if (threadIdx.x == 0) p.part_tokens[blockIdx.x] = counts[p.G];
        } else {
            finish_in_cluster(p, sums, counts);
        }
    }
}

// The CTAs' sums to counts, dprob and the loss: one cluster; a CTA takes 32 experts at a time, a lane
// each, and its warps share the parts.  FP64 sums in a fixed order.
__global__ void __cluster_dims__(kFinishCtas, 1, 1) __launch_bounds__(kFinishThreads)
    route_finish_kernel(const float *__restrict__ part_p, const int32_t *__restrict__ part_count,
                        const int32_t *__restrict__ part_tokens, int parts, int G, int k,
                        int32_t *__restrict__ counts, float *__restrict__ loss, float *__restrict__ dprob) {
    constexpr int kWarps = kFinishThreads / 32;
    __shared__ double warp_p[kWarps][32], warp_loss[kWarps], cta_loss[kFinishCtas];
    __shared__ int warp_count[kWarps][32], warp_tokens[kWarps];
    cluster_arrive_relaxed();  // this CTA runs
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
    cluster_wait();  // all of them do: a CTA without experts comes here at once
    loss_of_cluster<kFinishCtas>(mine, warp_loss, cta_loss, loss);
}

struct RouteBackwardParams {
    const void *logits;
    const int32_t *ids;
    const float *dweights, *dprob, *dloss;
    int64_t T;
    int G, k;
    WarpShare share;
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
// CTAs of an SM, as the registers allow: none waits for another to end.
constexpr int backward_ctas(int per) { return per <= 8 ? 4 : per <= 16 ? 2 : 1; }

template <int PER, bool ROWS>
__global__ void __launch_bounds__(256, backward_ctas(PER)) route_backward_kernel(const RouteBackwardParams p) {
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

    // the warp's tokens, 32 / width at a time: their slots side by side, their rows one after another
    const int me = static_cast<int>(blockIdx.x) * warps + warp, width = 1 << p.share.shift, batch = 32 >> p.share.shift;
    const int segment = lane >> p.share.shift, slot = lane & (width - 1);
    int64_t t0 = p.share.first(me);
    const int64_t end = t0 + p.share.count(me);
    for (; t0 < end; t0 += batch) {
        const int tokens = static_cast<int>(end - t0 < batch ? end - t0 : batch);
        const bool here = segment < tokens && slot < p.k;
        const int64_t at_slot = (t0 + segment) * p.k + slot;
        const int id = here ? __ldg(p.ids + at_slot) : -1;
        const bool ok = id >= 0 && id < p.G;
        const float dw = ok && p.dweights ? __ldg(p.dweights + at_slot) : 0.0f;
        const float z_id = ok ? load_score(p.logits, p.bf16, (t0 + segment) * p.G + id) : 0.0f;
        const uint32_t oks = __ballot_sync(kAll, ok);
        const float m = p.renormalize || !p.sigmoid ? segment_max(ok ? z_id : -CUDART_INF_F, width) : 0.0f;
        float a, token_a = 0.0f;  // A_j; softmax without renormalization: over e^(m - top) / sum, with its sum over the slots
        if (p.renormalize) {
            const float v = share_of_chosen(z_id, ok, p.sigmoid, m, width);
            const float mean = segment_sum(ok ? dw * v : 0.0f, width);
            a = ok ? p.scale * v * (dw - mean) : 0.0f;
        } else {
            a = ok ? p.scale * dw * (p.sigmoid ? sigmoid_of(z_id) : expf(z_id - m)) : 0.0f;
            if (!p.sigmoid) token_a = segment_sum(a, width);
        }
        float my_r = 0.0f, my_base = 0.0f, my_top = 0.0f;  // of the lane's token
        bool my_exponential = false;
        const uint32_t segment_lanes = width == 32 ? kAll : (1u << width) - 1u;
        for (int b = 0; b < tokens; ++b) {
            const int64_t row = (t0 + b) * p.G;
            const bool routed = (oks >> (b * width)) & segment_lanes;
            float q[PER], ns[PER];  // what p is proportional to, and 1 - sigmoid; then the gradient
            float top = -CUDART_INF_F, r = 0.0f, base = 0.0f;
            bool exponential = !p.sigmoid;
            if (ROWS && routed) {
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
                if (!p.sigmoid && !p.renormalize)
                    base += __shfl_sync(kAll, token_a, b * width) * (expf(__shfl_sync(kAll, m, b * width) - top) * r);
                if (segment == b) {
                    my_r = r;
                    my_base = base;
                    my_top = top;
                    my_exponential = exponential;
                }
            }
            // every expert's part; the chosen ones' whole gradient follows over it
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                q[i] = ROWS && routed ? q[i] * r * (dp[i] - base) : 0.0f;
                if (ROWS && routed && p.sigmoid) q[i] *= ns[i];
            }
            if (p.bf16) {
                __nv_bfloat16 *at = static_cast<__nv_bfloat16 *>(p.dlogits) + row + lane;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (lane + 32 * i < p.G) at[32 * i] = __float2bfloat16(q[i]);
            } else {
                float *at = static_cast<float *>(p.dlogits) + row + lane;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (lane + 32 * i < p.G) at[32 * i] = q[i];
            }
        }
        if (oks == 0u) continue;
        if (!p.renormalize && !p.sigmoid) a *= expf(m - my_top) * my_r;
        // an expert that a token names twice gets both slots' parts
        const uint32_t same = __match_any_sync(kAll, ok ? segment * 1024 + id : -1 - lane);
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
            g += unnormalized(z_id, my_top, my_exponential) * my_r * (d - my_base);
        }
        if (p.sigmoid) {
            const float e = fminf(exp_fast(-z_id), 0x1p125f);
            g *= e * reciprocal(1.0f + e);
        }
        __syncwarp();  // the rows' stores come first
        if (ok) store_score(p.dlogits, p.bf16, (t0 + segment) * p.G + id, g);
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

// Few tokens are taken by one cluster of sixteen CTAs alone, where a pass is bound by host time: a launch and an
// allocation less (1000 tokens of 64 experts: 10.2 -> 8.2 us a call among others, though 5.9 -> 7.7 on the GPU; 100 tokens 5.0 -> 4.5 there).
// With more experts or tokens the cluster itself takes longer than that (1000 of 256: 15 us).
bool one_cluster(int64_t T, int G) { return T * per_lane(G) <= 2048; }

// A CTA per SM with as many warps as there are tokens for, up to 32: fewer parts to add up.
RouteShape balance_shape(int64_t T, int G) {
    const int64_t most = route_max_threads(per_lane(G)) / 32;
    if (one_cluster(T, G)) {
        const int64_t warps = (T + kClusterCtas - 1) / kClusterCtas;
        return {static_cast<int>(warps < 4 ? 4 : warps > most ? most : warps) * 32, kClusterCtas};
    }
    int64_t warps = (T + kSms - 1) / kSms;
    warps = warps < 4 ? 4 : warps > most ? most : warps;
    const int64_t grid = (T + warps - 1) / warps, limit = kSms;
    return {static_cast<int>(warps) * 32, static_cast<int>(grid < 1 ? 1 : grid > limit ? limit : grid)};
}

// As few lanes for a token's slots as hold them, and at least as many as leave a warp no more
// tokens at a time than it has.
WarpShare share_out(int64_t T, int k, int64_t warps) {
    const int64_t per = T / warps;
    const int extra = static_cast<int>(T - per * warps), most = per < 16 ? static_cast<int>(per) + (extra != 0) : 16;
    int shift = 0;
    while ((1 << shift) < k || (shift < 5 && most <= (16 >> shift))) ++shift;
    return {per, extra, shift};
}

}  // namespace

// As many parts as any T up to this one gives: a workspace for the largest batch serves smaller ones.
int64_t route_workspace(int64_t T, int G) {
    if (one_cluster(T, G)) return 0;
    const int64_t most = (T + 3) / 4, limit = kSms;
    return (most < limit ? most : limit) * (G * 8 + 4);
}

template <int PER, bool BIAS, bool BALANCE, bool CLUSTER>
static dg_status_t launch_route_impl(const RouteParams &p, const RouteShape &s, cudaStream_t stream) {
    auto kernel = route_kernel<PER, BIAS, BALANCE, CLUSTER>;
    const size_t smem = BALANCE ? (static_cast<size_t>(s.threads / 32) * p.G + p.G + 1) * 4 : 0;
    if (smem > 48 * 1024) {
        static thread_local int configured_device = -1;
        const dg_status_t st = allow_smem(kernel, (static_cast<size_t>(route_max_threads(PER) / 32 + 1) * 32 * PER + 1) * 4,
                                          configured_device);
        if (st != DG_OK) return st;
    }
    if (!CLUSTER) return launch_pdl(kernel, s.grid, s.threads, smem, stream, p);
    static thread_local int wide_device = -1;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return DG_ERR_CUDA;
    if (wide_device != device) {  // clusters of more than eight need the kernel's consent
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return DG_ERR_CUDA;
        wide_device = device;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(s.grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(s.threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(s.grid);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

template <int PER, bool BIAS>
static dg_status_t launch_route_per(const RouteParams &p, bool balance, const RouteShape &s, cudaStream_t stream) {
    if (!balance) return launch_route_impl<PER, BIAS, false, false>(p, s, stream);
    return p.part_p ? launch_route_impl<PER, BIAS, true, false>(p, s, stream) : launch_route_impl<PER, BIAS, true, true>(p, s, stream);
}

template <int PER>
static dg_status_t launch_route_per(const RouteParams &p, bool balance, const RouteShape &s, cudaStream_t stream) {
    return p.bias ? launch_route_per<PER, true>(p, balance, s, stream) : launch_route_per<PER, false>(p, balance, s, stream);
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
        p.counts = a.counts;
        p.loss = a.loss;
        p.dprob = a.dprob;
        if (!one_cluster(a.T, a.G)) {
            p.part_p = static_cast<float *>(a.workspace);
            p.part_count = reinterpret_cast<int32_t *>(p.part_p + static_cast<int64_t>(s.grid) * a.G);
            p.part_tokens = p.part_count + static_cast<int64_t>(s.grid) * a.G;
        }
    } else {
        const int64_t want = (a.T + 3) / 4, most = 8 * static_cast<int64_t>(dev.num_sms);
        s = {128, static_cast<int>(want < most ? want : most)};
    }
    p.share = share_out(a.T, a.k, static_cast<int64_t>(s.grid) * (s.threads / 32));
    dg_status_t st;
    switch (per_lane(a.G)) {
    case 1: st = launch_route_per<1>(p, balance, s, stream); break;
    case 2: st = launch_route_per<2>(p, balance, s, stream); break;
    case 4: st = launch_route_per<4>(p, balance, s, stream); break;
    case 8: st = launch_route_per<8>(p, balance, s, stream); break;
    case 16: st = launch_route_per<16>(p, balance, s, stream); break;
    default: st = launch_route_per<32>(p, balance, s, stream); break;
    }
    if (st != DG_OK || !p.part_p) return st;
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
    const int64_t want = (a.T + 7) / 8, most = backward_ctas(per_lane(a.G)) * static_cast<int64_t>(dev.num_sms);
    const int grid = static_cast<int>(want < most ? want : most);
    const RouteBackwardParams p = {a.logits, a.ids, a.dweights, a.dprob, a.dloss, a.T, a.G, a.k,
                                   share_out(a.T, a.k, static_cast<int64_t>(grid) * 8),
                                   a.bf16, a.sigmoid, a.renormalize, a.scale, a.dlogits};
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

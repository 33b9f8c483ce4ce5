// The global norm of many gradient tensors, sqrt(sum g^2), and clipping by it:
//   g *= max_norm / norm  where norm > max_norm (a norm that is not finite clips nothing).
//
// The tensors' addresses and sizes travel in the kernel's parameters, so a captured graph
// keeps them and no copy has to finish first.  Tensors are cut into chunks of kChunk elements;
// a CTA takes every grid-th chunk of the list, and its sum goes to its own word, so the norm
// does not depend on the launch.  Clipping walks the chunks backwards: the gradients read last
// for the norm are still in L2.
#include <cuda_bf16.h>

#include "dg_device.cuh"
#include "train_internal.h"

namespace dg {

constexpr int kNormThreads = 256;
constexpr int kChunk = 8192;
constexpr int kGradCtas = 148 * 4;  // CTAs of a launch at most; the workspace holds as many sums

// 28 bytes a tensor; parameters may take 32764 bytes.
template <int N>
struct GradTable {
    const void *in[N];
    void *out[N];
    int64_t size[N];
    int32_t chunk_end[N];  // chunks up to and with this tensor; bf16 in the top bit of `kind`
    uint32_t kind[(N + 31) / 32];
    int tensors, chunks;
};

struct Chunk {
    const void *in;
    void *out;
    int64_t first;
    int count;
    bool bf16;
};

template <int N>
__device__ __forceinline__ Chunk find_chunk(const GradTable<N> &t, int c) {
    int lo = 0, hi = t.tensors - 1;  // the first tensor whose chunk_end lies past c
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t.chunk_end[mid] > c) hi = mid; else lo = mid + 1;
    }
    Chunk k;
    k.in = t.in[lo];
    k.out = t.out[lo];
    k.bf16 = (t.kind[lo >> 5] >> (lo & 31)) & 1u;
    k.first = static_cast<int64_t>(c - (lo ? t.chunk_end[lo - 1] : 0)) * kChunk;
    const int64_t left = t.size[lo] - k.first;
    k.count = left < kChunk ? static_cast<int>(left) : kChunk;
    return k;
}

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Squares of a few values in FP32 are good while their sum neither overflows nor comes near the
// subnormals; otherwise they are squared in FP64.  `bits`: all values' bits or-ed, signs off.
struct SquareSum {
    double total = 0.0;

    template <typename F>
    __device__ __forceinline__ void add(float s, uint32_t bits, F each_in_fp64) {
        if (s >= 0x1p-80f && s <= 0x1p126f)
            total += static_cast<double>(s);
        else if (bits != 0)
            each_in_fp64();
    }
};

__device__ __forceinline__ void add_words(SquareSum &sum, const uint4 *v, int n, bool bf16) {
    // n <= 4 pieces of 16 bytes
    float s = 0.0f;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= n) break;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bits |= w[j];
            if (bf16) {
                s = fmaf(bf16_low(w[j]), bf16_low(w[j]), s);
                s = fmaf(bf16_high(w[j]), bf16_high(w[j]), s);
            } else {
                s = fmaf(__uint_as_float(w[j]), __uint_as_float(w[j]), s);
            }
        }
    }
    sum.add(s, bits & (bf16 ? 0x7FFF7FFFu : 0x7FFFFFFFu), [&] {
        for (int i = 0; i < n; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            for (int j = 0; j < 4; ++j) {
                const double a = bf16 ? bf16_low(w[j]) : __uint_as_float(w[j]), b = bf16 ? bf16_high(w[j]) : 0.0f;
                sum.total += a * a + b * b;
            }
        }
    });
}

__device__ __forceinline__ float element(const Chunk &k, int64_t i) {
    return k.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(k.in)[i]) : static_cast<const float *>(k.in)[i];
}

// A CTA's sum of doubles, the same in every thread's order.
__device__ __forceinline__ double cta_sum_f64(double v, double *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane_id() == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) v += red[i];
    return v;
}

template <int N>
__global__ void __launch_bounds__(kNormThreads) grad_squares_kernel(const __grid_constant__ GradTable<N> t, double *part) {
    __shared__ double red[kNormThreads / 32];
    const int tid = static_cast<int>(threadIdx.x);
    grid_dep_wait();
    grid_dep_launch_dependents();
    SquareSum sum;
    for (int c = static_cast<int>(blockIdx.x); c < t.chunks; c += static_cast<int>(gridDim.x)) {
        const Chunk k = find_chunk(t, c);
        const int per = k.bf16 ? 8 : 4;  // elements of a 16-byte piece
        const uint8_t *base = static_cast<const uint8_t *>(k.in) + k.first * (k.bf16 ? 2 : 4);
        int done = 0;
        if ((reinterpret_cast<uintptr_t>(base) & 15) == 0) {
            const uint4 *v = reinterpret_cast<const uint4 *>(base);
            const int pieces = k.count / per;
            int i = tid;
            for (; i + 3 * kNormThreads < pieces; i += 4 * kNormThreads) {
                const uint4 w[4] = {__ldg(v + i), __ldg(v + i + kNormThreads), __ldg(v + i + 2 * kNormThreads),
                                    __ldg(v + i + 3 * kNormThreads)};
                add_words(sum, w, 4, k.bf16);
            }
            for (; i < pieces; i += kNormThreads) {
                const uint4 w = __ldg(v + i);
                add_words(sum, &w, 1, k.bf16);
            }
            done = pieces * per;
        }
        for (int i = done + tid; i < k.count; i += kNormThreads) {
            const float x = element(k, k.first + i);
            sum.add(x * x, __float_as_uint(x) & 0x7FFFFFFFu, [&] { sum.total += static_cast<double>(x) * x; });
        }
    }
    const double s = cta_sum_f64(sum.total, red);
    if (tid == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ float norm_of(const double *part, int parts, double *red) {
    double s = 0.0;
    for (int i = static_cast<int>(threadIdx.x); i < parts; i += kNormThreads) s += part[i];
    return static_cast<float>(sqrt(cta_sum_f64(s, red)));
}

__global__ void __launch_bounds__(kNormThreads) grad_norm_kernel(const double *part, int parts, float *norm) {
    __shared__ double red[kNormThreads / 32];
    grid_dep_wait();
    grid_dep_launch_dependents();
    const float n = norm_of(part, parts, red);
    if (threadIdx.x == 0) *norm = n;
}

// part == nullptr: `norm` is given.  Otherwise every CTA adds up the sums itself, and the
// first writes the norm if `write` is set.
template <int N>
__global__ void __launch_bounds__(kNormThreads) grad_clip_kernel(const __grid_constant__ GradTable<N> t, const double *part,
                                                                 int parts, float *norm, bool write, float max_norm) {
    __shared__ double red[kNormThreads / 32];
    const int tid = static_cast<int>(threadIdx.x);
    grid_dep_wait();
    grid_dep_launch_dependents();
    const float n = part ? norm_of(part, parts, red) : *norm;
    if (part && write && blockIdx.x == 0 && tid == 0) *norm = n;
    const float coef = n > max_norm && n <= 3.402823466e38f ? __fdiv_rn(max_norm, n) : 1.0f;
    for (int c = t.chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= static_cast<int>(gridDim.x)) {
        const Chunk k = find_chunk(t, c);
        if (coef == 1.0f && k.in == k.out) continue;
        const int size = k.bf16 ? 2 : 4, per = 16 / size;
        const uint8_t *in = static_cast<const uint8_t *>(k.in) + k.first * size;
        uint8_t *out = static_cast<uint8_t *>(k.out) + k.first * size;
        int done = 0;
        if (((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
            const uint4 *v = reinterpret_cast<const uint4 *>(in);
            uint4 *o = reinterpret_cast<uint4 *>(out);
            const int pieces = k.count / per;
            auto scaled = [&](uint4 w) {
                auto one = [&](uint32_t x) {
                    return k.bf16 ? pack_bf16x2(bf16_low(x) * coef, bf16_high(x) * coef)
                                  : __float_as_uint(__uint_as_float(x) * coef);
                };
                return make_uint4(one(w.x), one(w.y), one(w.z), one(w.w));
            };
            int i = tid;
            for (; i + 3 * kNormThreads < pieces; i += 4 * kNormThreads) {
                const uint4 a = v[i], b = v[i + kNormThreads], d = v[i + 2 * kNormThreads], e = v[i + 3 * kNormThreads];
                o[i] = scaled(a);
                o[i + kNormThreads] = scaled(b);
                o[i + 2 * kNormThreads] = scaled(d);
                o[i + 3 * kNormThreads] = scaled(e);
            }
            for (; i < pieces; i += kNormThreads) o[i] = scaled(v[i]);
            done = pieces * per;
        }
        for (int i = done + tid; i < k.count; i += kNormThreads) {
            const float x = element(k, k.first + i) * coef;
            if (k.bf16)
                reinterpret_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16(x);
            else
                reinterpret_cast<float *>(out)[i] = x;
        }
    }
}

namespace {

constexpr int kTable = 1024;      // tensors of a launch at most
constexpr int kSmallTable = 64;   // parameters cost host time: 2 KB for few tensors instead of 29

int64_t chunks_of(int64_t size) { return (size + kChunk - 1) / kChunk; }

// Calls launch(table, grid) for runs of at most kTable tensors that have elements.
template <int N, typename F>
dg_status_t walk_tables(const GradList &g, F launch) {
    // filled from scratch for each run; too large for some threads' stacks twice over
    GradTable<N> t;
    t.tensors = t.chunks = 0;
    for (uint32_t &w : t.kind) w = 0;
    auto flush = [&] {
        if (t.tensors == 0) return DG_OK;
        const dg_status_t st = launch(t, t.chunks < kGradCtas ? t.chunks : kGradCtas);
        t.tensors = t.chunks = 0;
        for (uint32_t &w : t.kind) w = 0;
        return st;
    };
    for (int64_t i = 0; i < g.count; ++i) {
        if (g.sizes[i] == 0) continue;
        const int64_t chunks = chunks_of(g.sizes[i]);
        if (t.tensors == N || t.chunks + chunks > 0x3FFFFFFFLL) {
            const dg_status_t st = flush();
            if (st != DG_OK) return st;
        }
        const int at = t.tensors++;
        t.in[at] = g.in[i];
        t.out[at] = g.out ? g.out[i] : const_cast<void *>(g.in[i]);
        t.size[at] = g.sizes[i];
        t.chunks += static_cast<int>(chunks);
        t.chunk_end[at] = t.chunks;
        if (g.bf16[i]) t.kind[at >> 5] |= 1u << (at & 31);
    }
    return flush();
}

template <int N>
dg_status_t squares(const GradList &g, double *part, int &parts, cudaStream_t stream) {
    parts = 0;
    return walk_tables<N>(g, [&](const GradTable<N> &t, int grid) {
        const dg_status_t st = launch_pdl(grad_squares_kernel<N>, grid, kNormThreads, 0, stream, t, part + parts);
        parts += grid;
        return st;
    });
}

template <int N>
dg_status_t clip(const GradList &g, const double *part, int parts, float *norm, float max_norm, cudaStream_t stream) {
    bool first = true;
    return walk_tables<N>(g, [&](const GradTable<N> &t, int grid) {
        const dg_status_t st = launch_pdl(grad_clip_kernel<N>, grid, kNormThreads, 0, stream, t, part, parts, norm, first, max_norm);
        first = false;
        return st;
    });
}

int64_t with_elements(const GradList &g) {
    int64_t n = 0;
    for (int64_t i = 0; i < g.count; ++i) n += g.sizes[i] != 0;
    return n;
}

}  // namespace

int64_t grad_norm_workspace(int64_t count) { return (count / kTable + 1) * kGradCtas * 8; }

dg_status_t launch_grad_norm(const GradList &g, float *norm, void *workspace, cudaStream_t stream) {
    double *part = static_cast<double *>(workspace);
    int parts = 0;
    const dg_status_t st = with_elements(g) <= kSmallTable ? squares<kSmallTable>(g, part, parts, stream)
                                                           : squares<kTable>(g, part, parts, stream);
    if (st != DG_OK) return st;
    return launch_pdl(grad_norm_kernel, 1, kNormThreads, 0, stream, static_cast<const double *>(part), parts, norm);
}

dg_status_t launch_grad_clip(const GradList &g, const float *norm, float max_norm, cudaStream_t stream) {
    float *n = const_cast<float *>(norm);  // only read: no partial sums are given
    return with_elements(g) <= kSmallTable ? clip<kSmallTable>(g, nullptr, 0, n, max_norm, stream)
                                           : clip<kTable>(g, nullptr, 0, n, max_norm, stream);
}

dg_status_t launch_grad_norm_clip(const GradList &g, float max_norm, float *norm, void *workspace, cudaStream_t stream) {
    double *part = static_cast<double *>(workspace);
    int parts = 0;
    const int64_t n = with_elements(g);
    if (n == 0) return launch_grad_norm(g, norm, workspace, stream);
    dg_status_t st = n <= kSmallTable ? squares<kSmallTable>(g, part, parts, stream) : squares<kTable>(g, part, parts, stream);
    if (st != DG_OK) return st;
    return n <= kSmallTable ? clip<kSmallTable>(g, part, parts, norm, max_norm, stream)
                            : clip<kTable>(g, part, parts, norm, max_norm, stream);
}

}  // namespace dg

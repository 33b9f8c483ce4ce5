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
template <int N, int DEEP>
__global__ void __launch_bounds__(kNormThreads) grad_clip_kernel(const __grid_constant__ GradTable<N> t, const double *part,
                                                                 int parts, float *norm, bool write, float max_norm) {
    __shared__ double red[kNormThreads / 32];
    const int tid = static_cast<int>(threadIdx.x);
    grid_dep_wait();
    grid_dep_launch_dependents();
    const float n = part ? norm_of(part, parts, red) : *norm;
    if (part && write && blockIdx.x == 0 && tid == 0) *norm = n;
    const float coef = n > max_norm && n <= 3.402823466e38f ? __fdiv_rn(max_norm, n) : 1.0f;
    // a subnormal quotient has lost bits that the product still needs: FP64 then, element by element
    const bool tiny = coef < 0x1p-126f && max_norm > 0.0f;
    const double ratio = tiny ? static_cast<double>(max_norm) / static_cast<double>(n) : 0.0;
    for (int c = t.chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= static_cast<int>(gridDim.x)) {
        const Chunk k = find_chunk(t, c);
        if (coef == 1.0f && k.in == k.out) continue;
        const int size = k.bf16 ? 2 : 4, per = 16 / size;
        const uint8_t *in = static_cast<const uint8_t *>(k.in) + k.first * size;
        uint8_t *out = static_cast<uint8_t *>(k.out) + k.first * size;
        int done = 0;
        if (!tiny && ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
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
            for (; i + (DEEP - 1) * kNormThreads < pieces; i += DEEP * kNormThreads) {
                uint4 w[DEEP];
#pragma unroll
                for (int j = 0; j < DEEP; ++j) w[j] = v[i + j * kNormThreads];
#pragma unroll
                for (int j = 0; j < DEEP; ++j) o[i + j * kNormThreads] = scaled(w[j]);
            }
            for (; i < pieces; i += kNormThreads) o[i] = scaled(v[i]);
            done = pieces * per;
        }
        for (int i = done + tid; i < k.count; i += kNormThreads) {
            float x = element(k, k.first + i);
            x = tiny ? static_cast<float>(x * ratio) : x * coef;
            if (k.bf16)
                reinterpret_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16(x);
            else
                reinterpret_cast<float *>(out)[i] = x;
        }
    }
}

namespace {

// Tensors of a launch at most.  Parameters cost host time: 2 or 9 KB for fewer tensors instead of 27.
constexpr int kTable = 960, kMiddleTable = 320, kSmallTable = 64;

int64_t chunks_of(int64_t size) { return (size + kChunk - 1) / kChunk; }

// The gradients, table after table.  One that holds them all is built once and serves both launches.
template <int N>
class Tables {
public:
    explicit Tables(const GradList &g) : g_(g) {}

    // launch(table, grid) for each.
    template <typename F>
    dg_status_t each(F launch) {
        if (whole_) return launch(t_, ctas_);
        int64_t next = 0;
        while (next < g_.count) {
            const bool first = next == 0;
            next = fill(next);
            if (t_.tensors == 0) break;
            whole_ = first && next == g_.count;
            t_.chunks = t_.chunk_end[t_.tensors - 1];
            ctas_ = t_.chunks < kGradCtas ? t_.chunks : kGradCtas;
            const dg_status_t st = launch(t_, ctas_);
            if (st != DG_OK) return st;
        }
        return DG_OK;
    }

private:
    // Tensors from `next` on, as many as fit; returns the first that is left.
    int64_t fill(int64_t next) {
        t_.tensors = 0;
        for (uint32_t &w : t_.kind) w = 0;
        int64_t chunks = 0;
        for (; next < g_.count; ++next) {
            const int64_t size = g_.sizes[next], n = chunks_of(size);
            if (size == 0) continue;
            if (t_.tensors == N || chunks + n > 0x3FFFFFFFLL) break;
            const int at = t_.tensors++;
            t_.in[at] = g_.in[next];
            t_.out[at] = g_.out ? g_.out[next] : const_cast<void *>(g_.in[next]);
            t_.size[at] = size;
            t_.chunk_end[at] = static_cast<int32_t>(chunks += n);
            if (g_.bf16[next]) t_.kind[at >> 5] |= 1u << (at & 31);
        }
        while (next < g_.count && g_.sizes[next] == 0) ++next;
        return next;
    }

    const GradList &g_;
    GradTable<N> t_;
    int ctas_ = 0;
    bool whole_ = false;
};

// launch_pdl takes its arguments by value; a table is better not copied once more.
template <typename Kernel, typename... Args>
dg_status_t launch_table(Kernel kernel, int grid, cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kNormThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *pointers[] = {const_cast<void *>(static_cast<const void *>(&args))...};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(kernel), pointers) == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

template <int N>
dg_status_t squares(Tables<N> &tables, double *part, int &parts, cudaStream_t stream) {
    parts = 0;
    return tables.each([&](const GradTable<N> &t, int ctas) {
        double *const to = part + parts;
        parts += ctas;
        return launch_table(grad_squares_kernel<N>, ctas, stream, t, to);
    });
}

// Gradients that outgrow the L2: reads further ahead of the writes cost bandwidth (1.6 GB of FP32 with four pieces a
// thread 540 us, with two 497, with one 602); smaller ones are done sooner with four (300 tensors 6.5 us against 7.0,
// 100 MB 34.7 against 35.7).
constexpr int kManyChunks = 8 * kGradCtas;

template <int N>
dg_status_t clip(Tables<N> &tables, const double *part, int parts, float *norm, float max_norm, cudaStream_t stream) {
    bool first = true;
    return tables.each([&](const GradTable<N> &t, int ctas) {
        const bool write = first;
        first = false;
        return t.chunks > kManyChunks
            ? launch_table(grad_clip_kernel<N, 2>, ctas, stream, t, part, parts, norm, write, max_norm)
            : launch_table(grad_clip_kernel<N, 4>, ctas, stream, t, part, parts, norm, write, max_norm);
    });
}

template <int N>
dg_status_t norm_of_list(const GradList &g, float *norm, double *part, cudaStream_t stream) {
    Tables<N> tables(g);
    int parts = 0;
    const dg_status_t st = squares<N>(tables, part, parts, stream);
    if (st != DG_OK) return st;
    return launch_pdl(grad_norm_kernel, 1, kNormThreads, 0, stream, static_cast<const double *>(part), parts, norm);
}

template <int N>
dg_status_t clip_list(const GradList &g, float max_norm, float *norm, double *part, cudaStream_t stream) {
    Tables<N> tables(g);
    int parts = 0;
    const dg_status_t st = squares<N>(tables, part, parts, stream);
    return st != DG_OK ? st : clip<N>(tables, part, parts, norm, max_norm, stream);
}

int64_t with_elements(const GradList &g) {
    int64_t n = 0;
    for (int64_t i = 0; i < g.count; ++i) n += g.sizes[i] != 0;
    return n;
}

}  // namespace

// A table ends early only where its chunks outrun 30 bits: 2^43 elements, more than a GPU holds.
int64_t grad_norm_workspace(int64_t count) { return (count / kTable + 1) * kGradCtas * 8; }

dg_status_t launch_grad_norm(const GradList &g, float *norm, void *workspace, cudaStream_t stream) {
    double *part = static_cast<double *>(workspace);
    const int64_t n = with_elements(g);
    if (n <= kSmallTable) return norm_of_list<kSmallTable>(g, norm, part, stream);
    return n <= kMiddleTable ? norm_of_list<kMiddleTable>(g, norm, part, stream) : norm_of_list<kTable>(g, norm, part, stream);
}

template <int N>
static dg_status_t clip_by(const GradList &g, const float *norm, float max_norm, cudaStream_t stream) {
    Tables<N> tables(g);
    return clip<N>(tables, nullptr, 0, const_cast<float *>(norm), max_norm, stream);  // only read: no partial sums are given
}

dg_status_t launch_grad_clip(const GradList &g, const float *norm, float max_norm, cudaStream_t stream) {
    const int64_t n = with_elements(g);
    if (n <= kSmallTable) return clip_by<kSmallTable>(g, norm, max_norm, stream);
    return n <= kMiddleTable ? clip_by<kMiddleTable>(g, norm, max_norm, stream) : clip_by<kTable>(g, norm, max_norm, stream);
}

dg_status_t launch_grad_norm_clip(const GradList &g, float max_norm, float *norm, void *workspace, cudaStream_t stream) {
    double *part = static_cast<double *>(workspace);
    const int64_t n = with_elements(g);
    if (n == 0) return launch_grad_norm(g, norm, workspace, stream);
    if (n <= kSmallTable) return clip_list<kSmallTable>(g, max_norm, norm, part, stream);
    return n <= kMiddleTable ? clip_list<kMiddleTable>(g, max_norm, norm, part, stream)
                             : clip_list<kTable>(g, max_norm, norm, part, stream);
}

}  // namespace dg

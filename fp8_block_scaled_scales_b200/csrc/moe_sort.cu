// Tokens sorted by expert: a stable counting sort of the T x k routing slots, into the
// grouped-contiguous layout (each expert's rows start at a multiple of 128) or into the
// masked layout (a slab of M_max rows per expert).
//
//   e(s)   = topk_ids[s] (outside [0, G): the slot is dropped)
//   rank   = number of slots s' < s with e(s') = e(s)
//   row(s) = off[e] + rank, off the prefix sum of the experts' counts rounded up to 128
//            (masked: e * M_max + rank, dropped when rank >= M_max)
//
// Ranks come without atomics, so the order is fixed: a warp takes 32 consecutive slots, finds
// the lanes with its own expert from one ballot per bit of the id, and its count per expert
// goes into a table that is summed over the warps in order.  (match.any in place of the
// ballots was several times slower: 52 us for 131072 slots, 256 experts, with one cluster of
// 8 CTAs.)
//
// Up to kSortOneCta slots one CTA does it all: a decode step's cost is one launch.  Beyond
// that, two launches over consecutive chunks, one CTA each: the first ranks the slots inside
// their chunk and writes the chunk's counts; in the second every CTA adds up the counts of
// all chunks (a few hundred KB from L2) and hands out the rows.  Bound by latency: in a graph
// 3.3 us for 8 slots into 64 slabs of 128 rows, 7.9 us for 131072 slots of 256 experts.
//
// The form goes by the slots alone, and the one CTA also writes the row map of all slabs: 8 slots
// into 64 slabs of 1024 rows take 10.7 us, of 4096 rows 37 us, 2048 slots into 8 slabs of 6912
// rows 10.7 us; 2050 slots, in two launches, 7.7 us.
#include "dg_device.cuh"
#include "train_internal.h"

namespace dg {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxG = 1024;  // one thread per expert in the scans
constexpr int kSortSteps = 2;    // slots a thread of the one-CTA form holds
constexpr int64_t kSortOneCta = kSortSteps * kSortThreads;
static_assert(kSortMaxG <= kSortThreads, "one thread per expert");

template <typename IdT>
__device__ __forceinline__ int expert_of(const IdT *ids, int64_t s, bool there, int G) {
    const IdT v = there ? __ldg(ids + s) : IdT(-1);
    return (v >= 0 && v < IdT(G)) ? static_cast<int>(v) : -1;
}

// Lanes of the warp with this lane's expert (0 for a dropped slot).
__device__ __forceinline__ uint32_t lanes_with(int e, int bits) {
    uint32_t peers = __ballot_sync(0xFFFFFFFFu, e >= 0);
    for (int b = 0; b < bits; ++b) {
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, (e >> b) & 1);
        peers &= ((e >> b) & 1) ? m : ~m;
    }
    return e >= 0 ? peers : 0u;
}

// Ranks of one step of 1024 slots among the slots of the same expert since `base` was zero:
// base[e] (shared, one per expert) is advanced by the step's counts.  hist: [active][G] words.
// Called by all threads; `active` warps hold slots.  Returns the rank (e >= 0).
__device__ __forceinline__ int rank_step(int e, int G, int bits, int active, int *hist, int *base) {
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < active * G; i += kSortThreads) hist[i] = 0;
    const uint32_t peers = lanes_with(e, bits);
    const int in_warp = __popc(peers & ((1u << lane) - 1u));
    __syncthreads();
    if (e >= 0 && in_warp == 0) hist[warp * G + e] = __popc(peers);
    __syncthreads();
    if (tid < G) {
        int run = base[tid];
        for (int w0 = 0; w0 < active; w0 += 8) {  // eight loads at a time: each alone waits for shared memory
            int c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = w0 + i < active ? hist[(w0 + i) * G + tid] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (w0 + i < active) hist[(w0 + i) * G + tid] = run;
                run += c[i];
            }
        }
        base[tid] = run;
    }
    __syncthreads();
    return e >= 0 ? hist[warp * G + e] + in_warp : -1;
}

// First row of each expert from the counts (one thread per expert, all threads call it):
// masked: e * rows; contiguous: the prefix sum of the counts rounded up to 128, into off[0..G]
// as well.  scan: 32 words.
template <bool MASKED>
__device__ __forceinline__ void first_rows(int all, int G, int rows, int *first, int *scan) {
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    if (MASKED) {
        if (tid < G) first[tid] = tid * rows;
        return;
    }
    const int padded = tid < G ? (all + 127) / 128 * 128 : 0;
    int incl = padded;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += scan[w];
    if (tid < G) {
        first[tid] = before + incl - padded;
        if (tid == G - 1) first[G] = before + incl;
    }
}

// The row of rank `rank` of expert e.
template <bool MASKED>
__device__ __forceinline__ int row_of(int e, int rank, const int *first, int rows) {
    if (e < 0 || (MASKED && rank >= rows)) return -1;
    return first[e] + rank;
}

// -1 into the rows without a slot (count: slots per expert that have a row), by `ctas` CTAs.
template <bool MASKED>
__device__ __forceinline__ void fill_empty_rows(int G, int rows, const int *first, const int *count, int cta, int ctas,
                                                int32_t *slot_of_row) {
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    if (!MASKED) {
        for (int e = cta * kSortWarps + warp; e < G; e += ctas * kSortWarps)
            for (int r = first[e] + count[e] + lane; r < first[e + 1]; r += 32) slot_of_row[r] = -1;
    }
    // masked: all slabs; contiguous: past the last expert
    const int64_t end = MASKED ? static_cast<int64_t>(G) * rows : rows;
    for (int64_t r = (MASKED ? 0 : first[G]) + static_cast<int64_t>(cta) * kSortThreads + tid; r < end;
         r += static_cast<int64_t>(ctas) * kSortThreads) {
        if (MASKED) {
            const int e = static_cast<int>(r) / rows;
            if (static_cast<int>(r) - e * rows < count[e]) continue;
        }
        slot_of_row[r] = -1;
    }
}

// offsets (contiguous: first[0..G]) or counts (masked) out.
template <bool MASKED>
__device__ __forceinline__ void write_offsets(int G, const int *first, const int *count, int32_t *offsets) {
    const int tid = static_cast<int>(threadIdx.x);
    if (tid < G) offsets[tid] = MASKED ? count[tid] : first[tid];
    if (!MASKED && tid == 0) offsets[G] = first[G];
}

template <typename IdT, bool MASKED>
__global__ void __launch_bounds__(kSortThreads, 1)
    moe_sort_kernel(const IdT *__restrict__ ids, int slots, int G, int bits, int rows, int32_t *__restrict__ offsets,
                    int32_t *__restrict__ row_of_slot, int32_t *__restrict__ slot_of_row) {
    extern __shared__ int sm[];
    int *base = sm;               // [G] slots per expert so far
    int *first = base + G;        // [G+1]
    int *scan = first + G + 1;    // [32]
    int *hist = scan + 32;        // [warps with slots][G]
    const int tid = static_cast<int>(threadIdx.x);
    if (tid < G) base[tid] = 0;
    grid_dep_launch_dependents();
    grid_dep_wait();  // the ids may come from the previous kernel
    int e[kSortSteps], rank[kSortSteps];
#pragma unroll
    for (int i = 0; i < kSortSteps; ++i)
        e[i] = expert_of(ids, i * kSortThreads + tid, i * kSortThreads + tid < slots, G);
#pragma unroll
    for (int i = 0; i < kSortSteps; ++i) {
        const int left = slots - i * kSortThreads;
        if (left <= 0) break;
        __syncthreads();
        rank[i] = rank_step(e[i], G, bits, min(kSortWarps, (left + 31) / 32), hist, base);
    }
    __syncthreads();
    const int all = tid < G ? base[tid] : 0;
    first_rows<MASKED>(all, G, rows, first, scan);
    if (MASKED && tid < G) base[tid] = min(all, rows);
    __syncthreads();
    write_offsets<MASKED>(G, first, base, offsets);
#pragma unroll
    for (int i = 0; i < kSortSteps; ++i) {
        const int s = i * kSortThreads + tid;
        if (s < slots) {
            const int row = row_of<MASKED>(e[i], rank[i], first, rows);
            row_of_slot[s] = row;
            if (row >= 0) slot_of_row[row] = s;
        }
    }
    fill_empty_rows<MASKED>(G, rows, first, base, 0, 1, slot_of_row);
}

// First launch of two: ranks inside the chunk into row_of_slot, counts into counts[chunk][4 Gq]
// (zeros past G).
template <typename IdT>
__global__ void __launch_bounds__(kSortThreads, 1)
    moe_rank_kernel(const IdT *__restrict__ ids, int64_t slots, int64_t chunk, int G, int bits,
                    int32_t *__restrict__ row_of_slot, int32_t *__restrict__ counts) {
    extern __shared__ int sm[];
    int *base = sm, *hist = sm + G;
    const int tid = static_cast<int>(threadIdx.x);
    if (tid < G) base[tid] = 0;
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int64_t begin = blockIdx.x * chunk, end = min(begin + chunk, slots);
    int next = expert_of(ids, begin + tid, begin + tid < end, G);
    for (int64_t b = begin; b < end; b += kSortThreads) {
        const int e = next;
        next = expert_of(ids, b + kSortThreads + tid, b + kSortThreads + tid < end, G);
        __syncthreads();
        const int rank = rank_step(e, G, bits, static_cast<int>(min(int64_t(kSortWarps), (end - b + 31) / 32)), hist, base);
        if (b + tid < end) row_of_slot[b + tid] = rank;
    }
    __syncthreads();
    const int row = (G + 3) / 4 * 4;
    if (tid < row) counts[static_cast<int64_t>(blockIdx.x) * row + tid] = tid < G ? base[tid] : 0;
}

// Second launch: rows from the ranks.  Gq: ceil(G / 4), the table's row in 16-byte pieces.
template <typename IdT, bool MASKED>
__global__ void __launch_bounds__(kSortThreads, 1)
    moe_place_kernel(const IdT *__restrict__ ids, int64_t slots, int64_t chunk, int G, int Gq, int rows,
                     const int32_t *__restrict__ counts, int32_t *__restrict__ offsets,
                     int32_t *__restrict__ row_of_slot, int32_t *__restrict__ slot_of_row) {
    __shared__ int count[kSortMaxG], below[kSortMaxG], first[kSortMaxG + 1], scan[32];
    const int tid = static_cast<int>(threadIdx.x);
    count[tid] = below[tid] = 0;
    grid_dep_launch_dependents();
    grid_dep_wait();
    __syncthreads();
    const int me = static_cast<int>(blockIdx.x), chunks = static_cast<int>(gridDim.x);
    const int64_t begin = me * chunk, end = min(begin + chunk, slots);
    // this thread's first slot, loaded under the sums
    int e = expert_of(ids, begin + tid, begin + tid < end, G);
    int rank = begin + tid < end ? row_of_slot[begin + tid] : -1;
    // Each warp adds up every 32nd chunk's row, four experts a lane and four rows in flight:
    // all CTAs read the same table, and one word a load took 12 us of 19 for 128 chunks.
    const int4 *table = reinterpret_cast<const int4 *>(counts);
    for (int q = tid & 31; q < Gq; q += 32) {
        int4 all = make_int4(0, 0, 0, 0), before = make_int4(0, 0, 0, 0);
#pragma unroll 4
        for (int c = tid >> 5; c < chunks; c += kSortWarps) {
            const int4 v = __ldcg(table + static_cast<int64_t>(c) * Gq + q);
            all.x += v.x, all.y += v.y, all.z += v.z, all.w += v.w;
            if (c < me) before.x += v.x, before.y += v.y, before.z += v.z, before.w += v.w;
        }
        // integers: the order does not matter
        atomicAdd(&count[4 * q], all.x), atomicAdd(&below[4 * q], before.x);
        atomicAdd(&count[4 * q + 1], all.y), atomicAdd(&below[4 * q + 1], before.y);
        atomicAdd(&count[4 * q + 2], all.z), atomicAdd(&below[4 * q + 2], before.z);
        atomicAdd(&count[4 * q + 3], all.w), atomicAdd(&below[4 * q + 3], before.w);
    }
    __syncthreads();
    const int all = tid < G ? count[tid] : 0;
    first_rows<MASKED>(all, G, rows, first, scan);
    if (MASKED && tid < G) count[tid] = min(all, rows);
    __syncthreads();
    if (me == 0) write_offsets<MASKED>(G, first, count, offsets);
    for (int64_t s = begin + tid; s < end; s += kSortThreads) {
        const int row = e >= 0 ? row_of<MASKED>(e, rank + below[e], first, rows) : -1;
        row_of_slot[s] = row;
        if (row >= 0) slot_of_row[row] = static_cast<int32_t>(s);
        if (s + kSortThreads < end) {
            e = expert_of(ids, s + kSortThreads, true, G);
            rank = row_of_slot[s + kSortThreads];
        }
    }
    fill_empty_rows<MASKED>(G, rows, first, count, me, chunks, slot_of_row);
}

// Slots per CTA of the two-launch form: a step of 1024, or more so that there are at most
// kSortChunks chunks (each CTA of the second launch reads every chunk's counts).
constexpr int64_t kSortChunks = 148;
static int64_t chunk_of(int64_t slots) {
    const int64_t steps = (slots + kSortThreads - 1) / kSortThreads;
    return (steps + kSortChunks - 1) / kSortChunks * kSortThreads;
}

int64_t moe_sort_workspace(int64_t slots, int G) {
    if (slots <= kSortOneCta) return 0;
    const int64_t chunk = chunk_of(slots);
    return (slots + chunk - 1) / chunk * ((G + 3) / 4) * static_cast<int64_t>(sizeof(int4));
}

template <typename IdT, bool MASKED>
static dg_status_t launch_sort_impl(const IdT *ids, int64_t slots, int G, int64_t rows, int32_t *offsets,
                                    int32_t *row_of_slot, int32_t *slot_of_row, int32_t *workspace,
                                    cudaStream_t stream) {
    int bits = 0;
    while ((1 << bits) < G) ++bits;
    if (slots <= kSortOneCta) {
        static thread_local int configured_device = -1;
        const size_t fixed = sizeof(int) * (2 * static_cast<size_t>(G) + 1 + 32);
        const size_t warps = slots < kSortThreads ? (slots + 31) / 32 : kSortWarps;
        const dg_status_t st = allow_smem(moe_sort_kernel<IdT, MASKED>, sizeof(int) * ((kSortWarps + 2) * kSortMaxG + 33),
                                          configured_device);
        if (st != DG_OK) return st;
        return launch_pdl(moe_sort_kernel<IdT, MASKED>, 1, kSortThreads, fixed + sizeof(int) * warps * G, stream, ids,
                          static_cast<int>(slots), G, bits, static_cast<int>(rows), offsets, row_of_slot, slot_of_row);
    }
    static thread_local int configured_device = -1;
    const size_t smem = sizeof(int) * static_cast<size_t>(kSortWarps + 1) * G;
    dg_status_t st = allow_smem(moe_rank_kernel<IdT>, sizeof(int) * (kSortWarps + 1) * kSortMaxG, configured_device);
    if (st != DG_OK) return st;
    const int64_t chunk = chunk_of(slots);
    const int n = static_cast<int>((slots + chunk - 1) / chunk);
    st = launch_pdl(moe_rank_kernel<IdT>, n, kSortThreads, smem, stream, ids, slots, chunk, G, bits, row_of_slot,
                    workspace);
    if (st != DG_OK) return st;
    return launch_pdl(moe_place_kernel<IdT, MASKED>, n, kSortThreads, 0, stream, ids, slots, chunk, G, (G + 3) / 4,
                      static_cast<int>(rows), static_cast<const int32_t *>(workspace), offsets, row_of_slot,
                      slot_of_row);
}

dg_status_t launch_moe_sort(const void *ids, bool ids64, int64_t slots, int G, bool masked, int64_t rows,
                            int32_t *offsets, int32_t *row_of_slot, int32_t *slot_of_row, int32_t *workspace,
                            cudaStream_t stream) {
    if (ids64) {
        const int64_t *p = static_cast<const int64_t *>(ids);
        return masked ? launch_sort_impl<int64_t, true>(p, slots, G, rows, offsets, row_of_slot, slot_of_row, workspace, stream)
                      : launch_sort_impl<int64_t, false>(p, slots, G, rows, offsets, row_of_slot, slot_of_row, workspace, stream);
    }
    const int32_t *p = static_cast<const int32_t *>(ids);
    return masked ? launch_sort_impl<int32_t, true>(p, slots, G, rows, offsets, row_of_slot, slot_of_row, workspace, stream)
                  : launch_sort_impl<int32_t, false>(p, slots, G, rows, offsets, row_of_slot, slot_of_row, workspace, stream);
}

}  // namespace dg

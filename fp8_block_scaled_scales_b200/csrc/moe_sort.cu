// Tokens sorted by expert: a stable counting sort of the T x k routing slots, into the
// grouped-contiguous layout (each expert's rows start at a multiple of 128) or into the
// masked layout (a slab of M_max rows per expert).
//
//   e(s)   = topk_ids[s] (outside [0, G): the slot is dropped)
//   rank   = number of slots s' < s with e(s') = e(s)
//   row(s) = off[e] + rank, off the prefix sum of the experts' counts rounded up to 128
//            (masked: e * M_max + rank, dropped when rank >= M_max)
//
// One launch of one thread-block cluster: the slots are cut into consecutive pieces, one
// per warp.  Each warp counts its piece per expert (32 slots at a time, equal experts found
// with match.any, so no atomics and the order is fixed); a scan over the warps and, through
// distributed shared memory, over the CTAs turns the counts into each warp's first row per
// expert; a second pass over the piece hands the rows out.  Needs no scratch memory and no
// second launch.  A few slots (a decode step) take a single CTA, whose cost is latency.
#include "dg_device.cuh"
#include "train_internal.h"

namespace dg {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 8;
constexpr int kSortMaxG = 1024;  // one thread per expert in the scans
constexpr int kSortBatch = 8;    // ids a lane loads ahead
// Up to this many slots one CTA is used.
constexpr int64_t kSortOneCta = 4096;

static_assert(kSortMaxG <= kSortThreads, "one thread per expert");

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

template <typename IdT, bool MASKED>
__global__ void __launch_bounds__(kSortThreads, 1)
    moe_sort_kernel(const IdT *__restrict__ ids, int slots, int per_warp, int G, int rows,
                    int32_t *__restrict__ offsets, int32_t *__restrict__ row_of_slot,
                    int32_t *__restrict__ slot_of_row, int ctas) {
    extern __shared__ int sm[];
    int *hist = sm;                       // [active warps][G]
    int *total = hist + kSortWarps * G;   // [G] this CTA's slots per expert
    int *count = total + G;               // [G] all slots per expert
    int *off = count + G;                 // [G+1] first row of each expert
    int *scan = off + G + 1;              // [32]

    const int tid = static_cast<int>(threadIdx.x);
    const int warp = tid >> 5, lane = tid & 31;
    const int rank = ctas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int gw = rank * kSortWarps + warp;
    const uint32_t lower = (1u << lane) - 1u;

    // warps of this CTA that have a piece
    const int left = slots - rank * kSortWarps * per_warp;
    const int active = left <= 0 ? 0 : min(kSortWarps, (left + per_warp - 1) / per_warp);
    for (int i = tid; i < active * G; i += kSortThreads) hist[i] = 0;
    grid_dep_launch_dependents();
    grid_dep_wait();  // the ids may come from the previous kernel
    __syncthreads();

    const int begin = static_cast<int>(min(static_cast<int64_t>(gw) * per_warp, static_cast<int64_t>(slots)));
    const int end = min(begin + per_warp, slots);
    int *mine = hist + warp * G;

    // visits the piece 32 slots at a time: f(slot, expert or -1, peers)
    auto visit = [&](auto f) {
        for (int b = begin; b < end; b += 32 * kSortBatch) {
            int e[kSortBatch];
#pragma unroll
            for (int j = 0; j < kSortBatch; ++j) {
                const int s = b + j * 32 + lane;
                const IdT v = s < end ? __ldg(ids + s) : IdT(-1);
                e[j] = (v >= 0 && v < IdT(G)) ? static_cast<int>(v) : -1;
            }
#pragma unroll
            for (int j = 0; j < kSortBatch; ++j) {
                if (b + j * 32 >= end) break;
                const uint32_t peers = __match_any_sync(0xFFFFFFFFu, e[j]);
                f(b + j * 32 + lane, e[j], peers);
                __syncwarp();
            }
        }
    };

    visit([&](int, int e, uint32_t peers) {
        if (e >= 0 && (peers & lower) == 0) mine[e] += __popc(peers);
    });
    __syncthreads();

    // per expert: exclusive scan over the warps, then over the CTAs
    int below = 0, all = 0;
    if (tid < G) {
        int run = 0;
        for (int w = 0; w < active; ++w) {
            const int c = hist[w * G + tid];
            hist[w * G + tid] = run;
            run += c;
        }
        total[tid] = all = run;
    }
    if (ctas > 1) {
        cluster_sync();
        if (tid < G) {
            all = 0;
            for (int c = 0; c < ctas; ++c) {
                const int v = ld_cluster_s32(mapa_shared(smem_u32(total + tid), static_cast<uint32_t>(c)));
                if (c < rank) below += v;
                all += v;
            }
        }
    }
    // first row of each expert
    int first = 0;
    if (MASKED) {
        first = tid * rows;
        if (tid < G) count[tid] = min(all, rows);
    } else {
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
        first = before + incl - padded;
        if (tid < G) {
            count[tid] = all;
            off[tid] = first;
            if (tid == G - 1) off[G] = first + padded;
        }
    }
    if (tid < G) {
        // masked: hist keeps ranks inside the expert, so that rank >= M_max can be seen
        const int base = below + (MASKED ? 0 : first);
        for (int w = 0; w < active; ++w) hist[w * G + tid] += base;
    }
    __syncthreads();
    if (rank == 0) {
        if (MASKED) {
            if (tid < G) offsets[tid] = count[tid];
        } else {
            if (tid < G) offsets[tid] = off[tid];
            if (tid == 0) offsets[G] = off[G];
        }
    }

    visit([&](int s, int e, uint32_t peers) {
        int row = -1;
        if (e >= 0) {
            const int at = mine[e];
            row = at + __popc(peers & lower);
            if (MASKED) row = row < rows ? e * rows + row : -1;
            __syncwarp(peers);
            if ((peers & lower) == 0) mine[e] = at + __popc(peers);
        }
        if (s < end) {
            row_of_slot[s] = row;
            if (row >= 0) slot_of_row[row] = s;
        }
    });

    // rows without a slot
    if (MASKED) {
        const int n = G * rows;
        for (int r = rank * kSortThreads + tid; r < n; r += ctas * kSortThreads) {
            const int e = r / rows;
            if (r - e * rows >= count[e]) slot_of_row[r] = -1;
        }
    } else {
        for (int e = gw; e < G; e += ctas * kSortWarps)
            for (int r = off[e] + count[e] + lane; r < off[e + 1]; r += 32) slot_of_row[r] = -1;
        for (int r = off[G] + rank * kSortThreads + tid; r < rows; r += ctas * kSortThreads) slot_of_row[r] = -1;
    }
    if (ctas > 1) cluster_sync();  // no CTA leaves while another may read its totals
}

template <typename IdT, bool MASKED>
static dg_status_t launch_sort_impl(const void *ids, int64_t slots, int G, int64_t rows, int32_t *offsets,
                                    int32_t *row_of_slot, int32_t *slot_of_row, cudaStream_t stream) {
    auto kernel = moe_sort_kernel<IdT, MASKED>;
    const int ctas = slots <= kSortOneCta ? 1 : kSortCluster;
    const int64_t pieces = static_cast<int64_t>(ctas) * kSortWarps;
    const int per_warp = static_cast<int>(((slots + pieces - 1) / pieces + 31) / 32 * 32);
    const size_t smem = sizeof(int) * (static_cast<size_t>(kSortWarps) * G + 3 * G + 1 + 32);
    static thread_local int configured_device = -1;
    int device = 0;
    cudaGetDevice(&device);
    if (configured_device != device) {
        const int most = static_cast<int>(sizeof(int) * ((kSortWarps + 3) * kSortMaxG + 33));
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
            return DG_ERR_CUDA;
        configured_device = device;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(kSortThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const IdT *>(ids), static_cast<int>(slots), per_warp, G,
                              static_cast<int>(rows), offsets, row_of_slot, slot_of_row, ctas) == cudaSuccess
               ? DG_OK
               : DG_ERR_CUDA;
}

dg_status_t launch_moe_sort(const void *ids, bool ids64, int64_t slots, int G, bool masked, int64_t rows,
                            int32_t *offsets, int32_t *row_of_slot, int32_t *slot_of_row, const DeviceInfo &dev,
                            cudaStream_t stream) {
    (void)dev;
    if (ids64)
        return masked ? launch_sort_impl<int64_t, true>(ids, slots, G, rows, offsets, row_of_slot, slot_of_row, stream)
                      : launch_sort_impl<int64_t, false>(ids, slots, G, rows, offsets, row_of_slot, slot_of_row, stream);
    return masked ? launch_sort_impl<int32_t, true>(ids, slots, G, rows, offsets, row_of_slot, slot_of_row, stream)
                  : launch_sort_impl<int32_t, false>(ids, slots, G, rows, offsets, row_of_slot, slot_of_row, stream);
}

}  // namespace dg

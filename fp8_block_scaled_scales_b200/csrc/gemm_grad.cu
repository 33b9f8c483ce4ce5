// The two gradient products of a block-scaled FP8 layer C = A B^T, dense and MoE
// grouped-contiguous, from the codes exactly as the forward pass and the quantizers left
// them (row-major, 128x128 block scales): nothing is transposed in memory.
//
//   dgrad: dX[m][k] = sum_nb sdY[m/128][nb] * sW[nb][k/128] * sum_{n in nb} dY[m][n] * W[n][k]
//   wgrad: dW[n][k] = sum_mb sdY[mb][n/128] * sX[mb][k/128] * sum_{m in mb} dY[m][n] * X[m][k]
//
// A block scale is constant over a 128-deep block of either contraction, because the blocks
// are square: that is why the codes of the forward pass serve the backward pass unchanged
// (an 8-bit activation checkpoint that costs nothing to use).
//
// Only the operands' majorness differs from the forward product.  A 128-deep block of an
// operand whose contraction index is the row is a box of 128 rows x 128 bytes; TMA lays it
// out with the 128-byte swizzle, and the MMA reads it as an M- or N-major operand: swizzle
// atoms of 8 contraction rows x 128 bytes, 1024 bytes from one group of 8 rows to the next,
// and the next 128 columns in the next box.  dgrad: dY K-major, W N-major; wgrad: both.
//
// Structure as in the forward tile kernel (one persistent CTA per SM, two TMA producer
// threads, two MMA-issuing threads, eight epilogue warps that scale each 128-deep partial
// in FP32 registers); what differs is the walk: a wgrad tile's contraction runs over its
// expert's row blocks, so its length varies from tile to tile and may be zero (an expert
// without tokens: zeros are stored), and the scales step by a row of the scale arrays.
//
// Measured one call at a time, in brackets twenty in a graph, where the power cap tells: dgrad of 8
// experts, N = K = 4096, 16384 rows in equal parts 241 us (2280 TFLOP/s; the forward product of that
// size 241), 16384 slots in unequal parts 264 (276); dense 4096^3 70 (65), 8192^3 479 (511), forward
// 64 (61) and 444 (460): bound, as the forward kernel, by the round trip of a partial through tensor
// memory (tensor pipe 59 % active).  wgrad dense 4096^3 77 (72), 8192^3 510 (525); in BF16 70 (66) and
// 486 (518): as dgrad but for the wider output's stores.  wgrad of 64 experts, N = 2048, K = 7168, 32768
// slots in FP32 1056 (1138), accumulating, which reads the output too, 1717 (1720), in BF16 735 (846):
// 3.8 GB of FP32 output stored by the warps that also scale the partials, 575 us without the stores,
// 635 us of stores alone.
#include <cuda_bf16.h>

#include "dg_device.cuh"
#include "train_internal.h"

namespace dg {

enum GradMode { kDgrad = 0, kWgrad = 1 };

struct GradParams {
    const float *sA;  // scales of dY [.][Nb]
    const float *sB;  // dgrad: W [G][Nb][Kc]; wgrad: X [.][Kc]
    const int32_t *offsets;  // null: dense
    int G;
    int cap;       // rows of dY
    int N, K;      // dims of W
    int Nb, Kc;    // ceil(N/128), ceil(K/128)
    int num_m;     // dgrad: m-blocks of the allocation; wgrad: row tiles of one expert's dW
    int num_k;     // 256-column tiles of the output
    int splits;    // parts of the contraction, each with an output of its own
    int c_rows;    // output rows from one part (wgrad: and expert) to the next
    int c_end;     // rows of the output in all
    int accumulate;
    uint64_t timeout_ns;
    int *status;
    int debug_flags;
};

constexpr int kGradThreads = 384;
constexpr int kGradRegsLaunch = 168;   // 65536 / 384 rounded down to a multiple of 8
constexpr int kGradRegsProducer = 56;  // warpgroup 0
constexpr int kGradRegsEpilogue = 224; // warpgroups 1, 2
static_assert(128 * kGradRegsProducer + 256 * kGradRegsEpilogue <= kGradThreads * kGradRegsLaunch,
              "setmaxnreg split exceeds the registers the block is launched with");
constexpr int kGradBufs = 2;
constexpr uint32_t kGradUnitBytes = 24;
constexpr int kGradUnits = 8;  // units an epilogue warp works out at a time, one a lane
constexpr uint32_t kGradBHalf = 128 * 128;  // one 128-column box of B

// STAGES operand stages in the ring; BOXES output boxes of 4 KB for each epilogue warp.
template <int STAGES, int BOXES>
struct GradSmem {
    static constexpr uint32_t kABytes = 128 * 128;
    static constexpr uint32_t kBHalf = kGradBHalf;
    static constexpr uint32_t kBBytes = 2 * kBHalf;
    static constexpr uint32_t kCBoxBytes = 32 * 128;  // 32 rows x 128 bytes
    static constexpr uint32_t kOffA = 0;
    static constexpr uint32_t kOffB = kOffA + STAGES * kABytes;
    static constexpr uint32_t kOffC = kOffB + STAGES * kBBytes;
    static constexpr uint32_t kOffBar = kOffC + 8 * BOXES * kCBoxBytes;
    static constexpr uint32_t kNumBars = 3 * STAGES + 2 * kGradBufs + 2;
    // iterations between two uses of a `full` barrier by its MMA thread
    static constexpr int kPeriod = STAGES % 2 ? 2 * STAGES : STAGES;
    static constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;
    static constexpr uint32_t kOffUnits = kOffMisc + 16;  // a table of units for each epilogue warp
    static constexpr uint32_t kBytes = kOffUnits + 8 * kGradUnits * kGradUnitBytes;
    static constexpr uint32_t kDynamicBytes = kBytes + 1024;  // slack for 1024-byte alignment
};

// Shared-memory descriptor of an operand stored with its M or N index contiguous: rows of
// 128 bytes (one contraction index each) with the 128-byte swizzle.  Leading byte offset:
// from one 128-byte-wide column of atoms to the next (the next box, kBHalf); stride byte
// offset: from 8 contraction rows to the next 8 (1024).  32 rows on (one MMA) is 4096 bytes.
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(kGradBHalf >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// Instruction descriptor bits for M- / N-major operands.
constexpr uint32_t kIdescAMajorM = 1u << 15;
constexpr uint32_t kIdescBMajorN = 1u << 16;

__device__ __forceinline__ void tma_store_add_2d(const CUtensorMap *map, const void *smem_src, int32_t c0,
                                                 int32_t c1) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(smem_src)), "r"(c0), "r"(c1)
                 : "memory");
}

// Block scales along a contraction whose blocks are `sa` / `sb` floats apart; otherwise as
// ScaleStream: lane l holds the product of block (base + l), the next 32 are loaded ahead.
struct StridedScales {
    const float *a;
    const float *b;
    int64_t sa, sb;
    int end;
    float cur, next;

    __device__ __forceinline__ float load(int base) const {
        const int k = base + lane_id();
        return k < end ? __ldg(a + k * sa) * __ldg(b + k * sb) : 0.0f;
    }
    __device__ __forceinline__ void set(const float *a0, const float *b0, int64_t step_a, int64_t step_b, int n) {
        a = a0;
        b = b0;
        sa = step_a;
        sb = step_b;
        end = n;
    }
    __device__ __forceinline__ float scale(int i) {
        if ((i & 31) == 0 && i > 0) {
            cur = next;
            next = load(i + 32);
        }
        return __shfl_sync(0xFFFFFFFFu, cur, i & 31);
    }
};

// What the epilogue needs of a unit.
struct UnitEntry {
    int blocks, c_row, c_col, narrow, sa_at, sb_row;
};
static_assert(sizeof(UnitEntry) == kGradUnitBytes, "table size");

// One unit of work: a 128 x 256 output tile or a 128 x 128 half of one.
struct GradUnit {
    int blocks;    // 128-deep blocks of the contraction
    int a_row, a_col;  // TMA coordinates of dY at block 0; block i adds 128 * i to the row or the column
    int b_row, b_col;              // of B; block i adds 128 * i to the row
    int c_row, c_col;              // of the output
    bool narrow;                   // 128 columns only
    int sa_at;                     // index into dY's scales at block 0 (its step: 1 or Nb)
    int sb_row;                    // row of B's scales at block 0
};

// Row tiles of a raster group: as in the forward kernel 32 dense (8192^3, side by side: dgrad 450 us
// against 463 with 8, wgrad 5 % shorter), 8 grouped.
__device__ __forceinline__ int grad_raster(const GradParams &p) { return p.offsets ? 8 : 32; }

template <int MODE>
__device__ __forceinline__ GradUnit grad_unit(const GradParams &p, int num_m, int t, int h) {
    GradUnit u;
    int g = 0, mb, kt;
    if (MODE == kDgrad) {
        const int per = num_m * p.num_k, part = t / per;
        t -= part * per;
        const int b0 = p.Nb * part / p.splits;
        // m-block fastest inside raster groups, so that a group's tiles of W are read from L2
        const int kRaster = grad_raster(p);
        const int group = t / (kRaster * p.num_k);
        const int first = group * kRaster;
        const int gm = min(kRaster, num_m - first);
        const int local = t - group * kRaster * p.num_k;
        mb = first + local % gm;
        kt = local / gm;
        if (p.offsets) {
            int lo = 0, hi = p.G;  // the g with off[g] <= 128 mb < off[g+1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(p.offsets + mid) <= mb * 128) lo = mid; else hi = mid;
            }
            g = lo;
        }
        u.blocks = p.Nb * (part + 1) / p.splits - b0;
        u.a_row = mb * 128;
        u.a_col = b0 * 128;
        u.b_row = g * p.N + b0 * 128;
        u.c_row = part * p.c_rows + mb * 128;
        u.sa_at = mb * p.Nb + b0;
        u.sb_row = g * p.Nb + b0;
    } else {
        const int kRaster = grad_raster(p);
        const int per = p.num_m * p.num_k;
        const int slice = t / per;  // part of an expert's rows
        t -= slice * per;
        g = slice / p.splits;
        const int part = slice - g * p.splits;
        const int group = t / (kRaster * p.num_k);
        const int first = group * kRaster;
        const int gm = min(kRaster, p.num_m - first);
        const int local = t - group * kRaster * p.num_k;
        mb = first + local % gm;
        kt = local / gm;
        const int m0 = p.offsets ? __ldg(p.offsets + g) : 0;
        const int m1 = p.offsets ? __ldg(p.offsets + g + 1) : p.cap;
        const int blocks = (m1 - m0 + 127) / 128, b0 = blocks * part / p.splits;
        u.blocks = blocks * (part + 1) / p.splits - b0;
        u.a_row = m0 + b0 * 128;
        u.a_col = mb * 128;
        u.b_row = u.a_row;
        u.c_row = slice * p.c_rows + mb * 128;
        u.sa_at = (m0 / 128 + b0) * p.Nb + mb;
        u.sb_row = m0 / 128 + b0;
    }
    const int col = kt * 256 + (h > 0 ? 128 : 0);
    u.narrow = h >= 0 || col + 128 >= p.K;
    if (col >= p.K) u.blocks = -1;  // the second half of a tile that has none: nothing to do
    u.b_col = u.c_col = col;
    return u;
}

template <int MODE, bool F32, int STAGES, int BOXES>
__global__ void __launch_bounds__(kGradThreads, 1)
    grad_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const GradParams p) {
    using L = GradSmem<STAGES, BOXES>;
    constexpr int kColsPerWarp = 128;
    constexpr uint32_t kTmemCols = tmem_cols_for(kGradBufs * 256);
    constexpr uint32_t kMajor = kIdescBMajorN | (MODE == kWgrad ? kIdescAMajorM : 0u);
    constexpr uint32_t kIdescWide = idesc_e4m3_f32(128, 256) | kMajor;
    constexpr uint32_t kIdescNarrow = idesc_e4m3_f32(128, 128) | kMajor;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
    uint64_t *empty = full + 2 * STAGES;
    uint64_t *tfull = empty + STAGES;
    uint64_t *tempty = tfull + kGradBufs;
    uint64_t *mdone = tempty + kGradBufs;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffMisc + 4);
    volatile int *groups_bad = reinterpret_cast<volatile int *>(smem + L::kOffMisc + 8);

    const int warp = static_cast<int>(threadIdx.x >> 5);
    const int lane = lane_id();

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 2);
            mbar_init(&full[STAGES + s], 2);
            mbar_init(&empty[s], 1);
        }
        for (int q = 0; q < 2; ++q) mbar_init(&mdone[q], 1);
        for (int b = 0; b < kGradBufs; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 8);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmC);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    grid_dep_wait();  // inputs and outputs are touched only from here on
    grid_dep_launch_dependents();
    if (warp == 3) {
        // the contract of group_offsets, as in the forward product: a violation computes nothing.
        // This warp alone writes the flag, so that no other thread's first value can follow it.
        bool bad = false;
        for (int g = lane; p.offsets && g <= p.G; g += 32) {
            const int o = __ldg(p.offsets + g);
            const int prev = g > 0 ? __ldg(p.offsets + g - 1) : 0;
            bad |= (o & 127) != 0 || o < prev || o > p.cap || (g == 0 && o != 0);
        }
        bad = __any_sync(0xFFFFFFFFu, bad);
        if (lane == 0) {
            *groups_bad = bad ? 1 : 0;
            if (bad && blockIdx.x == 0) record_failure(p.status, kStatusBadGroups, 3, -1);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const int num_m = MODE == kDgrad && p.offsets ? __ldg(p.offsets + p.G) / 128 : p.num_m;
    const int num_tiles = *groups_bad ? 0 : (MODE == kWgrad ? p.G : 1) * p.splits * num_m * p.num_k;
    // a last round that would keep at most half the CTAs busy runs as half tiles
    const int grid = static_cast<int>(gridDim.x);
    int tiles_wide = num_tiles, num_units = num_tiles;
    if (num_tiles > 0) {
        const int last_round = num_tiles - ((num_tiles - 1) / grid) * grid;
        if (2 * last_round <= grid) {
            tiles_wide = num_tiles - last_round;
            num_units = num_tiles + last_round;
        }
    }
    auto unit_at = [&](int u) {
        return u < tiles_wide
                   ? grad_unit<MODE>(p, num_m, u, -1)
                   : grad_unit<MODE>(p, num_m, tiles_wide + (u - tiles_wide) / 2, (u - tiles_wide) & 1);
    };

    if (warp < 4) {
        regs_dealloc<kGradRegsProducer>();
        if ((warp == 0 || warp == 3) && lane == 0) {
            // ----------------------------------------------------------- producers
            // One thread loads dY, the other B's one or two boxes, for every iteration: both
            // see every phase of `empty` in order, whatever the number of stages.  A stage
            // has two `full` barriers, one for each MMA thread, so that each of those is
            // waited on by one thread alone and in order too.
            const bool loads_a = warp == 0;
            uint32_t issued = 0, parity_bits = 0;  // per full barrier: its last phase
            int it = 0, s = 0, q = 0;
            uint32_t v = 0, x = 0;  // it / STAGES, it / kPeriod
            bool ok = true;
            for (int w = static_cast<int>(blockIdx.x); w < num_units && ok; w += grid) {
                const GradUnit u = unit_at(w);
                for (int i = 0; i < u.blocks; ++i, ++it) {
                    if (!mbar_wait(&empty[s], (v & 1u) ^ 1u, abort_flag, p.timeout_ns)) {
                        record_failure(p.status, kStatusTimeout, 0, it);
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    const int bar = q * STAGES + s;
                    if (!((p.debug_flags & 1) && it == 0)) {  // test hook: never fill stage 0
                        if (loads_a) {
                            mbar_arrive_expect_tx(&full[bar], L::kABytes);
                            uint8_t *dst = smem + L::kOffA + s * L::kABytes;
                            if (MODE == kDgrad)
                                tma_load_2d(dst, &tmA, &full[bar], u.a_col + i * 128, u.a_row);
                            else
                                tma_load_2d(dst, &tmA, &full[bar], u.a_col, u.a_row + i * 128);
                        } else {
                            mbar_arrive_expect_tx(&full[bar], u.narrow ? L::kBHalf : L::kBBytes);
                            uint8_t *dst = smem + L::kOffB + s * L::kBBytes;
                            tma_load_2d(dst, &tmB, &full[bar], u.b_col, u.b_row + i * 128);
                            if (!u.narrow)
                                tma_load_2d(dst + L::kBHalf, &tmB, &full[bar], u.b_col + 128, u.b_row + i * 128);
                        }
                        issued |= 1u << bar;
                        parity_bits = (parity_bits & ~(1u << bar)) | ((x & 1u) << bar);
                    }
                    q ^= 1;
                    if (++s == STAGES) {
                        s = 0;
                        ++v;
                        if (it % L::kPeriod == L::kPeriod - 1) ++x;
                    }
                }
            }
            // every load issued must land before the CTA may exit
            const int never = 0;
            for (int bar = 0; bar < 2 * STAGES; ++bar)
                if (issued & (1u << bar))
                    if (!mbar_wait(&full[bar], (parity_bits >> bar) & 1u, &never, p.timeout_ns))
                        record_failure(p.status, kStatusTimeout, 0, -1 - bar);
        } else if ((warp == 1 || warp == 2) && lane == 0) {
            // ------------------------------------------------------- MMA (two threads)
            const int q = warp - 1;
            const uint32_t a0 = smem_u32(smem + L::kOffA);
            const uint32_t b0 = smem_u32(smem + L::kOffB);
            bool any = false, ok = true;
            int it = 0;
            for (int w = static_cast<int>(blockIdx.x); w < num_units && ok; w += grid) {
                const GradUnit u = unit_at(w);
                const uint32_t idesc = u.narrow ? kIdescNarrow : kIdescWide;
                for (int i = 0; i < u.blocks; ++i, ++it) {
                    if ((it & 1) != q) continue;
                    const int s = it % STAGES;
                    const uint32_t v = static_cast<uint32_t>(it / L::kPeriod);  // phase of this thread's barrier
                    const int buf = it % kGradBufs;
                    const uint32_t x = static_cast<uint32_t>(it / kGradBufs);
                    const uint64_t adesc = MODE == kDgrad ? sdesc_kmajor_sw128(a0 + s * L::kABytes)
                                                          : sdesc_mnmajor_sw128(a0 + s * L::kABytes);
                    const uint64_t bdesc = sdesc_mnmajor_sw128(b0 + s * L::kBBytes);
                    const uint32_t d = tmem_base + static_cast<uint32_t>(buf * 256);
                    if (!mbar_wait(&full[q * STAGES + s], v & 1u, abort_flag, p.timeout_ns) ||
                        !mbar_wait(&tempty[buf], (x & 1u) ^ 1u, abort_flag, p.timeout_ns)) {
                        record_failure(p.status, kStatusTimeout, 1, it);
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // 32 contraction indices an instruction: 32 bytes along a K-major row, or
                    // 32 rows of 128 bytes
                    constexpr uint32_t kStepA = MODE == kDgrad ? 32u >> 4 : 4096u >> 4;
                    constexpr uint32_t kStepB = 4096u >> 4;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_e4m3(d, adesc + kStepA * k, bdesc + kStepB * k, idesc, k > 0 ? 1u : 0u);
                    umma_commit(&empty[s]);
                    umma_commit(&tfull[buf]);
                    any = true;
                }
            }
            if (any) {  // the tensor memory may only be released once every MMA issued is done
                const int never = 0;
                umma_commit(&mdone[q]);
                if (!mbar_wait(&mdone[q], 0, &never, p.timeout_ns)) record_failure(p.status, kStatusTimeout, 1, -1);
            }
        }
    } else {
        regs_alloc<kGradRegsEpilogue>();
        // -------------------------------------------------------------- epilogue
        const int ew = warp - 4;
        const int quarter = warp & 3;
        const int half = ew >> 2;
        uint8_t *boxes = smem + L::kOffC + ew * BOXES * L::kCBoxBytes;
        // Working out a unit (divisions, offsets) takes 700 cycles and its first scales as many
        // again, which a tile of a few blocks would wait for; so lanes work out the next eight
        // units at once, and a tile's first scales are loaded before the tile before it is stored.
        UnitEntry *table = reinterpret_cast<UnitEntry *>(smem + L::kOffUnits) + ew * kGradUnits;
        const int my_units = static_cast<int>(blockIdx.x) < num_units
                                 ? (num_units - 1 - static_cast<int>(blockIdx.x)) / grid + 1
                                 : 0;
        StridedScales scales;
        float first_scales = 0.0f;
        auto prepare = [&](int n) {  // unit n of this CTA: its table entry and its first scales
            if (n >= my_units) return;
            if (n % kGradUnits == 0) {
                __syncwarp();
                if (lane < kGradUnits && n + lane < my_units) {
                    const GradUnit u = unit_at(static_cast<int>(blockIdx.x) + (n + lane) * grid);
                    table[lane] = UnitEntry{u.blocks, u.c_row, u.c_col, u.narrow ? 1 : 0, u.sa_at, u.sb_row};
                }
                __syncwarp();
            }
            const UnitEntry e = table[n % kGradUnits];
            const int col0 = e.c_col + half * (e.narrow ? kColsPerWarp / 2 : kColsPerWarp);
            const bool valid = col0 < p.K;
            scales.set(p.sA + e.sa_at, p.sB + static_cast<int64_t>(e.sb_row) * p.Kc + (valid ? col0 / 128 : 0),
                       MODE == kDgrad ? 1 : p.Nb, p.Kc, valid ? e.blocks : 0);
            first_scales = scales.load(0);
        };
        float2 acc[kColsPerWarp / 2];
        int it = 0;
        bool ok = true;
        prepare(0);
        for (int n = 0; n < my_units && ok; ++n) {
            const UnitEntry u = table[n % kGradUnits];
            if (u.blocks < 0 || (MODE == kWgrad && u.blocks == 0 && p.accumulate)) {
                prepare(n + 1);
                continue;
            }
            const int ncols = u.narrow ? kColsPerWarp / 2 : kColsPerWarp;
            const int col0 = u.c_col + half * ncols;
            scales.cur = first_scales;
            scales.next = scales.load(32);
#pragma unroll
            for (int j = 0; j < kColsPerWarp / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
            for (int i = 0; i < u.blocks; ++i, ++it) {
                const int buf = it % kGradBufs;
                const uint32_t x = static_cast<uint32_t>(it / kGradBufs);
                const float scale = scales.scale(i);
                const float2 s2 = make_float2(scale, scale);
                if (!mbar_wait(&tfull[buf], x & 1u, abort_flag, p.timeout_ns)) {
                    record_failure(p.status, kStatusTimeout, 2, it);
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                       static_cast<uint32_t>(buf * 256 + half * ncols);
                promote_kblock<kColsPerWarp, kPromoChunk>(taddr, s2, acc, ncols / kPromoChunk, [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tempty[buf]);
                });
            }
            if (!ok) break;
            prepare(n + 1);
            // rows c_row + 32 * quarter + lane; one box of 32 rows x 128 bytes at a time
            constexpr int kBoxCols = F32 ? 32 : 64;
            const int row0 = u.c_row + quarter * 32;
#pragma unroll
            for (int j = 0; j < kColsPerWarp / kBoxCols; ++j) {
                if (j * kBoxCols >= ncols) break;
                uint8_t *cstage = boxes + (j % BOXES) * L::kCBoxBytes;
                // the store before the last BOXES - 1 has finished reading this box
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(BOXES - 1) : "memory");
                __syncwarp();
                uint8_t *rowp = cstage + lane * 128;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint4 o;
                    if (F32) {
                        const float2 *y = acc + j * 16 + c * 2;
                        o = make_uint4(__float_as_uint(y[0].x), __float_as_uint(y[0].y), __float_as_uint(y[1].x),
                                       __float_as_uint(y[1].y));
                    } else {
                        const float2 *y = acc + j * 32 + c * 4;
                        o = make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y),
                                       pack_bf16x2(y[2].x, y[2].y), pack_bf16x2(y[3].x, y[3].y));
                    }
                    *reinterpret_cast<uint4 *>(rowp + ((c ^ (lane & 7)) << 4)) = o;
                }
                fence_async_smem();
                __syncwarp();
                // a box that starts past the matrix edge is skipped, not clipped
                if (lane == 0 && col0 + j * kBoxCols < p.K && row0 < p.c_end) {
                    if (F32 && p.accumulate)
                        tma_store_add_2d(&tmC, cstage, col0 + j * kBoxCols, row0);
                    else
                        tma_store_2d(&tmC, cstage, col0 + j * kBoxCols, row0);
                }
                if (lane == 0) bulk_commit();  // an empty group keeps the count
            }
        }
        if (lane == 0) bulk_wait_all0();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

// The parts of a split product added up in order: out = sum_s parts[s] (+ out), four columns a
// thread; a part is `stride` floats.
template <bool F32>
__global__ void __launch_bounds__(256)
    grad_join_kernel(const float *__restrict__ parts, int splits, int64_t stride, int64_t quads, int accumulate,
                     void *__restrict__ out) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= quads) return;
    const float4 *p = reinterpret_cast<const float4 *>(parts) + i;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (F32 && accumulate) sum = reinterpret_cast<const float4 *>(out)[i];
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
        const float4 v = __ldcg(p + s * (stride / 4));
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
    if (F32)
        reinterpret_cast<float4 *>(out)[i] = sum;
    else
        reinterpret_cast<uint2 *>(out)[i] = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
}

// Parts that a dense product's contraction of `blocks` 128-deep blocks is cut into: as many
// as leave no half tile without an SM, of four blocks at least.  A block takes 0.4 us on the
// way through a tile, the sums' launch 2 us, so short contractions stay whole.  wgrad (whole and
// split): 256 x 256 from 4096 rows 16.0 and 8.3 us, 512 x 512 from 8192 27 and 12, from 2048
// 10.4 and 8.5, 528 x 784 from 1000 (8 blocks) 7.8 and 8.8; dgrad of 16 rows, N = K = 4096, 13.8
// and 11.4.  Parts of two or six blocks were no faster.
constexpr int kSplitBlocks = 4, kSplitMost = 16, kSplitFrom = 12;
constexpr int64_t kSplitSms = 148;
static int grad_splits(int64_t rows, int64_t cols, int64_t blocks) {
    const int64_t tiles = ((rows + 127) / 128) * ((cols + 255) / 256);
    if (blocks < kSplitFrom) return 1;
    int64_t n = kSplitSms / (2 * tiles);
    if (n > blocks / kSplitBlocks) n = blocks / kSplitBlocks;
    if (n > kSplitMost) n = kSplitMost;
    return n < 2 ? 1 : static_cast<int>(n);
}

int64_t grad_workspace(bool wgrad, int64_t M, int64_t N, int64_t K) {
    const int64_t rows = wgrad ? N : M, n = grad_splits(rows, K, ((wgrad ? M : N) + 127) / 128);
    return n > 1 ? n * ((rows + 127) / 128 * 128) * K * 4 : 0;
}

template <int MODE, bool F32, int STAGES, int BOXES>
static dg_status_t launch_grad_impl(const GradArgs &a, int splits, const DeviceInfo &dev, cudaStream_t stream) {
    using L = GradSmem<STAGES, BOXES>;
    static_assert(L::kDynamicBytes <= 232448, "shared memory budget");
    static_assert(kGradBufs % 2 == 0, "each MMA thread must own its buffers");
    CUtensorMap tmA, tmB, tmC;
    const uint64_t b_rows = MODE == kDgrad ? static_cast<uint64_t>(a.G) * a.N : static_cast<uint64_t>(a.M);
    // rows of one output; a split product's parts are padded to whole tiles
    const int64_t out_rows = MODE == kDgrad ? a.M : a.N;
    const int64_t part_rows = splits > 1 ? (out_rows + 127) / 128 * 128 : out_rows;
    const uint64_t c_rows = static_cast<uint64_t>(part_rows) * splits * (MODE == kWgrad ? a.G : 1);
    dg_status_t st = make_tmap_2d(&tmA, a.dY, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.M, a.N, 128, 128,
                                  CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != DG_OK) return st;
    st = make_tmap_2d(&tmB, a.B, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, b_rows, a.K, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != DG_OK) return st;
    st = F32 ? make_tmap_2d(&tmC, a.C, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, c_rows, a.K, 32, 32,
                            CU_TENSOR_MAP_SWIZZLE_128B)
             : make_tmap_2d(&tmC, a.C, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c_rows, a.K, 32, 64,
                            CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != DG_OK) return st;

    const KernelControl ctl = kernel_control();
    GradParams p;
    p.sA = a.sdY;
    p.sB = a.sB;
    p.offsets = a.offsets;
    p.G = a.G;
    p.cap = static_cast<int>(a.M);
    p.N = static_cast<int>(a.N);
    p.K = static_cast<int>(a.K);
    p.Nb = static_cast<int>((a.N + 127) / 128);
    p.Kc = static_cast<int>((a.K + 127) / 128);
    p.num_m = MODE == kDgrad ? static_cast<int>((a.M + 127) / 128) : p.Nb;
    p.num_k = static_cast<int>((a.K + 255) / 256);
    p.splits = splits;
    p.c_rows = static_cast<int>(part_rows);
    p.c_end = static_cast<int>(c_rows);
    p.accumulate = a.accumulate ? 1 : 0;
    p.timeout_ns = ctl.timeout_ns;
    p.status = ctl.status;
    p.debug_flags = ctl.debug_flags;

    auto kernel = grad_gemm_kernel<MODE, F32, STAGES, BOXES>;
    static thread_local int configured_device = -1;
    int device = 0;
    cudaGetDevice(&device);
    if (configured_device != device) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(L::kDynamicBytes)) != cudaSuccess)
            return DG_ERR_CUDA;
        // the register split inside the kernel must fit what a launch provides
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) return DG_ERR_CUDA;
        if (128 * kGradRegsProducer + 256 * kGradRegsEpilogue > kGradThreads * fa.numRegs) return DG_ERR_CUDA;
        configured_device = device;
    }
    const int64_t tiles = static_cast<int64_t>(MODE == kWgrad ? a.G : 1) * splits * p.num_m * p.num_k;
    if (tiles > 0x3FFFFFFFLL) return DG_ERR_SHAPE;
    // twice the tiles: a single partial round may run as half tiles
    const int grid = static_cast<int>(2 * tiles < dev.num_sms ? 2 * tiles : dev.num_sms);
    return launch_pdl(kernel, grid, kGradThreads, L::kDynamicBytes, stream, tmA, tmB, tmC, p);
}

// A split product: parts into the workspace, then their sums.
template <int MODE>
static dg_status_t launch_split(const GradArgs &a, int splits, const DeviceInfo &dev, cudaStream_t stream) {
    GradArgs part = a;
    part.C = a.workspace;
    part.accumulate = false;
    dg_status_t st = launch_grad_impl<MODE, true, 4, 1>(part, splits, dev, stream);
    if (st != DG_OK) return st;
    const int64_t rows = MODE == kDgrad ? a.M : a.N, quads = rows * a.K / 4;
    const int64_t stride = (rows + 127) / 128 * 128 * a.K;
    return launch_pdl(a.fp32 ? grad_join_kernel<true> : grad_join_kernel<false>, static_cast<int>((quads + 255) / 256), 256,
                      0, stream, static_cast<const float *>(a.workspace), splits, stride, quads, a.accumulate ? 1 : 0,
                      a.C);
}

dg_status_t launch_dgrad(const GradArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    const int splits = a.offsets ? 1 : grad_splits(a.M, a.K, (a.N + 127) / 128);
    return splits > 1 ? launch_split<kDgrad>(a, splits, dev, stream)
                      : launch_grad_impl<kDgrad, false, 4, 1>(a, 1, dev, stream);
}

// Operand stages against output boxes.  An output tile is 128 KB (FP32): with few blocks of
// contraction a tile its stores matter more than a fourth stage, with many the stages do.
// Measured side by side, back to back (three stages and two boxes, four and one): 64 experts of N = 2048, K = 7168 over
// 32768 slots, 4 blocks a tile on average, 975-1045 and 1090-1120 us; 8 experts of 4096^2, 16
// blocks, 320 and 320; 4096^3, 32 blocks, 79.8 and 75.7; 8192^3, 64 blocks, 535 and 525.
constexpr int64_t kWgradLongBlocks = 24;

template <bool F32>
static dg_status_t launch_wgrad_impl(const GradArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    return a.M / 128 > kWgradLongBlocks * a.G ? launch_grad_impl<kWgrad, F32, 4, 1>(a, 1, dev, stream)
                                              : launch_grad_impl<kWgrad, F32, 3, 2>(a, 1, dev, stream);
}

dg_status_t launch_wgrad(const GradArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    const int splits = a.offsets ? 1 : grad_splits(a.N, a.K, (a.M + 127) / 128);
    if (splits > 1) return launch_split<kWgrad>(a, splits, dev, stream);
    return a.fp32 ? launch_wgrad_impl<true>(a, dev, stream) : launch_wgrad_impl<false>(a, dev, stream);
}

}  // namespace dg

// Matrix products grouped by expert, with ragged numbers of rows: out_r = W_e x_r for the rows r of every
// expert e, and the gate/up pair of them with SwiGLU, on the tcgen05 tensor cores.
//
// A tile is up to 128 rows of one expert (the MMA's M) by NT rows of its matrix (the MMA's N: 256, or 128
// where 256 would leave SMs without a tile). A persistent CTA per SM takes tiles blockIdx, blockIdx + grid,
// ...: every role finds a tile's expert in a prefix table of row tiles that the CTA makes from `offsets` when
// it starts. Roles, one warp each unless said otherwise:
//   - producer: tiled TMA loads of 128 bytes of k per row into a ring of stages. Weight rows come by two boxes
//     (for SwiGLU: the gate rows and the up rows of the same 128 columns of h, so that one thread has both for
//     its row), input rows that follow one another by boxes of 32;
//   - four warps gather the input rows of an index with 16-byte asynchronous copies, 8 lanes a row, in the
//     layout that TMA writes. (Gathering TMA loads of four rows were tried first: 32 of them per stage took
//     about 2700 cycles to issue, five times the MMAs of a q8 stage.) Rows that no expert has are not loaded;
//   - q8: two warps bring the scale bytes (one word per row and stage) into the order the tensor cores take;
//   - MMA: one thread; four K slices per stage, accumulators in tensor memory. bf16 has two accumulators of
//     NT columns. q8 needs tensor memory for scales too, so its two accumulators of 256 share 32 columns:
//     the next tile starts once the epilogue has read those, which it does first;
//   - epilogue, four warps (one per quarter of the tensor-memory lanes = 32 rows): SwiGLU and the rounding on
//     registers (a thread has 32 neighbouring columns of one row: a whole q8 block), then through shared
//     memory so that rows are stored in pieces of 128 bytes.
// Every wait is bounded; a wait that runs out is recorded (pmoe_grouped_error) and the CTA's roles finish in
// turn, after their copies and MMAs in flight have landed.
#include <cuda_bf16.h>

#include <atomic>

#include "common.h"
#include "layer.cuh"
#include "q8.cuh"
#include "tma.cuh"
#include "umma.cuh"

namespace pmoe {

namespace {

constexpr int kMaxDenseExperts = 2048;
constexpr int kRows = 128;      // rows of a tile
constexpr int kRowBytes = 128;  // bytes of k per row and stage
constexpr int kGatherWarps = 4;
constexpr int kThreads = 256 + 32 * kGatherWarps; // producer, MMA, two scale warps, epilogue (4), gather (4)
constexpr int kStageRowBytes = 128; // epilogue staging: bytes per row
constexpr uint64_t kDrainNs = 1000ull * 1000 * 1000;

// code of the first wait that ran out in any grouped product since pmoe_grouped_error last read it
__device__ int g_grouped_error[2];

struct Grouped {
    int E, N, K, n, rows, width, iters, ntiles; // width: output columns; iters: stages per tile
    const uint8_t *x, *ws, *xs;
    const int32_t *index, *offsets;
    void *out;
    uint8_t *out_scales;
    uint64_t limit_ns;
};

template <bool Q8IN, int NT> struct Shape {
    static constexpr int kA = kRows * kRowBytes, kB = NT * kRowBytes;
    static constexpr int kScales = Q8IN ? (kRows + NT) * 4 : 0;
    static constexpr int kStages = NT == 256 ? 4 : 6;
    // tensor memory: two accumulators; q8 with 256 columns: the second starts 32 columns early
    static constexpr bool kOverlap = Q8IN && NT == 256;
    static constexpr int kSecond = kOverlap ? NT - 32 : NT;
    static constexpr int kScaleCols = kSecond + NT; // then two sets of scale columns
    static constexpr int kTmemCols = kScaleCols + (Q8IN ? 32 : 0) <= 256 ? 256 : 512;
    static_assert(kScaleCols + (Q8IN ? 32 : 0) <= 512, "tensor memory");
    static constexpr int kStageAt = kStages * (kA + kB);
    static constexpr int kStagingAt = kStageAt + kStages * kScales;
    static constexpr int kBarAt = kStagingAt + 4 * 32 * kStageRowBytes;
    static constexpr int kTableAt = kBarAt + 512;
    static constexpr size_t smem(int E) { return (size_t)kTableAt + 4 * (E + 1) + 1024; } // 1024: alignment
};
static_assert(Shape<true, 256>::smem(kMaxDenseExperts) <= 227 * 1024, "shared memory");
static_assert(Shape<true, 128>::smem(kMaxDenseExperts) <= 227 * 1024, "shared memory");

struct Bars {
    uint64_t full[6], gathered[6], scales[6], empty[6], acc_full[2], acc_free[2], done;
    uint32_t tmem;
    int abort;
    int part[kThreads / 32];
};
static_assert(sizeof(Bars) <= 512, "barriers");

// A wait that gives up after limit_ns, or as soon as another role has given up.
struct Waiter {
    Bars *b;
    uint64_t limit_ns;
    __device__ bool operator()(uint64_t *bar, uint32_t parity, int where) const
    {
        if (pipe::mbar_try_wait(bar, parity))
            return true;
        const uint64_t deadline = pipe::globaltimer() + limit_ns;
        for (int it = 1;; ++it) {
            if (pipe::mbar_try_wait(bar, parity))
                return true;
            if ((it & 3) == 0) {
                if (*reinterpret_cast<volatile int *>(&b->abort))
                    return false;
                if (pipe::globaltimer() > deadline) {
                    *reinterpret_cast<volatile int *>(&b->abort) = 1;
                    if (atomicCAS(&g_grouped_error[0], 0, 3) == 0)
                        g_grouped_error[1] = where;
                    return false;
                }
            }
        }
    }
};

// The same for a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool warp_wait(const Waiter &wait, uint64_t *bar, uint32_t parity, int where)
{
    return __all_sync(0xffffffffu, wait(bar, parity, where));
}

// After a role has given up: until the barrier's phase completes, with a long bound.
__device__ void drain(uint64_t *bar, uint32_t parity)
{
    const uint64_t deadline = pipe::globaltimer() + kDrainNs;
    while (!pipe::mbar_try_wait(bar, parity) && pipe::globaltimer() < deadline) {
    }
}

// One tile: its expert, rows and first matrix row (or h column).
struct Tile {
    int e, row0, rows, col0;
};

// Rows of expert e as far as `offsets` is sound: [first, last) within [0, rows).
__device__ __forceinline__ int2 expert_rows(const Grouped &g, int e)
{
    const int a = max(0, __ldg(g.offsets + e)), b = min(g.rows, __ldg(g.offsets + e + 1));
    return make_int2(a, max(a, b));
}

__device__ __forceinline__ Tile tile_at(const Grouped &g, const int *first, int t, int cols)
{
    const int m = t / g.ntiles;
    int lo = 0, hi = g.E; // first[lo] <= m < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (first[mid] <= m)
            lo = mid;
        else
            hi = mid;
    }
    const int2 r = expert_rows(g, lo);
    Tile T;
    T.e = lo;
    T.row0 = r.x + (m - first[lo]) * kRows;
    T.rows = min(kRows, r.y - T.row0);
    T.col0 = (t % g.ntiles) * cols;
    return T;
}

// Prefix sums of the experts' row tiles, first[0..E]; all threads.
__device__ void row_tiles(const Grouped &g, int *first, int *part)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (g.E + kThreads - 1) / kThreads;
    const int e0 = min(g.E, tid * per), e1 = min(g.E, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        const int2 r = expert_rows(g, e);
        sum += (r.y - r.x + kRows - 1) / kRows;
    }
    int inc = sum;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, inc, s);
        inc += lane >= s ? n : 0;
    }
    if (lane == 31)
        part[warp] = inc;
    __syncthreads();
    int at = inc - sum;
    for (int w = 0; w < warp; ++w)
        at += part[w];
    for (int e = e0; e < e1; ++e) {
        first[e] = at;
        const int2 r = expert_rows(g, e);
        at += (r.y - r.x + kRows - 1) / kRows;
    }
    if (tid == kThreads - 1)
        first[g.E] = at; // the last thread's range ends at E
    __syncthreads();
}

// 16 bytes to shared memory, the first `bytes` of them (16 or 0) from src and the rest zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// An arrival once all of this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(pipe::smem_u32(bar)) : "memory");
}

// With the fast exponential and quotient (2 + |g| and 2 units in the last place of a float): far below the
// rounding of h, and free of branches, so that a thread's 32 columns overlap. (expf and the exact quotient
// made the epilogue of a 2048-deep q8 tile twice as long as its products.)
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

__device__ __forceinline__ uint32_t bf16x2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <bool Q8IN, bool SWIGLU, int NT, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                   const __grid_constant__ Grouped g)
{
    using S = Shape<Q8IN, NT>;
    constexpr int kCols = SWIGLU ? NT / 2 : NT; // output columns of a tile
    constexpr int kElem = Q8IN ? 1 : 2;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (pipe::smem_u32(raw) & 1023)) & 1023);
    Bars *bars = reinterpret_cast<Bars *>(smem + S::kBarAt);
    int *first = reinterpret_cast<int *>(smem + S::kTableAt);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            pipe::mbar_init(&bars->full[s], 1);
            pipe::mbar_init(&bars->gathered[s], 32 * kGatherWarps);
            pipe::mbar_init(&bars->scales[s], 2);
            pipe::mbar_init(&bars->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            pipe::mbar_init(&bars->acc_full[i], 1);
            pipe::mbar_init(&bars->acc_free[i], 4);
        }
        pipe::mbar_init(&bars->done, 1);
        bars->abort = 0;
        pipe::fence_barrier_init();
        tma::prefetch_map(&xmap);
        tma::prefetch_map(&wmap);
    }
    if (warp == 1) {
        umma::tmem_alloc(&bars->tmem, S::kTmemCols);
        umma::tmem_relinquish();
    }
    umma::fence_before_sync();
    row_tiles(g, first, bars->part); // ends with the block's barrier
    umma::fence_after_sync();
    const uint32_t tmem = bars->tmem;
    const int tiles = first[g.E] * g.ntiles;
    const Waiter wait{bars, g.limit_ns};

    if (warp == 0) {
        // ---- producer
        int it = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
            const Tile T = tile_at(g, first, t, kCols);
            const int loads = g.index ? 0 : (T.rows + 31) / 32;
            const uint32_t bytes = (uint32_t)(loads * 32 * kRowBytes + S::kB);
            const int second = SWIGLU ? g.width + T.col0 : T.col0 + NT / 2;
            for (int i = 0; i < g.iters; ++i, ++it) {
                const int s = it % S::kStages, u = it / S::kStages;
                if (u > 0 && !warp_wait(wait, &bars->empty[s], (u - 1) & 1, 1))
                    goto produced;
                uint8_t *a = smem + s * (S::kA + S::kB), *b = a + S::kA;
                const int x = i * (kRowBytes / kElem);
                if (lane == 0)
                    pipe::mbar_arrive_expect_tx(&bars->full[s], bytes);
                __syncwarp();
                if (lane < 2)
                    tma::load_3d(b + lane * (NT / 2) * kRowBytes, &wmap, x, lane ? second : T.col0, T.e,
                                 &bars->full[s]);
                if (lane < loads)
                    tma::load_2d(a + lane * 32 * kRowBytes, &xmap, x, T.row0 + 32 * lane, &bars->full[s]);
                __syncwarp();
            }
        }
    produced:
        __syncwarp();
        // what was issued has to land before the CTA's shared memory goes
        for (int j = max(0, it - S::kStages); j < it; ++j)
            drain(&bars->full[j % S::kStages], (j / S::kStages) & 1);
    } else if (warp == 1) {
        // ---- MMA
        if (lane == 0) {
            int it = 0, i = 0;
            for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++i) {
                // the accumulator this tile takes: free since the epilogue's read of the last tile's shared
                // columns (q8, 256 columns), or of all of the tile before that
                const int free = S::kOverlap ? i - 1 : i - 2;
                if (free >= 0 && !wait(&bars->acc_free[free & 1], (free >> 1) & 1, 2))
                    break;
                umma::fence_after_sync();
                const uint32_t d = tmem + (i & 1) * S::kSecond;
                bool ok = true;
                for (int k = 0; k < g.iters; ++k, ++it) {
                    const int s = it % S::kStages, u = it / S::kStages;
                    if (!wait(&bars->full[s], u & 1, 3) || (Q8IN && !wait(&bars->scales[s], u & 1, 4)) ||
                        (g.index && !wait(&bars->gathered[s], u & 1, 8))) {
                        ok = false;
                        break;
                    }
                    if (Q8IN || g.index) // what other threads stored is seen by the tensor cores from here on
                        umma::fence_smem_async();
                    umma::fence_after_sync();
                    const uint8_t *a = smem + s * (S::kA + S::kB), *b = a + S::kA;
                    const uint64_t ad = umma::smem_desc_sw128(a), bd = umma::smem_desc_sw128(b);
                    if (Q8IN) {
                        // two sets of scale columns: the MMAs that read this one are two stages back
                        if (it >= 2 && !wait(&bars->empty[(it - 2) % S::kStages], ((it - 2) / S::kStages) & 1, 5)) {
                            ok = false;
                            break;
                        }
                        const uint32_t sa = tmem + S::kScaleCols + 4 * (it & 1);
                        const uint32_t sb = tmem + S::kScaleCols + 8 + 8 * (it & 1);
                        const uint8_t *sc = smem + S::kStageAt + s * S::kScales;
                        umma::copy_scales(sa, sc);
                        for (int j = 0; j < NT / 128; ++j)
                            umma::copy_scales(sb + 4 * j, sc + 512 * (j + 1));
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            umma::mma_mxf8(d, ad + 2 * j, bd + 2 * j, umma::idesc_mxf8(kRows, NT, j), sa, sb,
                                           (k | j) != 0);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            umma::mma_f16(d, ad + 2 * j, bd + 2 * j, umma::idesc_bf16(kRows, NT), (k | j) != 0);
                    }
                    umma::commit(&bars->empty[s]);
                }
                if (!ok)
                    break;
                umma::commit(&bars->acc_full[i & 1]);
            }
            umma::commit(&bars->done);
            drain(&bars->done, 0);
        }
        __syncwarp();
    } else if (warp < 4) {
        // ---- scale bytes: warp 2 the input rows', warp 3 the matrix rows'. A lane has rows lane + 32 j; a
        // group of four stages' words (16 bytes per row) is loaded while the group before is handed over.
        if (Q8IN) {
            constexpr int kMost = NT / 32;
            const bool mine = warp == 2; // input rows
            const int have = mine ? 4 : kMost;
            const int64_t words = g.K / 128;
            const int groups = (g.iters + 3) / 4;
            const bool wide = g.iters % 4 == 0; // rows of scales are 16-byte aligned
            const uint8_t *row[kMost < 4 ? 4 : kMost];
            uint4 next[kMost < 4 ? 4 : kMost];
            const uint32_t kOnes = 0x7f7f7f7fu;

            auto rows_of = [&](int t) {
                const Tile T = tile_at(g, first, t, kCols);
#pragma unroll
                for (int j = 0; j < (kMost < 4 ? 4 : kMost); ++j) {
                    if (j >= have)
                        break;
                    const int r = lane + 32 * j;
                    row[j] = nullptr;
                    if (mine) {
                        if (r < T.rows) {
                            const int i = g.index ? __ldg(g.index + T.row0 + r) : T.row0 + r;
                            if ((uint32_t)i < (uint32_t)g.n)
                                row[j] = g.xs + (int64_t)i * words * 4;
                        }
                    } else {
                        const int c = r < NT / 2 ? T.col0 + r
                                                 : (SWIGLU ? g.width + T.col0 : T.col0 + NT / 2) + r - NT / 2;
                        if (c < g.N)
                            row[j] = g.ws + ((int64_t)T.e * g.N + c) * words * 4;
                    }
                }
            };
            auto load = [&](int group) {
#pragma unroll
                for (int j = 0; j < (kMost < 4 ? 4 : kMost); ++j) {
                    if (j >= have)
                        break;
                    uint4 v = make_uint4(kOnes, kOnes, kOnes, kOnes);
                    if (row[j]) {
                        const uint32_t *p = reinterpret_cast<const uint32_t *>(row[j]) + 4 * group;
                        if (wide) {
                            v = __ldg(reinterpret_cast<const uint4 *>(p));
                        } else {
                            const int left = g.iters - 4 * group;
                            v.x = __ldg(p);
                            v.y = left > 1 ? __ldg(p + 1) : kOnes;
                            v.z = left > 2 ? __ldg(p + 2) : kOnes;
                            v.w = left > 3 ? __ldg(p + 3) : kOnes;
                        }
                    }
                    next[j] = v;
                }
            };

            int it = 0, t = blockIdx.x, group = 0;
            if (t < tiles) {
                rows_of(t);
                load(0);
            }
            while (t < tiles) {
                uint4 now[kMost < 4 ? 4 : kMost];
#pragma unroll
                for (int j = 0; j < (kMost < 4 ? 4 : kMost); ++j)
                    now[j] = next[j];
                const int count = min(4, g.iters - 4 * group);
                if (++group == groups) {
                    group = 0;
                    t += gridDim.x;
                    if (t < tiles)
                        rows_of(t);
                }
                if (t < tiles)
                    load(group);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q >= count)
                        break;
                    const int s = it % S::kStages, u = it / S::kStages;
                    if (u > 0 && !warp_wait(wait, &bars->empty[s], (u - 1) & 1, 6))
                        goto scaled;
                    uint8_t *sc = smem + S::kStageAt + s * S::kScales + (mine ? 0 : 512) + lane * 16;
#pragma unroll
                    for (int j = 0; j < (kMost < 4 ? 4 : kMost); j += 4) {
                        if (j >= have)
                            break;
                        auto word = [&](const uint4 &v) { return q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w; };
                        *reinterpret_cast<uint4 *>(sc + 512 * (j / 4)) =
                            make_uint4(word(now[j]), word(now[j + 1]), word(now[j + 2]), word(now[j + 3]));
                    }
                    __syncwarp();
                    if (lane == 0)
                        pipe::mbar_arrive(&bars->scales[s]);
                    ++it;
                }
            }
        scaled:
            __syncwarp();
        }
    } else if (warp >= 8) {
        // ---- gathered input rows: a thread has one 16-byte chunk of rows r0, r0 + 16, ...
        if (g.index) {
            const int r0 = (warp - 8) * 4 + lane / 8, chunk = lane & 7;
            const int64_t pitch = (int64_t)g.K * kElem;
            const uint32_t at = (uint32_t)(r0 * kRowBytes + ((chunk ^ (r0 & 7)) << 4)); // 16 more rows: 2 KB more
            int it = 0;
            for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
                const Tile T = tile_at(g, first, t, kCols);
                const uint8_t *src[kRows / 16];
#pragma unroll
                for (int j = 0; j < kRows / 16; ++j) {
                    const int r = r0 + 16 * j;
                    src[j] = nullptr;
                    if (r < T.rows) {
                        const int i = __ldg(g.index + T.row0 + r);
                        if ((uint32_t)i < (uint32_t)g.n)
                            src[j] = g.x + i * pitch + 16 * chunk;
                    }
                }
                for (int i = 0; i < g.iters; ++i, ++it) {
                    const int s = it % S::kStages, u = it / S::kStages;
                    if (u > 0 && !warp_wait(wait, &bars->empty[s], (u - 1) & 1, 9))
                        goto gathered;
                    const uint32_t dst = pipe::smem_u32(smem + s * (S::kA + S::kB)) + at;
                    const bool in = i * kRowBytes + 16 * chunk < pitch;
#pragma unroll
                    for (int j = 0; j < kRows / 16; ++j)
                        if (r0 + 16 * j < T.rows) // rows outside x, and k behind K, are filled with zeros
                            copy16(dst + j * 16 * kRowBytes, src[j] && in ? src[j] + i * kRowBytes : g.x,
                                   src[j] && in ? 16 : 0);
                    copies_arrive(&bars->gathered[s]);
                }
            }
        gathered:
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
        }
    } else {
        // ---- epilogue
        constexpr int kChunks = kCols / 32;
        constexpr int kUnits = OUT == PMOE_TYPE_F32 ? 8 : OUT == PMOE_TYPE_BF16 ? 4 : 2; // 16-byte units of a chunk
        constexpr int kPer = kChunks < 8 / kUnits ? kChunks : 8 / kUnits;                // chunks stored together
        constexpr int kPitch = kPer * kUnits;                                            // units of a staged row
        constexpr int kUnitCols = 32 / kUnits;
        const int q = warp & 3;
        uint8_t *stage = smem + S::kStagingAt + q * 32 * kStageRowBytes;
        auto place = [&](int r, int unit) { return stage + (r * kPitch + (unit ^ (r & (kPitch - 1)))) * 16; };
        int i = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++i) {
            const Tile T = tile_at(g, first, t, kCols);
            if (!warp_wait(wait, &bars->acc_full[i & 1], (i >> 1) & 1, 7))
                break;
            umma::fence_after_sync();
            const uint32_t acc = tmem + (i & 1) * S::kSecond + ((uint32_t)(32 * q) << 16);
            const bool any = 32 * q < T.rows;
            const bool backwards = S::kOverlap && (i & 1) == 0; // the shared columns first
#pragma unroll 1
            for (int j = 0; j < kChunks; ++j) {
                const int c = backwards ? kChunks - 1 - j : j;
                float v[32], w[32];
                if (any) {
                    umma::ld32(acc + 32 * c, v);
                    if (SWIGLU)
                        umma::ld32(acc + NT / 2 + 32 * c, w);
                }
                if (j == (S::kOverlap ? 0 : kChunks - 1)) {
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        pipe::mbar_arrive(&bars->acc_free[i & 1]);
                }
                if (!any || T.col0 + 32 * c >= g.width)
                    continue;
                if (SWIGLU) {
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        v[x] = silu(v[x]) * w[x];
                }
                const int base = (c % kPer) * kUnits;
                if (OUT == PMOE_TYPE_F32) {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        *reinterpret_cast<float4 *>(place(lane, base + x)) =
                            make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                } else if (OUT == PMOE_TYPE_BF16) {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        *reinterpret_cast<uint4 *>(place(lane, base + x)) =
                            make_uint4(bf16x2(v[8 * x], v[8 * x + 1]), bf16x2(v[8 * x + 2], v[8 * x + 3]),
                                       bf16x2(v[8 * x + 4], v[8 * x + 5]), bf16x2(v[8 * x + 6], v[8 * x + 7]));
                } else {
                    uint32_t top = 0;
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        top = max(top, q8::magnitude(v[x]));
                    const uint32_t byte = q8::scale_byte(top);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t o[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            o[y] = q8::codes4(v[16 * x + 4 * y], v[16 * x + 4 * y + 1], v[16 * x + 4 * y + 2],
                                              v[16 * x + 4 * y + 3], byte);
                        *reinterpret_cast<uint4 *>(place(lane, base + x)) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    if (32 * q + lane < T.rows)
                        g.out_scales[(int64_t)(T.row0 + 32 * q + lane) * (g.width / 32) + T.col0 / 32 + c] =
                            (uint8_t)byte;
                }
                // the group's last chunk in this order, or the last one inside the matrix
                const bool last = backwards ? c % kPer == 0
                                            : c % kPer == kPer - 1 || T.col0 + 32 * (c + 1) >= g.width;
                if (!last)
                    continue;
                __syncwarp();
                const int unit = lane % kPitch;
                const int col = T.col0 + 32 * (c - c % kPer) + unit * kUnitCols;
#pragma unroll
                for (int x = 0; x < kPitch; ++x) {
                    const int r = lane / kPitch + x * (32 / kPitch);
                    if (32 * q + r < T.rows && col < g.width)
                        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(g.out) +
                                                   ((int64_t)(T.row0 + 32 * q + r) * g.width + col) *
                                                       (16 / kUnitCols)) =
                            *reinterpret_cast<const uint4 *>(place(r, unit));
                }
                __syncwarp();
            }
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, S::kTmemCols);
    }
}

template <bool Q8IN, bool SWIGLU, int NT, int OUT>
pmoe_status launch(const CUtensorMap &xmap, const CUtensorMap &wmap, const Grouped &g, int64_t tiles, cudaStream_t st)
{
    using S = Shape<Q8IN, NT>;
    auto *kernel = grouped_kernel<Q8IN, SWIGLU, NT, OUT>;
    static std::atomic<uint64_t> ready{0}; // devices whose shared-memory limit of this kernel is set
    int dev = 0;
    PMOE_CUDA(cudaGetDevice(&dev));
    if (dev >= 64 || !(ready.load() >> dev & 1)) {
        PMOE_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)S::smem(kMaxDenseExperts)));
        if (dev < 64)
            ready.fetch_or(1ull << dev);
    }
    kernel<<<(unsigned)(tiles < kNumSMs ? tiles : kNumSMs), kThreads, S::smem(g.E), st>>>(xmap, wmap, g);
    return launch_status();
}

template <bool Q8IN, int NT>
pmoe_status launch_out(bool swiglu, int out_type, const CUtensorMap &xmap, const CUtensorMap &wmap, const Grouped &g,
                       int64_t tiles, cudaStream_t st)
{
    if (swiglu)
        return out_type == PMOE_TYPE_Q8 ? launch<Q8IN, true, NT, PMOE_TYPE_Q8>(xmap, wmap, g, tiles, st)
                                        : launch<Q8IN, true, NT, PMOE_TYPE_BF16>(xmap, wmap, g, tiles, st);
    return out_type == PMOE_TYPE_F32 ? launch<Q8IN, false, NT, PMOE_TYPE_F32>(xmap, wmap, g, tiles, st)
                                     : launch<Q8IN, false, NT, PMOE_TYPE_BF16>(xmap, wmap, g, tiles, st);
}

pmoe_status grouped(const pmoe_dense *W, const pmoe_rows *X, const int32_t *offsets, int rows, int out_type, void *out,
                    uint8_t *out_scales, bool swiglu, pmoe_stream stream)
{
    if (!W || !X || !W->w || !offsets || rows < 0 || X->n < 0 || (rows && (!out || (X->n && !X->x))) || W->E < 1 ||
        W->N < 1 || W->K < 1 || W->N % 8 || X->type != W->type || (W->type != PMOE_TYPE_BF16 && W->type != PMOE_TYPE_Q8))
        return PMOE_ERR_INVALID_ARG;
    const bool is_q8 = W->type == PMOE_TYPE_Q8;
    if (is_q8 ? (W->K % 128 || !W->scales || (X->n && !X->scales)) : (W->K % 8 || W->scales || X->scales))
        return PMOE_ERR_INVALID_ARG;
    if (!X->index && X->n < rows)
        return PMOE_ERR_INVALID_ARG;
    const int width = swiglu ? W->N / 2 : W->N;
    if (swiglu ? (W->N % 16 || (out_type != PMOE_TYPE_BF16 && out_type != PMOE_TYPE_Q8))
               : (out_type != PMOE_TYPE_BF16 && out_type != PMOE_TYPE_F32))
        return PMOE_ERR_INVALID_ARG;
    if (out_type == PMOE_TYPE_Q8 ? (width % 32 || (rows && !out_scales)) : out_scales != nullptr)
        return PMOE_ERR_INVALID_ARG;
    if (!aligned(W->w, 16) || !aligned(W->scales, 16) || !aligned(X->x, 16) || !aligned(X->scales, 16) ||
        !aligned(X->index, 4) || !aligned(offsets, 4) || !aligned(out, 16) || !aligned(out_scales, 4))
        return PMOE_ERR_INVALID_ARG;
    if (W->E > kMaxDenseExperts)
        return PMOE_ERR_UNSUPPORTED;
    if (rows == 0)
        return PMOE_OK;
    PMOE_TRY(on_current_device({W->w, W->scales, X->x, X->scales, X->index, offsets, out, out_scales}));

    // Row tiles: at most one ragged one per expert. Narrow weight tiles where wide ones leave SMs idle.
    const int64_t most = (int64_t)rows / kRows + (W->E < rows ? W->E : rows);
    const int wide = swiglu ? 128 : 256;
    const bool narrow = most * ((width + wide - 1) / wide) < 2 * kNumSMs;
    const int cols = narrow ? wide / 2 : wide;
    const int ntiles = (width + cols - 1) / cols;
    // offsets that overlap could name every row for every expert: even those tiles are counted in an int
    if (((int64_t)rows + kRows - 1) / kRows * W->E * ntiles > INT32_MAX)
        return PMOE_ERR_UNSUPPORTED;
    const int elem = is_q8 ? 1 : 2;
    const uint64_t K = (uint64_t)W->K;
    CUtensorMap xmap, wmap;
    // no input rows at all: every index is outside, the map's one row is never read
    const void *x = X->n ? X->x : W->w;
    const uint64_t xd[2] = {K, (uint64_t)(X->n ? X->n : 1)}, xstride[1] = {K * elem};
    const uint32_t xbox[2] = {(uint32_t)(kRowBytes / elem), 32u};
    PMOE_TRY(tma::make_map(&xmap, elem, 2, x, xd, xstride, xbox));
    const uint64_t wd[3] = {K, (uint64_t)W->N, (uint64_t)W->E}, wstride[2] = {K * elem, K * elem * W->N};
    const uint32_t wbox[3] = {(uint32_t)(kRowBytes / elem), narrow ? 64u : 128u, 1u};
    PMOE_TRY(tma::make_map(&wmap, elem, 3, W->w, wd, wstride, wbox));
    const Grouped g{W->E,      W->N,     W->K,      X->n,    rows, width,      (int)((K * elem + kRowBytes - 1) / kRowBytes),
                    ntiles, static_cast<const uint8_t *>(x), W->scales, X->scales, X->index, offsets, out, out_scales,
                    wait_limit_ns()};
    const int64_t tiles = most * ntiles;
    const cudaStream_t st = (cudaStream_t)stream;
    if (is_q8)
        return narrow ? launch_out<true, 128>(swiglu, out_type, xmap, wmap, g, tiles, st)
                      : launch_out<true, 256>(swiglu, out_type, xmap, wmap, g, tiles, st);
    return narrow ? launch_out<false, 128>(swiglu, out_type, xmap, wmap, g, tiles, st)
                  : launch_out<false, 256>(swiglu, out_type, xmap, wmap, g, tiles, st);
}

} // namespace
} // namespace pmoe

using namespace pmoe;

extern "C" {

pmoe_status pmoe_grouped_matmul(const pmoe_dense *W, const pmoe_rows *X, const int32_t *offsets, int rows, int out_type,
                                void *out, pmoe_stream stream)
{
    return grouped(W, X, offsets, rows, out_type, out, nullptr, false, stream);
}

pmoe_status pmoe_grouped_swiglu(const pmoe_dense *W, const pmoe_rows *X, const int32_t *offsets, int rows, int out_type,
                                void *h, uint8_t *h_scales, pmoe_stream stream)
{
    return grouped(W, X, offsets, rows, out_type, h, h_scales, true, stream);
}

pmoe_status pmoe_grouped_error(int *code, int *detail, pmoe_stream stream)
{
    if (!code)
        return PMOE_ERR_INVALID_ARG;
    int f[2];
    void *p = nullptr;
    PMOE_CUDA(cudaGetSymbolAddress(&p, g_grouped_error));
    PMOE_CUDA(cudaMemcpyAsync(f, p, sizeof(f), cudaMemcpyDeviceToHost, (cudaStream_t)stream));
    PMOE_CUDA(cudaMemsetAsync(p, 0, sizeof(f), (cudaStream_t)stream));
    PMOE_CUDA(cudaStreamSynchronize((cudaStream_t)stream));
    *code = f[0];
    if (detail)
        *detail = f[1];
    return PMOE_OK;
}

} // extern "C"

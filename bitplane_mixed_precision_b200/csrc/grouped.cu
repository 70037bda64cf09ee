// Matrix products grouped by expert, with ragged numbers of rows: out_r = W_e x_r for the rows r of every
// expert e, and the gate/up pair of them with SwiGLU, on the tcgen05 tensor cores.
//
// A tile is up to ROWS rows of one expert (the MMA's M: 128 tensor-memory lanes) by NT rows of its matrix (the
// MMA's N). An MMA takes about 128 cycles for its 4 KB of A however small N is, so the matrix rows are N: 256 of
// them (128 where 256 would leave SMs idle) stream through at full rate whether an expert has 1 row or 128. (The
// other way round, with N following the number of rows, cost 20 to 50 % more at 40 and 320 rows an expert, and
// bound single rows by the MMAs.) For SwiGLU the NT rows alternate between 32 gate rows and the up rows of the same
// columns of h, so that one thread has both.
// An SM takes in about 64 bytes per cycle: 48 KB take longer than the stage's MMAs (768 against 512 cycles at least),
// which is what bounds long prompts. (Pairs of SMs sharing 256 x 256 tiles, 32 KB per SM and stage, gained 6 to 8 %
// where experts have multiples of 256 rows and nothing on average over ragged ones.)
// Measured: 16 experts of 1024 rows, 2048 x 4096: bf16 219 us (1258 TFLOP/s), q8 124 us (2221), with gathered rows 223
// and 131 us; 300 experts of 40 rows, 4096 x 1024: 404 and 214 us (6.2 and 6.1 TB/s of weights); one token of ten
// experts, q8 gate, up and SwiGLU, 2 x 1024 x 4096: 21 us (bf16 37), of which the weights stream for 13 (6.6 TB/s).
// A persistent CTA per SM takes tiles at a stride of all of them: every role finds a tile's expert in a prefix
// table of row tiles that the CTA makes from `offsets` when it starts. Roles, one warp each unless said otherwise:
//   - producer: tiled TMA loads of 128 bytes of k per row into a ring of stages: the matrix rows and rows of x that
//     follow one another by few and large boxes (the SM's TMA unit is busy for 85 cycles or more per instruction,
//     whatever its size);
//   - four warps gather the rows of x of an index with 16-byte asynchronous copies, 8 lanes a row, in the layout
//     that TMA writes. (Gathering TMA loads of four rows were tried first: 32 of them per stage took about 2700
//     cycles to issue, five times the MMAs of a stage.) Rows that no expert has are not loaded. A fifth warp hands
//     them over as they land (2 to 4 % faster than the four waiting for copies of their own two stages back);
//   - q8: two warps bring the scale bytes (one word per row and stage) into the order the tensor cores take, loaded
//     several stages ahead;
//   - MMA: one elected lane issues, its warp waits for one barrier per stage with it (a second wait and a fence of its
//     own per stage cost the q8 products 10 to 20 %: everybody else fences and arrives on that one barrier; and behind
//     a branch on the lane's number instead of an election, in a warp that does not stay together, the same
//     instructions took 10 % longer); four K slices per stage,
//     accumulators in tensor memory: two of NT columns. q8 needs tensor memory for scales too, so its two of 256 share
//     64 columns: the next tile starts once the epilogue has read those, which it does first;
//   - epilogue, four warps (one per quarter of the tensor-memory lanes = 32 rows): SwiGLU and the rounding on
//     registers (a thread has 32 neighbouring columns of one row: a whole q8 block), then through shared memory so
//     that rows are stored in pieces of 128 bytes.
// Every wait is bounded; a wait that runs out is recorded (pmoe_rows.error, or the device's record) and the CTA's roles
// finish in turn, after their copies and MMAs in flight have landed.
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>

#include "common.h"
#include "layer.cuh"
#include "q8.cuh"
#include "tma.cuh"
#include "umma.cuh"

namespace pmoe {

namespace {

constexpr int kMaxDenseExperts = 2048;
constexpr int kRowBytes = 128; // bytes of k per row and stage
constexpr int kGatherWarps = 4;
constexpr int kThreads = 256 + 32 * kGatherWarps + 32; // producer, MMA, two scale warps, epilogue (4), gather (4 + 1)
constexpr int kLanes = 128;                       // the MMA's M
constexpr int kStageRowBytes = 128;               // epilogue staging: bytes per row
constexpr uint64_t kDrainNs = 1000ull * 1000 * 1000;

// A record of the first wait that ran out, {code 3, which}, as one word that is written and taken in one step. This one
// is for calls without a record of their own, since pmoe_grouped_error last took it.
using Record = unsigned long long;
__device__ Record g_grouped_error;
__device__ Record g_taken; // pmoe_grouped_error's answer, one caller at a time

struct Grouped {
    int E, N, K, n, rows, width, iters, ntiles; // width: output columns; iters: stages per tile
    const uint8_t *x, *ws, *xs;
    const int32_t *index, *offsets;
    void *out;
    uint8_t *out_scales;
    Record *error; // NULL: the device's
    uint64_t limit_ns;
};

constexpr int kMostStages = 12;
constexpr int64_t kNone = INT64_MAX;

template <bool Q8IN, int ROWS, int NT> struct Shape {
    static constexpr int kA = kLanes * kRowBytes, kB = NT * kRowBytes;
    static constexpr int kAtoms = NT / 128; // scale blocks of 128 matrix rows
    static constexpr int kScales = Q8IN ? 512 * (1 + kAtoms) : 0;
    static constexpr int kStagingPitch = 132; // ROWS = 32: floats of a staged row of 128 columns
    static constexpr int kStaging = ROWS == 32 ? 32 * kStagingPitch * 4 : 4 * 32 * kStageRowBytes;
    static constexpr int kRoom = 227 * 1024 - 1024 - 1024 - 4 * (kMaxDenseExperts + 1) - kStaging;
    static constexpr int kFit = kRoom / (kA + kB + kScales);
    static constexpr int kStages = kFit < kMostStages ? kFit : kMostStages;
    // tensor memory: two accumulators; q8 with 256 columns: the second starts 64 columns early, which leaves room
    // for the scales of five stages
    static constexpr bool kOverlap = Q8IN && NT == 256;
    static constexpr int kShared = kOverlap ? 64 : 0;
    static constexpr int kSecond = NT - kShared;
    static constexpr int kScaleCols = kSecond + NT; // then the sets of scale columns
    static constexpr int kSets = kStages, kSetCols = 4 + 4 * kAtoms; // a set for each stage
    static constexpr int kTmemUsed = kScaleCols + (Q8IN ? kSets * kSetCols : 0);
    static constexpr int kTmemCols = kTmemUsed <= 256 ? 256 : 512;
    static_assert(kTmemUsed <= 512, "tensor memory");
    static_assert(kStages >= 4, "stages");
    static constexpr int kScalesAt = kStages * (kA + kB);
    static constexpr int kStagingAt = kScalesAt + kStages * kScales;
    static constexpr int kBarAt = kStagingAt + kStaging;
    static constexpr int kTableAt = kBarAt + 1024;
    static constexpr size_t smem(int E) { return (size_t)kTableAt + 4 * (E + 1) + 1024; } // 1024: alignment
    static_assert(kTableAt + 4 * (kMaxDenseExperts + 1) + 1024 <= 227 * 1024, "shared memory");
};

struct Bars {
    uint64_t full[kMostStages]; // a stage is complete
    uint64_t gathered[kMostStages]; // its gathered rows have landed
    uint64_t empty[kMostStages];
    uint64_t acc_full[2], acc_free[2], done;
    uint32_t tmem;
    int abort;
    int part[kThreads / 32];
    // stages that a role had arrived for when it gave up (kNone: it did not, or has no part)
    int64_t full_by[4];               // producer, scale warps, hand-over
    int64_t gathered_by[kGatherWarps];
};
static_assert(sizeof(Bars) <= 1024, "barriers");

// One lane of a whole warp, the same every time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "elect.sync _|p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r));
    return r != 0;
}

// mbar_try_wait that comes back after half a microsecond or so (without a hint it may take several).
__device__ __forceinline__ bool mbar_try_wait_briefly(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(pipe::smem_u32(bar)), "r"(parity), "r"(500u)
                 : "memory");
    return ok != 0;
}

// A wait that gives up after limit_ns, or as soon as another role has given up.
struct Waiter {
    Bars *b;
    uint64_t limit_ns;
    Record *error;
    __device__ bool operator()(uint64_t *bar, uint32_t parity, int where) const
    {
        if (pipe::mbar_try_wait(bar, parity))
            return true;
        const uint64_t start = pipe::globaltimer();
        while (!mbar_try_wait_briefly(bar, parity)) {
            if (*reinterpret_cast<volatile int *>(&b->abort))
                return false;
            if (pipe::globaltimer() - start >= limit_ns) {
                *reinterpret_cast<volatile int *>(&b->abort) = 1;
                atomicCAS(error ? error : &g_grouped_error, 0ull, 3ull | (Record)where << 32);
                return false;
            }
        }
        return true;
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

// After all roles have finished, some of them early: one thread waits for the copies that nobody waited for. They count
// towards their stages' barriers, so it makes the arrivals that are owed there (`each` by an owner that stopped before
// that stage). No owner is a whole turn of the ring ahead of another, so a barrier is at the phase of the last stage of
// `end` that it belongs to, or behind it.
template <int STAGES>
__device__ __noinline__ void land(uint64_t *bars, int64_t end, const int64_t *stopped, int owners, uint32_t each,
                                  uint64_t deadline)
{
    for (int64_t n = end > STAGES ? end - STAGES : 0; n < end; ++n) {
        uint64_t *bar = bars + n % STAGES;
        uint32_t owed = 0;
        for (int i = 0; i < owners; ++i)
            owed += stopped[i] <= n ? each : 0;
        if (owed)
            asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(pipe::smem_u32(bar)),
                         "r"(owed)
                         : "memory");
        while (!pipe::mbar_try_wait(bar, (uint32_t)(n / STAGES) & 1) && pipe::globaltimer() < deadline) {
        }
    }
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Stages of this CTA's tiles t0, t0 + step, ... before tile t. (Out of line, like land(): inside the roles' loops these
// two, which no call needs that ends well, cost 0.5 of 16.3 us of a one-round product and 2 of 78 us of a q8 SwiGLU.)
__device__ __noinline__ int64_t stages_before(const Grouped &g, int t, int t0, int step)
{
    return (int64_t)((t - t0) / step) * g.iters;
}

// The ring's stages in order: stage s for the (phase)th time.
template <int STAGES> struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++s == STAGES) {
            s = 0;
            phase ^= 1;
        }
    }
    // whether the MMAs that read the stage before have finished; at once the first time round
    __device__ __forceinline__ bool free(const Waiter &wait, Bars *bars, int where) const
    {
        return warp_wait(wait, &bars->empty[s], phase ^ 1, where);
    }
};

// One tile: its expert, rows of x (sorted rows row0 .. row0 + rows - 1) and first output column.
struct Tile {
    int e, row0, rows, col0;
};

// Rows of expert e as far as `offsets` is sound: [first, last) within [0, rows).
__device__ __forceinline__ int2 expert_rows(const Grouped &g, int e)
{
    const int a = max(0, g.offsets[e]), b = min(g.rows, g.offsets[e + 1]);
    return make_int2(a, max(a, b));
}

// A warp's walk through tiles of ascending number (weight tiles of a row tile follow one another); all lanes.
template <int ROWS> struct Walk {
    const Grouped &g;
    const int *first;
    int cols, e;
    __device__ Walk(const Grouped &G, const int *f, int c) : g(G), first(f), cols(c), e(0) {}
    __device__ __forceinline__ Tile operator()(int t)
    {
        const int m = t / g.ntiles, lane = threadIdx.x & 31;
        int end = g.E; // first[e] <= m < first[end]: 32 places of the range at a time
        while (end - e > 1) {
            const int span = (end - e + 31) / 32, at = min(e + (lane + 1) * span, end);
            const int below = __popc(__ballot_sync(0xffffffffu, first[at] <= m));
            e += below * span;
            end = min(e + span, end);
        }
        const int2 r = expert_rows(g, e);
        Tile T;
        T.e = e;
        T.row0 = r.x + (m - first[e]) * ROWS;
        T.rows = min(ROWS, r.y - T.row0);
        T.col0 = (t % g.ntiles) * cols;
        return T;
    }
};

// Prefix sums of the experts' row tiles, first[0..E]; all threads.
template <int ROWS> __device__ void row_tiles(const Grouped &g, int *first, int *part)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (g.E + kThreads - 1) / kThreads;
    const int e0 = min(g.E, tid * per), e1 = min(g.E, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        const int2 r = expert_rows(g, e);
        sum += (r.y - r.x + ROWS - 1) / ROWS;
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
        at += (r.y - r.x + ROWS - 1) / ROWS;
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

// g / (1 + exp(-g)) through e = exp(-|g|) <= 1: (g or g * e) / (1 + e), whose denominator lies in 1..2 whatever g is.
// e = 2^(2t) * exp(-|g| - 2t * ln 2) with t = -|g| * log2(e) / 2 rounded: the second factor, 1 + what its exponent is,
// takes back the rounding of t (Cody and Waite's residual), so that the error does not grow with |g| but for ln 2's own
// rounding. 2^t is squared because it would be flushed to zero from 2^-126 on, where 2^(2t) ends in the subnormals.
// In half units of a float: the exponential 4, squared 9; residual |g| / 20, its sum 1; g * e, 1 + e, their quotient
// and the products 7, so at most 17 + |g| / 20; a subnormal e is off by a step of the subnormals (2^-149). All of it is
// far below the rounding of h, and free of branches, so that a thread's columns overlap. (q8 SwiGLU
// 16384 x 2048 x 1536: 93.3 us against 91.8 with the plain fast exponential, whose error grows by 2.3 half units with
// |g|, and quotient, which is 0 below g = -87; expf and the reciprocal 2.9 us, expf and the fast quotient 7.6 us more
// than that.)
__device__ __forceinline__ float silu(float g)
{
    const float a = fminf(fabsf(g), 512.0f), t = a * -0.72134752f; // 512: exp(-512) is 0, and infinities stay out
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    e *= e;
    e = fmaf(e, fmaf(t, -1.38629436f, -a), e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return (g >= 0.0f ? g : g * e) * r;
}

// Barrier of the four epilogue warps; between two of them none waits for anything that has a limit.
__device__ __forceinline__ void epilogue_sync() { pipe::named_bar(1, 128); }

// The same, with one answer for all: whether all are to go on.
__device__ __forceinline__ bool epilogue_all(bool ok)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.u32 p, %1, 0;\n\t"
                 "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)ok)
                 : "memory");
    return r != 0;
}

// The scale warps: 32 * ROWS rows, a lane has rows lane + 32 j. The words of four stages (16 bytes of a row) are
// loaded together, while those of the four before are handed over. (Two or three such groups ahead, or a loop
// unrolled over them, were 1 to 8 % slower.) rows_of(T, j) is the row's scale bytes, or NULL where
// the values are zeros or not used (scale 1, so that zeros stay zeros).
template <class S, int ROWS, class RowsOf, class Tiles>
__device__ __forceinline__ void scale_warp(const Grouped &g, Bars *bars, const Waiter &wait, uint8_t *dst, int tiles,
                                           int t0, int step, int where, int64_t *stopped, const RowsOf &rows_of,
                                           Tiles tile)
{
    const int lane = threadIdx.x & 31;
    const int groups = (g.iters + 3) / 4;
    const bool wide = g.iters % 4 == 0; // rows of scales are 16-byte aligned
    constexpr uint32_t kOnes = 0x7f7f7f7fu;
    const uint8_t *row[ROWS];
    uint4 next[ROWS];
    int at = t0, group = 0; // the next group to load
    auto load = [&] {
        if (at >= tiles)
            return;
        if (group == 0) {
            const Tile T = tile(at);
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
                row[j] = rows_of(T, lane + 32 * j);
        }
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            next[j] = make_uint4(kOnes, kOnes, kOnes, kOnes);
            if (row[j]) {
                const uint32_t *p = reinterpret_cast<const uint32_t *>(row[j]) + 4 * group;
                if (wide) {
                    next[j] = *reinterpret_cast<const uint4 *>(p);
                } else {
                    const int left = g.iters - 4 * group;
                    next[j].x = p[0];
                    next[j].y = left > 1 ? p[1] : kOnes;
                    next[j].z = left > 2 ? p[2] : kOnes;
                    next[j].w = left > 3 ? p[3] : kOnes;
                }
            }
        }
        if (++group == groups) {
            group = 0;
            at += step;
        }
    };
    load();
    Ring<S::kStages> ring;
    for (int t = t0; t < tiles; t += step) {
        for (int k = 0; k < g.iters; k += 4) {
            uint4 now[ROWS];
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
                now[j] = next[j];
            load();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (k + q >= g.iters)
                    break;
                if (!ring.free(wait, bars, where)) {
                    if (lane == 0)
                        *stopped = stages_before(g, t, t0, step) + k + q;
                    return;
                }
                auto word = [&](int j) {
                    return j >= ROWS ? kOnes : q == 0 ? now[j].x : q == 1 ? now[j].y : q == 2 ? now[j].z : now[j].w;
                };
#pragma unroll
                for (int j = 0; j < ROWS; j += 4)
                    *reinterpret_cast<uint4 *>(dst + ring.s * S::kScales + 512 * (j / 4) + lane * 16) =
                        make_uint4(word(j), word(j + 1), word(j + 2), word(j + 3));
                umma::fence_smem_async();
                __syncwarp();
                if (lane == 0)
                    pipe::mbar_arrive(&bars->full[ring.s]);
                ring.next();
            }
        }
    }
}

template <bool Q8IN, bool SWIGLU, int ROWS, int NT, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap xwide,
                   const __grid_constant__ CUtensorMap wmap, const __grid_constant__ Grouped g)
{
    using S = Shape<Q8IN, ROWS, NT>;
    constexpr int kCols = SWIGLU ? NT / 2 : NT; // output columns of a tile
    constexpr int kElem = Q8IN ? 1 : 2;
    constexpr int kBoxRows = SWIGLU ? 64 : 128, kBoxCols = SWIGLU ? 32 : 128; // a box of matrix rows, its columns
    constexpr int kBoxes = NT / kBoxRows;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (pipe::smem_u32(raw) & 1023)) & 1023);
    Bars *bars = reinterpret_cast<Bars *>(smem + S::kBarAt);
    int *first = reinterpret_cast<int *>(smem + S::kTableAt);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            // the producer with its bytes, two scale warps, the gather warps
            pipe::mbar_init(&bars->full[s], 1 + (Q8IN ? 2 : 0) + (g.index ? 1 : 0));
            pipe::mbar_init(&bars->gathered[s], 32 * kGatherWarps);
            pipe::mbar_init(&bars->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            pipe::mbar_init(&bars->acc_full[i], 1);
            pipe::mbar_init(&bars->acc_free[i], 4);
        }
        pipe::mbar_init(&bars->done, 1);
        bars->abort = 0;
        for (int i = 0; i < 4; ++i)
            bars->full_by[i] = kNone;
        for (int i = 0; i < kGatherWarps; ++i)
            bars->gathered_by[i] = kNone;
        pipe::fence_barrier_init();
        if (!g.index)
            tma::prefetch_map(&xmap);
        tma::prefetch_map(&wmap);
    }
    if (warp == 1) {
        umma::tmem_alloc(&bars->tmem, S::kTmemCols);
        umma::tmem_relinquish();
        // only now: a launch behind this one that takes tensor memory early would keep it until this one has finished
        pipe::launch_dependents();
    }
    // Zeros where no row of x will be: an MMA multiplies 128 rows whatever a tile has, and back to back these calls run
    // at the power limit, where zeros in place of what happened to lie there gain 1 to 4 %.
    for (int i = threadIdx.x; i < S::kStages * (S::kA / 16); i += kThreads)
        *reinterpret_cast<uint4 *>(smem + i / (S::kA / 16) * (S::kA + S::kB) + i % (S::kA / 16) * 16) =
            make_uint4(0, 0, 0, 0);
    umma::fence_smem_async();
    pipe::wait_prerequisites(); // nothing of another launch is read or written before this
    umma::fence_before_sync();
    row_tiles<ROWS>(g, first, bars->part); // ends with the block's barrier
    umma::fence_after_sync();
    const uint32_t tmem = bars->tmem;
    const int tiles = first[g.E] * g.ntiles, t0 = blockIdx.x, step = gridDim.x;
    const Waiter wait{bars, g.limit_ns, g.error};
    Walk<ROWS> tile(g, first, kCols);

    if (warp == 0) {
        // ---- producer
        const bool leader = elect_one();
        Ring<S::kStages> ring;
        for (int t = t0; t < tiles; t += step) {
            const Tile T = tile(t);
            const bool one = ROWS == 128 && T.rows > 64; // one box of 128 rows
            const int loads = g.index ? 0 : one ? 1 : (T.rows + 31) / 32;
            const uint32_t bytes = (uint32_t)(loads * (one ? 128 : 32) * kRowBytes + S::kB);
            for (int i = 0; i < g.iters; ++i, ring.next()) {
                const int s = ring.s;
                if (!ring.free(wait, bars, 1)) {
                    if (lane == 0)
                        bars->full_by[0] = stages_before(g, t, t0, step) + i;
                    goto produced;
                }
                uint8_t *a = smem + s * (S::kA + S::kB), *b = a + S::kA;
                const int x = i * (kRowBytes / kElem);
                if (leader) {
                    pipe::mbar_arrive_expect_tx(&bars->full[s], bytes);
#pragma unroll
                    for (int j = 0; j < kBoxes; ++j)
                        tma::load_4d(b + j * kBoxRows * kRowBytes, &wmap, x, T.col0 + j * kBoxCols, 0, T.e,
                                     &bars->full[s]);
                    for (int j = 0; j < loads; ++j)
                        tma::load_2d(a + j * 32 * kRowBytes, one ? &xwide : &xmap, x, T.row0 + 32 * j, &bars->full[s]);
                }
                __syncwarp();
            }
        }
    produced:
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA: the warp goes through the stages together, one lane issues
        {
            const bool leader = elect_one();
            Ring<S::kStages> ring;
            const uint64_t a0 = umma::smem_desc_sw128(smem), b0 = umma::smem_desc_sw128(smem + S::kA);
            bool ok = true;
            int i = 0;
            for (int t = t0; ok && t < tiles; t += step, ++i) {
                // the accumulator this tile takes: free since the epilogue's read of the last tile's shared
                // columns (q8, 256 columns), or of all of the tile before that
                const int free = S::kOverlap ? i - 1 : i - 2;
                ok = free < 0 || warp_wait(wait, &bars->acc_free[free & 1], (free >> 1) & 1, 2);
                umma::fence_after_sync();
                const uint32_t d = tmem + (i & 1) * S::kSecond;
                for (int k = 0; ok && k < g.iters; ++k, ring.next()) {
                    const int s = ring.s;
                    ok = warp_wait(wait, &bars->full[s], ring.phase, 3);
                    if (!ok)
                        break;
                    umma::fence_after_sync();
                    const uint64_t ad = a0 + s * ((S::kA + S::kB) >> 4), bd = b0 + s * ((S::kA + S::kB) >> 4);
                    if (leader) {
                        if (Q8IN) {
                            // a set of scale columns per stage: what read it last has finished, or the stage would
                            // not be there
                            const uint32_t sa = tmem + S::kScaleCols + 4 * s;
                            const uint32_t sb = tmem + S::kScaleCols + 4 * S::kSets + 4 * S::kAtoms * s;
                            const uint8_t *sc = smem + S::kScalesAt + s * S::kScales;
                            umma::copy_scales(sa, sc);
                            for (int j = 0; j < S::kAtoms; ++j)
                                umma::copy_scales(sb + 4 * j, sc + 512 * (j + 1));
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                umma::mma_mxf8(d, ad + 2 * j, bd + 2 * j, umma::idesc_mxf8(kLanes, NT, j), sa, sb,
                                               (k | j) != 0);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                umma::mma_f16(d, ad + 2 * j, bd + 2 * j, umma::idesc_bf16(kLanes, NT), (k | j) != 0);
                        }
                        umma::commit(&bars->empty[s]);
                        if (k == g.iters - 1)
                            umma::commit(&bars->acc_full[i & 1]);
                    }
                    __syncwarp();
                }
            }
            if (leader) {
                umma::commit(&bars->done);
                drain(&bars->done, 0);
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---- scale bytes of the rows of x
        if (Q8IN)
            scale_warp<S, ROWS / 32>(
                g, bars, wait, smem + S::kScalesAt, tiles, t0, step, 6, &bars->full_by[1],
                [&](const Tile &T, int r) -> const uint8_t * {
                    if (r >= T.rows)
                        return nullptr;
                    const int i = g.index ? g.index[T.row0 + r] : T.row0 + r;
                    return (uint32_t)i < (uint32_t)g.n ? g.xs + (int64_t)i * (g.K / 32) : nullptr;
                },
                tile);
        __syncwarp();
    } else if (warp == 3) {
        // ---- scale bytes of the matrix rows
        if (Q8IN)
            scale_warp<S, NT / 32>(
                g, bars, wait, smem + S::kScalesAt + 512, tiles, t0, step, 7, &bars->full_by[2],
                [&](const Tile &T, int r) -> const uint8_t * {
                    const bool up = SWIGLU && (r & 32);
                    const int c = T.col0 + (SWIGLU ? (r / 64) * 32 + (r & 31) : r);
                    return c < g.width ? g.ws + ((int64_t)T.e * g.N + c + (up ? g.width : 0)) * (g.K / 32) : nullptr;
                },
                tile);
        __syncwarp();
    } else if (warp == 8 + kGatherWarps) {
        // ---- hands gathered rows over: the copies land as other threads' writes, which the tensor cores see behind
        // this fence
        if (g.index) {
            Ring<S::kStages> ring;
            const bool leader = elect_one();
            for (int t = t0; t < tiles; t += step)
                for (int i = 0; i < g.iters; ++i, ring.next()) {
                    if (!warp_wait(wait, &bars->gathered[ring.s], ring.phase, 11)) {
                        if (lane == 0)
                            bars->full_by[3] = stages_before(g, t, t0, step) + i;
                        goto handed;
                    }
                    if (leader) {
                        umma::fence_smem_async();
                        pipe::mbar_arrive(&bars->full[ring.s]);
                    }
                    __syncwarp();
                }
        }
    handed:
        __syncwarp();
    } else if (warp >= 8) {
        // ---- gathered rows of x: a thread has one 16-byte chunk of rows r0, r0 + 16, ...
        if (g.index) {
            const int r0 = (warp - 8) * 4 + lane / 8, chunk = lane & 7;
            const int64_t pitch = (int64_t)g.K * kElem;
            const uint32_t at = (uint32_t)(r0 * kRowBytes + ((chunk ^ (r0 & 7)) << 4)); // 16 more rows: 2 KB more
            Ring<S::kStages> ring;
            for (int t = t0; t < tiles; t += step) {
                const Tile T = tile(t);
                const uint8_t *src[ROWS / 16];
                uint32_t live = 0; // rows inside x
#pragma unroll
                for (int j = 0; j < ROWS / 16; ++j) {
                    const int r = r0 + 16 * j;
                    src[j] = g.x + 16 * chunk;
                    if (r < T.rows) {
                        const int from = g.index[T.row0 + r];
                        if ((uint32_t)from < (uint32_t)g.n) {
                            src[j] += from * pitch;
                            live |= 1u << j;
                        }
                    }
                }
                for (int i = 0; i < g.iters; ++i, ring.next()) {
                    if (!ring.free(wait, bars, 9)) {
                        if (lane == 0)
                            bars->gathered_by[warp - 8] = stages_before(g, t, t0, step) + i;
                        goto gathered;
                    }
                    const uint32_t dst = pipe::smem_u32(smem + ring.s * (S::kA + S::kB)) + at;
                    const uint32_t off = (uint32_t)i * kRowBytes;
                    const bool in = off + 16 * chunk < pitch;
#pragma unroll
                    for (int j = 0; j < ROWS / 16; ++j)
                        // rows outside x, and k behind K, are filled with zeros; so is, the first time round, what the
                        // last tile left behind this one's rows
                        if (r0 + 16 * j < T.rows || i < S::kStages)
                            copy16(dst + j * 16 * kRowBytes, src[j] + off, in && (live >> j & 1) ? 16 : 0);
                    copies_arrive(&bars->gathered[ring.s]);
                }
            }
        gathered:
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
        }
    } else if (ROWS == 32) {
        // ---- epilogue of few rows: one warp has them all in its lanes, so it only brings the accumulators to
        // shared memory, 128 columns at a time, and all four warps go on from there (one warp alone took 3.8 us
        // for a row of 256 columns with SwiGLU and q8)
        constexpr int kParts = NT / 128, kGroups = SWIGLU ? 16 : 32; // four output columns each
        const int q = warp & 3;
        float *stage = reinterpret_cast<float *>(smem + S::kStagingAt);
        int i = 0;
        for (int t = t0; t < tiles; t += step, ++i) {
            const Tile T = tile(t);
            if (!epilogue_all(warp_wait(wait, &bars->acc_full[i & 1], (i >> 1) & 1, 10)))
                break;
            umma::fence_after_sync();
            const bool backwards = S::kOverlap && (i & 1) == 0; // the shared columns first
#pragma unroll 1
            for (int j = 0; j < kParts; ++j) {
                const int part = backwards ? kParts - 1 - j : j;
                if (q == 0) {
                    const uint32_t acc = tmem + (i & 1) * S::kSecond + 128 * part;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float v[64];
                        umma::ld64(acc + 64 * half, v);
                        if (lane < T.rows)
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                *reinterpret_cast<float4 *>(stage + lane * S::kStagingPitch + 64 * half + 4 * x) =
                                    make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                    }
                }
                if (j == (S::kOverlap ? 0 : kParts - 1)) { // kOverlap: the shared 64 columns are in the first part
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        pipe::mbar_arrive(&bars->acc_free[i & 1]);
                }
                epilogue_sync();
                for (int at0 = 32 * q; at0 < T.rows * kGroups; at0 += 128) {
                    const int at = at0 + lane, r = at / kGroups, group = at % kGroups;
                    const int staged = SWIGLU ? group / 8 * 64 + group % 8 * 4 : 4 * group;
                    const int col = T.col0 + 4 * (part * kGroups + group);
                    const bool in = r < T.rows && col < g.width;
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (in) {
                        const float *p = stage + r * S::kStagingPitch + staged;
                        v = *reinterpret_cast<const float4 *>(p);
                        if (SWIGLU) {
                            const float4 u = *reinterpret_cast<const float4 *>(p + 32);
                            v = make_float4(silu(v.x) * u.x, silu(v.y) * u.y, silu(v.z) * u.z, silu(v.w) * u.w);
                        }
                    }
                    const int64_t o = (int64_t)(T.row0 + r) * g.width + col;
                    if (OUT == PMOE_TYPE_F32) {
                        if (in)
                            *reinterpret_cast<float4 *>(static_cast<float *>(g.out) + o) = v;
                    } else if (OUT == PMOE_TYPE_BF16) {
                        if (in)
                            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(g.out) + o) =
                                make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
                    } else { // 8 lanes have a block
                        const uint32_t byte = q8::scale_byte(q8::top_of_8_lanes(q8::top4(v.x, v.y, v.z, v.w)));
                        if (in) {
                            *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(g.out) + o) =
                                q8::codes4(v.x, v.y, v.z, v.w, byte);
                            if (lane % 8 == 0)
                                g.out_scales[o / 32] = (uint8_t)byte;
                        }
                    }
                }
                epilogue_sync();
            }
        }
    } else {
        // ---- epilogue, 64 accumulator columns at a time: 64 output columns, or 32 of a SwiGLU
        constexpr int kChunks = NT / 64, kHalves = SWIGLU ? 1 : 2; // halves: 32 output columns
        constexpr int kUnits = OUT == PMOE_TYPE_F32 ? 8 : OUT == PMOE_TYPE_BF16 ? 4 : 2; // 16-byte units of a half
        constexpr int kAll = kChunks * kHalves;
        constexpr int kPer = kAll < 8 / kUnits ? kAll : 8 / kUnits; // halves stored together
        constexpr int kPitch = kPer * kUnits;                       // units of a staged row
        constexpr int kUnitCols = 32 / kUnits;
        const int q = warp & 3;
        uint8_t *stage = smem + S::kStagingAt + q * 32 * kStageRowBytes;
        auto place = [&](int r, int unit) { return stage + (r * kPitch + (unit ^ (r & (kPitch - 1)))) * 16; };
        int i = 0;
        for (int t = t0; t < tiles; t += step, ++i) {
            const Tile T = tile(t);
            if (!warp_wait(wait, &bars->acc_full[i & 1], (i >> 1) & 1, 10))
                break;
            umma::fence_after_sync();
            const uint32_t acc = tmem + (i & 1) * S::kSecond + ((uint32_t)(32 * q) << 16);
            const bool any = 32 * q < T.rows;
            const bool backwards = S::kOverlap && (i & 1) == 0; // the shared columns first
#pragma unroll 1
            for (int j = 0; j < kChunks; ++j) {
                const int c = backwards ? kChunks - 1 - j : j;
                float v[64];
                if (any)
                    umma::ld64(acc + 64 * c, v);
                if (j == (S::kOverlap ? 0 : kChunks - 1)) {
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        pipe::mbar_arrive(&bars->acc_free[i & 1]);
                }
                if (!any)
                    continue;
#pragma unroll
                for (int half = 0; half < kHalves; ++half) {
                    const int h = kHalves * c + half; // 32 output columns
                    if (T.col0 + 32 * h >= g.width)
                        continue;
                    float *o = v + 32 * half;
                    if (SWIGLU) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            o[x] = silu(o[x]) * v[32 + x];
                    }
                    const int base = (h % kPer) * kUnits;
                    if (OUT == PMOE_TYPE_F32) {
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            *reinterpret_cast<float4 *>(place(lane, base + x)) =
                                make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                    } else if (OUT == PMOE_TYPE_BF16) {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            *reinterpret_cast<uint4 *>(place(lane, base + x)) =
                                make_uint4(bf16x2(o[8 * x], o[8 * x + 1]), bf16x2(o[8 * x + 2], o[8 * x + 3]),
                                           bf16x2(o[8 * x + 4], o[8 * x + 5]), bf16x2(o[8 * x + 6], o[8 * x + 7]));
                    } else {
                        uint32_t top = 0;
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            top = max(top, q8::magnitude(o[x]));
                        const uint32_t byte = q8::scale_byte(top);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t w[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                w[y] = q8::codes4(o[16 * x + 4 * y], o[16 * x + 4 * y + 1], o[16 * x + 4 * y + 2],
                                                  o[16 * x + 4 * y + 3], byte);
                            *reinterpret_cast<uint4 *>(place(lane, base + x)) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        if (32 * q + lane < T.rows)
                            g.out_scales[(int64_t)(T.row0 + 32 * q + lane) * (g.width / 32) + T.col0 / 32 + h] =
                                (uint8_t)byte;
                    }
                    // stored together with the last half of the group in this order (or of the matrix)
                    const bool last = backwards && kHalves == 1
                                          ? h % kPer == 0
                                          : h % kPer == kPer - 1 || T.col0 + 32 * (h + 1) >= g.width;
                    if (!last)
                        continue;
                    __syncwarp();
                    const int unit = lane % kPitch;
                    const int col = T.col0 + 32 * (h - h % kPer) + unit * kUnitCols;
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
    }
    __syncwarp();
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, S::kTmemCols);
    }
    if (threadIdx.x == 0 && bars->abort) {
        const uint64_t deadline = pipe::globaltimer() + kDrainNs;
        const int64_t all = t0 < tiles ? stages_before(g, tiles - 1, t0, step) + g.iters : 0;
        land<S::kStages>(bars->full, min(all, bars->full_by[0]), bars->full_by, 4, 1, deadline);
        if (g.index) {
            int64_t end = 0;
            for (int i = 0; i < kGatherWarps; ++i)
                end = max(end, min(all, bars->gathered_by[i]));
            land<S::kStages>(bars->gathered, end, bars->gathered_by, kGatherWarps, 32, deadline);
        }
    }
}

__global__ void take_error_kernel() { g_taken = atomicExch(&g_grouped_error, 0ull); }

struct Maps {
    CUtensorMap x, xwide, w;
};

template <bool Q8IN, bool SWIGLU, int ROWS, int NT, int OUT>
pmoe_status launch(const Maps &m, const Grouped &g, int64_t tiles, cudaStream_t st)
{
    using S = Shape<Q8IN, ROWS, NT>;
    auto *kernel = grouped_kernel<Q8IN, SWIGLU, ROWS, NT, OUT>;
    static std::atomic<uint64_t> ready{0}; // devices whose shared-memory limit of this kernel is set
    int dev = 0;
    PMOE_CUDA(cudaGetDevice(&dev));
    if (dev >= 64 || !(ready.load() >> dev & 1)) {
        PMOE_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)S::smem(kMaxDenseExperts)));
        if (dev < 64)
            ready.fetch_or(1ull << dev);
    }
    return launch_early(kernel, dim3((unsigned)(tiles < kNumSMs ? tiles : kNumSMs)), kThreads, S::smem(g.E), st, m.x,
                        m.xwide, m.w, g);
}

template <bool Q8IN, int ROWS, int NT>
pmoe_status launch_out(bool swiglu, int out_type, const Maps &m, const Grouped &g, int64_t tiles, cudaStream_t st)
{
    if (swiglu)
        return out_type == PMOE_TYPE_Q8 ? launch<Q8IN, true, ROWS, NT, PMOE_TYPE_Q8>(m, g, tiles, st)
                                        : launch<Q8IN, true, ROWS, NT, PMOE_TYPE_BF16>(m, g, tiles, st);
    return out_type == PMOE_TYPE_F32 ? launch<Q8IN, false, ROWS, NT, PMOE_TYPE_F32>(m, g, tiles, st)
                                     : launch<Q8IN, false, ROWS, NT, PMOE_TYPE_BF16>(m, g, tiles, st);
}

template <bool Q8IN>
pmoe_status launch_shape(int tile_rows, int nt, bool swiglu, int out_type, const Maps &m, const Grouped &g,
                         int64_t tiles, cudaStream_t st)
{
    if (tile_rows == 32)
        return nt == 128 ? launch_out<Q8IN, 32, 128>(swiglu, out_type, m, g, tiles, st)
                         : launch_out<Q8IN, 32, 256>(swiglu, out_type, m, g, tiles, st);
    return nt == 128 ? launch_out<Q8IN, 128, 128>(swiglu, out_type, m, g, tiles, st)
                     : launch_out<Q8IN, 128, 256>(swiglu, out_type, m, g, tiles, st);
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
        !aligned(X->index, 4) || !aligned(X->error, 8) || !aligned(offsets, 4) || !aligned(out, 16) ||
        !aligned(out_scales, 4))
        return PMOE_ERR_INVALID_ARG;
    if (W->E > kMaxDenseExperts)
        return PMOE_ERR_UNSUPPORTED;
    if (rows == 0)
        return PMOE_OK;

    // Rows of x per tile by the rows an expert has on average: at 16, tiles of 32 against 128 took 181 against 176 us
    // (q8, 256 experts of 4096 x 1024), 177 against 187 (q8 SwiGLU), 333 against 339 (bf16); at 32, 227 against 182 and
    // 386 against 352. The mean does not see crowded experts: 512 tokens of ten of 512 under a Zipf load (exponent 1.1,
    // mean 10, one of 457) take 634 against 619 us (q8 SwiGLU) and 330 against 317 (q8, 4096 x 1024), 256 tokens 512
    // against 510 and 265 against 262, 64 tokens 274 against 278. Matrix rows per tile by whether 256 give half of the
    // SMs a tile: one row for each of 9 experts, 2048 x 4096, 18.4 us with 128 against 19.5 (72 tiles), of 10 experts
    // 29.0 against 21.6 (80 tiles).
    const int hit = W->E < rows ? W->E : rows;
    const int tile_rows = rows <= 16 * (int64_t)hit ? 32 : 128;
    const int64_t most = (int64_t)rows / tile_rows + hit; // at most one ragged row tile per expert
    const int wide = swiglu ? 128 : 256;
    const int nt = most * ((width + wide - 1) / wide) < kNumSMs / 2 ? 128 : 256;
    const int cols = swiglu ? nt / 2 : nt;
    const int ntiles = (width + cols - 1) / cols;
    // offsets that overlap could name every row for every expert: even those tiles are counted in an int, which a role's
    // last step past them must not leave; nor may the rows of a tile behind the last row
    if (((int64_t)rows + tile_rows - 1) / tile_rows * W->E * ntiles > INT32_MAX - kNumSMs || rows > INT32_MAX - kLanes)
        return PMOE_ERR_UNSUPPORTED;
    PMOE_TRY(on_current_device({W->w, W->scales, X->x, X->scales, X->index, X->error, offsets, out, out_scales}));
    const int elem = is_q8 ? 1 : 2;
    const uint64_t K = (uint64_t)W->K;
    Maps m{}; // no maps of x where it is gathered
    // no input rows at all: every index is outside, the map's one row is never read
    const void *x = X->n ? X->x : W->w;
    const uint64_t xd[2] = {K, (uint64_t)(X->n ? X->n : 1)}, xstride[1] = {K * elem};
    const uint32_t xbox[2] = {(uint32_t)(kRowBytes / elem), 32}, xwbox[2] = {(uint32_t)(kRowBytes / elem), 128};
    if (!X->index) {
        PMOE_TRY(tma::make_map(&m.x, elem, 2, x, xd, xstride, xbox));
        PMOE_TRY(tma::make_map(&m.xwide, elem, 2, x, xd, xstride, xwbox));
    }
    // [E][gate, up][I][K] in boxes of 32 gate rows and the up rows of the same columns, or [E][1][N][K]
    const uint64_t halves = swiglu ? 2 : 1;
    const uint64_t wd[4] = {K, (uint64_t)width, halves, (uint64_t)W->E};
    const uint64_t wstride[3] = {K * elem, K * elem * width, K * elem * W->N};
    const uint32_t wbox[4] = {(uint32_t)(kRowBytes / elem), swiglu ? 32u : 128u, (uint32_t)halves, 1};
    PMOE_TRY(tma::make_map(&m.w, elem, 4, W->w, wd, wstride, wbox));
    const Grouped g{W->E,      W->N,     W->K,      X->n,    rows, width,      (int)((K * elem + kRowBytes - 1) / kRowBytes),
                    ntiles, static_cast<const uint8_t *>(x), W->scales, X->scales, X->index, offsets, out, out_scales,
                    reinterpret_cast<Record *>(X->error), wait_limit_ns()};
    const int64_t tiles = most * ntiles;
    const cudaStream_t st = (cudaStream_t)stream;
    return is_q8 ? launch_shape<true>(tile_rows, nt, swiglu, out_type, m, g, tiles, st)
                 : launch_shape<false>(tile_rows, nt, swiglu, out_type, m, g, tiles, st);
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
    static std::mutex one; // g_taken is the caller's from the exchange to the copy
    const std::lock_guard<std::mutex> lock(one);
    const cudaStream_t st = (cudaStream_t)stream;
    Record r = 0;
    void *p = nullptr;
    PMOE_CUDA(cudaGetSymbolAddress(&p, g_taken));
    take_error_kernel<<<1, 1, 0, st>>>();
    PMOE_TRY(launch_status());
    PMOE_CUDA(cudaMemcpyAsync(&r, p, sizeof(r), cudaMemcpyDeviceToHost, st));
    PMOE_CUDA(cudaStreamSynchronize(st));
    *code = (int)(uint32_t)r;
    if (detail)
        *detail = (int)(r >> 32);
    return PMOE_OK;
}

} // extern "C"

// The two ends of a grouped product: the routed pairs sorted by expert, and every token's weighted sum
// of its pairs' rows.
#include <cuda_bf16.h>

#include "common.h"
#include "pipe.cuh"

namespace pmoe {

namespace {

constexpr int kMaxGroupExperts = 2048;
constexpr int kGroupWarps = 16;
constexpr int kGroupThreads = 32 * kGroupWarps;
constexpr int kBatch = 8; // batches of 32 pairs whose loads a warp has in flight together

// Blocks that sort P pairs: one alone, in one launch, up to 2048 pairs; then blocks of 2048 (40,960 pairs of 512
// experts: 8.6 us against 11.9 in blocks of 4096), but no more than 40 of them before each has 8192, because every
// block reads all blocks' histograms (163,840 pairs: 13.0 us in 40 blocks, 13.8 in 80; 11.4 since those reads have
// 20 in flight).
inline int group_blocks(int64_t P)
{
    const int64_t small = (P + 2047) / 2048, large = (P + 8191) / 8192;
    const int64_t b = small < 40 ? small : large > 40 ? large : 40;
    return (int)(b < 1 ? 1 : b < kNumSMs ? b : kNumSMs);
}

__global__ void __launch_bounds__(kGroupThreads) group_histogram_kernel(const int32_t *ids, int P, int E, int chunk,
                                                                        int32_t *__restrict__ hist)
{
    extern __shared__ int32_t h[];
    for (int e = threadIdx.x; e < E; e += kGroupThreads)
        h[e] = 0;
    pipe::launch_dependents();
    pipe::wait_prerequisites();
    __syncthreads();
    const int p0 = blockIdx.x * chunk, p1 = min(P - p0, chunk) + p0;
#pragma unroll 8
    for (int p = p0 + threadIdx.x; p < p1; p += kGroupThreads) {
        const uint32_t e = (uint32_t)ids[p];
        if (e < (uint32_t)E)
            atomicAdd(&h[e], 1); // whole numbers: the order does not show
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kGroupThreads)
        hist[(int64_t)blockIdx.x * E + e] = h[e];
}

// kBatch batches of 32 pairs, p, p + 32, ... < end: a lane's ids (all ones where that is no expert) and the lanes with
// the same one, by a ballot per bit of the ids, several batches at a time. (The match instruction took some 700 cycles
// for 32 different experts.) bits: a multiple of 4 that no expert's id has all set.
__device__ __forceinline__ void load_batches(const int32_t *ids, int p, int end, int E, int bits, uint32_t (&id)[kBatch],
                                             unsigned (&same)[kBatch])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
        id[j] = p + 32 * j + lane < end ? (uint32_t)ids[p + 32 * j + lane] : 0xffffffffu;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
        id[j] = id[j] < (uint32_t)E ? id[j] : 0xffffffffu;
        same[j] = 0xffffffffu;
    }
#pragma unroll
    for (int j = 0; j < kBatch; j += 2) {
        if (p + 32 * j >= end)
            break;
        for (int b = 0; b < bits; b += 4)
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const bool set = id[j + c % 2] >> (b + c / 2) & 1;
                const unsigned with = __ballot_sync(0xffffffffu, set);
                same[j + c % 2] &= set ? with : ~with;
            }
    }
}

// A stable counting sort, bound by the latency of its steps (12 bytes a pair move: 320 pairs take 2.9 us, 163,840
// pairs 11.4 us with the histograms). Every block takes `chunk` consecutive pairs, every warp of it a consecutive
// sixteenth. Places: all pairs of lower experts, then the blocks before, the warps before, and inside a
// warp, 32 pairs at a time, the lanes before with the same expert. hist (one row per block) is NULL when
// one block has all pairs.
__global__ void __launch_bounds__(kGroupThreads)
    group_scatter_kernel(const int32_t *ids, int P, int k, int E, int chunk, const int32_t *hist,
                         int32_t *__restrict__ offsets, int32_t *__restrict__ row_of, int32_t *__restrict__ token_of)
{
    extern __shared__ int32_t cnt[]; // [kGroupWarps][E]
    __shared__ int32_t scan[kGroupWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int p0 = blockIdx.x * chunk, p1 = min(P - p0, chunk) + p0;
    const int bits = (35 - __clz(E)) / 4 * 4; // ids 0..E-1 never have all of them set; no expert's id has
    const int per = (chunk / kGroupWarps + 31) / 32 * 32;
    const int w0 = min(p0 + warp * per, p1), w1 = min(w0 + per, p1);
    for (int i = tid; i < kGroupWarps * E; i += kGroupThreads)
        cnt[i] = 0;
    pipe::launch_dependents();
    pipe::wait_prerequisites();
    __syncthreads();
    int32_t *mine = cnt + warp * E;
    uint32_t id[kBatch];
    unsigned same[kBatch];
    for (int p = w0; p < w1; p += 32 * kBatch) {
        load_batches(ids, p, w1, E, bits, id, same);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (p + 32 * j >= w1)
                break;
            if (id[j] < (uint32_t)E && lane == __ffs(same[j]) - 1)
                mine[id[j]] += __popc(same[j]);
            __syncwarp();
        }
    }
    __syncthreads();
    // first places, 512 experts at a time
    int32_t below = 0;
    for (int e0 = 0; e0 < E; e0 += kGroupThreads) {
        const int e = e0 + tid;
        int32_t total = 0, before = 0;
        if (e < E) {
            if (hist == nullptr) {
#pragma unroll
                for (int w = 0; w < kGroupWarps; ++w)
                    total += cnt[w * E + e];
            } else {
                for (int b0 = 0; b0 < (int)gridDim.x; b0 += 20) { // 20 loads in flight
                    int32_t n[20];
#pragma unroll
                    for (int j = 0; j < 20; ++j)
                        n[j] = b0 + j < (int)gridDim.x ? hist[(int64_t)(b0 + j) * E + e] : 0;
#pragma unroll
                    for (int j = 0; j < 20; ++j) {
                        total += n[j];
                        before += b0 + j < (int)blockIdx.x ? n[j] : 0;
                    }
                }
            }
        }
        int32_t inc = total;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int32_t n = __shfl_up_sync(0xffffffffu, inc, s);
            inc += lane >= s ? n : 0;
        }
        if (lane == 31)
            scan[warp] = inc;
        __syncthreads();
        int32_t base = below, all = 0;
        for (int w = 0; w < kGroupWarps; ++w) {
            base += w < warp ? scan[w] : 0;
            all += scan[w];
        }
        below += all;
        if (e < E) {
            int32_t at = base + inc - total;
            if (blockIdx.x == 0) {
                offsets[e] = at;
                if (e == E - 1)
                    offsets[E] = at + total;
            }
            at += before;
            int32_t n[kGroupWarps];
#pragma unroll
            for (int w = 0; w < kGroupWarps; ++w)
                n[w] = cnt[w * E + e];
#pragma unroll
            for (int w = 0; w < kGroupWarps; ++w) {
                cnt[w * E + e] = at;
                at += n[w];
            }
        }
        __syncthreads();
    }
    for (int p = w0; p < w1; p += 32 * kBatch) {
        if (w1 - w0 > 32 * kBatch) // else they are at hand
            load_batches(ids, p, w1, E, bits, id, same);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int pair = p + 32 * j + lane;
            if (p + 32 * j >= w1)
                break;
            int32_t row = -1;
            if (id[j] < (uint32_t)E)
                row = mine[id[j]] + __popc(same[j] & ((1u << lane) - 1u));
            __syncwarp();
            if (id[j] < (uint32_t)E && lane == __ffs(same[j]) - 1)
                mine[id[j]] += __popc(same[j]);
            __syncwarp();
            if (pair < w1) {
                row_of[pair] = row;
                if (row >= 0)
                    token_of[row] = pair / k;
            }
        }
    }
}

__device__ __forceinline__ void load8(const void *rows, int64_t at, float (&v)[8], bool bf16)
{
    if (bf16) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(rows) + at);
        const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(q[i] << 16);
            v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
        }
    } else {
        const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(rows) + at);
        const float4 a = f[0], b = f[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

// A thread has 8 columns of one token and adds its k rows in slot order, four rows' loads in flight. Bound by memory:
// 4096 tokens of 10 bf16 rows of 4096 take 66 us, 5.8 TB/s of what has to be read and written.
template <bool BF16>
__global__ void __launch_bounds__(128)
    combine_rows_kernel(const void *rows, const int32_t *row_of, const float *w, int P, int k, int H, int chunks,
                        float *__restrict__ y)
{
    const int t = blockIdx.x / chunks;
    const int c = 8 * ((blockIdx.x % chunks) * 128 + threadIdx.x);
    if (c >= H)
        return;
    float s[8] = {};
    pipe::launch_dependents();
    pipe::wait_prerequisites();
#pragma unroll 4
    for (int i = 0; i < k; ++i) {
        const int row = row_of[(int64_t)t * k + i];
        if ((uint32_t)row >= (uint32_t)P)
            continue;
        const float wt = w[(int64_t)t * k + i];
        float v[8];
        load8(rows, (int64_t)row * H + c, v, BF16);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[j] = fmaf(wt, v[j], s[j]);
    }
    float4 *o = reinterpret_cast<float4 *>(y + (int64_t)t * H + c);
    o[0] = make_float4(s[0], s[1], s[2], s[3]);
    o[1] = make_float4(s[4], s[5], s[6], s[7]);
}

} // namespace
} // namespace pmoe

using namespace pmoe;

extern "C" {

size_t pmoe_group_workspace_bytes(int T, int k, int E)
{
    if (T < 0 || k < 1 || E < 1)
        return 0;
    const int b = group_blocks((int64_t)T * k);
    return b > 1 ? (size_t)b * E * sizeof(int32_t) : 0;
}

pmoe_status pmoe_group_pairs(const int32_t *ids, int T, int k, int E, int32_t *offsets, int32_t *row_of,
                             int32_t *token_of, void *ws, size_t ws_bytes, pmoe_stream stream)
{
    const int64_t P = (int64_t)T * k;
    if (!offsets || T < 0 || k < 1 || k > 32 || E < 1 || P > (1 << 30) || (P && (!ids || !row_of || !token_of)) ||
        !aligned(ids, 4) || !aligned(offsets, 4) || !aligned(row_of, 4) || !aligned(token_of, 4) || !aligned(ws, 4))
        return PMOE_ERR_INVALID_ARG;
    if (E > kMaxGroupExperts)
        return PMOE_ERR_UNSUPPORTED;
    const size_t need = pmoe_group_workspace_bytes(T, k, E);
    if (need > ws_bytes || (need && !ws))
        return PMOE_ERR_WORKSPACE;
    const int blocks = group_blocks(P);
    PMOE_TRY(on_current_device({ids, offsets, row_of, token_of, need ? ws : nullptr}));
    const int chunk = (int)(((P + blocks - 1) / blocks + 32 * kGroupWarps - 1) / (32 * kGroupWarps) * (32 * kGroupWarps));
    const size_t smem = (size_t)kGroupWarps * E * sizeof(int32_t);
    const cudaStream_t st = (cudaStream_t)stream;
    if (smem + kGroupWarps * sizeof(int32_t) > 48 * 1024) // with the scan's static words
        PMOE_CUDA(cudaFuncSetAttribute(group_scatter_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kGroupWarps * kMaxGroupExperts * (int)sizeof(int32_t)));
    int32_t *hist = blocks > 1 ? static_cast<int32_t *>(ws) : nullptr;
    if (hist)
        PMOE_TRY(launch_early(group_histogram_kernel, dim3(blocks), kGroupThreads, E * sizeof(int32_t), st, ids, (int)P,
                              E, chunk, hist));
    return launch_early(group_scatter_kernel, dim3(blocks), kGroupThreads, smem, st, ids, (int)P, k, E, chunk, hist,
                        offsets, row_of, token_of);
}

pmoe_status pmoe_combine_rows(const void *rows, int rows_are_bf16, const int32_t *row_of, const float *w, int T, int k,
                              int H, float *y, pmoe_stream stream)
{
    const int64_t P = (int64_t)T * k;
    if (T < 0 || k < 1 || k > 32 || H <= 0 || H % 8 || P > (1 << 30) || (T && (!rows || !row_of || !w || !y)) ||
        !aligned(rows, 16) || !aligned(y, 16) || !aligned(row_of, 4) || !aligned(w, 4))
        return PMOE_ERR_INVALID_ARG;
    const int chunks = (H / 8 + 127) / 128;
    if ((int64_t)T * chunks > INT32_MAX)
        return PMOE_ERR_UNSUPPORTED;
    if (T == 0)
        return PMOE_OK;
    PMOE_TRY(on_current_device({rows, row_of, w, y}));
    return launch_early(rows_are_bf16 ? combine_rows_kernel<true> : combine_rows_kernel<false>, dim3(T * chunks), 128, 0,
                        (cudaStream_t)stream, rows, row_of, w, (int)P, k, H, chunks, y);
}

} // extern "C"

// Residual addition and root-mean-square norm with an output in 8 bits (q8 rows), and the plain
// conversion of rows to q8.
#include <cuda_bf16.h>

#include <cfloat>

#include "common.h"
#include "pipe.cuh"
#include "q8.cuh"

namespace pmoe {

namespace {

constexpr int kMaxNormThreads = 1024;

__device__ __forceinline__ uint2 bf16x4(float4 v)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// The block's largest value (as bits of a magnitude, so that a NaN is the largest); all threads.
__device__ __forceinline__ uint32_t block_top(uint32_t top, uint32_t *part)
{
    const int lane = threadIdx.x & 31;
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0)
        part[threadIdx.x >> 5] = top;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < (int)(blockDim.x >> 5) ? part[lane] : 0u);
}

// The block's sum, in a fixed order; all threads.
__device__ __forceinline__ float block_sum(float s, float *part)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0)
        part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = lane < (int)(blockDim.x >> 5) ? part[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}

template <int V> __device__ __forceinline__ float squares(const float4 (&v)[V])
{
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        ss = fmaf(v[j].x, v[j].x, ss);
        ss = fmaf(v[j].y, v[j].y, ss);
        ss = fmaf(v[j].z, v[j].z, ss);
        ss = fmaf(v[j].w, v[j].w, ss);
    }
    return ss;
}

// One block per token, V float4 of the row per thread, held in registers between the sum of squares and
// the output: r and y are read once and r written once. 8 neighbouring lanes hold one 32-column block. Bound by memory:
// 4096 x 4096 takes 39.2 us, 5.6 TB/s of the 13 bytes an element that have to move (r and y pass through the L2 as
// streams, which leaves its room to the codes that the next call reads: 0.9 us less; the branch for rows whose squares
// leave the floats costs 0.5 us).
template <int V>
__global__ void __launch_bounds__(kMaxNormThreads)
    residual_norm_q8_kernel(float *__restrict__ r, const float *y, const float *gain, float eps, int H,
                            uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, uint16_t *__restrict__ x)
{
    __shared__ float part[32], sums[32];
    __shared__ uint32_t tops[32];
    const int tid = threadIdx.x, lane = tid & 31, n4 = H / 4;
    const int64_t row = (int64_t)blockIdx.x * H;
    float4 v[V];
    pipe::launch_dependents();
    pipe::wait_prerequisites();
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = tid + j * blockDim.x;
        v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < n4) {
            v[j] = __ldcs(reinterpret_cast<const float4 *>(r + row + 4 * i));
            if (y != nullptr) {
                const float4 d = __ldcs(reinterpret_cast<const float4 *>(y + row + 4 * i));
                v[j].x += d.x;
                v[j].y += d.y;
                v[j].z += d.z;
                v[j].w += d.w;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = tid + j * blockDim.x;
        if (y != nullptr && i < n4)
            __stcs(reinterpret_cast<float4 *>(r + row + 4 * i), v[j]);
    }
    const float all = block_sum(squares(v), part);
    const float ms = all / (float)H + eps;
    float inv = ms == 0.0f ? 0.0f : 1.0f / sqrtf(ms);
    // Where squares of finite values leave the floats, or what underflowed of them (2^-150 each) is not far below the
    // rest, the row is multiplied by a power of two first, which brings its largest magnitude to 1..2, or eps to at most
    // 2 where that comes first. The whole block takes this path or not.
    if (!(all <= FLT_MAX) || all + (float)H * eps < 0x1p-100f) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < V; ++j)
            top = max(top, q8::top4(v[j].x, v[j].y, v[j].z, v[j].w));
        top = block_top(top, tops);
        if (top < 0x7f800000u && top != 0u) {
            int up = max(-126, 127 - (int)(top >> 23));
            if (eps > 0.0f)
                up = min(up, (128 - (int)(__float_as_uint(eps) >> 23)) / 2);
            const float by = __uint_as_float((uint32_t)(up + 127) << 23);
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[j] = make_float4(v[j].x * by, v[j].y * by, v[j].z * by, v[j].w * by);
            inv = 1.0f / sqrtf(block_sum(squares(v), sums) / (float)H + by * eps * by);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = tid + j * blockDim.x;
        if (i >= n4) // whole warps where codes are made: H % 128 == 0
            break;
        float4 o = make_float4(v[j].x * inv, v[j].y * inv, v[j].z * inv, v[j].w * inv);
        if (gain != nullptr) {
            const float4 g = *reinterpret_cast<const float4 *>(gain + 4 * i);
            o = make_float4(o.x * g.x, o.y * g.y, o.z * g.z, o.w * g.w);
        }
        if (x != nullptr)
            *reinterpret_cast<uint2 *>(x + row + 4 * i) = bf16x4(o);
        if (codes != nullptr) {
            const uint32_t byte = q8::scale_byte(q8::top_of_8_lanes(q8::top4(o.x, o.y, o.z, o.w)));
            *reinterpret_cast<uint32_t *>(codes + row + 4 * i) = q8::codes4(o.x, o.y, o.z, o.w, byte);
            // the warp's four scale bytes as one word
            const uint32_t b1 = __shfl_sync(0xffffffffu, byte, 8), b2 = __shfl_sync(0xffffffffu, byte, 16),
                           b3 = __shfl_sync(0xffffffffu, byte, 24);
            if (lane == 0)
                *reinterpret_cast<uint32_t *>(scales + row / 32 + i / 8) = byte | (b1 << 8) | (b2 << 16) | (b3 << 24);
        }
    }
}

template <bool BF16>
__global__ void __launch_bounds__(256) quantize_q8_kernel(const void *w, int64_t n4, uint8_t *__restrict__ codes,
                                                          uint8_t *__restrict__ scales)
{
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    pipe::launch_dependents();
    pipe::wait_prerequisites();
    for (int64_t i0 = (int64_t)blockIdx.x * blockDim.x; i0 < n4; i0 += step) { // the whole block takes every step
        const int64_t i = i0 + threadIdx.x;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < n4) {
            if (BF16) {
                const uint2 u = reinterpret_cast<const uint2 *>(w)[i];
                o = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                                __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
            } else {
                o = reinterpret_cast<const float4 *>(w)[i];
            }
        }
        const uint32_t byte = q8::scale_byte(q8::top_of_8_lanes(q8::top4(o.x, o.y, o.z, o.w)));
        if (i < n4) {
            *reinterpret_cast<uint32_t *>(codes + 4 * i) = q8::codes4(o.x, o.y, o.z, o.w, byte);
            if ((i & 7) == 0)
                scales[i / 8] = (uint8_t)byte;
        }
    }
}

} // namespace
} // namespace pmoe

using namespace pmoe;

extern "C" {

pmoe_status pmoe_quantize_q8(const void *w, int w_is_bf16, int64_t rows, int K, uint8_t *codes, uint8_t *scales,
                             pmoe_stream stream)
{
    if (!w || !codes || !scales || rows < 0 || K <= 0 || K % 32 || !aligned(w, 16) || !aligned(codes, 4) ||
        rows > (INT64_MAX / 8) / K)
        return PMOE_ERR_INVALID_ARG;
    if (rows == 0)
        return PMOE_OK;
    PMOE_TRY(on_current_device({w, codes, scales}));
    const int64_t n4 = rows * K / 4;
    const int64_t blocks = (n4 + 255) / 256;
    const int grid = (int)(blocks < 16 * kNumSMs ? blocks : 16 * kNumSMs);
    return launch_early(w_is_bf16 ? quantize_q8_kernel<true> : quantize_q8_kernel<false>, dim3(grid), 256, 0,
                        (cudaStream_t)stream, w, n4, codes, scales);
}

pmoe_status pmoe_residual_norm_q8(float *r, const float *y, const float *gain, float eps, int T, int H, uint8_t *codes,
                                  uint8_t *scales, uint16_t *x, pmoe_stream stream)
{
    if (!r || T < 0 || H <= 0 || H % (codes ? 128 : 8) || !(eps >= 0.0f) || (!codes != !scales) || (!codes && !x) ||
        !aligned(r, 16) || !aligned(y, 16) || !aligned(gain, 16) || !aligned(codes, 16) || !aligned(scales, 4) ||
        !aligned(x, 16))
        return PMOE_ERR_INVALID_ARG;
    if (H > 32768)
        return PMOE_ERR_UNSUPPORTED;
    if (T == 0)
        return PMOE_OK;
    PMOE_TRY(on_current_device({r, y, gain, codes, scales, x}));
    // 512 threads a row where it is long enough: at 4096 x 4096, 38.8 us (5.6 TB/s) against 40.6 with 256 threads
    // (their 3.5 rounds of blocks end in half a round), 43.1 with 1024 and 49.1 with 128.
    const int n4 = H / 4;
    int V = 1;
    while (V < 8 && n4 > V * 512)
        V *= 2;
    while (n4 > V * kMaxNormThreads)
        V *= 2;
    const int threads = ((n4 + V - 1) / V + 31) / 32 * 32;
    auto *kernel = V == 1   ? residual_norm_q8_kernel<1>
                   : V == 2 ? residual_norm_q8_kernel<2>
                   : V == 4 ? residual_norm_q8_kernel<4>
                            : residual_norm_q8_kernel<8>;
    return launch_early(kernel, dim3(T), threads, 0, (cudaStream_t)stream, r, y, gain, eps, H, codes, scales, x);
}

} // extern "C"

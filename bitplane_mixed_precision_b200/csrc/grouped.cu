// Matrix products grouped by expert, with ragged numbers of rows: out_r = W_e x_r for the rows r of every
// expert e, and the gate/up pair of them with SwiGLU.
#include <cuda_bf16.h>

#include "common.h"
#include "q8.cuh"

namespace pmoe {

namespace {

constexpr int kMaxDenseExperts = 2048;
constexpr int kTile = 64, kStep = 32;

__device__ __forceinline__ float load_value(const void *x, const uint8_t *scales, bool is_q8, int64_t row, int K, int k)
{
    if (!is_q8)
        return __uint_as_float((uint32_t) static_cast<const uint16_t *>(x)[row * K + k] << 16);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t *>(x)[row * K + k], __NV_E4M3);
    return __half2float(__half(h)) * q8::value(scales[row * (K / 32) + k / 32]);
}

struct Grouped {
    int E, N, K, n, rows, is_q8, out_type, width; // width: output columns (N, or I of a swiglu)
    const void *w, *x;
    const uint8_t *ws, *xs;
    const int32_t *index, *offsets;
    void *out;
    uint8_t *out_scales;
};

// One block: 64 rows x 32 output columns (of a swiglu: 32 gate and 32 up columns), or 64 plain columns.
template <bool SWIGLU>
__global__ void __launch_bounds__(256) grouped_kernel(const Grouped g)
{
    __shared__ float xt[kStep][kTile + 1], wt[kStep][kTile + 1];
    __shared__ float res[kTile][kTile + 1];
    int blk = blockIdx.x, e = 0, r0 = 0, r1 = 0;
    for (; e < g.E; ++e) {
        r0 = max(0, g.offsets[e]);
        r1 = min(g.rows, g.offsets[e + 1]);
        const int n = r1 > r0 ? (r1 - r0 + kTile - 1) / kTile : 0;
        if (blk < n)
            break;
        blk -= n;
    }
    if (e == g.E)
        return;
    r0 += blk * kTile;
    const int cols = SWIGLU ? kTile / 2 : kTile, c0 = blockIdx.y * cols;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < g.K; k0 += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
            const int k = k0 + i % kStep, r = i / kStep;
            int src = -1;
            if (r0 + r < r1)
                src = g.index ? g.index[r0 + r] : r0 + r;
            xt[i % kStep][r] = k < g.K && src >= 0 && src < g.n ? load_value(g.x, g.xs, g.is_q8, src, g.K, k) : 0.0f;
            int c = c0 + r;
            bool in = c < g.N;
            if (SWIGLU) {
                c = c0 + r % cols;
                in = c < g.width;
                c += r < cols ? 0 : g.width;
            }
            wt[i % kStep][r] = k < g.K && in ? load_value(g.w, g.ws, g.is_q8, (int64_t)e * g.N + c, g.K, k) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kStep; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(xt[k][ty + 16 * i], wt[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            res[ty + 16 * i][tx + 16 * j] = acc[i][j];
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * cols; i += 256) { // a warp: 32 columns of one row
        const int r = i / cols, c = i % cols;
        const bool in = r0 + r < r1 && c0 + c < g.width;
        float v = res[r][c];
        if (SWIGLU)
            v = v / (1.0f + expf(-v)) * res[r][c + cols];
        const int64_t at = (int64_t)(r0 + r) * g.width + c0 + c;
        if (g.out_type == PMOE_TYPE_Q8) {
            const uint32_t byte = q8::scale_byte(__reduce_max_sync(0xffffffffu, q8::magnitude(v)));
            const uint32_t code = q8::codes4(v, 0.0f, 0.0f, 0.0f, byte) & 0xffu;
            if (in) {
                static_cast<uint8_t *>(g.out)[at] = (uint8_t)code;
                if (c % 32 == 0)
                    g.out_scales[at / 32] = (uint8_t)byte;
            }
        } else if (in) {
            if (g.out_type == PMOE_TYPE_BF16)
                static_cast<__nv_bfloat16 *>(g.out)[at] = __float2bfloat16(v);
            else
                static_cast<float *>(g.out)[at] = v;
        }
    }
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
    Grouped g{W->E, W->N,      W->K, X->n,      rows,     is_q8,   out_type, width,
              W->w, X->x, W->scales, X->scales, X->index, offsets, out,      out_scales};
    const int cols = swiglu ? kTile / 2 : kTile;
    const dim3 grid((unsigned)((rows + kTile - 1) / kTile + W->E), (unsigned)((width + cols - 1) / cols));
    if (swiglu)
        grouped_kernel<true><<<grid, 256, 0, (cudaStream_t)stream>>>(g);
    else
        grouped_kernel<false><<<grid, 256, 0, (cudaStream_t)stream>>>(g);
    return launch_status();
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

} // extern "C"

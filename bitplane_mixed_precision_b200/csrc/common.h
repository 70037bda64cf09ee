// Host-side helpers shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/pmoe.h"

namespace pmoe {

void set_cuda_error(cudaError_t e);

// Records a CUDA failure and returns PMOE_ERR_CUDA, or PMOE_OK.
inline pmoe_status cuda_status(cudaError_t e)
{
    if (e == cudaSuccess)
        return PMOE_OK;
    set_cuda_error(e);
    return PMOE_ERR_CUDA;
}

inline pmoe_status launch_status() { return cuda_status(cudaGetLastError()); }

// Launches a kernel that may start before the launch in front of it on the stream has finished, up to its
// pipe::wait_prerequisites(): its setup then overlaps that one's end. Every such kernel calls that before it touches
// global memory, and reads by plain loads: what the launch in front writes is not read-only while this one is resident,
// which is what __ldg, and a pointer that is const and __restrict__, would promise.
template <class... P, class... A>
pmoe_status launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...));
}

#define PMOE_TRY(expr)                                                                             \
    do {                                                                                           \
        pmoe_status _s = (expr);                                                                   \
        if (_s != PMOE_OK)                                                                         \
            return _s;                                                                             \
    } while (0)

#define PMOE_CUDA(expr) PMOE_TRY(::pmoe::cuda_status(expr))

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// PMOE_OK if every pointer that is not null is memory of the current device (or managed memory).
pmoe_status on_current_device(std::initializer_list<const void *> ptrs);

// Gaussian helpers (host, double): own implementations, see format.cu.
double norm_ppf(double p);
void tree_codebook(float *cb510);
void quantile_thresholds(double *t256);

// Device-side budget rule shared by host and device selection code.
inline int select_budget(int k, float avg_bits)
{
    double b = (double)avg_bits * (double)k + 1e-4;
    int B = (int)b;
    if ((double)B > b)
        B -= 1;
    if (B < k)
        B = k;
    if (B > 8 * k)
        B = 8 * k;
    return B;
}

constexpr int kNumSMs = 148;

} // namespace pmoe

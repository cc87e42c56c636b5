// experts.cu -- FP8 products of experts in blocks of 128, and the weight
// gradients of experts: the entry points, and the kernel for few rows an expert.
// Products of more rows and the weight gradients run on gemm.cu's CTA-pair
// kernels.
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/fp8linear.h"
#include "experts.cuh"
#include "hostops.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowops.cuh"

namespace fp8 {
namespace {

constexpr int64_t kLimit = (int64_t{1} << 31) - 1024;   // coordinates and units are 32-bit

// What both calls check.  rows: the dimension that the offsets cut; m, n, k in
// the GEMM's own order.
int check(const char* what, const uint8_t* A, const uint8_t* B, int fa, int fb, const float* sa, const float* sb,
          const void* D, const int32_t* offsets, int experts, int64_t rows) {
    if ((fa != FP8_E4M3 && fa != FP8_E5M2) || (fb != FP8_E4M3 && fb != FP8_E5M2))
        return set_error(FP8_ERR_INVALID_ARG, "%s: unknown FP8 format", what);
    if (experts < 1 || experts > kMaxGemmExperts)
        return set_error(FP8_ERR_SHAPE, "%s: experts in 1..%d", what, kMaxGemmExperts);
    if (!offsets) return set_error(FP8_ERR_INVALID_ARG, "%s: offsets is NULL", what);
    if (rows && (!A || !B || !sa || !sb || !D)) return set_error(FP8_ERR_INVALID_ARG, "%s: NULL pointer", what);
    for (const void* t : {static_cast<const void*>(A), static_cast<const void*>(B), D})
        if (!host::aligned(t, 16)) return set_error(FP8_ERR_ALIGN, "%s: tensors must be 16-byte aligned", what);
    for (const void* t : {static_cast<const void*>(sa), static_cast<const void*>(sb),
                          static_cast<const void*>(offsets)})
        if (!host::aligned(t, 4))
            return set_error(FP8_ERR_ALIGN, "%s: factors and offsets must be 4-byte aligned", what);
    return FP8_OK;
}

}  // namespace
}  // namespace fp8

using namespace fp8;
using namespace fp8::host;

extern "C" {

int fp8_gemm_experts(const fp8_gemm_experts_args_t* a, void* stream) {
    const char* what = "fp8_gemm_experts";
    if (!a) return set_error(FP8_ERR_INVALID_ARG, "%s: args is NULL", what);
    if (a->M < 0 || a->N < 128 || a->K < 128 || a->N % 128 || a->K % 128)
        return set_error(FP8_ERR_SHAPE, "%s: M must be >= 0, N and K positive multiples of 128", what);
    if (a->out != FP8_OUT_BF16 && a->out != FP8_OUT_F32)
        return set_error(FP8_ERR_INVALID_ARG, "%s: unknown output type", what);
    int r = check(what, a->A, a->B, a->fa, a->fb, a->scale_inv_a, a->scale_inv_b, a->d, a->offsets, a->experts, a->M);
    if (r != FP8_OK) return r;
    if (a->M > kLimit || a->K > kLimit || a->N > kLimit / a->experts ||
        (a->M / 16 + a->experts) * (a->N / 128) > kLimit)
        return set_error(FP8_ERR_SHAPE, "%s: dimensions out of range", what);
    if (a->M == 0) return FP8_OK;
    const ExpertGemm g{a->A, a->fa, a->B, a->fb, a->M, a->N, a->K, a->scale_inv_a, a->scale_inv_b, a->d, a->out, 0,
                       a->pow2, a->offsets, a->experts};
    r = launch_gemm_by_rows(g, as_stream(stream));
    return r != FP8_OK ? r : launch_status(what);
}

int fp8_wgrad_experts(const fp8_wgrad_experts_args_t* a, void* stream) {
    const char* what = "fp8_wgrad_experts";
    if (!a) return set_error(FP8_ERR_INVALID_ARG, "%s: args is NULL", what);
    if (a->M < 0 || a->M % 128 || a->N < 128 || a->K < 128 || a->N % 128 || a->K % 128)
        return set_error(FP8_ERR_SHAPE, "%s: M, N and K must be multiples of 128, N and K positive", what);
    int r = check(what, a->dY_t, a->X_t, a->f_dy, a->f_x, a->scale_inv_dy, a->scale_inv_x, a->dW, a->offsets,
                  a->experts, a->M);
    if (r != FP8_OK) return r;
    if (a->M > kLimit || a->K > kLimit || a->N > kLimit / a->experts ||
        (a->N / 256 + 1) * (a->K / 256 + 1) > kLimit / a->experts)
        return set_error(FP8_ERR_SHAPE, "%s: dimensions out of range", what);
    cudaStream_t st = as_stream(stream);
    if (!a->dW) return set_error(FP8_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if (a->M == 0) {   // no tokens at all
        if (a->accumulate) return FP8_OK;
        const size_t bytes = static_cast<size_t>(a->experts) * static_cast<size_t>(a->N) * static_cast<size_t>(a->K) * 4;
        const cudaError_t e = cudaMemsetAsync(a->dW, 0, bytes, st);
        return e == cudaSuccess ? FP8_OK : set_error(FP8_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    }
    const ExpertGemm g{a->dY_t, a->f_dy, a->X_t, a->f_x, a->N, a->K, a->M, a->scale_inv_dy, a->scale_inv_x, a->dW,
                       FP8_OUT_F32, a->accumulate != 0, a->pow2, a->offsets, a->experts};
    r = launch_gemm_by_tokens(g, st);
    return r != FP8_OK ? r : launch_status(what);
}

}  // extern "C"

// rowops.cuh -- device helpers shared by the kernels that work on rows (norm.cu,
// moe.cu, the activation gradient of gemm_act.cu): 8-element pieces of a row
// as fp32, streaming loads and stores, reductions, the FP8 cast.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace fp8 {
namespace row {

constexpr uint32_t kAll = 0xFFFFFFFFu;

// 16-byte streaming load: read once, so it is not kept in L1, where the rows'
// shared vectors (norm weights, gates) live.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void unpack8(float (&v)[8], const uint4& w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = bf_lo(u[e]);
        v[2 * e + 1] = bf_hi(u[e]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                      pack_bf16(v[6], v[7]));
}

// Two fp32 -> two FP8 codes (the first in the low byte), round to nearest
// even, saturating.
template <int FMT>
__device__ __forceinline__ uint32_t cvt_pair(float lo, float hi) {
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE,
                                                          FMT == 0 ? __NV_E4M3 : __NV_E5M2));
}

__device__ __forceinline__ uint32_t cvt_pair(int fmt, float lo, float hi) {
    return fmt == 0 ? cvt_pair<0>(lo, hi) : cvt_pair<1>(lo, hi);
}

__device__ __forceinline__ uint2 cvt8(int fmt, const float (&v)[8], float s) {
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        c[e] = cvt_pair(fmt, __fmul_rn(v[2 * e], s), __fmul_rn(v[2 * e + 1], s));
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// |v| as an unsigned integer that orders like the magnitude, NaN above all.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Raise *amax (fp32, non-negative) to the magnitude with these bits.  Most
// callers find it already higher and save the atomic.
__device__ __forceinline__ void raise_amax(float* amax, uint32_t bits) {
    unsigned* a = reinterpret_cast<unsigned*>(amax);
    if (bits > *static_cast<volatile unsigned*>(a)) atomicMax(a, bits);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Sums of N values over the CTA's threads (a multiple of 32), the same bits
// in every thread.  One barrier a call; `part` is this call's own buffer of
// N x 32 floats: a caller alternates between two.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = warp_sum(v[i]);
        if (lane == 0) part[i * 32 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < nw ? part[i * 32 + lane] : 0.0f);
}

}  // namespace row
}  // namespace fp8

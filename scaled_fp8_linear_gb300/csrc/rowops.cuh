// rowops.cuh -- device helpers shared by the kernels that work on rows (norm.cu,
// moe.cu, the activation gradient of gemm_act.cu): 8-element pieces of a row
// as fp32, streaming loads and stores, reductions, the FP8 cast.
#pragma once

#include <cfloat>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace fp8 {
namespace row {

constexpr uint32_t kAll = 0xFFFFFFFFu;

// 16-byte streaming load: read once, so it is not kept in L1, where the rows'
// shared vectors (norm weights, gates) live.  A plain load, not one of the
// read-only path: some outputs may be an input itself.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
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

// ------------------------------------------------ pairs of fp32 in one register pair
// Packed instructions do two elements at a time: the norms' kernels are near
// the issue limit without them.

using f2 = uint64_t;

__device__ __forceinline__ f2 mk2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f2 all2(float v) { return mk2(v, v); }
__device__ __forceinline__ float lo2(f2 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi2(f2 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) { return ptx::fmul2(a, b); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) { return ptx::ffma2(a, b, c); }
__device__ __forceinline__ f2 bf2(uint32_t w) { return mk2(bf_lo(w), bf_hi(w)); }
__device__ __forceinline__ uint32_t pack_bf16(f2 v) { return pack_bf16(lo2(v), hi2(v)); }

// Eight elements, as loaded (bf16: one 16-byte word, fp32: two) and as pairs.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = ld_stream(p); }
    __device__ __forceinline__ void load_shared(const __nv_bfloat16* p) {
        w = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ void pairs(f2 (&v)[4]) const {
        v[0] = bf2(w.x); v[1] = bf2(w.y); v[2] = bf2(w.z); v[3] = bf2(w.w);
    }
};
template <>
struct Raw8<float> {
    uint4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const float* p) {
        a = ld_stream(p);
        b = ld_stream(p + 4);
    }
    __device__ __forceinline__ void load_shared(const float* p) {
        a = *reinterpret_cast<const uint4*>(p);
        b = *reinterpret_cast<const uint4*>(p + 4);
    }
    __device__ __forceinline__ void pairs(f2 (&v)[4]) const {
        v[0] = mk2(__uint_as_float(a.x), __uint_as_float(a.y));
        v[1] = mk2(__uint_as_float(a.z), __uint_as_float(a.w));
        v[2] = mk2(__uint_as_float(b.x), __uint_as_float(b.y));
        v[3] = mk2(__uint_as_float(b.z), __uint_as_float(b.w));
    }
};

__device__ __forceinline__ void store_pairs(__nv_bfloat16* p, const f2 (&v)[4]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(v[0]), pack_bf16(v[1]), pack_bf16(v[2]), pack_bf16(v[3]));
}
__device__ __forceinline__ void store_pairs(float* p, const f2 (&v)[4]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(lo2(v[0]), hi2(v[0]), lo2(v[1]), hi2(v[1]));
    reinterpret_cast<float4*>(p)[1] = make_float4(lo2(v[2]), hi2(v[2]), lo2(v[3]), hi2(v[3]));
}

// Eight elements of a vector that every row shares, through L1.
__device__ __forceinline__ void shared_pairs(f2 (&v)[4], const float* p) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = mk2(a.x, a.y); v[1] = mk2(a.z, a.w); v[2] = mk2(b.x, b.y); v[3] = mk2(b.z, b.w);
}
__device__ __forceinline__ void shared_pairs(f2 (&v)[4], const __nv_bfloat16* p) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
    v[0] = bf2(w.x); v[1] = bf2(w.y); v[2] = bf2(w.z); v[3] = bf2(w.w);
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

template <int FMT>
__device__ __forceinline__ uint2 cvt8(const float (&v)[8], float s) {
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        c[e] = cvt_pair<FMT>(__fmul_rn(v[2 * e], s), __fmul_rn(v[2 * e + 1], s));
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ uint2 cvt8(int fmt, const float (&v)[8], float s) {
    return fmt == 0 ? cvt8<0>(v, s) : cvt8<1>(v, s);
}

// Codes of eight pairs-packed values.
template <int FMT>
__device__ __forceinline__ uint2 cvt8(const f2 (&v)[4], f2 s) {
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f2 t = mul2(v[e], s);
        c[e] = cvt_pair<FMT>(lo2(t), hi2(t));
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// |v| as an unsigned integer that orders like the magnitude, NaN above all.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// max(top, |v|), NaN if either is: abs_bits() of the result orders above all.
__device__ __forceinline__ float max_abs(float top, float v) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(top), "f"(fabsf(v)));
    return m;
}

// A row's scale from the bits of its largest magnitude, by the per-row cast's
// rule: 1 for a row that is all zero or not finite.
__device__ __forceinline__ float block_scale(uint32_t top, int fmt, int pow2) {
    const float a = __uint_as_float(top);
    if (!(a > 0.0f && a <= FLT_MAX)) return 1.0f;
    float s = __fdiv_rn(fmt == FP8_E4M3 ? 448.0f : 57344.0f, a);
    s = fminf(fmaxf(s, FLT_MIN), FLT_MAX);
    return pow2 ? __uint_as_float(__float_as_uint(s) & 0xFF800000u) : s;
}

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

// The same for CTAs of at most 16 warps: every thread adds the warps' values
// itself, four at a load, which is a third of a second shuffle tree's
// latency.  `part`: N x 16 floats, zero past the CTA's warps.
template <int N>
__device__ __forceinline__ void block_sum16(float (&v)[N], float* part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = warp_sum(v[i]);
        if (lane == 0) part[i * 16 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float4* q = reinterpret_cast<const float4*>(part + i * 16);
        const float4 a = q[0], b = q[1], c = q[2], d = q[3];
        const f2 s = add2(add2(add2(mk2(a.x, a.y), mk2(a.z, a.w)), add2(mk2(b.x, b.y), mk2(b.z, b.w))),
                          add2(add2(mk2(c.x, c.y), mk2(c.z, c.w)), add2(mk2(d.x, d.y), mk2(d.z, d.w))));
        v[i] = lo2(s) + hi2(s);
    }
}

}  // namespace row
}  // namespace fp8

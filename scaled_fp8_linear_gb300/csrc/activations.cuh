// activations.cuh -- the activations and their derivatives on pairs of fp32, for
// the products' epilogues (gemm_act.cu) and the elementwise kernels
// (gemm_act.cu, act_block.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/fp8linear.h"
#include "rowops.cuh"

namespace fp8 {
namespace {

using row::f2;

__device__ __forceinline__ float ex2(float x) {   // 2^x
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC = 0.7978845608028654f, kGeluA = 0.044715f;   // sqrt(2 / pi)
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// 1 / (1 + exp(-k x)) for a pair, `scale` = -k log2(e).  Far out, 2^x runs to
// infinity or zero and the result to 0 (past k x = -87.3, where it would be a
// subnormal) or 1.  The exponent's rounding comes back as
// a relative error: where the result is small, 2^-24 |k x| and 2^-22 of the two
// approximations, 17 2^-24 at -20.  Outputs of 16 and 8 bits do not see it: SiLU's
// gradient of 16384 x 2048 gated over four seeds, 3630 of 268 million codes other than
// 64 bits', 3611 with the library's exp and an IEEE division.  With the exponent's
// remainder added to 2^x, which leaves 4 2^-24, 3633, and a Newton step of the reciprocal
// besides 3646; 32768 x 2048 then takes 167 and 175 us for 160.
__device__ __forceinline__ f2 sigmoid2(f2 x, float scale) {
    const f2 t = row::mul2(x, row::all2(scale));
    return row::mk2(rcp(1.0f + ex2(row::lo2(t))), rcp(1.0f + ex2(row::hi2(t))));
}

// The argument of GELU's tanh form: z + 0.044715 z^3; 1 + tanh(u) = 2 / (1 + exp(-2u)).
__device__ __forceinline__ f2 gelu_arg2(f2 z) {
    return row::mul2(z, row::fma2(row::mul2(z, z), row::all2(kGeluA), row::all2(1.0f)));
}

// Phi(z) of a pair, and e = exp(-z^2 / 2).  (1 + erf(z / sqrt(2))) / 2 would
// cancel on the negative side (nothing is left of it at -5.5), so the tail
// h = Phi(-|z|) is taken as e t P(t), t = 1 / (1 + 0.305 |z|), the form of
// Abramowitz and Stegun 7.1.26, with a P of degree 7 fitted here to the least
// relative error over |z| <= 13.2 (1.4e-7 with these fp32 coefficients, 0.5 + 7e-8 at
// 0; 5e-7 with fp32's roundings up to 2, 3e-6 at 8, where e's exponent is 46).  e serves the derivative as well, and P
// runs on pairs: 8192 x 11008 gated to codes 115 us (127 with erff, 179 with erfcf).
__device__ __forceinline__ f2 normal_cdf2(f2 z, f2& e) {
    constexpr float P[8] = {1.216366664e-01f, 1.225134656e-01f, 1.031311154e-01f, 1.219759211e-01f,
                            -3.978091478e-02f, 1.876799166e-01f, -1.541295797e-01f, 3.697348014e-02f};
    const f2 one = row::all2(1.0f);
    const f2 d = row::fma2(z & 0x7FFFFFFF7FFFFFFFull, row::all2(0.305f), one);   // |z| in both halves
    const f2 t = row::mk2(rcp(row::lo2(d)), rcp(row::hi2(d)));
    const f2 x = row::mul2(row::mul2(z, z), row::all2(-0.5f * kLog2e));
    e = row::mk2(ex2(row::lo2(x)), ex2(row::hi2(x)));
    f2 h = row::all2(P[7]);
#pragma unroll
    for (int i = 6; i >= 0; --i) h = row::fma2(h, t, row::all2(P[i]));
    h = row::mul2(row::mul2(h, t), e);
    const f2 rest = row::fma2(h, row::all2(-1.0f), one);
    return row::mk2(row::lo2(z) < 0.0f ? row::lo2(h) : row::lo2(rest),
                    row::hi2(z) < 0.0f ? row::hi2(h) : row::hi2(rest));
}

__device__ __forceinline__ float relu(float z) { return z > 0.0f ? z : (z != z ? z : 0.0f); }

template <int ACT>
__device__ __forceinline__ f2 act2(f2 z) {
    if constexpr (ACT == FP8_ACT_RELU) return row::mk2(relu(row::lo2(z)), relu(row::hi2(z)));
    if constexpr (ACT == FP8_ACT_SILU) return row::mul2(z, sigmoid2(z, -kLog2e));
    if constexpr (ACT == FP8_ACT_GELU) {
        f2 e;
        return row::mul2(z, normal_cdf2(z, e));
    }
    if constexpr (ACT == FP8_ACT_GELU_TANH)
        return row::mul2(z, sigmoid2(gelu_arg2(z), -2.0f * kGeluC * kLog2e));
    return z;
}

// act(z) and its derivative.
template <int ACT>
__device__ __forceinline__ void act_and_grad2(f2 z, f2& a, f2& g) {
    const f2 one = row::all2(1.0f), minus = row::all2(-1.0f);
    if constexpr (ACT == FP8_ACT_RELU) {
        a = act2<ACT>(z);
        g = row::mk2(row::lo2(z) > 0.0f ? 1.0f : 0.0f, row::hi2(z) > 0.0f ? 1.0f : 0.0f);
    } else if constexpr (ACT == FP8_ACT_SILU) {
        const f2 s = sigmoid2(z, -kLog2e);
        a = row::mul2(z, s);
        g = row::fma2(a, row::fma2(s, minus, one), s);   // s + z s (1 - s)
    } else if constexpr (ACT == FP8_ACT_GELU) {
        f2 e;
        const f2 cdf = normal_cdf2(z, e);
        a = row::mul2(z, cdf);
        g = row::fma2(row::mul2(z, row::all2(kInvSqrt2Pi)), e, cdf);
    } else if constexpr (ACT == FP8_ACT_GELU_TANH) {
        // s + z s (1 - s) u', u' = 2 sqrt(2/pi) (1 + 3 0.044715 z^2).  Past |z| = 100
        // s (1 - s) is 0 in fp32, so z stays there: 0 times z^2's overflow is NaN.
        const f2 s = sigmoid2(gelu_arg2(z), -2.0f * kGeluC * kLog2e);
        a = row::mul2(z, s);
        const f2 c = row::mk2(fminf(fmaxf(row::lo2(z), -100.0f), 100.0f), fminf(fmaxf(row::hi2(z), -100.0f), 100.0f));
        const f2 du = row::fma2(row::mul2(c, c), row::all2(6.0f * kGeluC * kGeluA), row::all2(2.0f * kGeluC));
        g = row::fma2(row::mul2(row::mul2(c, s), du), row::fma2(s, minus, one), s);
    } else {
        a = z;
        g = one;
    }
}

template <int ACT, int N>
__device__ __forceinline__ void act_all(float (&v)[N]) {
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const f2 a = act2<ACT>(row::mk2(v[j], v[j + 1]));
        v[j] = row::lo2(a);
        v[j + 1] = row::hi2(a);
    }
}

template <int N>
__device__ __forceinline__ void apply_act(int act, float (&v)[N]) {
    switch (act) {   // uniform over the grid
        case FP8_ACT_RELU: act_all<FP8_ACT_RELU>(v); break;
        case FP8_ACT_SILU: act_all<FP8_ACT_SILU>(v); break;
        case FP8_ACT_GELU: act_all<FP8_ACT_GELU>(v); break;
        case FP8_ACT_GELU_TANH: act_all<FP8_ACT_GELU_TANH>(v); break;
        default: break;
    }
}

}  // namespace
}  // namespace fp8

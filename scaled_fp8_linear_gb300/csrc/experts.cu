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

// ------------------------------------------------------------------ few rows an expert

// Tokens of decoding or of a prompt's chunk: reading the weights is the floor,
// and a 256-row tile would be nearly empty.  So the operands change sides: 128
// rows of the weights are the MMA's M, TN tokens its N.  A weight tile is one
// 128x128 block a K step, so its factor is one number, and a token's is a
// column's.
//   warp 0      TMA producer (one thread): weight and token tiles into a ring;
//   warp 1      MMA issuer: each 128-deep K block to a TMEM buffer of TN columns;
//   warp 2      TMEM allocation;
//   warp 3      factors: per four K blocks the products (token x weight block)
//               of TN tokens, one group ahead;
//   warps 4-    promotion: a weight row a thread, its sums with TN (16) or TN / 2
//               tokens in registers, 16 partial sums on their way from TMEM while
//               16 are added; at the tile's end a token's 32 neighbouring columns
//               a store.
// One CTA an SM; the ring holds 160 KB or more in flight, so that waiting for the
// sums of one tile does not stop the next tile's weights.
constexpr int BK = 128, UMMA_K = 32;
constexpr int kFewSets = 3;   // factor groups in flight

template <int TN>
struct Few {
    static constexpr int EPI = TN == 16 ? 4 : 8;   // promotion warps: two a lane quarter take half of the tokens each
    static constexpr int CW = TN * 4 / EPI;        // tokens of one
    static constexpr int THREADS = (4 + EPI) * 32;
    static constexpr int NBUF = TN <= 64 ? 4 : 512 / TN;
    static constexpr uint32_t TMEM_COLS = NBUF * TN < 32 ? 32 : NBUF * TN;
    static constexpr int W_BYTES = 128 * BK, T_BYTES = TN * BK;
    static constexpr int STAGE_BYTES = W_BYTES + T_BYTES;
    static constexpr int STAGES = 184 * 1024 / STAGE_BYTES;
    static constexpr int SET_BYTES = 4 * TN * 4;   // [4 K blocks][TN]
    static constexpr int BARS = 2 * STAGES + 2 * NBUF + 2 * kFewSets + 1;
    static constexpr int SMEM = STAGES * STAGE_BYTES + kFewSets * SET_BYTES + BARS * 8 + 16 +
                                static_cast<int>(sizeof(Units)) + 1024;
    static_assert(T_BYTES % 1024 == 0 && SMEM <= 227 * 1024, "swizzle atoms, shared memory");
};

struct FewParams {
    int M, N, num_n, num_kb;
    int fa, fb;
    const float* sa;
    const float* sb;
    void* D;
    int out;
    const int32_t* offsets;
    int experts;
    int vec_a, vec_b;
    unsigned* status;
};

struct FewTile {
    int expert, n_blk, t0, t_end;   // first token, end of the expert's
};

template <int TN>
__device__ __forceinline__ FewTile few_tile(int unit, const Units* u, const FewParams& p) {
    FewTile t;
    t.expert = expert_of(unit, u, p.experts);
    const int local = unit - u->first[t.expert];
    const int num_t = (u->end[t.expert] - u->begin[t.expert] + TN - 1) / TN;
    t.n_blk = local / num_t;   // token tiles innermost: they share the weights in L2
    t.t0 = u->begin[t.expert] + (local - t.n_blk * num_t) * TN;
    t.t_end = u->end[t.expert];
    return t;
}

// Four factors of a row of K blocks from kb on, 0 past the last.
__device__ __forceinline__ float4 factors4(const float* s, int kb, int KB, bool vec) {
    if (kb >= KB) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (vec) return *reinterpret_cast<const float4*>(s + kb);
    return make_float4(s[kb], kb + 1 < KB ? s[kb + 1] : 0.0f, kb + 2 < KB ? s[kb + 2] : 0.0f,
                       kb + 3 < KB ? s[kb + 3] : 0.0f);
}

template <int TN>
__global__ void __launch_bounds__(Few<TN>::THREADS, 1)
    gemm_experts_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT,
                            const __grid_constant__ FewParams p) {
    using L = Few<TN>;
    constexpr int STAGES = L::STAGES, NBUF = L::NBUF;
    ptx::griddep_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float* sets = reinterpret_cast<float*>(ring + STAGES * L::STAGE_BYTES);
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sets) + kFewSets * L::SET_BYTES);
    uint64_t* empty = full + STAGES;
    uint64_t* tfull = empty + STAGES;
    uint64_t* tempty = tfull + NBUF;
    uint64_t* ffull = tempty + NBUF;
    uint64_t* fempty = ffull + kFewSets;
    uint64_t* done = fempty + kFewSets;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    Units* units = reinterpret_cast<Units*>(reinterpret_cast<uint8_t*>(full) + L::BARS * 8 + 16);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < NBUF; ++b) {
            ptx::mbar_init(&tfull[b], 1);
            ptx::mbar_init(&tempty[b], L::EPI);   // promotion warps
        }
        for (int b = 0; b < kFewSets; ++b) {
            ptx::mbar_init(&ffull[b], 1);
            ptx::mbar_init(&fempty[b], L::EPI);
        }
        ptx::mbar_init(done, 1);
        *abort_flag = 0;
        ptx::fence_barrier_init();
        ptx::tma_prefetch_desc(&tmW);
        ptx::tma_prefetch_desc(&tmT);
    }
    if (warp == 2) {
        ptx::tmem_alloc(tmem_slot, L::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::griddep_wait();
    make_units(units, p.M, p.offsets, p.experts, p.num_n, kAllRows, TN);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int num_units = units->first[p.experts], KB = p.num_kb;
    const int u0 = blockIdx.x, step = gridDim.x;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int u = u0; ok && u < num_units; u += step) {
                const FewTile t = few_tile<TN>(u, units, p);
                const int yw = t.expert * p.N + t.n_blk * 128;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!ptx::mbar_wait<true>(&empty[stage], phase ^ 1u, abort_flag)) { ok = false; break; }
                    uint8_t* s = ring + stage * L::STAGE_BYTES;
                    ptx::mbar_arrive_expect_tx(&full[stage], L::STAGE_BYTES);
                    ptx::tma_load_2d(s, &tmW, &full[stage], kb * BK, yw);
                    ptx::tma_load_2d(s + L::W_BYTES, &tmT, &full[stage], kb * BK, t.t0);
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            uint32_t never = 0;   // drain: the last copies into each slot have landed
            for (int s = 0; s < STAGES; ++s) {
                if (issued <= s && issued < STAGES) break;
                ptx::mbar_wait<true>(&full[s], static_cast<uint32_t>(s) < stage ? phase : phase ^ 1u, &never);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = ptx::idesc_f8f6f4(p.fb, p.fa, 128, TN);
            uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
            bool ok = true;
            for (int u = u0; ok && u < num_units; u += step) {
                for (int kb = 0; kb < KB; ++kb) {
                    if (!ptx::mbar_wait<true>(&tempty[buf], buf_phase ^ 1u, abort_flag)) { ok = false; break; }
                    if (!ptx::mbar_wait<true>(&full[stage], phase, abort_flag)) { ok = false; break; }
                    ptx::tc_fence_after();
                    uint8_t* s = ring + stage * L::STAGE_BYTES;
                    const uint64_t wd = ptx::sdesc_kmajor_sw128(ptx::smem_u32(s));
                    const uint64_t td = ptx::sdesc_kmajor_sw128(ptx::smem_u32(s + L::W_BYTES));
#pragma unroll
                    for (int k = 0; k < BK / UMMA_K; ++k)
                        ptx::mma_f8f6f4(tmem_base + buf * TN, wd + (k * UMMA_K >> 4), td + (k * UMMA_K >> 4), idesc,
                                        k != 0);
                    ptx::mma_commit(&empty[stage]);
                    ptx::mma_commit(&tfull[buf]);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    if (++buf == NBUF) { buf = 0; buf_phase ^= 1u; }
                }
            }
            uint32_t never = 0;
            ptx::mma_commit(done);
            ptx::mbar_wait<true>(done, 0, &never);
        }
    } else if (warp == 3) {
        constexpr int PER = TN < 32 ? 1 : TN / 32;   // tokens a lane
        uint32_t set = 0, phase = 0;
        bool ok = true;
        for (int u = u0; ok && u < num_units; u += step) {
            const FewTile t = few_tile<TN>(u, units, p);
            const float* sw = p.sb + (static_cast<int64_t>(t.expert) * p.num_n + t.n_blk) * KB;
            auto token = [&](int i) {   // tokens past the last row are read at it
                return p.sa + static_cast<int64_t>(min(t.t0 + i * 32 + lane, p.M - 1)) * KB;
            };
            float4 w = factors4(sw, 0, KB, p.vec_b), f[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) f[i] = factors4(token(i), 0, KB, p.vec_a);
            for (int kb = 0; kb < KB; kb += 4) {
                ok = lane == 0 ? ptx::mbar_wait<true>(&fempty[set], phase ^ 1u, abort_flag) : false;
                ok = __shfl_sync(row::kAll, ok, 0);
                if (!ok) break;
                float* to = sets + set * (L::SET_BYTES / 4) + lane;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    if (TN >= 32 || lane < TN) {
                        to[32 * i] = __fmul_rn(f[i].x, w.x);
                        to[TN + 32 * i] = __fmul_rn(f[i].y, w.y);
                        to[2 * TN + 32 * i] = __fmul_rn(f[i].z, w.z);
                        to[3 * TN + 32 * i] = __fmul_rn(f[i].w, w.w);
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&ffull[set]);
                if (++set == kFewSets) { set = 0; phase ^= 1u; }
                w = factors4(sw, kb + 4, KB, p.vec_b);
#pragma unroll
                for (int i = 0; i < PER; ++i) f[i] = factors4(token(i), kb + 4, KB, p.vec_a);
            }
        }
    } else if (warp >= 4) {
        constexpr int CW = L::CW, STEPS = CW / 16;
        const int c0 = (warp - 4) / 4 * CW;   // this warp's first token
        const uint32_t tcol = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0;
        uint32_t buf = 0, buf_phase = 0, set = 0, set_phase = 0;
        bool ok = true;
        for (int u = u0; u < num_units; u += step) {
            float acc[CW];
#pragma unroll
            for (int c = 0; c < CW; ++c) acc[c] = 0.0f;
            for (int kb = 0; kb < KB; ++kb) {
                if ((kb & 3) == 0) {
                    ok = __all_sync(row::kAll, ptx::mbar_wait<true>(&ffull[set], set_phase, abort_flag));
                    if (!ok) break;
                }
                const float* f = sets + set * (L::SET_BYTES / 4) + (kb & 3) * TN + c0;
                ok = lane == 0 ? ptx::mbar_wait<true>(&tfull[buf], buf_phase, abort_flag) : false;
                ok = __shfl_sync(row::kAll, ok, 0);
                if (!ok) break;
                __syncwarp();
                ptx::tc_fence_after();
                uint32_t r[2][16];
                ptx::tmem_ld_32x32b_x16(tcol + buf * TN, r[0]);
#pragma unroll
                for (int j = 0; j < STEPS; ++j) {
                    float4 w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(f + 16 * j + 4 * i);
                    ptx::tmem_wait_ld();
                    if (j + 1 < STEPS) {
                        ptx::tmem_ld_32x32b_x16(tcol + buf * TN + 16 * (j + 1), r[(j + 1) & 1]);
                    } else {
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&tempty[buf]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float* a = acc + 16 * j + 4 * i;
                        const uint32_t* v = r[j & 1] + 4 * i;
                        a[0] = __fmaf_rn(__uint_as_float(v[0]), w[i].x, a[0]);
                        a[1] = __fmaf_rn(__uint_as_float(v[1]), w[i].y, a[1]);
                        a[2] = __fmaf_rn(__uint_as_float(v[2]), w[i].z, a[2]);
                        a[3] = __fmaf_rn(__uint_as_float(v[3]), w[i].w, a[3]);
                    }
                }
                if (++buf == NBUF) { buf = 0; buf_phase ^= 1u; }
                if ((kb & 3) == 3 || kb == KB - 1) {
                    __syncwarp();   // the set has been read
                    if (lane == 0) ptx::mbar_arrive(&fempty[set]);
                    if (++set == kFewSets) { set = 0; set_phase ^= 1u; }
                }
            }
            if (!ok) break;
            const FewTile t = few_tile<TN>(u, units, p);
            const int rows = t.t_end - t.t0 - c0;
            const int64_t at = static_cast<int64_t>(t.t0 + c0) * p.N + t.n_blk * 128 + (warp & 3) * 32 + lane;
            if (p.out == FP8_OUT_BF16) {
                __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.D) + at;
#pragma unroll
                for (int c = 0; c < CW; ++c)
                    if (c < rows) d[static_cast<int64_t>(c) * p.N] = __float2bfloat16_rn(acc[c]);
            } else {
                float* d = static_cast<float*>(p.D) + at;
#pragma unroll
                for (int c = 0; c < CW; ++c)
                    if (c < rows) d[static_cast<int64_t>(c) * p.N] = acc[c];
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem_base, L::TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag && p.status) atomicOr(p.status, 1u);
}

template <int TN>
int launch_few(const ExpertGemm& g, cudaStream_t stream) {
    using L = Few<TN>;
    CUtensorMap tmW, tmT;
    int r = make_kmajor_map(&tmW, g.B, g.N * g.experts, g.K, 128);
    if (r == FP8_OK) r = make_kmajor_map(&tmT, g.A, g.M, g.K, TN);
    static host::SmemAllowance allowance;
    auto k = gemm_experts_few_kernel<TN>;
    if (r == FP8_OK) r = host::allow_smem(k, L::SMEM, allowance);
    if (r != FP8_OK) return r;
    FewParams p{};
    p.M = static_cast<int>(g.M); p.N = static_cast<int>(g.N);
    p.num_n = static_cast<int>(g.N / 128); p.num_kb = static_cast<int>(g.K / BK);
    p.fa = g.fa; p.fb = g.fb; p.sa = g.sa; p.sb = g.sb;
    p.D = g.D; p.out = g.out; p.offsets = g.offsets; p.experts = g.experts;
    p.vec_a = p.num_kb % 4 == 0 && host::aligned(g.sa, 16);
    p.vec_b = p.num_kb % 4 == 0 && host::aligned(g.sb, 16);
    p.status = device_status_word();
    // at most this many tiles, however the rows are cut
    const int64_t busy = g.M < g.experts ? g.M : g.experts;
    const int64_t tiles = ((g.M - busy) / TN + busy) * p.num_n;
    const int sms = num_sms();
    launch_pdl(k, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), dim3(L::THREADS), L::SMEM, stream, tmW, tmT,
               p);
    return host::launch_status("fp8_gemm_experts");
}

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
    // rows an expert on average: the tile that holds them
    const int64_t rows = (a->M + a->experts - 1) / a->experts;
    cudaStream_t st = as_stream(stream);
    if (rows <= 8) return launch_few<16>(g, st);
    if (rows <= 16) return launch_few<32>(g, st);
    if (rows <= 40) return launch_few<64>(g, st);
    if (rows <= 112) return launch_few<128>(g, st);
    r = launch_gemm_by_rows(g, st);
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

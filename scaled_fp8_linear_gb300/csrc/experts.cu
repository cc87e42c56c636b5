// experts.cu -- FP8 products of experts in blocks of 128, and the weight
// gradients of experts: the entry points, and the kernel for few rows an expert.
// Products of more rows and the weight gradients run on gemm.cu's CTA-pair
// kernels.
#include <atomic>
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

// Tokens of decoding or of a prompt's chunk: reading the weights is the floor.
// 128 x 128 weight blocks against TN tokens a tile, one factor of the weights a K
// step; the products of its token factors and that one are made once a tile.
//   TN = 128   tokens on the MMA's M side: a promotion thread has a token and half
//              of its columns, so one factor serves all that it adds;
//   TN = 16    the weights on the M side, 16 tokens its N: a thread has one weight
//              row and all 16 tokens, a factor each.  An eighth of the shared
//              memory for tokens leaves more for weights on their way.
//   warp 0      TMA producer (one thread): weight and token tiles into a ring;
//   warp 1      MMA issuer: each 128-deep K block to a TMEM buffer of TN columns;
//   warp 2      TMEM allocation;
//   warp 3      factors: per four K blocks the products (token x weight block)
//               of TN tokens, one group ahead;
//   warps 4-    promotion, 16 partial sums on their way from TMEM while 16 are
//               added.
// One CTA an SM; the ring holds 180 KB or more in flight, so that waiting for the
// sums of one tile does not stop the next tile's weights.
// Measured (and without the 256 MB that the timing left dirty in L2, some 20 us
// less): 64 tokens to 28 of 32 experts of 4096 x 7168 147 us (823 MB read, 6.7
// TB/s); 32 experts of 4096 x 4096 with 8 rows each 108, 24 rows 112, 64 rows
// 116-118, 96 rows 141.  With the weights on the M side at 128 tokens the last two
// took 142 and 171: each thread reads 64 factors from shared memory a K block, 512
// cycles an SM.  Sixteen promotion warps instead of eight 126 for 118.  CTA pairs
// that share the tokens, so that a quarter less goes into the SMs: level.
constexpr int BK = 128, UMMA_K = 32;
constexpr int kFewSets = 3;   // factor groups in flight

template <int TN>
struct Few {
    static constexpr bool ROWS = TN == 128;       // tokens on the M side
    static constexpr int EPI = ROWS ? 8 : 4;      // promotion warps: two a lane quarter take half of the columns each
    static constexpr int CW = TN * 4 / EPI;       // columns of one
    static constexpr int THREADS = (4 + EPI) * 32;
    static constexpr int NBUF = 4;
    static constexpr uint32_t TMEM_COLS = NBUF * TN;
    static constexpr int W_BYTES = 128 * BK, T_BYTES = TN * BK;
    static constexpr int STAGE_BYTES = W_BYTES + T_BYTES;
    static constexpr int STAGES = 192 * 1024 / STAGE_BYTES;
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

// acc += partial sums x factors, W columns of a lane: f[c] for column c.
// Sixteen are on their way from TMEM while sixteen are added.
template <int W, typename Release>
__device__ __forceinline__ void add_columns(row::f2 (&acc)[W / 2], uint32_t tmem, const float* f, Release release) {
    uint32_t r[2][16];
    ptx::tmem_ld_32x32b_x16(tmem, r[0]);
#pragma unroll
    for (int j = 0; j < W / 16; ++j) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(f + 16 * j + 4 * i);
        ptx::tmem_wait_ld();
        if (j + 1 < W / 16) ptx::tmem_ld_32x32b_x16(tmem + 16 * (j + 1), r[(j + 1) & 1]);
        else release();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            row::f2* a = acc + 8 * j + 2 * i;
            const uint32_t* v = r[j & 1] + 4 * i;
            a[0] = row::fma2(row::mk2(__uint_as_float(v[0]), __uint_as_float(v[1])), row::mk2(w[i].x, w[i].y), a[0]);
            a[1] = row::fma2(row::mk2(__uint_as_float(v[2]), __uint_as_float(v[3])), row::mk2(w[i].z, w[i].w), a[1]);
        }
    }
}

// The same with one factor for all of a lane's columns.
template <int W, typename Release>
__device__ __forceinline__ void add_rows(row::f2 (&acc)[W / 2], uint32_t tmem, row::f2 f, Release release) {
    uint32_t r[2][16];
    ptx::tmem_ld_32x32b_x16(tmem, r[0]);
#pragma unroll
    for (int j = 0; j < W / 16; ++j) {
        ptx::tmem_wait_ld();
        if (j + 1 < W / 16) ptx::tmem_ld_32x32b_x16(tmem + 16 * (j + 1), r[(j + 1) & 1]);
        else release();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t* v = r[j & 1] + 2 * i;
            acc[8 * j + i] = row::fma2(row::mk2(__uint_as_float(v[0]), __uint_as_float(v[1])), f, acc[8 * j + i]);
        }
    }
}

// W neighbouring columns of one row of D, from element `at` on.
template <int W>
__device__ __forceinline__ void put_row(const FewParams& p, const row::f2 (&acc)[W / 2], int64_t at) {
    if (p.out == FP8_OUT_BF16) {
        uint4* d = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.D) + at);
        auto pair = [](row::f2 v) { return row::pack_bf16(row::lo2(v), row::hi2(v)); };
#pragma unroll
        for (int i = 0; i < W / 8; ++i)
            d[i] = make_uint4(pair(acc[4 * i]), pair(acc[4 * i + 1]), pair(acc[4 * i + 2]), pair(acc[4 * i + 3]));
    } else {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.D) + at);
#pragma unroll
        for (int i = 0; i < W / 4; ++i)
            d[i] = make_float4(row::lo2(acc[2 * i]), row::hi2(acc[2 * i]), row::lo2(acc[2 * i + 1]),
                               row::hi2(acc[2 * i + 1]));
    }
}

// One column of the first `rows` of W rows of D, from element `at` on.
template <int W>
__device__ __forceinline__ void put_column(const FewParams& p, const row::f2 (&acc)[W / 2], int64_t at, int rows) {
    if (p.out == FP8_OUT_BF16) {
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.D) + at;
#pragma unroll
        for (int c = 0; c < W; ++c)
            if (c < rows)
                d[static_cast<int64_t>(c) * p.N] = __float2bfloat16_rn(c & 1 ? row::hi2(acc[c / 2]) : row::lo2(acc[c / 2]));
    } else {
        float* d = static_cast<float*>(p.D) + at;
#pragma unroll
        for (int c = 0; c < W; ++c)
            if (c < rows) d[static_cast<int64_t>(c) * p.N] = c & 1 ? row::hi2(acc[c / 2]) : row::lo2(acc[c / 2]);
    }
}

// A tile's sums over K, in parts [TN * 128 / 4] of four in each CTA's shared memory
// (tokens on the M side: columns 4 c .. of token r at 128 c + r; else tokens 4 c ..
// of column r): this CTA adds its share of them, in the order of the CTAs, and
// writes it.
template <int TN>
__device__ __forceinline__ void join_parts(const float4* part, const FewParams& p, const FewTile& t, uint32_t rank,
                                           uint32_t ctas) {
    using L = Few<TN>;
    constexpr uint32_t ALL = TN * 128 / 4;
    const uint32_t share = ALL / ctas;
    for (uint32_t i = rank * share + threadIdx.x; i < (rank + 1) * share; i += L::THREADS) {
        float4 v = ptx::ld_shared_cluster_f4(ptx::cluster_addr(part + i, 0));
        for (uint32_t c = 1; c < ctas; ++c) {
            const float4 w = ptx::ld_shared_cluster_f4(ptx::cluster_addr(part + i, c));
            v.x = __fadd_rn(v.x, w.x); v.y = __fadd_rn(v.y, w.y); v.z = __fadd_rn(v.z, w.z); v.w = __fadd_rn(v.w, w.w);
        }
        const row::f2 acc[2] = {row::mk2(v.x, v.y), row::mk2(v.z, v.w)};
        const int r = static_cast<int>(i & 127), c4 = static_cast<int>(i >> 7) * 4;
        if constexpr (L::ROWS) {
            const int token = t.t0 + r;
            const int64_t at = static_cast<int64_t>(token) * p.N + t.n_blk * 128 + c4;
            if (token >= t.t_end) continue;
            if (p.out == FP8_OUT_BF16)
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.D) + at) =
                    make_uint2(row::pack_bf16(v.x, v.y), row::pack_bf16(v.z, v.w));
            else
                *reinterpret_cast<float4*>(static_cast<float*>(p.D) + at) = v;
        } else {
            const int64_t at = static_cast<int64_t>(t.t0 + c4) * p.N + t.n_blk * 128 + r;
            put_column<4>(p, acc, at, t.t_end - t.t0 - c4);
        }
    }
}

// SPLIT: a cluster has one tile, each of its CTAs a range of K in groups of four
// K blocks, joined through distributed shared memory in the CTAs' order.  For
// products of few tiles, where the way through a tile's K is the time.
template <int TN, bool SPLIT>
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
    const uint32_t ctas = SPLIT ? ptx::cluster_nctarank() : 1, rank = SPLIT ? ptx::cluster_ctarank() : 0;
    const int u0 = static_cast<int>(blockIdx.x / ctas), step = static_cast<int>(gridDim.x / ctas);
    const int groups = (KB + 3) / 4;
    const int kb0 = SPLIT ? static_cast<int>(groups * rank / ctas) * 4 : 0;
    const int kb1 = SPLIT ? min(static_cast<int>(groups * (rank + 1) / ctas) * 4, KB) : KB;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int u = u0; ok && u < num_units; u += step) {
                const FewTile t = few_tile<TN>(u, units, p);
                const int yw = t.expert * p.N + t.n_blk * 128;
                for (int kb = kb0; kb < kb1; ++kb) {
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
            const uint32_t idesc = L::ROWS ? ptx::idesc_f8f6f4(p.fa, p.fb, 128, TN) : ptx::idesc_f8f6f4(p.fb, p.fa, 128, TN);
            uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
            bool ok = true;
            for (int u = u0; ok && u < num_units; u += step) {
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!ptx::mbar_wait<true>(&tempty[buf], buf_phase ^ 1u, abort_flag)) { ok = false; break; }
                    if (!ptx::mbar_wait<true>(&full[stage], phase, abort_flag)) { ok = false; break; }
                    ptx::tc_fence_after();
                    uint8_t* s = ring + stage * L::STAGE_BYTES;
                    const uint64_t wd = ptx::sdesc_kmajor_sw128(ptx::smem_u32(s));
                    const uint64_t td = ptx::sdesc_kmajor_sw128(ptx::smem_u32(s + L::W_BYTES));
#pragma unroll
                    for (int k = 0; k < BK / UMMA_K; ++k)
                        ptx::mma_f8f6f4(tmem_base + buf * TN, (L::ROWS ? td : wd) + (k * UMMA_K >> 4),
                                        (L::ROWS ? wd : td) + (k * UMMA_K >> 4), idesc, k != 0);
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
            float4 w = factors4(sw, kb0, KB, p.vec_b), f[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) f[i] = factors4(token(i), kb0, KB, p.vec_a);
            for (int kb = kb0; kb < kb1; kb += 4) {
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
        constexpr int CW = L::CW;
        const int quarter = warp & 3, c0 = (warp - 4) / 4 * CW;   // this warp's lanes and first column
        const uint32_t tcol = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + c0;
        const float* mine = sets + (L::ROWS ? quarter * 32 + lane : c0);
        uint32_t buf = 0, buf_phase = 0, set = 0, set_phase = 0;
        bool ok = true;
        for (int u = u0; u < num_units; u += step) {
            row::f2 acc[CW / 2];
#pragma unroll
            for (int c = 0; c < CW / 2; ++c) acc[c] = 0ull;
            for (int kb = kb0; kb < kb1; ++kb) {
                if ((kb & 3) == 0) {
                    ok = __all_sync(row::kAll, ptx::mbar_wait<true>(&ffull[set], set_phase, abort_flag));
                    if (!ok) break;
                }
                const float* f = mine + set * (L::SET_BYTES / 4) + (kb & 3) * TN;
                ok = lane == 0 ? ptx::mbar_wait<true>(&tfull[buf], buf_phase, abort_flag) : false;
                ok = __shfl_sync(row::kAll, ok, 0);
                if (!ok) break;
                __syncwarp();
                ptx::tc_fence_after();
                auto release = [&]() {   // the buffer has been read
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&tempty[buf]);
                };
                if constexpr (L::ROWS) add_rows<CW>(acc, tcol + buf * TN, row::all2(*f), release);
                else add_columns<CW>(acc, tcol + buf * TN, f, release);
                if (++buf == NBUF) { buf = 0; buf_phase ^= 1u; }
                if ((kb & 3) == 3 || kb == kb1 - 1) {
                    __syncwarp();   // the set has been read
                    if (lane == 0) ptx::mbar_arrive(&fempty[set]);
                    if (++set == kFewSets) { set = 0; set_phase ^= 1u; }
                }
            }
            if (!ok) break;
            const FewTile t = few_tile<TN>(u, units, p);
            if constexpr (SPLIT) {   // the ring is free: its last copies have been multiplied
                float4* to = reinterpret_cast<float4*>(ring) + c0 / 4 * 128 + quarter * 32 + lane;
#pragma unroll
                for (int i = 0; i < CW / 4; ++i)
                    to[128 * i] = make_float4(row::lo2(acc[2 * i]), row::hi2(acc[2 * i]), row::lo2(acc[2 * i + 1]),
                                              row::hi2(acc[2 * i + 1]));
            } else if constexpr (L::ROWS) {
                const int token = t.t0 + quarter * 32 + lane;
                if (token < t.t_end) put_row<CW>(p, acc, static_cast<int64_t>(token) * p.N + t.n_blk * 128 + c0);
            } else {
                const int64_t at = static_cast<int64_t>(t.t0 + c0) * p.N + t.n_blk * 128 + quarter * 32 + lane;
                put_column<CW>(p, acc, at, t.t_end - t.t0 - c0);
            }
        }
    }
    if constexpr (SPLIT) {
        __syncwarp();
        ptx::cluster_sync();   // every CTA's part is there
        if (u0 < num_units)
            join_parts<TN>(reinterpret_cast<const float4*>(ring), p, few_tile<TN>(u0, units, p), rank, ctas);
        __syncwarp();
        ptx::cluster_sync();   // and has been read
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem_base, L::TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag && p.status) atomicOr(p.status, 1u);
}

// How many clusters of `ctas` (2, 4, 8) CTAs of the split kernel the device holds at
// once; cached per device.  Fewer than its SMs would: a cluster is within one GPC.
template <int TN>
int few_clusters(int ctas) {
    static std::atomic<int> cache[64][4] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
    const bool known = dev >= 0 && dev < 64;   // other devices: asked at every call
    std::atomic<int>* c = known ? &cache[dev][ctas / 4 + 1] : nullptr;
    int n = known ? c->load(std::memory_order_relaxed) : 0;
    if (n) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas * 1024));
    cfg.blockDim = dim3(Few<TN>::THREADS);
    cfg.dynamicSmemBytes = Few<TN>::SMEM;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ctas);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, gemm_experts_few_kernel<TN, true>, &cfg) != cudaSuccess || n <= 0) {
        (void)cudaGetLastError();
        n = num_sms() / (2 * ctas);
    }
    if (known) c->store(n, std::memory_order_relaxed);
    return n;
}

// How many tiles of tn tokens there are at most, however the rows are cut.
int64_t most_tiles(const ExpertGemm& g, int tn) {
    const int64_t busy = g.M < g.experts ? g.M : g.experts;
    return ((g.M - busy) / tn + busy) * (g.N / 128);
}

template <int TN>
int launch_few(const ExpertGemm& g, cudaStream_t stream) {
    using L = Few<TN>;
    CUtensorMap tmW, tmT;
    int r = make_kmajor_map(&tmW, g.B, g.N * g.experts, g.K, 128);
    if (r == FP8_OK) r = make_kmajor_map(&tmT, g.A, g.M, g.K, TN);
    static host::SmemAllowance whole, split;
    if (r == FP8_OK) r = host::allow_smem(gemm_experts_few_kernel<TN, false>, L::SMEM, whole);
    if (r == FP8_OK) r = host::allow_smem(gemm_experts_few_kernel<TN, true>, L::SMEM, split);
    if (r != FP8_OK) return r;
    FewParams p{};
    p.M = static_cast<int>(g.M); p.N = static_cast<int>(g.N);
    p.num_n = static_cast<int>(g.N / 128); p.num_kb = static_cast<int>(g.K / BK);
    p.fa = g.fa; p.fb = g.fb; p.sa = g.sa; p.sb = g.sb;
    p.D = g.D; p.out = g.out; p.offsets = g.offsets; p.experts = g.experts;
    p.vec_a = p.num_kb % 4 == 0 && host::aligned(g.sa, 16);
    p.vec_b = p.num_kb % 4 == 0 && host::aligned(g.sb, 16);
    p.status = device_status_word();
    const int64_t tiles = most_tiles(g, TN), sms = num_sms();
    // As many CTAs a tile as groups of K blocks and all tiles' clusters at once allow.
    // (us with a launch's and a cold cache's 10, one CTA against 8, 4 or 2: 1 row of
    // 128 x 7168 28 against 13; 100 rows of 1024 x 7168 30 against 18, 16 of 2048 x
    // 7168 30 against 19, 64 of 4096 x 4096 22 against 18.  In two rounds 16 tiles of
    // 8 CTAs take 28.)
    const int groups = (p.num_kb + 3) / 4;
    int ctas = 8;
    while (ctas > 1 && (groups < ctas || tiles * ctas > sms || tiles > few_clusters<TN>(ctas))) ctas /= 2;
    if (ctas > 1)
        launch_pdl_cluster(gemm_experts_few_kernel<TN, true>, dim3(static_cast<unsigned>(tiles * ctas)), dim3(L::THREADS),
                           L::SMEM, ctas, stream, tmW, tmT, p);
    else
        launch_pdl(gemm_experts_few_kernel<TN, false>, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)),
                   dim3(L::THREADS), L::SMEM, stream, tmW, tmT, p);
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
    // By rows an expert on average (us, sizes as above).  Tiles of 16 tokens against
    // 128: 8 rows 108 against 108, 12 rows 115 against 110, and where one in eight
    // of 64 experts of 2048 x 7168 has a row, 36 against 44.  128 against CTA pairs of
    // 256: fp32 factors 160 rows 179 against 191, 224 rows 214 against 213, 288 rows
    // 252 against 249; with powers of two, which only the pairs hand to the tensor
    // core, 64 rows 118 against 120, 80 rows 126 against 120.  And tiles of 128 that
    // all run at once, of which the pairs would be half or a quarter of the CTAs: 300
    // rows of 1024 x 7168 20 against 42 (powers of two 32), 1000 rows of 2048 x 7168 32
    // against 42 (34), 2000 rows of 1024 x 2048 17 against 22 (22).
    const int64_t rows = (a->M + a->experts - 1) / a->experts;
    cudaStream_t st = as_stream(stream);
    if (rows <= 8) return launch_few<16>(g, st);
    if (rows <= (a->pow2 ? 72 : 224) || most_tiles(g, 128) <= num_sms()) return launch_few<128>(g, st);
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

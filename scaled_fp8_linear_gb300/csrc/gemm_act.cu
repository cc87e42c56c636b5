// gemm_act.cu -- FP8 GEMM with bias, activation and residual in its epilogue,
// dense or one product per expert, and the gradient of that epilogue.
//
//   z = s_a s_b A . B^T + bias;  v = act(z), or act(z_gate) z_up;  D = v + residual
//
// The products run as in gemm.cu: TMA tiles into a shared-memory ring, one
// thread issuing tcgen05.mma into one of two TMEM accumulators, epilogue
// warps on the other.  What is different here:
//   - gated: the accumulator's left half holds a tile of the gate's product
//     and the right half the same tile of the up product (the B rows of the
//     two are loaded side by side), so an epilogue thread has both in its row
//     and z_up never goes through memory;
//   - per expert: a unit of work is a tile of one expert's rows; the experts'
//     row offsets are read on the device, so no count comes to the host.  A
//     tile's rows past its expert's end are computed and not written; where
//     an expert ends within a stored box, the rows are stored one by one;
//   - eight epilogue warps: an activation costs more than a scale.
// z stays in fp32 from the accumulator to D; D, z and the codes are each
// rounded once.
// Measured on a GB300: gated 4096 x 28672 x 8192 with z kept 1.18 ms (3.27
// PFLOP/s, 0.86 of twice the bf16 cuBLAS burst rate), 4099 x 8192 x 28672 onto a
// residual 0.64 ms (3.0; the power limit sets the clock), 32 experts' gated
// products of 2048 x 4096 over 8192 rows to codes 138 us (2.0; 0.6 GB of weights,
// tiles bound by the 64 bytes a cycle that an SM takes in).
#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/fp8linear.h"
#include "activations.cuh"
#include "experts.cuh"
#include "hostops.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowops.cuh"

namespace fp8 {
namespace {

constexpr int BK = 128;       // FP8 elements of K per stage
constexpr int UMMA_K = 32;    // K of one kind::f8f6f4 instruction
constexpr int kEpiWarps = 8;
constexpr int kThreads = (4 + kEpiWarps) * 32;

struct ActParams {
    int64_t M, N, K;
    int num_n, num_kb;
    int fa, fb, ga, gb;
    const float* sa;
    const float* sb;
    int act;
    const __nv_bfloat16* bias;
    const __nv_bfloat16* residual;
    void* z;
    void* d;
    uint8_t* q;
    int q_fmt;
    const float* q_scale;
    float* amax;
    const int32_t* offsets;   // null: one product over all rows
    int experts;
    int group;                // raster group (row blocks)
    int part;                 // kAllRows, or which part of each product's rows
    unsigned* status;
};

// ------------------------------------------------------------------ units of work

__device__ __forceinline__ void make_units(Units* u, const ActParams& p, int rows_per_tile) {
    make_units(u, static_cast<int>(p.M), p.offsets, p.experts, p.num_n, p.part, rows_per_tile);
}

struct Tile {
    int expert;
    int row0, row_end;   // first row, end of the expert's rows
    int n_blk;
};

__device__ __forceinline__ Tile tile_of(int unit, const Units* u, const ActParams& p,
                                        int rows_per_tile) {
    const int lo = expert_of(unit, u, p.experts);
    const int local = unit - u->first[lo];
    const int num_m = (u->end[lo] - u->begin[lo] + rows_per_tile - 1) / rows_per_tile;
    // grouped raster: `group` row blocks down each column block, so that the
    // CTAs at work share A and B panels in L2
    const int per_group = p.group * p.num_n;
    const int g = local / per_group;
    const int size = min(num_m - g * p.group, p.group);
    const int in_g = local - g * per_group;
    Tile t;
    t.expert = lo;
    t.row0 = u->begin[lo] + (g * p.group + in_g % size) * rows_per_tile;
    t.row_end = u->end[lo];
    t.n_blk = in_g / size;
    return t;
}

// ------------------------------------------------------------------ the epilogue

// A warp's output staging: SLOTS boxes of 2 KB in turn, so that a box is filled
// while the copies of the ones before it read theirs.
constexpr int kSlotBytes = 2048;

template <int SLOTS>
struct Staging {
    uint8_t* base;
    uint32_t turn = 0;
    __device__ __forceinline__ uint8_t* next() {
        uint8_t* s = base + turn * kSlotBytes;
        turn = turn + 1 == SLOTS ? 0 : turn + 1;
        return s;
    }
};

// A warp's 32 rows of one tile: how a box of theirs is written.  kCopy: by the
// TMA, which leaves out rows and columns past the matrix.  kByRow: the product
// ends within the box and another's rows follow, so each row's thread stores
// its own.  kNone: nothing there to write.
enum class BoxMode { kNone, kCopy, kByRow };

// Fills the warp's next slot through `fill` and, in kCopy, sends its box.
template <int SLOTS, typename Fill>
__device__ __forceinline__ void emit(Staging<SLOTS>& staging, const CUtensorMap* map, int64_t x, int64_t y,
                                     BoxMode mode, Fill fill) {
    const int lane = threadIdx.x & 31;
    uint8_t* slot = staging.next();
    if (lane == 0) ptx::bulk_wait_group_read<SLOTS - 1>();   // the slot's last box has been read
    __syncwarp();
    fill(slot);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (mode == BoxMode::kCopy)
            ptx::tma_store_2d(map, ptx::smem_u32(slot), static_cast<int32_t>(x), static_cast<int32_t>(y));
        ptx::bulk_commit_group();
    }
}

// One row's 32 columns (n_left of them in the matrix, a multiple of 16).
__device__ __forceinline__ void store_row(void* row0, int64_t pitch, int64_t m, int64_t n0, int n_left,
                                          const uint4 (&w)[4]) {
    uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(row0) + m * pitch + n0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (8 * j < n_left) out[j] = w[j];
}

__device__ __forceinline__ void pack32(uint4 (&w)[4], const float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = make_uint4(row::pack_bf16(v[8 * j], v[8 * j + 1]), row::pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                          row::pack_bf16(v[8 * j + 4], v[8 * j + 5]),
                          row::pack_bf16(v[8 * j + 6], v[8 * j + 7]));
}

// 32 columns of this thread's row as bf16: 64 bytes, in the TMA's 64-byte
// swizzle (piece j of row r at j ^ ((r >> 1) & 3)), which spreads the banks.
template <int SLOTS>
__device__ __forceinline__ void emit_bf16(Staging<SLOTS>& staging, const float (&v)[32],
                                          const CUtensorMap* map, int64_t x, int64_t y, BoxMode mode) {
    emit(staging, map, x, y, mode, [&](uint8_t* slot) {
        const int lane = threadIdx.x & 31, swz = (lane >> 1) & 3;
        uint4 w[4];
        pack32(w, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(slot + lane * 64 + 16 * (j ^ swz)) = w[j];
    });
}

// The codes of 32 columns: 32 bytes.
template <int FMT>
__device__ __forceinline__ void codes32(uint4 (&w)[2], const float (&v)[32], float s) {
    const f2 ss = row::all2(s);
    uint2 c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f2 t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = row::mk2(v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
        c[j] = row::cvt8<FMT>(t, ss);
    }
    w[0] = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
    w[1] = make_uint4(c[2].x, c[2].y, c[3].x, c[3].y);
}

// z of 32 columns: accumulator times factors plus bias.  fa: the row's
// factor; `base`: where this expert's factors and bias of column n0 start.
// Columns at n_left and past are not read.
__device__ __forceinline__ void dequant(float (&z)[32], const uint32_t (&r)[32], float fa,
                                        int64_t base, int n_left, const ActParams& p, float sb0) {
    if (p.gb == FP8_GRAN_ROW) {
        const int lane = threadIdx.x & 31;
        const float sbv = lane < n_left ? p.sb[base + lane] : 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            z[j] = __fmul_rn(__uint_as_float(r[j]), __fmul_rn(fa, __shfl_sync(row::kAll, sbv, j)));
    } else {
        const float f = __fmul_rn(fa, sb0);
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = __fmul_rn(__uint_as_float(r[j]), f);
    }
    if (p.bias) {
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
            if (j < n_left) {   // n_left is a multiple of 16
                float b[8];
                row::unpack8(b, __ldg(reinterpret_cast<const uint4*>(p.bias + base + j)));
#pragma unroll
                for (int e = 0; e < 8; ++e) z[j + e] = __fadd_rn(z[j + e], b[e]);
            }
        }
    }
}

struct OutMaps {
    CUtensorMap z, z_up, d, q;
};

// The residual of a warp's 32 rows x 32 columns, as four coalesced loads a
// thread (four lanes a row: 64 bytes, eight rows a load).  Loaded by the rows'
// own threads instead, every 16 bytes would be a line of its own: 88 us
// against 37 for an 8192 x 4096 x 1024 product.
struct Residual {
    uint4 w[4];
    __device__ __forceinline__ void load(const ActParams& p, int64_t m0, int row_end, int64_t n0) {
        if (!p.residual) return;
        const int lane = threadIdx.x & 31;
        const int64_t n = n0 + 8 * (lane & 3);
        if (n >= p.N) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + 8 * i + (lane >> 2);
            if (m < row_end) w[i] = row::ld_stream(p.residual + m * p.N + n);
        }
    }
};

// D of 32 columns: adds the residual to v (handed to the rows' threads through
// the slot that D's box leaves from) and, where D is wanted, writes the box.
template <int SLOTS>
__device__ __forceinline__ void emit_d(Staging<SLOTS>& staging, float (&v)[32], const Residual& res,
                                       const ActParams& p, const CUtensorMap* map, int64_t x, int64_t y,
                                       BoxMode mode) {
    emit(staging, map, x, y, p.d ? mode : BoxMode::kNone, [&](uint8_t* slot) {
        const int lane = threadIdx.x & 31, swz = (lane >> 1) & 3;
        uint8_t* own = slot + lane * 64;
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * i + (lane >> 2);
                *reinterpret_cast<uint4*>(slot + r * 64 + 16 * ((lane & 3) ^ ((r >> 1) & 3))) = res.w[i];
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float t[8];
                row::unpack8(t, *reinterpret_cast<const uint4*>(own + 16 * (j ^ swz)));
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * j + e] += t[e];
            }
        }
        uint4 w[4];
        pack32(w, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(own + 16 * (j ^ swz)) = w[j];
    });
}

// The epilogue of a warp: 32 rows x COLS output columns of one tile, from
// TMEM column `tcol` (gated: the up product UP columns further on).  `res`
// holds the first chunk's residual; each later one is loaded a chunk ahead.
template <bool GATED, int UP, int COLS, int SLOTS>
__device__ __forceinline__ void epilogue(Staging<SLOTS>& staging, Residual& res, uint32_t tcol, const Tile& t,
                                         int64_t m0, int64_t n_first, const ActParams& p,
                                         const OutMaps& maps, float& top) {
    const int lane = threadIdx.x & 31;
    const int64_t m = m0 + lane;
    const bool live = m < t.row_end;
    const int64_t b_rows = GATED ? 2 * p.N : p.N;
    const float fa = p.ga == FP8_GRAN_ROW ? p.sa[live ? m : p.M - 1] : p.sa[0];
    const float sb0 = p.gb == FP8_GRAN_ROW ? 0.0f : p.sb[t.expert];
    const float qs = p.q ? p.q_scale[0] : 0.0f;
#pragma unroll 1
    for (int c = 0; c < COLS / 32; ++c) {
        const int64_t n0 = n_first + c * 32;
        const int n_left = static_cast<int>(min(p.N - n0, static_cast<int64_t>(32)));
        const BoxMode mode = m0 >= t.row_end || n_left <= 0 ? BoxMode::kNone
                             : m0 + 32 > t.row_end && t.row_end < p.M ? BoxMode::kByRow : BoxMode::kCopy;
        const bool by_row = mode == BoxMode::kByRow && live;
        uint4 w[4];
        float z[32];
        uint32_t r[32], r_up[GATED ? 32 : 1];
        ptx::tmem_ld_32x32b_x32(tcol + c * 32, r);
        if constexpr (GATED) ptx::tmem_ld_32x32b_x32(tcol + UP + c * 32, r_up);
        ptx::tmem_wait_ld();
        dequant(z, r, fa, t.expert * b_rows + n0, n_left, p, sb0);
        if (p.z) {
            emit_bf16(staging, z, &maps.z, n0, m0, mode);
            if (by_row) {
                pack32(w, z);
                store_row(p.z, b_rows, m, n0, n_left, w);
            }
        }
        apply_act(p.act, z);
        if constexpr (GATED) {
            float up[32];
            dequant(up, r_up, fa, t.expert * b_rows + p.N + n0, n_left, p, sb0);
            if (p.z) {
                emit_bf16(staging, up, &maps.z_up, n0, m0, mode);
                if (by_row) {
                    pack32(w, up);
                    store_row(p.z, b_rows, m, p.N + n0, n_left, w);
                }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] *= up[j];
        }
        if (p.d || p.residual) {
            emit_d(staging, z, res, p, &maps.d, n0, m0, mode);
            if (p.d && by_row) {
                pack32(w, z);
                store_row(p.d, p.N, m, n0, n_left, w);
            }
        }
        if (c + 1 < COLS / 32) res.load(p, m0, t.row_end, n0 + 32);
        if (p.q) {
            uint4 codes[2];
            if (p.q_fmt == FP8_E4M3) codes32<0>(codes, z, qs);   // tested once, not a pair
            else codes32<1>(codes, z, qs);
            emit(staging, &maps.q, n0, m0, mode, [&](uint8_t* slot) {
                reinterpret_cast<uint4*>(slot + lane * 32)[0] = codes[0];
                reinterpret_cast<uint4*>(slot + lane * 32)[1] = codes[1];
            });
            if (by_row) {
                uint4* out = reinterpret_cast<uint4*>(p.q + m * p.N + n0);
                out[0] = codes[0];
                if (n_left > 16) out[1] = codes[1];
            }
            if (p.amax && live) {
#pragma unroll
                for (int j = 0; j < 32; j += 16) {   // n_left is a multiple of 16
                    if (j >= n_left) continue;
#pragma unroll
                    for (int e = 0; e < 16; ++e) top = row::max_abs(top, z[j + e]);
                }
            }
        }
    }
}

// ------------------------------------------------------------------ CTA-pair kernel

// A cluster of two CTAs per 256-row tile of 256 accumulator columns (gated:
// 128 output columns; the even CTA holds their gate rows of B and the odd
// one their up rows, which is how cta_group::2 splits B).  Roles and
// barriers as in gemm.cu's pair kernel.
constexpr int kPairStages = 5, kPairSlots = 3;
constexpr int kHalf = 128;
constexpr int kPairTile = 256;
constexpr int kPairStageBytes = 2 * kHalf * BK;
constexpr int kPairSmem = kPairStages * kPairStageBytes + kEpiWarps * kPairSlots * kSlotBytes + 256 +
                          static_cast<int>(sizeof(Units)) + 1024;

template <bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_act_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ OutMaps maps, const __grid_constant__ ActParams p) {
    constexpr int TN = GATED ? kHalf : kPairTile;   // output columns of a tile
    constexpr uint32_t TMEM_COLS = 2 * kPairTile;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* slots = ring + kPairStages * kPairStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(slots + kEpiWarps * kPairSlots * kSlotBytes);
    uint64_t* empty = full + kPairStages;
    uint64_t* tfull = empty + kPairStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* done = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    Units* units = reinterpret_cast<Units*>(reinterpret_cast<uint8_t*>(full) + 256);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(&tfull[a], 1);
            ptx::mbar_init(&tempty[a], 2 * kEpiWarps);   // both CTAs' epilogue warps
        }
        ptx::mbar_init(done, 1);
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::tma_prefetch_desc(&tmA);
        ptx::tma_prefetch_desc(&tmB);
    }
    if (warp == 2) {
        ptx::tmem_alloc_pair(tmem_slot, TMEM_COLS);
        ptx::tmem_relinquish_pair();
    }
    ptx::griddep_wait();
    // only now: a remainder's launch does not wait for this one before it reads
    ptx::griddep_launch_dependents();
    make_units(units, p, kPairTile);
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int num_units = units->first[p.experts];
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int u = pair; ok && u < num_units; u += npairs) {
                const Tile t = tile_of(u, units, p, kPairTile);
                const int ya = t.row0 + static_cast<int>(rank) * kHalf;
                const int64_t yb64 =
                    GATED ? (2 * static_cast<int64_t>(t.expert) + rank) * p.N + t.n_blk * TN
                          : t.expert * p.N + t.n_blk * TN + rank * kHalf;
                const int yb = static_cast<int>(yb64);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!ptx::mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) { ok = false; break; }
                    uint8_t* sa = ring + stage * kPairStageBytes;
                    const uint32_t bar = ptx::cluster_addr(&full[stage], 0);
                    if (leader) ptx::mbar_arrive_expect_tx(&full[stage], 2 * kPairStageBytes);
                    ptx::tma_load_2d_pair(sa, &tmA, bar, kb * BK, ya);
                    ptx::tma_load_2d_pair(sa + kHalf * BK, &tmB, bar, kb * BK, yb);
                    ++issued;
                    if (++stage == kPairStages) { stage = 0; phase ^= 1u; }
                }
            }
            uint32_t never = 0;
            if (leader) {
                // drain: the last copies into each slot (both CTAs' bytes) have landed
                for (int s = 0; s < kPairStages; ++s) {
                    if (issued <= s && issued < kPairStages) break;
                    const uint32_t par = (static_cast<uint32_t>(s) < stage) ? phase : (phase ^ 1u);
                    ptx::mbar_wait(&full[s], par, &never);
                }
            } else if (!ok) {
                // copies signal the peer's barriers: after an abort, give those in
                // flight a bounded time to land before this CTA moves on
                const uint64_t t0 = ptx::globaltimer();
                while (ptx::globaltimer() - t0 < 1000000ull) {
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            const uint32_t idesc = ptx::idesc_f8f6f4(p.fa, p.fb, kPairTile, kPairTile);
            const uint64_t tmpl = ptx::sdesc_kmajor_sw128(0);
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            bool ok = true;
            for (int u = pair; ok && u < num_units; u += npairs) {
                if (!ptx::mbar_wait(&tempty[acc], acc_phase ^ 1u, abort_flag)) break;
                ptx::tc_fence_after();
                const uint32_t d = tmem_base + acc * kPairTile;
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!ptx::mbar_wait(&full[stage], phase, abort_flag)) { ok = false; break; }
                    ptx::tc_fence_after();
                    uint8_t* sa = ring + stage * kPairStageBytes;
                    const uint64_t ad = tmpl | ((ptx::smem_u32(sa) & 0x3FFFFu) >> 4);
                    const uint64_t bd = tmpl | ((ptx::smem_u32(sa + kHalf * BK) & 0x3FFFFu) >> 4);
#pragma unroll
                    for (int k = 0; k < BK / UMMA_K; ++k)
                        ptx::mma_f8f6f4_pair(d, ad + k * (UMMA_K >> 4), bd + k * (UMMA_K >> 4), idesc,
                                             (kb | k) != 0);
                    ptx::mma_commit_pair(&empty[stage], 0x3);
                    if (++stage == kPairStages) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                ptx::mma_commit_pair(&tfull[acc], 0x3);
                acc ^= 1u;
                if (acc == 0) acc_phase ^= 1u;
            }
            uint32_t never = 0;
            ptx::mma_commit_pair(done, 0x1);
            ptx::mbar_wait(done, 0, &never);
        }
    } else if (warp >= 4) {
        const int qd = warp & 3, side = (warp - 4) >> 2;   // TMEM lanes, half of the columns
        Staging<kPairSlots> staging{slots + (warp - 4) * kPairSlots * kSlotBytes};
        Residual res;
        uint32_t acc = 0, acc_phase = 0;
        float top = 0.0f;
        for (int u = pair; u < num_units; u += npairs) {
            const Tile t = tile_of(u, units, p, kPairTile);
            const int64_t m0 = t.row0 + rank * kHalf + qd * 32;
            const int64_t n0 = static_cast<int64_t>(t.n_blk) * TN + side * (TN / 2);
            res.load(p, m0, t.row_end, n0);
            bool ok = (lane == 0) ? ptx::mbar_wait(&tfull[acc], acc_phase, abort_flag) : false;
            ok = __shfl_sync(row::kAll, ok, 0);
            if (!ok) break;
            __syncwarp();
            ptx::tc_fence_after();
            const uint32_t tcol = tmem_base + (static_cast<uint32_t>(qd * 32) << 16) +
                                  acc * kPairTile + side * (TN / 2);
            epilogue<GATED, kHalf, TN / 2>(staging, res, tcol, t, m0, n0, p, maps, top);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_cluster_relaxed(ptx::cluster_addr(&tempty[acc], 0));
            acc ^= 1u;
            if (acc == 0) acc_phase ^= 1u;
        }
        if (lane == 0) ptx::bulk_wait_group_all();   // every TMA store has completed
        const uint32_t bits = __reduce_max_sync(row::kAll, row::abs_bits(top));
        if (p.amax && lane == 0) row::raise_amax(p.amax, bits);
        __syncwarp();
    }

    ptx::tc_fence_before();
    ptx::cluster_sync();   // the pair's MMAs, copies and remote arrivals are all done
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag && p.status) atomicOr(p.status, 1u);
}

// ------------------------------------------------------------------ single-CTA kernel

// 128 rows by BN accumulator columns (gated: BN / 2 of the gate's product and
// BN / 2 of the up product).  For problems whose tiles fit the SMs at once,
// where a tile's own latency is the cost (BN 64 or 128), and for experts with
// few rows each, where 256-row tiles would multiply too many absent rows.
template <int BN>
struct TileLayout {
    static constexpr int STAGES = BN == 256 ? 4 : BN == 128 ? 5 : 6;
    static constexpr int SLOTS = BN == 256 ? 1 : 3;

    static constexpr int A_BYTES = kHalf * BK, B_BYTES = BN * BK;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int SMEM = STAGES * STAGE_BYTES + kEpiWarps * SLOTS * kSlotBytes + 256 +
                                static_cast<int>(sizeof(Units)) + 1024;
};

template <int BN, bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_act_tile_kernel(const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ OutMaps maps, const __grid_constant__ ActParams p) {
    ptx::griddep_launch_dependents();
    using L = TileLayout<BN>;
    constexpr int STAGES = L::STAGES, SLOTS = L::SLOTS;
    constexpr int TN = GATED ? BN / 2 : BN;           // output columns of a tile
    constexpr int COLS = TN >= 64 ? TN / 2 : 32;      // of an epilogue warp
    constexpr int SIDES = TN / COLS;
    constexpr uint32_t TMEM_COLS = 2 * BN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* slots = ring + STAGES * L::STAGE_BYTES;
    uint64_t* full = reinterpret_cast<uint64_t*>(slots + kEpiWarps * SLOTS * kSlotBytes);
    uint64_t* empty = full + STAGES;
    uint64_t* tfull = empty + STAGES;
    uint64_t* tempty = tfull + 2;
    uint64_t* done = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    Units* units = reinterpret_cast<Units*>(reinterpret_cast<uint8_t*>(full) + 256);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(&tfull[a], 1);
            ptx::mbar_init(&tempty[a], 4 * SIDES);
        }
        ptx::mbar_init(done, 1);
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::tma_prefetch_desc(&tmA);
        ptx::tma_prefetch_desc(&tmB);
    }
    if (warp == 2) {
        ptx::tmem_alloc(tmem_slot, TMEM_COLS);
        ptx::tmem_relinquish();
    }
    // A remainder's launch runs beside the whole blocks' launch: that one's CTAs
    // have all waited for what came before, and the two write different rows.
    // It waits at its end, so that what follows it follows both.
    if (p.part != kRemainder) ptx::griddep_wait();
    ptx::tc_fence_before();
    make_units(units, p, kHalf);   // its barriers also cover the set-up above
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int num_units = units->first[p.experts];

    if (warp == 0) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int u = blockIdx.x; ok && u < num_units; u += gridDim.x) {
                const Tile t = tile_of(u, units, p, kHalf);
                const int64_t yb64 = static_cast<int64_t>(t.expert) * (GATED ? 2 : 1) * p.N + t.n_blk * TN;
                const int yb = static_cast<int>(yb64), yu = static_cast<int>(yb64 + p.N);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!ptx::mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) { ok = false; break; }
                    uint8_t* sa = ring + stage * L::STAGE_BYTES;
                    ptx::mbar_arrive_expect_tx(&full[stage], L::STAGE_BYTES);
                    ptx::tma_load_2d(sa, &tmA, &full[stage], kb * BK, t.row0);
                    ptx::tma_load_2d(sa + L::A_BYTES, &tmB, &full[stage], kb * BK, yb);
                    if constexpr (GATED)
                        ptx::tma_load_2d(sa + L::A_BYTES + L::B_BYTES / 2, &tmB, &full[stage], kb * BK, yu);
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            // drain: the last copies into each slot have landed
            uint32_t never = 0;
            for (int s = 0; s < STAGES; ++s) {
                if (issued <= s && issued < STAGES) break;
                const uint32_t par = (static_cast<uint32_t>(s) < stage) ? phase : (phase ^ 1u);
                ptx::mbar_wait(&full[s], par, &never);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = ptx::idesc_f8f6f4(p.fa, p.fb, kHalf, BN);
            const uint64_t tmpl = ptx::sdesc_kmajor_sw128(0);
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            bool ok = true;
            for (int u = blockIdx.x; ok && u < num_units; u += gridDim.x) {
                if (!ptx::mbar_wait(&tempty[acc], acc_phase ^ 1u, abort_flag)) break;
                ptx::tc_fence_after();
                const uint32_t d = tmem_base + acc * BN;
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!ptx::mbar_wait(&full[stage], phase, abort_flag)) { ok = false; break; }
                    ptx::tc_fence_after();
                    uint8_t* sa = ring + stage * L::STAGE_BYTES;
                    const uint64_t ad = tmpl | ((ptx::smem_u32(sa) & 0x3FFFFu) >> 4);
                    const uint64_t bd = tmpl | ((ptx::smem_u32(sa + L::A_BYTES) & 0x3FFFFu) >> 4);
#pragma unroll
                    for (int k = 0; k < BK / UMMA_K; ++k)
                        ptx::mma_f8f6f4(d, ad + k * (UMMA_K >> 4), bd + k * (UMMA_K >> 4), idesc,
                                        (kb | k) != 0);
                    ptx::mma_commit(&empty[stage]);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                ptx::mma_commit(&tfull[acc]);
                acc ^= 1u;
                if (acc == 0) acc_phase ^= 1u;
            }
            // every MMA issued by this thread must finish before TMEM is released
            uint32_t never = 0;
            ptx::mma_commit(done);
            ptx::mbar_wait(done, 0, &never);
        }
    } else if (warp >= 4 && (warp - 4) >> 2 < SIDES) {
        const int qd = warp & 3, side = (warp - 4) >> 2;
        Staging<SLOTS> staging{slots + (warp - 4) * SLOTS * kSlotBytes};
        Residual res;
        uint32_t acc = 0, acc_phase = 0;
        float top = 0.0f;
        for (int u = blockIdx.x; u < num_units; u += gridDim.x) {
            const Tile t = tile_of(u, units, p, kHalf);
            const int64_t m0 = t.row0 + qd * 32;
            const int64_t n0 = static_cast<int64_t>(t.n_blk) * TN + side * COLS;
            res.load(p, m0, t.row_end, n0);
            bool ok = (lane == 0) ? ptx::mbar_wait(&tfull[acc], acc_phase, abort_flag) : false;
            ok = __shfl_sync(row::kAll, ok, 0);
            if (!ok) break;
            __syncwarp();
            ptx::tc_fence_after();
            const uint32_t tcol = tmem_base + (static_cast<uint32_t>(qd * 32) << 16) + acc * BN + side * COLS;
            epilogue<GATED, BN / 2, COLS>(staging, res, tcol, t, m0, n0, p, maps, top);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&tempty[acc]);
            acc ^= 1u;
            if (acc == 0) acc_phase ^= 1u;
        }
        if (lane == 0) ptx::bulk_wait_group_all();   // every TMA store has completed
        const uint32_t bits = __reduce_max_sync(row::kAll, row::abs_bits(top));
        if (p.amax && lane == 0) row::raise_amax(p.amax, bits);
        __syncwarp();
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem_base, TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag && p.status) atomicOr(p.status, 1u);
    if (p.part == kRemainder) ptx::griddep_wait();
}

// ------------------------------------------------------------------ gradient of the epilogue

constexpr int kBwdRows = 64;   // rows a CTA: 8 warps, 8 rows each

struct ActBwd {
    const __nv_bfloat16* d;
    const __nv_bfloat16* z;
    __nv_bfloat16* dz;
    uint8_t* q;
    const float* q_scale;
    float* amax;
    float* part;      // [row blocks][N or 2N] partial column sums (BIAS)
    int64_t M, N;
    int64_t col_blocks;
    int q_fmt;
    const int32_t* offsets;   // EXPERTS: row blocks are cut within an expert's rows
    int experts;
    int32_t* first;           // EXPERTS and BIAS: [experts + 1] each expert's first row block, written here
};

// Elementwise, HBM-bound: D's gradient and z are read once, dz is written
// once, 256 columns a warp.  The pairs' packed instructions keep it off the
// issue limit: 8192 x 11008 gated to codes 111 us (6.5 TB/s; 138 with scalar
// ones).  BIAS: column sums stay in registers over the CTA's rows.  EXPERTS:
// only rows of the experts; a CTA's rows belong to one of them, and CTAs past
// the experts' row blocks have nothing to do.
template <int ACT, bool GATED, bool BIAS, bool EXPERTS>
__global__ void __launch_bounds__(256) act_bwd_kernel(const __grid_constant__ ActBwd p) {
    ptx::griddep_launch_dependents();
    __shared__ float sums[BIAS ? 8 : 1][256];
    ptx::griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t block_row = blockIdx.x / p.col_blocks;
    const int64_t c0 = (blockIdx.x - block_row * p.col_blocks) * 256, c = c0 + lane * 8;
    int64_t row0 = block_row * kBwdRows, row_end = p.M;
    if constexpr (EXPERTS) {
        __shared__ Units units;
        make_units(&units, static_cast<int>(p.M), p.offsets, p.experts, 1, kAllRows, kBwdRows);
        if (BIAS && blockIdx.x == 0)
            for (int e = threadIdx.x; e <= p.experts; e += 256) p.first[e] = units.first[e];
        if (block_row >= units.first[p.experts]) return;
        const int e = expert_of(static_cast<int>(block_row), &units, p.experts);
        row0 = units.begin[e] + (block_row - units.first[e]) * kBwdRows;
        row_end = units.end[e];
    }
    const int64_t width = GATED ? 2 * p.N : p.N;
    const bool on = c < p.N;   // N is a multiple of 16
    const f2 qs = row::all2(p.q ? p.q_scale[0] : 0.0f);
    f2 s0[4] = {}, s1[4] = {};
    float top = 0.0f;
    auto put = [&](const f2 (&v)[4], int64_t at) {
        if (p.dz) row::store_pairs(p.dz + at, v);
        if (p.q) {
            uint32_t code[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f2 t = row::mul2(v[e], qs);
                code[e] = row::cvt_pair(p.q_fmt, row::lo2(t), row::hi2(t));
                top = row::max_abs(row::max_abs(top, row::lo2(v[e])), row::hi2(v[e]));
            }
            *reinterpret_cast<uint2*>(p.q + at) = make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
        }
    };
    if (on) {
        const int64_t m0 = row0 + warp;
        // one row at a time: many warps hide its loads (116 us a pass with four
        // rows' loads in flight, 117 with one, 131 with two)
#pragma unroll 1
        for (int i = 0; i < kBwdRows / 8; ++i) {
            const int64_t m = m0 + i * 8;
            if (m >= row_end) break;
            row::Raw8<__nv_bfloat16> rd, rz, ru;
            rd.load(p.d + m * p.N + c);
            rz.load(p.z + m * width + c);
            if constexpr (GATED) ru.load(p.z + m * width + p.N + c);
            f2 d[4], z[4], u[4];
            rd.pairs(d);
            rz.pairs(z);
            if constexpr (GATED) ru.pairs(u);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f2 a, g;
                act_and_grad2<ACT>(z[e], a, g);
                if constexpr (GATED) {
                    z[e] = row::mul2(row::mul2(d[e], u[e]), g);
                    u[e] = row::mul2(d[e], a);
                    if constexpr (BIAS) s1[e] = row::add2(s1[e], u[e]);
                } else {
                    z[e] = row::mul2(d[e], g);
                }
                if constexpr (BIAS) s0[e] = row::add2(s0[e], z[e]);
            }
            put(z, m * width + c);
            if constexpr (GATED) put(u, m * width + p.N + c);
        }
    }
    if constexpr (BIAS) {
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sums[warp][lane * 8 + 2 * e] = row::lo2(h ? s1[e] : s0[e]);
                sums[warp][lane * 8 + 2 * e + 1] = row::hi2(h ? s1[e] : s0[e]);
            }
            __syncthreads();
            if (c0 + threadIdx.x < p.N) {
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < 8; ++w) s += sums[w][threadIdx.x];
                p.part[block_row * width + h * p.N + c0 + threadIdx.x] = s;
            }
        }
    }
    if (p.amax) {
        const uint32_t bits = __reduce_max_sync(row::kAll, row::abs_bits(top));
        if (lane == 0) row::raise_amax(p.amax, bits);
    }
}

// dbias[e][c] (+)= the sum of expert e's row blocks' partial sums: eight slices
// of the blocks first, then the slices, in a fixed order.  Four columns a
// thread: with many experts of few rows the CTAs' number is the cost (8192 x 2048
// gated, 256 experts, gradient and sums 44 us, 69 with one column a thread).
constexpr int kBiasCols = 128;   // a CTA

__global__ void __launch_bounds__(256)
    expert_bias_kernel(const float* part, const int32_t* first, int64_t width, float* dbias, int accumulate) {
    ptx::griddep_launch_dependents();
    __shared__ __align__(16) float sums[8][kBiasCols];
    ptx::griddep_wait();
    const int e = blockIdx.y, slice = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kBiasCols, c = c0 + 4 * lane;
    const int end = first[e + 1];
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < width) {   // a multiple of 16
#pragma unroll 4
        for (int i = first[e] + slice; i < end; i += 8) {
            const float4 v = *reinterpret_cast<const float4*>(part + i * width + c);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
    }
    *reinterpret_cast<float4*>(&sums[slice][4 * lane]) = s;
    __syncthreads();
    if (threadIdx.x < kBiasCols && c0 + threadIdx.x < width) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += sums[i][threadIdx.x];
        float* out = dbias + e * width + c0 + threadIdx.x;
        *out = accumulate ? *out + t : t;
    }
}

template <int ACT, bool EXPERTS>
void launch_act_bwd(const ActBwd& p, bool gated, unsigned ctas, cudaStream_t st) {
    if (gated) {
        if (p.part) launch_pdl(act_bwd_kernel<ACT, true, true, EXPERTS>, dim3(ctas), dim3(256), 0, st, p);
        else launch_pdl(act_bwd_kernel<ACT, true, false, EXPERTS>, dim3(ctas), dim3(256), 0, st, p);
    } else {
        if (p.part) launch_pdl(act_bwd_kernel<ACT, false, true, EXPERTS>, dim3(ctas), dim3(256), 0, st, p);
        else launch_pdl(act_bwd_kernel<ACT, false, false, EXPERTS>, dim3(ctas), dim3(256), 0, st, p);
    }
}

template <int ACT>
void launch_act_bwd(const ActBwd& p, bool gated, unsigned ctas, cudaStream_t st) {
    if (p.offsets) launch_act_bwd<ACT, true>(p, gated, ctas, st);
    else launch_act_bwd<ACT, false>(p, gated, ctas, st);
}

// ------------------------------------------------------------------ host side


// The kernel's dynamic shared memory allowed once per device, and how many of
// its clusters (or CTAs) run at once.
template <typename Kernel>
int kernel_slots(Kernel k, int id, int smem, int cluster, int* out) {
    static std::mutex mu;
    static int cache[64][8] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
    int uncached = 0;
    std::lock_guard<std::mutex> lock(mu);
    int& c = dev >= 0 && dev < 64 ? cache[dev][id] : uncached;
    if (c == 0) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return set_error(FP8_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        int n = num_sms() / cluster;
        if (cluster > 1) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2 * 1024);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = smem;
            int got = 0;
            if (cudaOccupancyMaxActiveClusters(&got, k, &cfg) == cudaSuccess && got > 0) n = got;
            else (void)cudaGetLastError();
        }
        c = n;
    }
    *out = c;
    return FP8_OK;
}

// Raster group: the group's A panels (256 rows by K bytes each) stay in L2
// beside the B panels in flight, as in gemm.cu.
int raster_group(int64_t K) {
    int g = 16;
    while (g > 4 && g * 256 * K > (int64_t{64} << 20)) g >>= 1;
    return g;
}

// At most this many blocks of `rows` rows, however the experts' rows are cut.
int64_t most_blocks(int64_t M, int rows, int experts) { return (M + rows - 1) / rows + experts - 1; }

// The same for tiles of `rows` rows and `cols` output columns.
int64_t most_tiles(const fp8_gemm_act_args_t* a, int rows, int cols) {
    return most_blocks(a->M, rows, a->experts) * ((a->N + cols - 1) / cols);
}

template <bool GATED>
int launch_pair(const fp8_gemm_act_args_t* a, ActParams& p, const OutMaps& maps, cudaStream_t st) {
    constexpr int TN = GATED ? kHalf : kPairTile;
    const int64_t b_rows = GATED ? 2 * a->N : a->N;
    CUtensorMap tmA, tmB;
    int r = make_kmajor_map(&tmA, a->A, a->M, a->K, kHalf);
    if (r == FP8_OK) r = make_kmajor_map(&tmB, a->B, b_rows * a->experts, a->K, kHalf);
    int clusters = 0;
    auto k = gemm_act_pair_kernel<GATED>;
    if (r == FP8_OK) r = kernel_slots(k, GATED, kPairSmem, 2, &clusters);
    if (r != FP8_OK) return r;
    p.num_n = static_cast<int>((a->N + TN - 1) / TN);
    const int64_t tiles = most_tiles(a, kPairTile, TN);
    const unsigned grid = 2 * static_cast<unsigned>(tiles < clusters ? tiles : clusters);
    launch_pdl(k, dim3(grid), dim3(kThreads), kPairSmem, st, tmA, tmB, maps, p);
    return host::launch_status("fp8_gemm_act");
}

template <int BN, bool GATED>
int launch_tile(const fp8_gemm_act_args_t* a, ActParams& p, const OutMaps& maps, cudaStream_t st) {
    constexpr int TN = GATED ? BN / 2 : BN, SMEM = TileLayout<BN>::SMEM;
    const int64_t b_rows = GATED ? 2 * a->N : a->N;
    CUtensorMap tmA, tmB;
    int r = make_kmajor_map(&tmA, a->A, a->M, a->K, kHalf);
    if (r == FP8_OK) r = make_kmajor_map(&tmB, a->B, b_rows * a->experts, a->K, TN);
    int ctas = 0;
    auto k = gemm_act_tile_kernel<BN, GATED>;
    constexpr int id = 2 + (BN == 64 ? 0 : BN == 128 ? 2 : 4) + GATED;
    if (r == FP8_OK) r = kernel_slots(k, id, SMEM, 1, &ctas);
    if (r != FP8_OK) return r;
    p.num_n = static_cast<int>((a->N + TN - 1) / TN);
    const int64_t tiles = p.part == kRemainder ? static_cast<int64_t>(a->experts) * p.num_n
                                               : most_tiles(a, kHalf, TN);
    const unsigned grid = static_cast<unsigned>(tiles < ctas ? tiles : ctas);
    launch_pdl(k, dim3(grid), dim3(kThreads), SMEM, st, tmA, tmB, maps, p);
    return host::launch_status("fp8_gemm_act");
}

template <bool GATED>
int launch_gemm_act(const fp8_gemm_act_args_t* a, ActParams& p, const OutMaps& maps, cudaStream_t st) {
    // The tile shape that finishes first: rounds over the SMs times a tile's
    // time, in units of a 128 x 256 tile's.  A CTA pair's 256 x 256 tile takes
    // 0.92 of it (half the B bytes an SM): 1177 against 1270 us for a gated
    // 4096 x 28672 x 8192 product; but its rows come in 256s, and a product of
    // 4099 x 8192 x 28672 takes 692 us in pairs and 640 us in 128 rows.  128 x 128
    // takes 0.67 and 128 x 64 0.60 (the A bytes are the same): 547 and 983 us
    // against 406 for gated products of 16384 x 4096 x 4096 over 16 experts, but
    // 8.9 and 6.8 us against 11.6 for 256 x 512 x 512.  An expert's last tile
    // is taken as half full, with no whole rounds.
    const int sms = num_sms();
    auto cost = [&](int rows, int acc_cols, int slots, double time) {
        const int64_t cols = GATED ? acc_cols / 2 : acc_cols;
        const double n = static_cast<double>((a->N + cols - 1) / cols);
        if (a->offsets)
            return (static_cast<double>(a->M) / rows + 0.5 * a->experts) * n / slots * time;
        const int64_t tiles = most_tiles(a, rows, static_cast<int>(cols));
        return static_cast<double>((tiles + slots - 1) / slots) * time;
    };
    const double c64 = cost(kHalf, 64, sms, 0.60), c128 = cost(kHalf, 128, sms, 0.67);
    const double c256 = cost(kHalf, 256, sms, 1.0), pair = cost(kPairTile, kPairTile, sms / 2, 0.92);
    // one product's whole blocks in pairs, its remainder in 128 x 256 tiles
    // beside them (4099 x 8192 x 28672: 632 us, against 686 for 128 x 256 alone;
    // experts' remainders, launched so, were 6% slower than all in 128 x 256)
    double split = 1e30;
    const int64_t rest = a->M % kPairTile;
    if (!a->offsets && a->M > kPairTile && rest > 0 && rest <= kHalf) {
        const int64_t n = (a->N + (GATED ? 127 : 255)) / (GATED ? 128 : 256);
        const int64_t blocks = a->M / kPairTile * n, slots = sms / 2;
        const double rounds = static_cast<double>((blocks + slots - 1) / slots) * 0.92;
        const double even = (static_cast<double>(blocks) * 2 * 0.92 + static_cast<double>(n)) / sms;
        split = even > rounds ? even : rounds;
    }
    if (c64 <= c128 && c64 <= c256 && c64 <= pair && c64 <= split)
        return launch_tile<64, GATED>(a, p, maps, st);
    if (c128 <= c256 && c128 <= pair && c128 <= split) return launch_tile<128, GATED>(a, p, maps, st);
    if (split < c256 && split < pair) {
        p.part = kWholeBlocks;
        const int r = launch_pair<GATED>(a, p, maps, st);
        if (r != FP8_OK) return r;
        p.part = kRemainder;
        return launch_tile<256, GATED>(a, p, maps, st);
    }
    if (c256 < pair) return launch_tile<256, GATED>(a, p, maps, st);
    return launch_pair<GATED>(a, p, maps, st);
}

}  // namespace
}  // namespace fp8

using namespace fp8;
using namespace fp8::host;

extern "C" {

int fp8_gemm_act(const fp8_gemm_act_args_t* a, void* stream) {
    const char* what = "fp8_gemm_act";
    if (!a) return set_error(FP8_ERR_INVALID_ARG, "%s: args is NULL", what);
    if ((a->fa != FP8_E4M3 && a->fa != FP8_E5M2) || (a->fb != FP8_E4M3 && a->fb != FP8_E5M2) ||
        (a->q && a->q_format != FP8_E4M3 && a->q_format != FP8_E5M2))
        return set_error(FP8_ERR_INVALID_ARG, "%s: unknown FP8 format", what);
    for (int g : {a->ga & ~FP8_SCALE_POW2, a->gb & ~FP8_SCALE_POW2}) {
        if (g < FP8_GRAN_TENSOR || g > FP8_GRAN_ROW)
            return set_error(FP8_ERR_INVALID_ARG, "%s: unknown scale granularity", what);
        if (g != FP8_GRAN_TENSOR && g != FP8_GRAN_ROW)
            return set_error(FP8_ERR_UNSUPPORTED, "%s: built for per-tensor and per-row scales", what);
    }
    if ((a->ga | a->gb) & FP8_SCALE_POW2)
        return set_error(FP8_ERR_INVALID_ARG, "%s: FP8_SCALE_POW2 is for block scales", what);
    if (a->act < FP8_ACT_NONE || a->act > FP8_ACT_GELU_TANH)
        return set_error(FP8_ERR_INVALID_ARG, "%s: unknown activation %d", what, a->act);
    if (a->M < 0 || a->N < 16 || a->K < 16 || a->N % 16 || a->K % 16)
        return set_error(FP8_ERR_SHAPE, "%s: M must be >= 0, N and K positive multiples of 16", what);
    if (a->experts < 1 || a->experts > kMaxGemmExperts || (!a->offsets && a->experts != 1))
        return set_error(FP8_ERR_SHAPE, "%s: experts in 1..%d, 1 without offsets", what, kMaxGemmExperts);
    const int64_t b_rows = a->gated ? 2 * a->N : a->N;
    const int64_t limit = (int64_t{1} << 31) - 1024;   // coordinates and units are 32-bit
    if (a->M > limit || b_rows > limit / a->experts || a->K > limit ||
        (a->M / 128 + a->experts) * (a->N / 32 + 1) > limit)
        return set_error(FP8_ERR_SHAPE, "%s: dimensions out of range", what);
    if (!a->scale_inv_a || !a->scale_inv_b || !a->B || (!a->A && a->M))
        return set_error(FP8_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if (!a->d && !a->q && a->M) return set_error(FP8_ERR_INVALID_ARG, "%s: d and q are NULL", what);
    if (a->q ? !a->q_scale : (a->M && (a->q_scale || a->amax)))
        return set_error(FP8_ERR_INVALID_ARG, "%s: q and q_scale go together, amax with them", what);
    for (const void* t : {static_cast<const void*>(a->A), static_cast<const void*>(a->B), a->bias,
                          a->residual, static_cast<const void*>(a->z), static_cast<const void*>(a->d),
                          static_cast<const void*>(a->q)})
        if (!aligned(t, 16)) return set_error(FP8_ERR_ALIGN, "%s: tensors must be 16-byte aligned", what);
    for (const void* t : {static_cast<const void*>(a->scale_inv_a), static_cast<const void*>(a->scale_inv_b),
                          static_cast<const void*>(a->q_scale), static_cast<const void*>(a->amax),
                          static_cast<const void*>(a->offsets)})
        if (!aligned(t, 4)) return set_error(FP8_ERR_ALIGN, "%s: scales and offsets must be 4-byte aligned", what);
    cudaStream_t st = as_stream(stream);
    if (a->amax) launch_zero_words(a->amax, 1, st);
    if (a->M == 0) return launch_status(what);

    ActParams p{};
    p.M = a->M; p.N = a->N; p.K = a->K;
    p.num_kb = static_cast<int>((a->K + BK - 1) / BK);
    p.fa = a->fa; p.fb = a->fb; p.ga = a->ga; p.gb = a->gb;
    p.sa = a->scale_inv_a; p.sb = a->scale_inv_b;
    p.act = a->act;
    p.bias = static_cast<const __nv_bfloat16*>(a->bias);
    p.residual = static_cast<const __nv_bfloat16*>(a->residual);
    p.z = a->z; p.d = a->d; p.q = a->q;
    p.q_fmt = a->q_format; p.q_scale = a->q_scale; p.amax = a->amax;
    p.offsets = a->offsets; p.experts = a->experts;
    p.group = raster_group(a->K);
    p.status = device_status_word();
    OutMaps maps{};
    int r = FP8_OK;
    const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const auto sw = CU_TENSOR_MAP_SWIZZLE_64B;
    if (a->z) r = make_output_map(&maps.z, a->z, a->M, a->N, b_rows * 2, bf, 32, sw);
    if (r == FP8_OK && a->z && a->gated)
        r = make_output_map(&maps.z_up, static_cast<__nv_bfloat16*>(a->z) + a->N, a->M, a->N,
                            b_rows * 2, bf, 32, sw);
    if (r == FP8_OK && a->d) r = make_output_map(&maps.d, a->d, a->M, a->N, a->N * 2, bf, 32, sw);
    if (r == FP8_OK && a->q)
        r = make_output_map(&maps.q, a->q, a->M, a->N, a->N, CU_TENSOR_MAP_DATA_TYPE_UINT8, 32,
                            CU_TENSOR_MAP_SWIZZLE_NONE);
    if (r != FP8_OK) return r;
    return a->gated ? launch_gemm_act<true>(a, p, maps, st) : launch_gemm_act<false>(a, p, maps, st);
}

size_t fp8_act_bwd_workspace_size(int64_t M, int64_t N, int gated) {
    if (M < 0 || N < 16 || N % 16) return 0;
    return static_cast<size_t>(most_blocks(M, kBwdRows, 1)) * static_cast<size_t>(gated ? 2 * N : N) * 4;
}

size_t fp8_act_bwd_experts_workspace_size(int64_t M, int64_t N, int gated, int experts) {
    if (M < 1 || N < 16 || N % 16 || experts < 1 || experts > kMaxGemmExperts) return 0;
    return static_cast<size_t>(most_blocks(M, kBwdRows, experts)) * static_cast<size_t>(gated ? 2 * N : N) * 4 +
           static_cast<size_t>(experts + 1) * 4;
}

int fp8_act_bwd(const fp8_act_bwd_args_t* a, void* workspace, size_t workspace_bytes, void* stream) {
    const char* what = "fp8_act_bwd";
    if (!a) return set_error(FP8_ERR_INVALID_ARG, "%s: args is NULL", what);
    if (a->act < FP8_ACT_NONE || a->act > FP8_ACT_GELU_TANH)
        return set_error(FP8_ERR_INVALID_ARG, "%s: unknown activation %d", what, a->act);
    if (a->M < 0 || a->N < 16 || a->N % 16 || a->N > (int64_t{1} << 30))
        return set_error(FP8_ERR_SHAPE, "%s: M must be >= 0, N a positive multiple of 16", what);
    if (a->offsets && (a->experts < 1 || a->experts > kMaxGemmExperts))
        return set_error(FP8_ERR_SHAPE, "%s: experts in 1..%d", what, kMaxGemmExperts);
    const int64_t limit = a->offsets ? (int64_t{1} << 31) - 1024 : int64_t{1} << 31;   // offsets are 32-bit
    if (a->M > limit) return set_error(FP8_ERR_SHAPE, "%s: dimensions out of range", what);
    const int64_t col_blocks = (a->N + 255) / 256;
    const int64_t row_blocks = most_blocks(a->M, kBwdRows, a->offsets ? a->experts : 1);
    if (row_blocks * col_blocks >= (int64_t{1} << 31))
        return set_error(FP8_ERR_SHAPE, "%s: dimensions out of range", what);
    if ((!a->dD || !a->z) && a->M) return set_error(FP8_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if (!a->dz && !a->q && !a->dbias && a->M)
        return set_error(FP8_ERR_INVALID_ARG, "%s: no output", what);
    if (a->q && a->q_format != FP8_E4M3 && a->q_format != FP8_E5M2)
        return set_error(FP8_ERR_INVALID_ARG, "%s: unknown FP8 format", what);
    if (a->q ? !a->q_scale : (a->M && (a->q_scale || a->amax)))
        return set_error(FP8_ERR_INVALID_ARG, "%s: q and q_scale go together, amax with them", what);
    const size_t need = !a->dbias ? 0
                        : a->offsets ? fp8_act_bwd_experts_workspace_size(a->M, a->N, a->gated, a->experts)
                                     : fp8_act_bwd_workspace_size(a->M, a->N, a->gated);
    if (need && (!workspace || workspace_bytes < need))
        return set_error(FP8_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", what,
                         workspace ? workspace_bytes : size_t{0}, need);
    for (const void* t : {a->dD, a->z, static_cast<const void*>(a->dz), static_cast<const void*>(a->q),
                          static_cast<const void*>(need ? workspace : nullptr)})
        if (!aligned(t, 16))
            return set_error(FP8_ERR_ALIGN, "%s: tensors and workspace must be 16-byte aligned", what);
    for (const void* t : {static_cast<const void*>(a->q_scale), static_cast<const void*>(a->amax),
                          static_cast<const void*>(a->dbias), static_cast<const void*>(a->offsets)})
        if (!aligned(t, 4))
            return set_error(FP8_ERR_ALIGN, "%s: q_scale, amax, dbias and offsets must be 4-byte aligned", what);
    cudaStream_t st = as_stream(stream);
    const int64_t width = a->gated ? 2 * a->N : a->N;
    if (a->amax) launch_zero_words(a->amax, 1, st);
    if (a->M) {
        ActBwd p{};
        p.d = static_cast<const __nv_bfloat16*>(a->dD);
        p.z = static_cast<const __nv_bfloat16*>(a->z);
        p.dz = static_cast<__nv_bfloat16*>(a->dz);
        p.q = a->q; p.q_scale = a->q_scale; p.q_fmt = a->q_format; p.amax = a->amax;
        p.part = a->dbias ? static_cast<float*>(workspace) : nullptr;
        p.M = a->M; p.N = a->N; p.col_blocks = col_blocks;
        p.offsets = a->offsets; p.experts = a->experts;
        if (p.part && a->offsets) p.first = reinterpret_cast<int32_t*>(p.part + row_blocks * width);
        const unsigned ctas = static_cast<unsigned>(row_blocks * col_blocks);
        const bool gated = a->gated != 0;
        switch (a->act) {
            case FP8_ACT_RELU: launch_act_bwd<FP8_ACT_RELU>(p, gated, ctas, st); break;
            case FP8_ACT_SILU: launch_act_bwd<FP8_ACT_SILU>(p, gated, ctas, st); break;
            case FP8_ACT_GELU: launch_act_bwd<FP8_ACT_GELU>(p, gated, ctas, st); break;
            case FP8_ACT_GELU_TANH: launch_act_bwd<FP8_ACT_GELU_TANH>(p, gated, ctas, st); break;
            default: launch_act_bwd<FP8_ACT_NONE>(p, gated, ctas, st); break;
        }
    }
    if (a->dbias && !a->offsets) {
        launch_column_sums(static_cast<const float*>(workspace), row_blocks, width, a->dbias,
                           a->accumulate, st);
    } else if (a->dbias && a->M) {
        const float* part = static_cast<const float*>(workspace);
        launch_pdl(expert_bias_kernel, dim3(static_cast<unsigned>((width + kBiasCols - 1) / kBiasCols), a->experts),
                   dim3(256), 0, st, part, reinterpret_cast<const int32_t*>(part + row_blocks * width), width, a->dbias,
                   a->accumulate != 0 ? 1 : 0);
    } else if (a->dbias && !a->accumulate) {   // no rows: zeros
        const cudaError_t e = cudaMemsetAsync(a->dbias, 0, static_cast<size_t>(a->experts) * width * 4, st);
        if (e != cudaSuccess) return set_error(FP8_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    }
    return launch_status(what);
}

}  // extern "C"

// act_block.cu -- the activation between two products in blocks of 128, with an
// 8-bit checkpoint for the backward pass, its gradient from the checkpoint, and
// the transposing re-cast of a kept input.
//
//   h = act(z_g) z_u,  q = codes of h,  z_q = codes of z        (1x128 blocks)
//   dz_g = dD z_u act'(z_g),  dz_u = dD act(z_g)                (from z_q)
//
// By rows (codes of rows only), eight lanes take a row's 128-column block, sixteen
// columns a lane: fewest instructions an element.  By tiles of 128 x 128 (codes
// along the tokens as well), a warp takes rows, four columns a lane: a row's
// maximum is one warp reduction, and a column's stays in the lane's registers
// over the rows.  Values are FP32 between the inputs and the one rounding of
// each code.
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
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

constexpr int kWarps = 8;        // of the kernels that go by rows
constexpr int kThreads = kWarps * 32;
constexpr int kTileWarps = 16;   // of the kernels that go by 128 x 128 tiles
constexpr int kTileThreads = kTileWarps * 32;
constexpr int kTileRows = 128 / kTileWarps;

// ------------------------------------------------------------------ four columns of a row

// Four elements as two pairs.
struct Quad {
    f2 v[2];
    __device__ __forceinline__ float at(int i) const { return i & 1 ? row::hi2(v[i >> 1]) : row::lo2(v[i >> 1]); }
};

__device__ __forceinline__ Quad zero4() { return Quad{{0ull, 0ull}}; }

// Four codes times a factor.
__device__ __forceinline__ Quad decode4(int fmt, uint32_t w, float inv) {
    Quad q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)),
                                                         fmt == 0 ? __NV_E4M3 : __NV_E5M2);
        const float2 f = __half22float2(__half2(h));
        q.v[i] = row::mul2(row::mk2(f.x, f.y), row::all2(inv));
    }
    return q;
}

__device__ __forceinline__ Quad from_bf16(uint2 w) { return Quad{{row::bf2(w.x), row::bf2(w.y)}}; }

// The four codes of q * s, the first in the low byte.
template <int FMT>
__device__ __forceinline__ uint32_t code4(const Quad& q, f2 s0, f2 s1) {
    const f2 a = row::mul2(q.v[0], s0), b = row::mul2(q.v[1], s1);
    return row::cvt_pair<FMT>(row::lo2(a), row::hi2(a)) | (row::cvt_pair<FMT>(row::lo2(b), row::hi2(b)) << 16);
}

// f(std::integral_constant<int, fmt>): the format is tested once, not at every code.
template <typename F>
__device__ __forceinline__ void by_format(int fmt, F f) {
    if (fmt == FP8_E4M3) f(std::integral_constant<int, FP8_E4M3>());
    else f(std::integral_constant<int, FP8_E5M2>());
}

// The largest magnitude of a row's 128 columns, in every lane: the bits of an
// fp32 order like its magnitude, NaN above all.
__device__ __forceinline__ uint32_t row_top(const Quad& q) {
    float m = row::max_abs(row::max_abs(0.0f, q.at(0)), q.at(1));
    m = row::max_abs(row::max_abs(m, q.at(2)), q.at(3));
    return __reduce_max_sync(row::kAll, row::abs_bits(m));
}

__device__ __forceinline__ void raise4(float (&top)[4], const Quad& q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) top[i] = row::max_abs(top[i], q.at(i));
}

__device__ __forceinline__ uint2 ld8(const void* p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld4(const void* p) {
    uint32_t v;
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// The experts' rows: begin .. end.  Every thread; ends with a barrier.  The kernels
// by rows pay for it in every CTA, those of rows without an expert too: 32768 x 2048
// gated with checkpoint 84 us without offsets, 92 with 32 experts' and 111 with 256
// experts' in a buffer of 65536 rows; the gradient's row codes 79, 88 and 106.  By tiles, a
// CTA an SM, it is level (160).
__device__ __forceinline__ int2 rows_of(const int32_t* offsets, int experts, int64_t M) {
    const int most = static_cast<int>(M);
    if (!offsets) return make_int2(0, most);
    __shared__ int ends[2];
    if (threadIdx.x < 32) {
        int end = 0;
        for (int i = threadIdx.x; i <= experts; i += 32) end = max(end, min(max(offsets[i], 0), most));
        end = __reduce_max_sync(row::kAll, end);
        if (threadIdx.x == 0) {
            ends[0] = min(max(offsets[0], 0), most);
            ends[1] = end;
        }
    }
    __syncthreads();
    return make_int2(ends[0], ends[1]);
}

// Row group (or tile row) and column block of a unit of work; units are fewer
// than 2^31, and 64-bit divisions would take as long as ten elements' work.
struct Place {
    uint32_t row;
    int blk;
};
__device__ __forceinline__ Place place(uint32_t unit, int blocks) {
    const uint32_t r = unit / static_cast<uint32_t>(blocks);
    return Place{r, static_cast<int>(unit - r * static_cast<uint32_t>(blocks))};
}

// ------------------------------------------------------------------ forward

struct ActBlock {
    const __nv_bfloat16* z;
    uint8_t* q;
    float* inv;
    uint8_t* zq;
    float* z_inv;
    int64_t M;
    int blocks;       // N / 128
    int fmt, pow2;
    const int32_t* offsets;
    int experts;
};

// A lane's sixteen columns of a row: eight from 8 (lane % 8) and eight 64 further.
struct Raw16 {
    uint4 w[2];
};

__device__ __forceinline__ uint4 ld16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void bf16_pairs(f2 (&v)[4], const uint4& w) {
    v[0] = row::bf2(w.x); v[1] = row::bf2(w.y); v[2] = row::bf2(w.z); v[3] = row::bf2(w.w);
}

// The largest magnitudes of a lane's sixteen bf16 in the low half of the word
// (the bits of a bf16 order like its magnitude, NaN above all).
__device__ __forceinline__ uint32_t top16(const Raw16& r) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        m = __vmaxu2(m, __vmaxu2(r.w[k].x & 0x7FFF7FFFu, r.w[k].y & 0x7FFF7FFFu));
        m = __vmaxu2(m, __vmaxu2(r.w[k].z & 0x7FFF7FFFu, r.w[k].w & 0x7FFF7FFFu));
    }
    return max(m >> 16, m & 0xFFFFu);
}

__device__ __forceinline__ uint32_t top16(const f2 (&v)[2][4]) {
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = row::max_abs(row::max_abs(m, row::lo2(v[k][i])), row::hi2(v[k][i]));
    return row::abs_bits(m);
}

// The largest over eight lanes, of a word or of its two halves.
__device__ __forceinline__ uint32_t eight_max(uint32_t m) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(row::kAll, m, o));
    return m;
}
__device__ __forceinline__ uint32_t eight_max2(uint32_t m) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(row::kAll, m, o));
    return m;
}

// Writes the codes of a lane's sixteen columns, v * s.
__device__ __forceinline__ void put16(uint8_t* to, int fmt, const f2 (&v)[2][4], float s) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
        *reinterpret_cast<uint2*>(to + 64 * k) =
            fmt == 0 ? row::cvt8<0>(v[k], row::all2(s)) : row::cvt8<1>(v[k], row::all2(s));
}

// Four rows of one 128-column block of h a warp.  The first lanes of a row's
// eight have the scales of its h, gate and up.  32768 x 2048 gated (SiLU) with the
// checkpoint: 83 us for 476 MB, 0.85 of the copy rate; a warp a row with four columns a lane
// spent twice the instructions on maxima and scales (144 us).  64 x 2048: 2 us,
// and the call around it 20.
template <int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads, 4) act_block_kernel(const __grid_constant__ ActBlock p) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int2 rows = rows_of(p.offsets, p.experts, p.M);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7;
    const Place at = place(blockIdx.x * kWarps + warp, p.blocks);
    const int64_t base = rows.x + static_cast<int64_t>(at.row) * 4, r = base + (lane >> 3);
    if (base >= rows.y) return;
    const int64_t N = static_cast<int64_t>(p.blocks) * 128, W = GATED ? 2 * N : N;
    const int wb = GATED ? 2 * p.blocks : p.blocks;   // factors a row of z
    const int c = at.blk * 128 + sub * 8;
    const bool on = r < rows.y;
    Raw16 g = {}, u = {};
    if (on) {
        const __nv_bfloat16* z = p.z + r * W + c;
        g.w[0] = ld16(z);
        g.w[1] = ld16(z + 64);
        if (GATED) {
            u.w[0] = ld16(z + N);
            u.w[1] = ld16(z + N + 64);
        }
    }
    f2 a[2][4], b[2][4], h[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        bf16_pairs(a[k], g.w[k]);
        if (GATED) bf16_pairs(b[k], u.w[k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[k][j] = act2<ACT>(a[k][j]);
            if (GATED) h[k][j] = row::mul2(h[k][j], b[k][j]);
        }
    }
    uint32_t mine = eight_max(top16(h));
    if (p.zq) {
        uint32_t m = top16(g);
        if (GATED) m |= top16(u) << 16;
        m = eight_max2(m);
        if (sub == 1) mine = m << 16;
        if (GATED && sub == 2) mine = m & 0xFFFF0000u;
    }
    const float s = row::block_scale(mine, sub == 0 ? p.fmt : FP8_E4M3, p.pow2);
    if (on && sub < 3) {
        const float f = __fdiv_rn(1.0f, s);
        if (sub == 0 && p.q) p.inv[r * p.blocks + at.blk] = f;
        if (sub == 1 && p.zq) p.z_inv[r * wb + at.blk] = f;
        if (GATED && sub == 2 && p.zq) p.z_inv[r * wb + p.blocks + at.blk] = f;
    }
    const int from = lane & 24;
    const float sh = __shfl_sync(row::kAll, s, from), sg = __shfl_sync(row::kAll, s, from + 1);
    const float su = __shfl_sync(row::kAll, s, from + 2);
    if (!on) return;
    if (p.q) put16(p.q + r * N + c, p.fmt, h, sh);
    if (p.zq) {
        put16(p.zq + r * W + c, FP8_E4M3, a, sg);
        if (GATED) put16(p.zq + r * W + N + c, FP8_E4M3, b, su);
    }
}

// ------------------------------------------------------------------ transposed codes of a 128 x 128 tile

// The codes of a lane's four columns over the warp's 8 rows: word r holds the
// columns of row r on the way in, word 2 c + k rows 4 k .. 4 k + 3 of column c
// on the way out.
__device__ __forceinline__ void turn8(uint32_t (&w)[kTileRows]) {
    uint32_t o[kTileRows];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t a = w[4 * k], b = w[4 * k + 1], c = w[4 * k + 2], d = w[4 * k + 3];
        const uint32_t ab = __byte_perm(a, b, 0x5140), cd = __byte_perm(c, d, 0x5140);
        const uint32_t AB = __byte_perm(a, b, 0x7362), CD = __byte_perm(c, d, 0x7362);
        o[k] = __byte_perm(ab, cd, 0x5410);
        o[2 + k] = __byte_perm(ab, cd, 0x7632);
        o[4 + k] = __byte_perm(AB, CD, 0x5410);
        o[6 + k] = __byte_perm(AB, CD, 0x7632);
    }
#pragma unroll
    for (int k = 0; k < kTileRows; ++k) w[k] = o[k];
}

// Puts a warp's turned codes into the tile [128 columns][128 rows]; a column's
// sixteen 8-byte pieces are at piece ^ ((column >> 2) & 15), so a half warp's
// writes (sixteen columns four apart) spread over the banks.
__device__ __forceinline__ void stage8(uint8_t* tile, const uint32_t (&w)[kTileRows], int warp, int lane) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint2*>(tile + (4 * lane + c) * 128 + 8 * (warp ^ (lane & 15))) =
            make_uint2(w[2 * c], w[2 * c + 1]);
}

// Writes the staged tile: column c's 128 codes to out + c * pitch.
__device__ __forceinline__ void write_tile(const uint8_t* tile, uint8_t* out, int64_t pitch) {
#pragma unroll
    for (int i = 0; i < 8192 / (8 * kTileThreads); ++i) {
        const int c = i * (kTileThreads / 8) + (threadIdx.x >> 3), piece = threadIdx.x & 7;   // 16 bytes of a column
        const int x = (c >> 2) & 15;
        const uint4 v = *reinterpret_cast<const uint4*>(tile + c * 128 + 16 * (piece ^ (x >> 1)));
        *reinterpret_cast<uint4*>(out + c * pitch + 16 * piece) = x & 1 ? make_uint4(v.z, v.w, v.x, v.y) : v;
    }
}

// The scales of T tensors' 128 columns from the warps' maxima `part`
// [16][T][128] into `scale` [T][128], and 1 / scale to inv[t] + c * pitch.
template <int T>
__device__ __forceinline__ void column_scales(const float* part, float* scale, float* const (&inv)[T],
                                              const int (&fmt)[T], int pow2, int64_t pitch) {
    for (int i = threadIdx.x; i < T * 128; i += kTileThreads) {
        const int t = i >> 7, c = i & 127;
        float* out = inv[0];
        int f = fmt[0];
#pragma unroll
        for (int k = 1; k < T; ++k)
            if (t == k) {
                out = inv[k];
                f = fmt[k];
            }
        if (!out) continue;   // uniform over a warp
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < kTileWarps; ++w) m = max(m, row::abs_bits(part[w * T * 128 + i]));
        const float s = row::block_scale(m, f, pow2);
        scale[i] = s;
        out[c * pitch] = __fdiv_rn(1.0f, s);
    }
}

// ------------------------------------------------------------------ gradient

struct ActBlockBwd {
    const __nv_bfloat16* d;
    const uint8_t* zq;
    const float* z_inv;
    uint8_t* q;
    float* inv;
    uint8_t* qt;
    float* inv_t;
    uint8_t* ht;
    float* h_inv_t;
    int64_t M;
    int blocks;
    int fmt, h_fmt, pow2;
    const int32_t* offsets;
    int experts;
    unsigned* status;
};

// What a lane reads of one row, and the values that come of it.
template <int ACT, bool GATED>
struct BwdRow {
    Quad dg, du, h;   // gradients of the gate's (or only) half and of the up half; act(z) z_u
    __device__ __forceinline__ void eval(uint2 d, uint32_t zg, uint32_t zu, float fg, float fu) {
        const Quad D = from_bf16(d), z = decode4(0, zg, fg);
        Quad u = zero4();
        if (GATED) u = decode4(0, zu, fu);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            f2 a, g;
            act_and_grad2<ACT>(z.v[j], a, g);
            if (GATED) {
                dg.v[j] = row::mul2(row::mul2(D.v[j], u.v[j]), g);
                du.v[j] = row::mul2(D.v[j], a);
                h.v[j] = row::mul2(a, u.v[j]);
            } else {
                dg.v[j] = row::mul2(D.v[j], g);
                h.v[j] = a;
            }
        }
    }
};

// Four rows of one 128-column block of dD a warp: row codes only.  The first two
// lanes of a row's eight have the scales of its gate's (or only) and up gradient.
// 4099 x 11008, GELU's tanh form: 45 us for 183 MB (0.61 of the copy rate).  No unit is
// near its limit (FMA pipe 57% busy, 26 instructions an element, 53% of the warps): a
// warp loads, computes and stores once, so only other warps cover its loads.
template <int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads, GATED ? 4 : 5) act_block_bwd_rows_kernel(const __grid_constant__ ActBlockBwd p) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int2 rows = rows_of(p.offsets, p.experts, p.M);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7;
    const Place at = place(blockIdx.x * kWarps + warp, p.blocks);
    const int64_t base = rows.x + static_cast<int64_t>(at.row) * 4, r = base + (lane >> 3);
    if (base >= rows.y) return;
    const int64_t N = static_cast<int64_t>(p.blocks) * 128, W = GATED ? 2 * N : N;
    const int wb = GATED ? 2 * p.blocks : p.blocks;
    const int c = at.blk * 128 + sub * 8;
    const bool on = r < rows.y;
    Raw16 d = {};
    uint2 zg[2] = {}, zu[2] = {};
    float fg = 0.0f, fu = 0.0f;
    if (on) {
        const uint8_t* z = p.zq + r * W + c;
        fg = p.z_inv[r * wb + at.blk];
        if (GATED) fu = p.z_inv[r * wb + p.blocks + at.blk];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            d.w[k] = ld16(p.d + r * N + c + 64 * k);
            zg[k] = ld8(z + 64 * k);
            if (GATED) zu[k] = ld8(z + N + 64 * k);
        }
    }
    f2 dg[2][4], du[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        f2 D[4];
        bf16_pairs(D, d.w[k]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const Quad z = decode4(0, h ? zg[k].y : zg[k].x, fg);
            Quad u = zero4();
            if (GATED) u = decode4(0, h ? zu[k].y : zu[k].x, fu);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f2 a, g;
                act_and_grad2<ACT>(z.v[j], a, g);
                dg[k][2 * h + j] = row::mul2(GATED ? row::mul2(D[2 * h + j], u.v[j]) : D[2 * h + j], g);
                if (GATED) du[k][2 * h + j] = row::mul2(D[2 * h + j], a);
            }
        }
    }
    uint32_t mine = eight_max(top16(dg));
    if constexpr (GATED) {
        const uint32_t m = eight_max(top16(du));
        if (sub == 1) mine = m;
    }
    const float s = row::block_scale(mine, p.fmt, p.pow2);
    if (on && sub < (GATED ? 2 : 1)) p.inv[r * wb + (sub ? p.blocks : 0) + at.blk] = __fdiv_rn(1.0f, s);
    const float sg = __shfl_sync(row::kAll, s, lane & 24), su = __shfl_sync(row::kAll, s, (lane & 24) + 1);
    if (!on) return;
    put16(p.q + r * W + c, p.fmt, dg, sg);
    if constexpr (GATED) put16(p.q + r * W + N + c, p.fmt, du, su);
}

// Shared memory of the tile kernel: two stages of inputs (dD, the gate's codes,
// the up product's), the warps' column maxima, three tiles of turned codes.
constexpr int kStageD = 128 * 128 * 2, kStageZ = 128 * 128, kStage = kStageD + 2 * kStageZ;
constexpr int kParts = kTileWarps * 3 * 128 * 4;
constexpr int kBwdSmem = 2 * kStage + kParts + 3 * 128 * 128 + 64 + 128;

// 128 x 128 tiles of dD, one CTA an SM, eight rows a warp.  A lane's values (8
// rows, 4 columns, three numbers each: 96 registers) are computed once and wait
// there for the rows' and the columns' scales; computed twice instead, with two
// CTAs an SM, 32768 x 2048 gated took 200 us.  The next tile's inputs come by TMA
// meanwhile.  That size with all outputs: 159 us for 619 MB (0.57 of the copy
// rate), bound by issue: 217 instructions a row of 128, at 0.6 a cycle since all
// warps are in the same part of a tile between its three barriers.
template <int ACT, bool GATED>
__global__ void __launch_bounds__(kTileThreads, 1)
    act_block_bwd_kernel(const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmZ,
                         const __grid_constant__ ActBlockBwd p) {
    ptx::griddep_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
    float* part = reinterpret_cast<float*>(smem + 2 * kStage);
    uint8_t* turned = smem + 2 * kStage + kParts;
    uint64_t* full = reinterpret_cast<uint64_t*>(turned + 3 * 128 * 128);
    __shared__ __align__(16) float scale[3][128];
    __shared__ uint32_t abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        ptx::mbar_init(&full[0], 1);
        ptx::mbar_init(&full[1], 1);
        abort_word = 0;
        ptx::fence_barrier_init();
    }
    ptx::griddep_wait();
    const int2 rows = rows_of(p.offsets, p.experts, p.M);
    __syncthreads();
    const int64_t N = static_cast<int64_t>(p.blocks) * 128, W = GATED ? 2 * N : N, tb = p.M >> 7;
    const int wb = GATED ? 2 * p.blocks : p.blocks;
    // the tiles with rows of experts
    const uint32_t tr0 = rows.x >> 7;
    const uint32_t tiles = rows.y > rows.x ? ((static_cast<uint32_t>(rows.y) + 127) / 128 - tr0) * p.blocks : 0;
    const uint32_t mine = blockIdx.x < tiles ? (tiles - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    auto issue = [&](uint32_t k) {   // one thread: this CTA's k-th tile into stage k & 1
        const Place at = place(blockIdx.x + k * gridDim.x, p.blocks);
        const int x = at.blk * 128, y = static_cast<int>((tr0 + at.row) * 128);
        uint8_t* st = smem + (k & 1) * kStage;
        ptx::mbar_arrive_expect_tx(&full[k & 1], GATED ? kStage : kStageD + kStageZ);
        ptx::tma_load_2d(st, &tmD, &full[k & 1], x, y);
        ptx::tma_load_2d(st + kStageD, &tmZ, &full[k & 1], x, y);
        if (GATED) ptx::tma_load_2d(st + kStageD + kStageZ, &tmZ, &full[k & 1], static_cast<int>(N) + x, y);
    };
    if (threadIdx.x == 0)
        for (uint32_t k = 0; k < mine && k < 2; ++k) issue(k);
    // a tile of this warp's: rows r0 + first .. r0 + last - 1 are the experts', lane
    // 2 i has row i's gate factor, lane 2 i + 1 its up factor
    struct Rows {
        int64_t tile_row, r0, at_factor;
        int blk, first, last;
        bool holds;
    };
    auto rows_at = [&](uint32_t k) {
        const Place here = place(blockIdx.x + k * gridDim.x, p.blocks);
        Rows t;
        t.blk = here.blk;
        t.tile_row = tr0 + here.row;
        t.r0 = t.tile_row * 128 + warp * kTileRows;
        t.first = static_cast<int>(rows.x > t.r0 ? (rows.x - t.r0 < kTileRows ? rows.x - t.r0 : kTileRows) : 0);
        t.last = static_cast<int>(rows.y > t.r0 ? (rows.y - t.r0 < kTileRows ? rows.y - t.r0 : kTileRows) : 0);
        t.holds = (lane >> 1) >= t.first && (lane >> 1) < t.last && (GATED || !(lane & 1));
        t.at_factor = (t.r0 + (lane >> 1)) * wb + (lane & 1 ? p.blocks : 0) + t.blk;
        return t;
    };
    uint32_t k = 0;
    auto factor_at = [&](uint32_t k) {
        if (k >= mine) return 0.0f;
        const Rows t = rows_at(k);
        return t.holds ? p.z_inv[t.at_factor] : 0.0f;
    };
    float next_factor = factor_at(0);
    for (; k < mine; ++k) {
        const Rows t = rows_at(k);
        const int64_t tile_row = t.tile_row, t0 = tile_row * 128, r0 = t.r0, at_factor = t.at_factor;
        const int blk = t.blk, first = t.first, last = t.last, c = blk * 128 + lane * 4;
        const bool holds = t.holds, whole = first == 0 && last == kTileRows;
        const float factor = next_factor;
        const bool ok = ptx::mbar_wait(&full[k & 1], (k >> 1) & 1u, &abort_word);
        const uint8_t* st = smem + (k & 1) * kStage;
        BwdRow<ACT, GATED> v[kTileRows];
        float tg[4] = {}, tu[4] = {}, th[4] = {};
        uint32_t top = 0;   // lane 2 i + k: the largest of row i's gate (k = 0) or up (1) gradient
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) {
            const int at = warp * kTileRows + i;
            uint2 d = *reinterpret_cast<const uint2*>(st + at * 256 + lane * 8);
            uint32_t zg = *reinterpret_cast<const uint32_t*>(st + kStageD + at * 128 + lane * 4);
            uint32_t zu = GATED ? *reinterpret_cast<const uint32_t*>(st + kStageD + kStageZ + at * 128 + lane * 4) : 0u;
            if (!whole && (i < first || i >= last)) {
                d = make_uint2(0, 0);
                zg = zu = 0;
            }
            v[i].eval(d, zg, zu, __shfl_sync(row::kAll, factor, 2 * i),
                      GATED ? __shfl_sync(row::kAll, factor, 2 * i + 1) : 0.0f);
            if (p.q) {
                const uint32_t m = row_top(v[i].dg);
                if (lane == 2 * i) top = m;
                if (GATED) {
                    const uint32_t n = row_top(v[i].du);
                    if (lane == 2 * i + 1) top = n;
                }
            }
            if (p.qt) {
                raise4(tg, v[i].dg);
                if (GATED) raise4(tu, v[i].du);
            }
            if (p.ht) raise4(th, v[i].h);
        }
        float4* mine4 = reinterpret_cast<float4*>(part + warp * 3 * 128) + lane;
        mine4[0] = make_float4(tg[0], tg[1], tg[2], tg[3]);
        mine4[32] = make_float4(tu[0], tu[1], tu[2], tu[3]);
        mine4[64] = make_float4(th[0], th[1], th[2], th[3]);
        // the stage has been read, the maxima are there, the last tile's codes have left `turned`
        if (!__syncthreads_and(ok)) break;
        if (threadIdx.x == 0 && k + 2 < mine) issue(k + 2);
        next_factor = factor_at(k + 1);
        float* const out[3] = {p.qt ? p.inv_t + static_cast<int64_t>(blk) * 128 * tb + tile_row : nullptr,
                               p.qt && GATED ? p.inv_t + (N + static_cast<int64_t>(blk) * 128) * tb + tile_row : nullptr,
                               p.ht ? p.h_inv_t + static_cast<int64_t>(blk) * 128 * tb + tile_row : nullptr};
        const int fmt[3] = {p.fmt, p.fmt, p.h_fmt};
        column_scales<3>(part, &scale[0][0], out, fmt, p.pow2, tb);
        if (p.q) {   // row codes while the other warps are at the columns' scales
            const float s_row = row::block_scale(top, p.fmt, p.pow2);
            if (holds) p.inv[at_factor] = __fdiv_rn(1.0f, s_row);
            uint8_t* q = p.q + r0 * W + c;
            by_format(p.fmt, [&](auto f) {
#pragma unroll
                for (int i = 0; i < kTileRows; ++i) {
                    const f2 a = row::all2(__shfl_sync(row::kAll, s_row, 2 * i));
                    const f2 b = row::all2(GATED ? __shfl_sync(row::kAll, s_row, 2 * i + 1) : 0.0f);
                    if (whole || (i >= first && i < last)) {
                        *reinterpret_cast<uint32_t*>(q) = code4<f.value>(v[i].dg, a, a);
                        if (GATED) *reinterpret_cast<uint32_t*>(q + N) = code4<f.value>(v[i].du, b, b);
                    }
                    q += W;
                }
            });
        }
        __syncthreads();
        // the codes of one tensor's columns, turned, into the tile `t`
        auto put_columns = [&](auto f, int t, auto value) {
            const float4 a = reinterpret_cast<const float4*>(scale[t])[lane];
            const f2 s0 = row::mk2(a.x, a.y), s1 = row::mk2(a.z, a.w);
            uint32_t w[kTileRows];
#pragma unroll
            for (int i = 0; i < kTileRows; ++i) w[i] = code4<f.value>(value(i), s0, s1);
            turn8(w);
            stage8(turned + t * 128 * 128, w, warp, lane);
        };
        if (p.qt)
            by_format(p.fmt, [&](auto f) {
                put_columns(f, 0, [&](int i) -> const Quad& { return v[i].dg; });
                if (GATED) put_columns(f, 1, [&](int i) -> const Quad& { return v[i].du; });
            });
        if (p.ht)
            by_format(p.h_fmt, [&](auto f) { put_columns(f, 2, [&](int i) -> const Quad& { return v[i].h; }); });
        __syncthreads();
        const int64_t out_at = static_cast<int64_t>(blk) * 128 * p.M + t0;
        if (p.qt) {
            write_tile(turned, p.qt + out_at, p.M);
            if (GATED) write_tile(turned + 128 * 128, p.qt + N * p.M + out_at, p.M);
        }
        if (p.ht) write_tile(turned + 2 * 128 * 128, p.ht + out_at, p.M);
    }
    if (threadIdx.x == 0 && k < mine) {
        // a wait gave up: let the copies already issued land before the CTA's
        // shared memory is released
        uint32_t never = 0;
        for (uint32_t j = k; j < mine && j < k + 2; ++j) ptx::mbar_wait(&full[j & 1], (j >> 1) & 1u, &never);
        if (p.status) atomicOr(p.status, 1u);
    }
}

// ------------------------------------------------------------------ a kept input, transposed

struct BlockTranspose {
    const uint8_t* q;
    const float* inv;
    uint8_t* qt;
    float* inv_t;
    int64_t rows;
    int blocks;   // cols / 128
    int pow2;
};

// Two CTAs an SM walk the tiles; a tile's codes are loaded while the one before
// it is cast.  32768 x 7168: 115 us for 485 MB (0.62 of the copy rate); the barriers
// around the columns' scales bound it (a CTA a tile 147 us; codes decoded
// twice, for fewer registers, 123).
template <int FMT>
__global__ void __launch_bounds__(kTileThreads, 2) block_transpose_kernel(const __grid_constant__ BlockTranspose p) {
    ptx::griddep_launch_dependents();
    __shared__ __align__(16) uint8_t turned[128 * 128];
    __shared__ __align__(16) float part[kTileWarps * 128];
    __shared__ __align__(16) float scale[128];
    ptx::griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t cols = static_cast<int64_t>(p.blocks) * 128, tb = p.rows >> 7;
    const uint32_t tiles = static_cast<uint32_t>(tb) * p.blocks;
    uint32_t next[kTileRows];
    float next_factor = 0.0f;
    auto load = [&](uint32_t tile) {
        if (tile >= tiles) return;
        const Place at = place(tile, p.blocks);
        const int blk = at.blk;
        const int64_t r0 = static_cast<int64_t>(at.row) * 128 + warp * kTileRows;
        const uint8_t* q = p.q + r0 * cols + blk * 128 + lane * 4;
#pragma unroll
        for (int i = 0; i < kTileRows; ++i, q += cols) next[i] = ld4(q);
        if (lane < kTileRows) next_factor = p.inv[(r0 + lane) * p.blocks + blk];
    };
    load(blockIdx.x);
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        uint32_t w[kTileRows];
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) w[i] = next[i];
        const float factor = next_factor;
        load(tile + gridDim.x);
        const Place here = place(tile, p.blocks);
        const int64_t tile_row = here.row;
        const int blk = here.blk;
        Quad v[kTileRows];
        float top[4] = {};
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) {
            v[i] = decode4(FMT, w[i], __shfl_sync(row::kAll, factor, i));
            raise4(top, v[i]);
        }
        reinterpret_cast<float4*>(part + warp * 128)[lane] = make_float4(top[0], top[1], top[2], top[3]);
        __syncthreads();   // also: the last tile's codes have left `turned`
        float* const out[1] = {p.inv_t + static_cast<int64_t>(blk) * 128 * tb + tile_row};
        const int fmt[1] = {FMT};
        column_scales<1>(part, scale, out, fmt, p.pow2, tb);
        __syncthreads();
        const float4 s = reinterpret_cast<const float4*>(scale)[lane];
        const f2 s0 = row::mk2(s.x, s.y), s1 = row::mk2(s.z, s.w);
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) w[i] = code4<FMT>(v[i], s0, s1);
        turn8(w);
        stage8(turned, w, warp, lane);
        __syncthreads();
        write_tile(turned, p.qt + static_cast<int64_t>(blk) * 128 * p.rows + tile_row * 128, p.rows);
    }
}

// ------------------------------------------------------------------ host side

// Four rows of one column block a warp.
dim3 row_grid(int64_t M, int64_t blocks) {
    return dim3(static_cast<unsigned>(((M + 3) / 4 * blocks + kWarps - 1) / kWarps));
}

template <int ACT>
int launch_fwd(const ActBlock& p, bool gated, cudaStream_t st) {
    const dim3 grid = row_grid(p.M, p.blocks), block(kThreads);
    if (gated) launch_pdl(act_block_kernel<ACT, true>, grid, block, 0, st, p);
    else launch_pdl(act_block_kernel<ACT, false>, grid, block, 0, st, p);
    return FP8_OK;
}

template <int ACT, bool GATED>
int launch_bwd(const ActBlockBwd& p, cudaStream_t st) {
    if (!p.qt && !p.ht) {
        launch_pdl(act_block_bwd_rows_kernel<ACT, GATED>, row_grid(p.M, p.blocks), dim3(kThreads), 0, st, p);
        return FP8_OK;
    }
    static host::SmemAllowance allowance;
    CUtensorMap tmD, tmZ;
    const int64_t N = static_cast<int64_t>(p.blocks) * 128;
    int r = make_bf16_box_map(&tmD, p.d, p.M, N, 128, 128);
    if (r == FP8_OK) r = make_codes_box_map(&tmZ, p.zq, p.M, GATED ? 2 * N : N, 128, 128);
    if (r == FP8_OK) r = host::allow_smem(act_block_bwd_kernel<ACT, GATED>, kBwdSmem, allowance);
    if (r != FP8_OK) return r;
    const int64_t tiles = p.M / 128 * p.blocks;
    const int sms = num_sms();
    launch_pdl(act_block_bwd_kernel<ACT, GATED>, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)),
               dim3(kTileThreads), kBwdSmem, st, tmD, tmZ, p);
    return FP8_OK;
}

template <int ACT>
int launch_bwd(const ActBlockBwd& p, bool gated, cudaStream_t st) {
    return gated ? launch_bwd<ACT, true>(p, st) : launch_bwd<ACT, false>(p, st);
}

// launch(std::integral_constant<int, act>) for the activation.
template <typename F>
int by_act(int act, F launch) {
    switch (act) {
        case FP8_ACT_RELU: return launch(std::integral_constant<int, FP8_ACT_RELU>());
        case FP8_ACT_SILU: return launch(std::integral_constant<int, FP8_ACT_SILU>());
        case FP8_ACT_GELU: return launch(std::integral_constant<int, FP8_ACT_GELU>());
        case FP8_ACT_GELU_TANH: return launch(std::integral_constant<int, FP8_ACT_GELU_TANH>());
        default: return launch(std::integral_constant<int, FP8_ACT_NONE>());
    }
}

// What the activation and its gradient both check.
int check_act(const char* what, int64_t M, int64_t N, int act, int gated, const int32_t* offsets, int experts) {
    if (act < FP8_ACT_NONE || act > FP8_ACT_GELU_TANH)
        return set_error(FP8_ERR_INVALID_ARG, "%s: unknown activation %d", what, act);
    if (M < 0 || N < 128 || N % 128)
        return set_error(FP8_ERR_SHAPE, "%s: M must be >= 0, N a positive multiple of 128", what);
    if (offsets && (experts < 1 || experts > kMaxGemmExperts))
        return set_error(FP8_ERR_SHAPE, "%s: experts in 1..%d", what, kMaxGemmExperts);
    const int64_t limit = (int64_t{1} << 31) - 1024;   // rows, columns and units are 32-bit
    if (M > limit || N > limit / (gated ? 2 : 1) || (M + 127) > limit / (N / 128))
        return set_error(FP8_ERR_SHAPE, "%s: dimensions out of range", what);
    return FP8_OK;
}

bool known(int fmt) { return fmt == FP8_E4M3 || fmt == FP8_E5M2; }

}  // namespace
}  // namespace fp8

using namespace fp8;
using namespace fp8::host;

extern "C" {

int fp8_act_block(const fp8_act_block_args_t* a, void* stream) {
    const char* what = "fp8_act_block";
    if (!a) return set_error(FP8_ERR_INVALID_ARG, "%s: args is NULL", what);
    const int r = check_act(what, a->M, a->N, a->act, a->gated, a->offsets, a->experts);
    if (r != FP8_OK) return r;
    if (a->q && !known(a->q_format)) return set_error(FP8_ERR_INVALID_ARG, "%s: unknown FP8 format", what);
    if (a->M && !a->z) return set_error(FP8_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if (a->M && !a->q && !a->z_q) return set_error(FP8_ERR_INVALID_ARG, "%s: no output", what);
    if (a->M && (!a->q != !a->scale_inv || !a->z_q != !a->z_scale_inv))
        return set_error(FP8_ERR_INVALID_ARG, "%s: codes and their factors go together", what);
    for (const void* t : {a->z, static_cast<const void*>(a->q), static_cast<const void*>(a->z_q)})
        if (!aligned(t, 16)) return set_error(FP8_ERR_ALIGN, "%s: tensors must be 16-byte aligned", what);
    for (const void* t : {static_cast<const void*>(a->scale_inv), static_cast<const void*>(a->z_scale_inv),
                          static_cast<const void*>(a->offsets)})
        if (!aligned(t, 4))
            return set_error(FP8_ERR_ALIGN, "%s: factors and offsets must be 4-byte aligned", what);
    if (a->M == 0) return FP8_OK;
    const ActBlock p{static_cast<const __nv_bfloat16*>(a->z), a->q, a->scale_inv, a->z_q, a->z_scale_inv, a->M,
                     static_cast<int>(a->N / 128), a->q_format, a->pow2, a->offsets, a->experts};
    by_act(a->act, [&](auto act) { return launch_fwd<decltype(act)::value>(p, a->gated != 0, as_stream(stream)); });
    return launch_status(what);
}

int fp8_act_block_bwd(const fp8_act_block_bwd_args_t* a, void* stream) {
    const char* what = "fp8_act_block_bwd";
    if (!a) return set_error(FP8_ERR_INVALID_ARG, "%s: args is NULL", what);
    int r = check_act(what, a->M, a->N, a->act, a->gated, a->offsets, a->experts);
    if (r != FP8_OK) return r;
    if (((a->q || a->q_t) && !known(a->q_format)) || (a->h_t && !known(a->h_format)))
        return set_error(FP8_ERR_INVALID_ARG, "%s: unknown FP8 format", what);
    if ((a->q_t || a->h_t) && a->M % 128)
        return set_error(FP8_ERR_SHAPE, "%s: q_t and h_t need M a multiple of 128", what);
    if (a->M && (!a->dD || !a->z_q || !a->z_scale_inv))
        return set_error(FP8_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if (a->M && !a->q && !a->q_t && !a->h_t) return set_error(FP8_ERR_INVALID_ARG, "%s: no output", what);
    if (a->M && (!a->q != !a->scale_inv || !a->q_t != !a->scale_inv_t || !a->h_t != !a->h_scale_inv_t))
        return set_error(FP8_ERR_INVALID_ARG, "%s: codes and their factors go together", what);
    for (const void* t : {a->dD, static_cast<const void*>(a->z_q), static_cast<const void*>(a->q),
                          static_cast<const void*>(a->q_t), static_cast<const void*>(a->h_t)})
        if (!aligned(t, 16)) return set_error(FP8_ERR_ALIGN, "%s: tensors must be 16-byte aligned", what);
    for (const void* t : {static_cast<const void*>(a->z_scale_inv), static_cast<const void*>(a->scale_inv),
                          static_cast<const void*>(a->scale_inv_t), static_cast<const void*>(a->h_scale_inv_t),
                          static_cast<const void*>(a->offsets)})
        if (!aligned(t, 4))
            return set_error(FP8_ERR_ALIGN, "%s: factors and offsets must be 4-byte aligned", what);
    if (a->M == 0) return FP8_OK;
    const ActBlockBwd p{static_cast<const __nv_bfloat16*>(a->dD), a->z_q, a->z_scale_inv, a->q, a->scale_inv,
                        a->q_t, a->scale_inv_t, a->h_t, a->h_scale_inv_t, a->M, static_cast<int>(a->N / 128),
                        a->q_format, a->h_format, a->pow2, a->offsets, a->experts, device_status_word()};
    r = by_act(a->act, [&](auto act) { return launch_bwd<decltype(act)::value>(p, a->gated != 0, as_stream(stream)); });
    return r != FP8_OK ? r : launch_status(what);
}

int fp8_block_transpose(const uint8_t* q, const float* scale_inv, int64_t rows, int64_t cols, int format, int pow2,
                        uint8_t* q_t, float* scale_inv_t, void* stream) {
    const char* what = "fp8_block_transpose";
    if (rows < 0 || cols < 128 || rows % 128 || cols % 128)
        return set_error(FP8_ERR_SHAPE, "%s: rows and cols must be multiples of 128, cols positive", what);
    if (!known(format)) return set_error(FP8_ERR_INVALID_ARG, "%s: unknown FP8 format", what);
    const int64_t limit = (int64_t{1} << 31) - 1024;
    if (rows > limit || cols > limit || rows / 128 > limit / (cols / 128))
        return set_error(FP8_ERR_SHAPE, "%s: dimensions out of range", what);
    if (rows && (!q || !scale_inv || !q_t || !scale_inv_t))
        return set_error(FP8_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if (!aligned(q, 16) || !aligned(q_t, 16))
        return set_error(FP8_ERR_ALIGN, "%s: tensors must be 16-byte aligned", what);
    if (!aligned(scale_inv, 4) || !aligned(scale_inv_t, 4))
        return set_error(FP8_ERR_ALIGN, "%s: factors must be 4-byte aligned", what);
    if (rows == 0) return FP8_OK;
    const BlockTranspose p{q, scale_inv, q_t, scale_inv_t, rows, static_cast<int>(cols / 128), pow2};
    const int64_t tiles = rows / 128 * p.blocks, slots = 2 * static_cast<int64_t>(num_sms());
    const dim3 grid(static_cast<unsigned>(tiles < slots ? tiles : slots)), block(kTileThreads);
    if (format == FP8_E4M3) launch_pdl(block_transpose_kernel<0>, grid, block, 0, as_stream(stream), p);
    else launch_pdl(block_transpose_kernel<1>, grid, block, 0, as_stream(stream), p);
    return launch_status(what);
}

}  // extern "C"

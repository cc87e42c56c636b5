// act_block.cu -- the activation between two products in blocks of 128, with an
// 8-bit checkpoint for the backward pass, its gradient from the checkpoint, and
// the transposing re-cast of a kept input.
//
//   h = act(z_g) z_u,  q = codes of h,  z_q = codes of z        (1x128 blocks)
//   dz_g = dD z_u act'(z_g),  dz_u = dD act(z_g)                (from z_q)
//
// A warp takes rows of one 128-column block, four columns a lane, so a row's
// maximum is one warp reduction and a column's stays in the lane's registers
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
__device__ __forceinline__ uint32_t code4(int fmt, const Quad& q, f2 s0, f2 s1) {
    const f2 a = row::mul2(q.v[0], s0), b = row::mul2(q.v[1], s1);
    return row::cvt_pair(fmt, row::lo2(a), row::hi2(a)) | (row::cvt_pair(fmt, row::lo2(b), row::hi2(b)) << 16);
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

// The experts' rows: begin .. end.  Every thread; ends with a barrier.
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

// R rows of one 128-column block of h a warp.
template <int ACT, bool GATED, int R>
__global__ void __launch_bounds__(kThreads, 4) act_block_kernel(const __grid_constant__ ActBlock p) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int2 rows = rows_of(p.offsets, p.experts, p.M);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int blk = static_cast<int>(unit % p.blocks);
    const int64_t r0 = rows.x + unit / p.blocks * R;
    if (r0 >= rows.y) return;
    const int64_t N = static_cast<int64_t>(p.blocks) * 128, W = GATED ? 2 * N : N;
    const int wb = GATED ? 2 * p.blocks : p.blocks;   // factors a row of z
    const int c = blk * 128 + lane * 4;
    uint2 g[R], u[GATED ? R : 1];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t r = r0 + i;
        g[i] = make_uint2(0, 0);
        if (GATED) u[i] = make_uint2(0, 0);
        if (r < rows.y) {
            g[i] = ld8(p.z + r * W + c);
            if (GATED) u[i] = ld8(p.z + r * W + N + c);
        }
    }
    // lane 4 i + k keeps the maximum of row i's h (k = 0), gate (1), up (2)
    Quad h[R];
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const Quad a = from_bf16(g[i]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            h[i].v[j] = act2<ACT>(a.v[j]);
            if (GATED) h[i].v[j] = row::mul2(h[i].v[j], from_bf16(u[i]).v[j]);
        }
        if (p.q) {
            const uint32_t m = row_top(h[i]);
            if (lane == 4 * i) mine = m;
        }
        if (p.zq) {
            const uint32_t m = row_top(a);
            if (lane == 4 * i + 1) mine = m;
            if (GATED) {
                const uint32_t n = row_top(from_bf16(u[i]));
                if (lane == 4 * i + 2) mine = n;
            }
        }
    }
    const int kind = lane & 3;
    const float s = row::block_scale(mine, kind == 0 ? p.fmt : FP8_E4M3, p.pow2);
    const int64_t mr = r0 + (lane >> 2);
    if ((lane >> 2) < R && mr < rows.y) {
        const float f = __fdiv_rn(1.0f, s);
        if (kind == 0 && p.q) p.inv[mr * p.blocks + blk] = f;
        if (kind == 1 && p.zq) p.z_inv[mr * wb + blk] = f;
        if (GATED && kind == 2 && p.zq) p.z_inv[mr * wb + p.blocks + blk] = f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float sh = __shfl_sync(row::kAll, s, 4 * i), sg = __shfl_sync(row::kAll, s, 4 * i + 1);
        const float su = GATED ? __shfl_sync(row::kAll, s, 4 * i + 2) : 0.0f;
        const int64_t r = r0 + i;
        if (r >= rows.y) break;
        if (p.q) *reinterpret_cast<uint32_t*>(p.q + r * N + c) = code4(p.fmt, h[i], row::all2(sh), row::all2(sh));
        if (p.zq) {
            *reinterpret_cast<uint32_t*>(p.zq + r * W + c) = code4(0, from_bf16(g[i]), row::all2(sg), row::all2(sg));
            if (GATED)
                *reinterpret_cast<uint32_t*>(p.zq + r * W + N + c) =
                    code4(0, from_bf16(u[i]), row::all2(su), row::all2(su));
        }
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

// R rows of one 128-column block of dD a warp: row codes only.
template <int ACT, bool GATED, int R>
__global__ void __launch_bounds__(kThreads, 4) act_block_bwd_rows_kernel(const __grid_constant__ ActBlockBwd p) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int2 rows = rows_of(p.offsets, p.experts, p.M);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int blk = static_cast<int>(unit % p.blocks);
    const int64_t r0 = rows.x + unit / p.blocks * R;
    if (r0 >= rows.y) return;
    const int64_t N = static_cast<int64_t>(p.blocks) * 128, W = GATED ? 2 * N : N;
    const int wb = GATED ? 2 * p.blocks : p.blocks;
    const int c = blk * 128 + lane * 4;
    uint2 d[R];
    uint32_t zg[R], zu[GATED ? R : 1];
    float fg[R], fu[GATED ? R : 1];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t r = r0 + i < rows.y ? r0 + i : r0;   // rows past the last are read again and not written
        d[i] = ld8(p.d + r * N + c);
        zg[i] = ld4(p.zq + r * W + c);
        fg[i] = p.z_inv[r * wb + blk];
        if (GATED) {
            zu[i] = ld4(p.zq + r * W + N + c);
            fu[i] = p.z_inv[r * wb + p.blocks + blk];
        }
    }
    // lane 2 i + k keeps the maximum of row i's gate (k = 0) or up (1) gradient
    BwdRow<ACT, GATED> v[R];
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        v[i].eval(d[i], zg[i], GATED ? zu[i] : 0, fg[i], GATED ? fu[i] : 0.0f);
        const uint32_t m = row_top(v[i].dg);
        if (lane == 2 * i) mine = m;
        if (GATED) {
            const uint32_t n = row_top(v[i].du);
            if (lane == 2 * i + 1) mine = n;
        }
    }
    const float s = row::block_scale(mine, p.fmt, p.pow2);
    const int64_t mr = r0 + (lane >> 1);
    if ((lane >> 1) < R && mr < rows.y && (GATED || !(lane & 1)))
        p.inv[mr * wb + (lane & 1 ? p.blocks : 0) + blk] = __fdiv_rn(1.0f, s);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const f2 sg = row::all2(__shfl_sync(row::kAll, s, 2 * i));
        const f2 su = row::all2(GATED ? __shfl_sync(row::kAll, s, 2 * i + 1) : 0.0f);
        const int64_t r = r0 + i;
        if (r >= rows.y) break;
        *reinterpret_cast<uint32_t*>(p.q + r * W + c) = code4(p.fmt, v[i].dg, sg, sg);
        if (GATED) *reinterpret_cast<uint32_t*>(p.q + r * W + N + c) = code4(p.fmt, v[i].du, su, su);
    }
}

constexpr int kBwdSmem = 3 * 128 * 128;   // three tiles of turned codes; the maxima before them

// One 128 x 128 tile of dD, eight rows a warp.  The values are computed twice, for
// the maxima and for the codes, from the inputs, which stay in registers as loaded
// (four bytes an element): FP32 values would take three times as many.
template <int ACT, bool GATED>
__global__ void __launch_bounds__(kTileThreads, 2) act_block_bwd_kernel(const __grid_constant__ ActBlockBwd p) {
    ptx::griddep_launch_dependents();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float scale[3][128];
    ptx::griddep_wait();
    const int2 rows = rows_of(p.offsets, p.experts, p.M);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tile_row = blockIdx.x / p.blocks;
    const int blk = static_cast<int>(blockIdx.x - tile_row * p.blocks);
    const int64_t t0 = tile_row * 128;
    if (t0 + 128 <= rows.x || t0 >= rows.y || rows.x >= rows.y) return;
    const int64_t N = static_cast<int64_t>(p.blocks) * 128, W = GATED ? 2 * N : N;
    const int wb = GATED ? 2 * p.blocks : p.blocks;
    const int c = blk * 128 + lane * 4;
    const int64_t r0 = t0 + warp * kTileRows;
    // rows r0 + first .. r0 + last - 1 are the experts'
    const int first = static_cast<int>(rows.x > r0 ? (rows.x - r0 < kTileRows ? rows.x - r0 : kTileRows) : 0);
    const int last = static_cast<int>(rows.y > r0 ? (rows.y - r0 < kTileRows ? rows.y - r0 : kTileRows) : 0);
    uint2 d[kTileRows];
    uint32_t zg[kTileRows], zu[GATED ? kTileRows : 1];
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        d[i] = make_uint2(0, 0);
        zg[i] = 0;
        if (GATED) zu[i] = 0;
        if (i >= first && i < last) {
            const int64_t r = r0 + i;
            d[i] = ld8(p.d + r * N + c);
            zg[i] = ld4(p.zq + r * W + c);
            if (GATED) zu[i] = ld4(p.zq + r * W + N + c);
        }
    }
    // lane 2 i has row i's gate factor, lane 2 i + 1 its up factor
    float factor = 0.0f;
    const bool holds = (lane >> 1) >= first && (lane >> 1) < last && (GATED || !(lane & 1));
    const int64_t at_factor = (r0 + (lane >> 1)) * wb + (lane & 1 ? p.blocks : 0) + blk;
    if (holds) factor = p.z_inv[at_factor];
    float tg[4] = {}, tu[4] = {}, th[4] = {};
    uint32_t mine = 0;   // lane 2 i + k: the largest of row i's gate (k = 0) or up (1) gradient
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        BwdRow<ACT, GATED> v;
        v.eval(d[i], zg[i], GATED ? zu[i] : 0, __shfl_sync(row::kAll, factor, 2 * i),
               GATED ? __shfl_sync(row::kAll, factor, 2 * i + 1) : 0.0f);
        if (p.q) {
            const uint32_t m = row_top(v.dg);
            if (lane == 2 * i) mine = m;
            if (GATED) {
                const uint32_t n = row_top(v.du);
                if (lane == 2 * i + 1) mine = n;
            }
        }
        if (p.qt) {
            raise4(tg, v.dg);
            if (GATED) raise4(tu, v.du);
        }
        if (p.ht) raise4(th, v.h);
        // the values are not kept for the second evaluation
        asm volatile("" : "+r"(d[i].x), "+r"(d[i].y), "+r"(zg[i]));
        if (GATED) asm volatile("" : "+r"(zu[i]));
    }
    float s_row = 1.0f;
    if (p.q) {
        s_row = row::block_scale(mine, p.fmt, p.pow2);
        if (holds) p.inv[at_factor] = __fdiv_rn(1.0f, s_row);
    }
    float* part = reinterpret_cast<float*>(smem);
    float4* mine4 = reinterpret_cast<float4*>(part + warp * 3 * 128) + lane;
    mine4[0] = make_float4(tg[0], tg[1], tg[2], tg[3]);
    mine4[32] = make_float4(tu[0], tu[1], tu[2], tu[3]);
    mine4[64] = make_float4(th[0], th[1], th[2], th[3]);
    __syncthreads();
    const int64_t tb = p.M >> 7;
    float* const out[3] = {p.qt ? p.inv_t + static_cast<int64_t>(blk) * 128 * tb + tile_row : nullptr,
                           p.qt && GATED ? p.inv_t + (N + static_cast<int64_t>(blk) * 128) * tb + tile_row : nullptr,
                           p.ht ? p.h_inv_t + static_cast<int64_t>(blk) * 128 * tb + tile_row : nullptr};
    const int fmt[3] = {p.fmt, p.fmt, p.h_fmt};
    column_scales<3>(part, &scale[0][0], out, fmt, p.pow2, tb);
    __syncthreads();   // the maxima have been read: their place takes the tiles
    const float4 a = reinterpret_cast<const float4*>(scale[0])[lane], b = reinterpret_cast<const float4*>(scale[1])[lane],
                 e = reinterpret_cast<const float4*>(scale[2])[lane];
    const f2 sg[2] = {row::mk2(a.x, a.y), row::mk2(a.z, a.w)}, su[2] = {row::mk2(b.x, b.y), row::mk2(b.z, b.w)};
    const f2 sh[2] = {row::mk2(e.x, e.y), row::mk2(e.z, e.w)};
    uint32_t wg[kTileRows], wu[kTileRows], wh[kTileRows];
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        BwdRow<ACT, GATED> v;
        v.eval(d[i], zg[i], GATED ? zu[i] : 0, __shfl_sync(row::kAll, factor, 2 * i),
               GATED ? __shfl_sync(row::kAll, factor, 2 * i + 1) : 0.0f);
        if (p.q) {
            const f2 a = row::all2(__shfl_sync(row::kAll, s_row, 2 * i));
            const f2 b = row::all2(GATED ? __shfl_sync(row::kAll, s_row, 2 * i + 1) : 0.0f);
            if (i >= first && i < last) {
                *reinterpret_cast<uint32_t*>(p.q + (r0 + i) * W + c) = code4(p.fmt, v.dg, a, a);
                if (GATED) *reinterpret_cast<uint32_t*>(p.q + (r0 + i) * W + N + c) = code4(p.fmt, v.du, b, b);
            }
        }
        if (p.qt) {
            wg[i] = code4(p.fmt, v.dg, sg[0], sg[1]);
            if (GATED) wu[i] = code4(p.fmt, v.du, su[0], su[1]);
        }
        if (p.ht) wh[i] = code4(p.h_fmt, v.h, sh[0], sh[1]);
    }
    if (p.qt) {
        turn8(wg);
        stage8(smem, wg, warp, lane);
        if (GATED) {
            turn8(wu);
            stage8(smem + 128 * 128, wu, warp, lane);
        }
    }
    if (p.ht) {
        turn8(wh);
        stage8(smem + 2 * 128 * 128, wh, warp, lane);
    }
    __syncthreads();
    const int64_t at = static_cast<int64_t>(blk) * 128 * p.M + t0;
    if (p.qt) {
        write_tile(smem, p.qt + at, p.M);
        if (GATED) write_tile(smem + 128 * 128, p.qt + N * p.M + at, p.M);
    }
    if (p.ht) write_tile(smem + 2 * 128 * 128, p.ht + at, p.M);
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

template <int FMT>
__global__ void __launch_bounds__(kTileThreads, 3) block_transpose_kernel(const __grid_constant__ BlockTranspose p) {
    ptx::griddep_launch_dependents();
    __shared__ __align__(16) uint8_t tile[128 * 128];   // the maxima, then the turned codes
    __shared__ __align__(16) float scale[128];
    ptx::griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tile_row = blockIdx.x / p.blocks;
    const int blk = static_cast<int>(blockIdx.x - tile_row * p.blocks);
    const int64_t cols = static_cast<int64_t>(p.blocks) * 128, r0 = tile_row * 128 + warp * kTileRows;
    const int c = blk * 128 + lane * 4;
    uint32_t w[kTileRows];
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) w[i] = ld4(p.q + (r0 + i) * cols + c);
    const float factor = lane < kTileRows ? p.inv[(r0 + lane) * p.blocks + blk] : 0.0f;
    float top[4] = {};
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        raise4(top, decode4(FMT, w[i], __shfl_sync(row::kAll, factor, i)));
        asm volatile("" : "+r"(w[i]));   // decoded again below
    }
    float* part = reinterpret_cast<float*>(tile);
    reinterpret_cast<float4*>(part + warp * 128)[lane] = make_float4(top[0], top[1], top[2], top[3]);
    __syncthreads();
    const int64_t tb = p.rows >> 7;
    float* const out[1] = {p.inv_t + static_cast<int64_t>(blk) * 128 * tb + tile_row};
    const int fmt[1] = {FMT};
    column_scales<1>(part, scale, out, fmt, p.pow2, tb);
    __syncthreads();
    const float4 s = reinterpret_cast<const float4*>(scale)[lane];
    const f2 s0 = row::mk2(s.x, s.y), s1 = row::mk2(s.z, s.w);
#pragma unroll
    for (int i = 0; i < kTileRows; ++i)
        w[i] = code4(FMT, decode4(FMT, w[i], __shfl_sync(row::kAll, factor, i)), s0, s1);
    turn8(w);
    stage8(tile, w, warp, lane);
    __syncthreads();
    write_tile(tile, p.qt + static_cast<int64_t>(blk) * 128 * p.rows + tile_row * 128, p.rows);
}

// ------------------------------------------------------------------ host side

constexpr int kRows = 4;   // rows a warp where there are many

// Whether kRows rows a warp still leave every SM several CTAs.
bool many_rows(int64_t M, int64_t blocks) {
    return M * blocks >= int64_t{kRows} * kWarps * 4 * num_sms();
}

dim3 row_grid(int64_t M, int64_t blocks, bool many) {
    const int64_t warps = (many ? (M + kRows - 1) / kRows : M) * blocks;
    return dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps));
}

template <int ACT>
int launch_fwd(const ActBlock& p, bool gated, cudaStream_t st) {
    const bool many = many_rows(p.M, p.blocks);
    const dim3 grid = row_grid(p.M, p.blocks, many), block(kThreads);
    if (gated) {
        if (many) launch_pdl(act_block_kernel<ACT, true, kRows>, grid, block, 0, st, p);
        else launch_pdl(act_block_kernel<ACT, true, 1>, grid, block, 0, st, p);
    } else {
        if (many) launch_pdl(act_block_kernel<ACT, false, kRows>, grid, block, 0, st, p);
        else launch_pdl(act_block_kernel<ACT, false, 1>, grid, block, 0, st, p);
    }
    return FP8_OK;
}

template <int ACT, bool GATED>
int launch_bwd(const ActBlockBwd& p, cudaStream_t st) {
    if (!p.qt && !p.ht) {
        const bool many = many_rows(p.M, p.blocks);
        const dim3 grid = row_grid(p.M, p.blocks, many), block(kThreads);
        if (many) launch_pdl(act_block_bwd_rows_kernel<ACT, GATED, kRows>, grid, block, 0, st, p);
        else launch_pdl(act_block_bwd_rows_kernel<ACT, GATED, 1>, grid, block, 0, st, p);
        return FP8_OK;
    }
    static host::SmemAllowance allowance;
    const int r = host::allow_smem(act_block_bwd_kernel<ACT, GATED>, kBwdSmem, allowance);
    if (r != FP8_OK) return r;
    const dim3 grid(static_cast<unsigned>(p.M / 128 * p.blocks)), block(kTileThreads);
    launch_pdl(act_block_bwd_kernel<ACT, GATED>, grid, block, kBwdSmem, st, p);
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
                        a->q_format, a->h_format, a->pow2, a->offsets, a->experts};
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
    const dim3 grid(static_cast<unsigned>(rows / 128 * p.blocks)), block(kTileThreads);
    if (format == FP8_E4M3) launch_pdl(block_transpose_kernel<0>, grid, block, 0, as_stream(stream), p);
    else launch_pdl(block_transpose_kernel<1>, grid, block, 0, as_stream(stream), p);
    return launch_status(what);
}

}  // extern "C"

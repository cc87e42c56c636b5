// norm.cu -- the norms around a block, fused with its gate and residual scale.
//
//   p  = N(h; w_post, b_post), or h            the block's output, normed or not
//   x' = alpha x + gate * p                    the residual stream
//   y  = N(x'; w_pre, b_pre)                   the next block's input, as bf16
//                                              and / or as FP8 codes
//   N(v; w, b) = w (v - m) r + b,  r = 1 / sqrt(mean((v - m)^2) + eps),
//   m = mean(v) (layer norm) or 0 (RMS norm)
//
// The forward reads x and h once and writes x' and y once: a row stays in
// registers between the two norms' statistics.  Everything between the loads
// and the stores is fp32: y comes from the unrounded x', and each output is
// rounded once.  The variance is the mean of squared distances from the mean
// (a second reduction over the registers), which does not cancel.
#include <cfloat>
#include <climits>
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/fp8linear.h"
#include "hostops.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowops.cuh"

namespace fp8 {

// Sets n 32-bit words to zero (an amax before the kernel that raises it).
__global__ void zero_words_kernel(uint32_t* p, int n) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    for (int i = threadIdx.x; i < n; i += blockDim.x) p[i] = 0u;
}

void launch_zero_words(void* p, int n, cudaStream_t stream) {
    launch_pdl(zero_words_kernel, dim3(1), dim3(32), 0, stream, static_cast<uint32_t*>(p), n);
}

namespace {

constexpr int64_t kMaxWidth = 16384;   // a row in the registers of 1024 threads
constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1025;   // row numbers, and a batch more, in 32 bits

struct NormFwd {
    const void* x;
    const __nv_bfloat16* h;
    const __nv_bfloat16* gate;
    const float *w_post, *b_post, *w_pre, *b_pre;
    void* x_out;
    __nv_bfloat16* y;
    uint8_t* q;
    const float* q_scale;
    float* q_scale_inv;
    float* amax;
    float* stats;
    int64_t rows, width, rows_per_gate;
    float alpha, eps;
    int post, q_fmt, q_rows, pow2;
};

// Sum of N values over the threads of a row: a warp, or the CTA.
template <bool WARP, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* part, int& turn) {
    if constexpr (WARP) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = row::warp_sum(v[i]);
    } else {
        row::block_sum<N>(v, part + (turn & 1) * 64);
        ++turn;
    }
}

template <bool WARP>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float* part, int& turn) {
    v = __reduce_max_sync(row::kAll, v);
    if constexpr (!WARP) {
        uint32_t* p = reinterpret_cast<uint32_t*>(part + (turn & 1) * 64);
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) p[warp] = v;
        __syncthreads();
        v = __reduce_max_sync(row::kAll, lane < static_cast<int>(blockDim.x >> 5) ? p[lane] : 0u);
        ++turn;
    }
    return v;
}

// A thread's eight elements of a piece: VEC, the 16 bytes at p (fp32: 32).
// Otherwise, for rows that do not start on 16 bytes, the n elements at p,
// p + step, ... (step: the threads of a row, so that a warp's loads are
// contiguous), zeros after them.
template <bool VEC>
__device__ __forceinline__ void load8(float (&v)[8], const __nv_bfloat16* p, int n, int step) {
    if constexpr (VEC) {
        row::unpack8(v, row::ld_stream(p));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? __bfloat162float(p[e * step]) : 0.0f;
    }
}

template <bool VEC>
__device__ __forceinline__ void load8(float (&v)[8], const float* p, int n, int step) {
    if constexpr (VEC) {
        const uint4 a = row::ld_stream(p), b = row::ld_stream(p + 4);
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
        v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
        v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e * step] : 0.0f;
    }
}

// The same where `on`, zeros elsewhere.
template <bool VEC, typename T>
__device__ __forceinline__ void load8(float (&v)[8], const T* p, int n, int step, bool on) {
    if (on) {
        load8<VEC>(v, p, n, step);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    }
}

// The same through L1, for the vectors that every row shares.
template <bool VEC, typename T>
__device__ __forceinline__ void shared8(float (&v)[8], const T* p, int n, int step) {
    if constexpr (VEC) {
        row::f2 t[4];
        row::shared_pairs(t, p);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = row::lo2(t[e]);
            v[2 * e + 1] = row::hi2(t[e]);
        }
    } else {
        load8<false>(v, p, n, step);
    }
}

__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8], int n, int step) {
    if constexpr (VEC) {
        const row::f2 t[4] = {row::mk2(v[0], v[1]), row::mk2(v[2], v[3]), row::mk2(v[4], v[5]),
                              row::mk2(v[6], v[7])};
        row::store_pairs(p, t);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) store1(p + e * step, v[e]);
    }
}

// First column of piece i of thread `at` of a row's `lanes` threads, and how
// many of its elements lie in the row.
template <bool VEC>
__device__ __forceinline__ int piece_col(int at, int i, int lanes) {
    return VEC ? 8 * (at + i * lanes) : at + 8 * i * lanes;
}
template <bool VEC>
__device__ __forceinline__ int piece_len(int col, int lanes, int64_t width) {
    const int left = static_cast<int>(width) - col;
    if (left <= 0) return 0;
    return min(8, VEC ? left : (left + lanes - 1) / lanes);
}

// Mean (layer norm) and 1/sqrt(variance + eps) of the row whose pieces the
// threads hold; elements past the row are zero in v and left out of the sums.
template <int VPT, bool WARP, bool LAYER>
__device__ __forceinline__ void row_stats(const float (&v)[VPT][8], const int (&n)[VPT], float inv_c,
                                          float eps, float* part, int& turn, float& mean,
                                          float& rstd) {
    mean = 0.0f;
    if constexpr (LAYER) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += v[i][e];
        row_sum<WARP>(s, part, turn);
        mean = s[0] * inv_c;
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = v[i][e] - mean;
            if (e < n[i]) s[0] = fmaf(d, d, s[0]);
        }
    row_sum<WARP>(s, part, turn);
    rstd = 1.0f / sqrtf(s[0] * inv_c + eps);
}

// v = w (v - mean) rstd + b on one piece.
__device__ __forceinline__ void apply_norm(float (&v)[8], const float* w, const float* b, int c,
                                           int n, int step, float mean, float rstd) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (v[e] - mean) * rstd;
    float s[8];
    if (w) {
        shared8<false>(s, w + c, n, step);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= s[e];
    }
    if (b) {
        shared8<false>(s, b + c, n, step);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += s[e];
    }
}

// The forward for rows that do not start on 16 bytes.
template <typename S, int VPT, bool WARP, bool LAYER, int THREADS>
__global__ void __launch_bounds__(THREADS)
    norm_fwd_any_kernel(const __grid_constant__ NormFwd p) {
    ptx::griddep_launch_dependents();
    __shared__ float part[128];
    ptx::griddep_wait();
    const int lanes = WARP ? 32 : static_cast<int>(blockDim.x);
    const int at = WARP ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
    const int64_t r = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)
                           : blockIdx.x;
    if (WARP && r >= p.rows) return;
    int turn = 0;
    const float inv_c = 1.0f / static_cast<float>(p.width);
    const int64_t base = r * p.width;
    const S* xin = static_cast<const S*>(p.x);

    float v[VPT][8], x[VPT][8];
    int n[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = piece_col<false>(at, i, lanes);
        n[i] = piece_len<false>(c, lanes, p.width);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = x[i][e] = 0.0f;
        if (n[i] > 0) {
            if (p.h) load8<false>(v[i], p.h + base + c, n[i], lanes);
            if (xin) load8<false>(x[i], xin + base + c, n[i], lanes);
        }
    }
    float mean_post = 0.0f, rstd_post = 0.0f, mean_pre = 0.0f, rstd_pre = 0.0f;
    if (p.post)
        row_stats<VPT, WARP, LAYER>(v, n, inv_c, p.eps, part, turn, mean_post, rstd_post);
    const __nv_bfloat16* gate =
        p.gate ? p.gate + (r / p.rows_per_gate) * p.width : nullptr;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = piece_col<false>(at, i, lanes);
        if (n[i] <= 0) continue;
        if (p.post) apply_norm(v[i], p.w_post, p.b_post, c, n[i], lanes, mean_post, rstd_post);
        if (gate) {
            float g[8];
            shared8<false>(g, gate + c, n[i], lanes);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[i][e] = e < n[i] ? fmaf(p.alpha, x[i][e], v[i][e]) : 0.0f;
        if (p.x_out) store8<false>(static_cast<S*>(p.x_out) + base + c, v[i], n[i], lanes);
    }
    if (p.y || p.q || p.stats)
        row_stats<VPT, WARP, LAYER>(v, n, inv_c, p.eps, part, turn, mean_pre, rstd_pre);
    if (p.stats && at == 0) {
        p.stats[r] = mean_post;
        p.stats[p.rows + r] = rstd_post;
        p.stats[2 * p.rows + r] = mean_pre;
        p.stats[3 * p.rows + r] = rstd_pre;
    }
    if (!p.y && !p.q) return;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = piece_col<false>(at, i, lanes);
        if (n[i] <= 0) continue;
        apply_norm(v[i], p.w_pre, p.b_pre, c, n[i], lanes, mean_pre, rstd_pre);
        if (p.y) store8<false>(p.y + base + c, v[i], n[i], lanes);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n[i]) top = max(top, row::abs_bits(v[i][e]));
    }
    if (!p.q) return;
    float s = 1.0f;
    if (p.q_rows || p.amax) top = row_max<WARP>(top, part, turn);
    if (p.q_rows) {
        s = row::block_scale(top, p.q_fmt, p.pow2);
        if (at == 0) p.q_scale_inv[r] = __fdiv_rn(1.0f, s);
    } else {
        s = p.q_scale[0];
        if (p.amax && at == 0) row::raise_amax(p.amax, top);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = piece_col<false>(at, i, lanes);
        if (n[i] <= 0) continue;
        const uint2 code = row::cvt8(p.q_fmt, v[i], s);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n[i])
                p.q[base + c + e * lanes] = static_cast<uint8_t>((e < 4 ? code.x : code.y) >> (8 * (e & 3)));
    }
}

// HAS of the resident kernels says at compile time which parts there are, for the usual calls: a row
// is then one stretch of code in which loads move ahead of their uses, where
// tests between them would hold them back.  0: all tested as the kernel runs.
constexpr int kHasAll = 1;    // forward: x, h, x', w_pre; backward: dy, x', dx', h, dx,
                              // dh, w_pre; whole rows (every thread's pieces
                              // lie within the row); the other parts by bits
constexpr int kHasPost = 2;   // with w_post
constexpr int kHasGate = 4;

// The forward for rows in 16-byte pieces: CTAs stay
// on the SM and walk the rows, each thread on its own columns, with the
// vectors of those columns in registers (RMS norm) and the next row's pieces
// loaded while the current row is reduced -- a row's loads cover the two
// reductions' latency.  WARP: a warp a row, else the CTA.
template <typename S, int VPT, bool WARP, bool LAYER, int THREADS, int HAS>
__global__ void __launch_bounds__(THREADS)
    norm_fwd_kernel(const __grid_constant__ NormFwd p) {
    using row::f2;
    ptx::griddep_launch_dependents();
    // sums: two buffers of 16 warps' values; the row maximum has its own
    __shared__ __align__(16) float part[2][16];
    __shared__ float part_max[128];
    constexpr bool KEEP = !LAYER && VPT <= 2;   // the vectors before the second norm
    constexpr bool KEEP_PRE = VPT <= 2;         // and its own
    constexpr bool ALL = (HAS & kHasAll) != 0;
    const bool has_h = ALL || p.h, has_x = ALL || p.x, has_x_out = ALL || p.x_out;
    const bool has_w_pre = ALL || p.w_pre;
    const bool post = ALL ? (HAS & kHasPost) != 0 : p.post != 0;
    const bool has_w_post = ALL ? (HAS & kHasPost) != 0 : p.w_post != nullptr;
    const bool gated = ALL ? (HAS & kHasGate) != 0 : p.gate != nullptr;
    if (!WARP && threadIdx.x < 32) part[threadIdx.x >> 4][threadIdx.x & 15] = 0.0f;
    if (!WARP) __syncthreads();
    const int lanes = WARP ? 32 : static_cast<int>(blockDim.x);
    const int at = WARP ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
    const int64_t stride = WARP ? static_cast<int64_t>(gridDim.x) * (THREADS / 32) : gridDim.x;
    int64_t r = WARP ? static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5)
                     : blockIdx.x;
    ptx::griddep_wait();
    if (r >= p.rows) return;
    int turn = 0, turn_max = 0;
    auto sum = [&](float (&s)[1]) {
        if constexpr (WARP) {
            s[0] = row::warp_sum(s[0]);
        } else {
            row::block_sum16<1>(s, part[turn]);
            turn ^= 1;
        }
    };
    const float inv_c = 1.0f / static_cast<float>(p.width);
    const S* xin = static_cast<const S*>(p.x);
    bool live[VPT];
    int col[VPT];
    row::Raw8<__nv_bfloat16> hn[VPT];
    row::Raw8<S> xn[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        col[i] = 8 * (at + i * lanes);
        live[i] = ALL || col[i] < p.width;
        hn[i].zero();
        xn[i].zero();
        if (live[i]) {
            if (has_h) hn[i].load(p.h + r * p.width + col[i]);
            if (has_x) xn[i].load(xin + r * p.width + col[i]);
        }
    }
    f2 wg[KEEP ? VPT : 1][4];   // w_post * gate
    f2 wp[KEEP_PRE ? VPT : 1][4], bp[KEEP_PRE && LAYER ? VPT : 1][4];   // w_pre, b_pre
    int64_t group = 0, group_end = 0;   // the gate row in use and the row after its last
    const bool scaled = has_w_post || gated;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (!KEEP_PRE || !live[i]) continue;
        if (has_w_pre) row::shared_pairs(wp[KEEP_PRE ? i : 0], p.w_pre + col[i]);
        if constexpr (LAYER) {
            if (p.b_pre) row::shared_pairs(bp[KEEP_PRE ? i : 0], p.b_pre + col[i]);
        }
    }
    const f2 alpha = row::all2(p.alpha);
    for (; r < p.rows; r += stride) {
        const int64_t base = r * p.width;
        if (r >= group_end) {
            group = r / p.rows_per_gate;
            group_end = (group + 1) * p.rows_per_gate;
            if (KEEP && scaled) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    if (!live[i]) continue;
                    if (has_w_post) row::shared_pairs(wg[KEEP ? i : 0], p.w_post + col[i]);
                    if (gated) {
                        f2 t[4];
                        row::shared_pairs(t, p.gate + group * p.width + col[i]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) wg[i][e] = has_w_post ? row::mul2(wg[i][e], t[e]) : t[e];
                    }
                }
            }
        }
        f2 v[VPT][4];
        row::Raw8<S> x[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            hn[i].pairs(v[i]);
            x[i] = xn[i];
        }
        if (r + stride < p.rows) {
            const int64_t next = base + stride * p.width;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (!live[i]) continue;
                if (has_h) hn[i].load(p.h + next + col[i]);
                if (has_x) xn[i].load(xin + next + col[i]);
            }
        }
        auto stats = [&](float& mean, float& rstd) {
            mean = 0.0f;
            if constexpr (LAYER) {
                f2 a = 0;
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) a = row::add2(a, v[i][e]);
                float s[1] = {row::lo2(a) + row::hi2(a)};
                sum(s);
                mean = s[0] * inv_c;
            }
            f2 a = 0;
            const f2 m = row::all2(-mean);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                f2 b = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f2 d = LAYER ? row::add2(v[i][e], m) : v[i][e];
                    b = row::fma2(d, d, b);
                }
                if (!LAYER || live[i]) a = row::add2(a, b);   // past the row v is 0, v - mean is not
            }
            float s[1] = {row::lo2(a) + row::hi2(a)};
            sum(s);
            rstd = rsqrtf(s[0] * inv_c + p.eps);
        };
        float mean_post = 0.0f, rstd_post = 0.0f, mean_pre = 0.0f, rstd_pre = 0.0f;
        if (post) stats(mean_post, rstd_post);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            f2 xs[4];
            x[i].pairs(xs);
            if (!live[i]) continue;
            if constexpr (KEEP) {
                const f2 rs = row::all2(post ? rstd_post : 1.0f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (scaled) v[i][e] = row::mul2(v[i][e], wg[i][e]);
                    v[i][e] = row::fma2(v[i][e], rs, row::mul2(xs[e], alpha));
                }
            } else {
                f2 t[4];
                if (post) {
                    const f2 m = row::all2(-mean_post), rs = row::all2(rstd_post);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[i][e] = row::mul2(row::add2(v[i][e], m), rs);
                    if (has_w_post) {
                        row::shared_pairs(t, p.w_post + col[i]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[i][e] = row::mul2(v[i][e], t[e]);
                    }
                    if (p.b_post) {
                        row::shared_pairs(t, p.b_post + col[i]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[i][e] = row::add2(v[i][e], t[e]);
                    }
                }
                if (gated) {
                    row::shared_pairs(t, p.gate + group * p.width + col[i]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[i][e] = row::mul2(v[i][e], t[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] = row::fma2(xs[e], alpha, v[i][e]);
            }
            if (has_x_out) row::store_pairs(static_cast<S*>(p.x_out) + base + col[i], v[i]);
        }
        if (p.y || p.q || p.stats) stats(mean_pre, rstd_pre);
        if (p.stats && at == 0) {
            p.stats[r] = mean_post;
            p.stats[p.rows + r] = rstd_post;
            p.stats[2 * p.rows + r] = mean_pre;
            p.stats[3 * p.rows + r] = rstd_pre;
        }
        if (!p.y && !p.q) continue;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (!live[i]) continue;
            const f2 rs = row::all2(rstd_pre), m = row::all2(-mean_pre);
            const int kept = KEEP_PRE ? i : 0;
            if constexpr (!KEEP_PRE) {
                if (has_w_pre) row::shared_pairs(wp[0], p.w_pre + col[i]);
                if (LAYER && p.b_pre) row::shared_pairs(bp[0], p.b_pre + col[i]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (LAYER) v[i][e] = row::add2(v[i][e], m);
                v[i][e] = row::mul2(v[i][e], rs);
                if (has_w_pre) v[i][e] = row::mul2(v[i][e], wp[kept][e]);
                if constexpr (LAYER) {
                    if (p.b_pre) v[i][e] = row::add2(v[i][e], bp[kept][e]);
                }
            }
            if (p.y) row::store_pairs(p.y + base + col[i], v[i]);
        }
        if (!p.q) continue;
        float s = 1.0f;
        if (p.q_rows || p.amax) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (!live[i]) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    m = row::max_abs(row::max_abs(m, row::lo2(v[i][e])), row::hi2(v[i][e]));
            }
            const uint32_t top = row_max<WARP>(row::abs_bits(m), part_max, turn_max);
            if (p.q_rows) {
                s = row::block_scale(top, p.q_fmt, p.pow2);
                if (at == 0) p.q_scale_inv[r] = __fdiv_rn(1.0f, s);
            } else if (at == 0) {
                row::raise_amax(p.amax, top);
            }
        }
        if (!p.q_rows) s = p.q_scale[0];
        const f2 ss = row::all2(s);
        // the format is tested once: a test a pair would convert to both
        auto codes = [&](auto fmt) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (live[i])
                    *reinterpret_cast<uint2*>(p.q + base + col[i]) = row::cvt8<decltype(fmt)::value>(v[i], ss);
        };
        if (p.q_fmt == FP8_E4M3) codes(std::integral_constant<int, 0>{});
        else codes(std::integral_constant<int, 1>{});
    }
}

// Rows in 16-byte pieces up to here: 512 threads with two pieces each and 128
// registers a thread.
constexpr int64_t kFastWidth = 8192;

template <typename S, bool LAYER>
void launch_fwd(const NormFwd& p, cudaStream_t st) {
    const int64_t pieces = (p.width + 7) / 8;
    const int threads = static_cast<int>(((pieces + 1) / 2 + 31) / 32 * 32);
    if (p.width % 8 == 0 && p.width <= kFastWidth) {
        // up to 512 columns a warp holds a row, without a CTA barrier
        const bool warp = pieces <= 64;
        const int64_t per_sm = warp ? 2 : 512 / threads;
        const int64_t want = warp ? (p.rows + 7) / 8 : p.rows, most = num_sms() * per_sm;
        const dim3 grid(static_cast<unsigned>(want < most ? want : most));
        if (pieces <= 32) {
            launch_pdl(norm_fwd_kernel<S, 1, true, LAYER, 256, 0>, grid, dim3(256), 0, st, p);
            return;
        }
        if (warp) {
            launch_pdl(norm_fwd_kernel<S, 2, true, LAYER, 256, 0>, grid, dim3(256), 0, st, p);
            return;
        }
        if (p.x && p.h && p.x_out && p.w_pre && (!p.post || p.w_post) && p.width == 16 * threads) {
            constexpr int A = kHasAll, P = kHasPost, G = kHasGate;
            if (p.post && p.gate)
                launch_pdl(norm_fwd_kernel<S, 2, false, LAYER, 512, A | P | G>, grid, dim3(threads), 0, st, p);
            else if (p.post)
                launch_pdl(norm_fwd_kernel<S, 2, false, LAYER, 512, A | P>, grid, dim3(threads), 0, st, p);
            else if (p.gate)
                launch_pdl(norm_fwd_kernel<S, 2, false, LAYER, 512, A | G>, grid, dim3(threads), 0, st, p);
            else
                launch_pdl(norm_fwd_kernel<S, 2, false, LAYER, 512, A>, grid, dim3(threads), 0, st, p);
            return;
        }
        launch_pdl(norm_fwd_kernel<S, 2, false, LAYER, 512, 0>, grid, dim3(threads), 0, st, p);
        return;
    }
    if (p.width % 8 == 0) {
        // wider rows: four pieces a thread, all vectors through L1
        const int t4 = static_cast<int>(((pieces + 3) / 4 + 31) / 32 * 32);
        const dim3 grid(static_cast<unsigned>(p.rows < num_sms() ? p.rows : num_sms()));
        launch_pdl(norm_fwd_kernel<S, 4, false, LAYER, 512, 0>, grid, dim3(t4), 0, st, p);
    } else if (pieces <= 64) {
        launch_pdl(norm_fwd_any_kernel<S, 2, true, LAYER, 256>,
                   dim3(static_cast<unsigned>((p.rows + 7) / 8)), dim3(256), 0, st, p);
    } else if (threads <= 512) {
        launch_pdl(norm_fwd_any_kernel<S, 2, false, LAYER, 512>,
                   dim3(static_cast<unsigned>(p.rows)), dim3(threads), 0, st, p);
    } else {
        launch_pdl(norm_fwd_any_kernel<S, 2, false, LAYER, 1024>,
                   dim3(static_cast<unsigned>(p.rows)), dim3(threads), 0, st, p);
    }
}

// ------------------------------------------------------------------ backward

// With g = w_pre dy, u = (x' - m) r and the norm's own gradient
//   D(g, u, r) = r (g - mean(g) - u mean(g u))     (RMS: without mean(g))
//   dX = dx' + D(g, u, r_pre)        the gradient of x' from both its uses
//   dx = alpha dX
//   dgate = sum dX p,  dp = gate dX
//   dh = D(w_post dp, hh, r_post), hh = (h - m_post) r_post     (or dp)
//   dw_pre = sum dy u,  db_pre = sum dy,  dw_post = sum dp hh,  db_post = sum dp
// One pass: a row is read once and both its norms' reductions run on the
// registers.  The sums over rows stay in registers (each thread owns its
// columns), one partial row a CTA at the end, added up by a second kernel in
// a fixed order.
struct NormBwd {
    const __nv_bfloat16* dy;
    const void* x_out;
    const void* dx_out;
    const __nv_bfloat16* h;
    const __nv_bfloat16* gate;
    const float *w_post, *b_post, *w_pre;
    const float* stats;
    void* dx;
    __nv_bfloat16* dh;
    float* dw_part;      // [4][ctas][width]: dw_pre, db_pre, dw_post, db_post
    float* dgate_part;   // [groups * parts][width], or dgate itself with one part
    int64_t rows, width, groups, parts;
    float alpha;
    int post, add_dgate;
    unsigned* status;
};

struct BwdPlan {
    bool warp;
    int vpt, threads, per_sm, ctas;
    int64_t groups, parts;
    size_t dw_floats, dgate_floats;
};

// Rows are cut into chunks that lie within one group of the gate: parts
// chunks a group, so that the chunks fill the grid once.
BwdPlan bwd_plan(int64_t rows, int64_t width, int64_t gate_rows) {
    BwdPlan b{};
    const int64_t pieces = (width + 7) / 8;
    b.warp = pieces <= 64;
    b.vpt = pieces <= 32 ? 1 : 2;
    b.threads = b.warp ? 256 : static_cast<int>(((pieces + 1) / 2 + 31) / 32 * 32);
    b.per_sm = b.warp ? 2 : (b.threads >= 512 ? 1 : 512 / b.threads);
    const int64_t target = num_sms() * b.per_sm;
    b.groups = gate_rows > 0 ? gate_rows : 1;
    const int64_t in_group = rows / b.groups;
    b.parts = b.groups >= target ? 1 : target / b.groups;
    if (b.warp && b.parts > (in_group + 7) / 8) b.parts = (in_group + 7) / 8;
    if (b.parts > in_group) b.parts = in_group;
    if (b.parts < 1) b.parts = 1;
    const int64_t chunks = b.groups * b.parts;
    b.ctas = rows == 0 ? 0 : static_cast<int>(chunks < target ? chunks : target);
    b.dw_floats = static_cast<size_t>(4) * b.ctas * width;
    b.dgate_floats = gate_rows > 0 && b.parts > 1 ? static_cast<size_t>(chunks) * width : 0;
    return b;
}

// Adds the CTA's rows of one accumulator (WARP: its eight warps' first) and
// writes the result to `out`; `add` adds to what is there.
template <int VPT, bool WARP, bool VEC>
__device__ __forceinline__ void flush(const float (&acc)[VPT][8], const int (&n)[VPT], int at,
                                      int lanes, int64_t width, float* out, bool add, float* buf) {
    if constexpr (WARP) {
        const int warp = threadIdx.x >> 5;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                buf[warp * 512 + piece_col<VEC>(at, i, 32) + (VEC ? e : e * 32)] = acc[i][e];
        __syncthreads();
        for (int64_t c = threadIdx.x; c < width; c += blockDim.x) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) s += buf[w * 512 + c];
            out[c] = add ? out[c] + s : s;
        }
    } else {
        const int step = VEC ? 1 : lanes;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (n[i] <= 0) continue;
            float* o = out + piece_col<VEC>(at, i, lanes);
            if (VEC && add) {
                float4* q = reinterpret_cast<float4*>(o);
                float4 a = q[0], b = q[1];
                a.x += acc[i][0]; a.y += acc[i][1]; a.z += acc[i][2]; a.w += acc[i][3];
                b.x += acc[i][4]; b.y += acc[i][5]; b.z += acc[i][6]; b.w += acc[i][7];
                q[0] = a;
                q[1] = b;
            } else if (add) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n[i]) o[e * step] += acc[i][e];
            } else {
                store8<VEC>(o, acc[i], n[i], lanes);
            }
        }
    }
}

// The gate is one row within a chunk, so with A = sum dX hh and B = sum dX over
// the chunk's rows  dgate = w_post A + b_post B,  dw_post = sum of gate A  and
// db_post = sum of gate B  over the chunks: one pair of running sums serves
// the gate's and the post norm's gradients.
//
// This kernel takes rows wider than kFastWidth (4096 x 16384: 288 us; its sums
// spill, 800 to 3712 bytes at 64 registers a thread and fewer), the resident one
// below the others.
template <typename S, bool VEC, bool LAYER>
__global__ void __launch_bounds__(1024)
    norm_bwd_any_kernel(const __grid_constant__ NormBwd p) {
    ptx::griddep_launch_dependents();
    __shared__ float part[128];
    ptx::griddep_wait();
    constexpr int VPT = 2;
    const int lanes = static_cast<int>(blockDim.x), at = static_cast<int>(threadIdx.x);
    const float inv_c = 1.0f / static_cast<float>(p.width);
    int turn = 0;

    float dw_pre[VPT][8], sum_a[VPT][8], db_pre[LAYER ? VPT : 1][8], sum_b[LAYER ? VPT : 1][8];
    int n[VPT], col[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        col[i] = piece_col<VEC>(at, i, lanes);
        n[i] = piece_len<VEC>(col[i], lanes, p.width);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw_pre[i][e] = sum_a[i][e] = 0.0f;
            if constexpr (LAYER) db_pre[i][e] = sum_b[i][e] = 0.0f;
        }
    }
    auto sum = [&](float (&s)[2]) {
        if constexpr (LAYER) {
            row_sum<false>(s, part, turn);
        } else {
            float t[1] = {s[0]};
            row_sum<false>(t, part, turn);
            s[0] = t[0];
            s[1] = 0.0f;
        }
    };
    const int64_t rows_of = static_cast<int64_t>(gridDim.x) * p.width;
    float* const my_sums = p.dw_part + static_cast<int64_t>(blockIdx.x) * p.width;

    const int64_t chunks = p.groups * p.parts, in_group = p.rows / p.groups;
    for (int64_t k = blockIdx.x; k < chunks; k += gridDim.x) {
        const int64_t group = k / p.parts, part_no = k % p.parts;
        const int64_t begin = group * in_group + part_no * in_group / p.parts;
        const int64_t end = group * in_group + (part_no + 1) * in_group / p.parts;
        const __nv_bfloat16* gate = p.gate ? p.gate + group * p.width : nullptr;
        for (int64_t r = begin; r < end; ++r) {
            const int64_t base = r * p.width;
            float d[VPT][8], u[VPT][8];
            float m_post = 0.0f, r_post = 1.0f;
            if (p.post) {
                m_post = LAYER ? p.stats[r] : 0.0f;
                r_post = p.stats[p.rows + r];
            }
            if (p.dy) {
                const float m_pre = LAYER ? p.stats[2 * p.rows + r] : 0.0f;
                const float r_pre = p.stats[3 * p.rows + r];
                float s[2] = {0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    load8<VEC>(d[i], p.dy + base + col[i], n[i], lanes, n[i] > 0);
                    load8<VEC>(u[i], static_cast<const S*>(p.x_out) + base + col[i], n[i], lanes, n[i] > 0);
                }
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    if (n[i] <= 0) continue;
                    float w[8];
                    if (p.w_pre) shared8<VEC>(w, p.w_pre + col[i], n[i], lanes);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        u[i][e] = VEC || e < n[i] ? (u[i][e] - m_pre) * r_pre : 0.0f;
                        dw_pre[i][e] = fmaf(d[i][e], u[i][e], dw_pre[i][e]);
                        if constexpr (LAYER) db_pre[i][e] += d[i][e];
                        if (p.w_pre) d[i][e] *= w[e];
                        s[0] = fmaf(d[i][e], u[i][e], s[0]);
                        s[1] += d[i][e];
                    }
                }
                float o[VPT][8];   // on its way while the row is summed
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    load8<VEC>(o[i], static_cast<const S*>(p.dx_out) + base + col[i], n[i], lanes,
                               p.dx_out && n[i] > 0);
                sum(s);
                const float su = s[0] * inv_c, sg = s[1] * inv_c;
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        d[i][e] = fmaf(r_pre, d[i][e] - sg - u[i][e] * su, o[i][e]);
            } else {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    load8<VEC>(d[i], static_cast<const S*>(p.dx_out) + base + col[i], n[i], lanes,
                               p.dx_out && n[i] > 0);
            }
            // d is dX (columns past the row hold values that no one uses); u
            // becomes the block's output, normed
            if (p.h) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    load8<VEC>(u[i], p.h + base + col[i], n[i], lanes, n[i] > 0);
            }
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (n[i] <= 0) continue;
                if (p.dx) {
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = p.alpha * d[i][e];
                    store8<VEC>(static_cast<S*>(p.dx) + base + col[i], o, n[i], lanes);
                }
                if (!p.h) continue;
                if (p.post) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[i][e] = (u[i][e] - m_post) * r_post;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sum_a[i][e] = fmaf(d[i][e], u[i][e], sum_a[i][e]);
                    if constexpr (LAYER) sum_b[i][e] += d[i][e];
                }
                float w[8];
                if (gate) {
                    shared8<VEC>(w, gate + col[i], n[i], lanes);
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[i][e] *= w[e];
                }
                if (p.post) {
                    if (p.w_post) shared8<VEC>(w, p.w_post + col[i], n[i], lanes);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (p.w_post) d[i][e] *= w[e];
                        if (!VEC && e >= n[i]) d[i][e] = 0.0f;
                        s[0] = fmaf(d[i][e], u[i][e], s[0]);
                        s[1] += d[i][e];
                    }
                }
            }
            if (!p.h) continue;
            if (p.post) sum(s);
            const float sh = s[0] * inv_c, sq = s[1] * inv_c;
            if (p.dh) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    if (n[i] <= 0) continue;
                    if (p.post) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            d[i][e] = r_post * (d[i][e] - sq - u[i][e] * sh);
                    }
                    store8<VEC>(p.dh + base + col[i], d[i], n[i], lanes);
                }
            }
        }
        if (!gate) continue;
        // the end of a chunk: its part of dgate, and of the post norm's sums
        if (p.dgate_part) {
            float t[VPT][8];
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float w[8], b[8];
                const bool on = n[i] > 0 && p.post;
                if (on && p.w_post) shared8<VEC>(w, p.w_post + col[i], n[i], lanes);
                if (on && p.b_post) shared8<VEC>(b, p.b_post + col[i], n[i], lanes);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    t[i][e] = on && p.w_post ? sum_a[i][e] * w[e] : sum_a[i][e];
                    if constexpr (LAYER) {
                        if (on && p.b_post) t[i][e] = fmaf(sum_b[i][e], b[e], t[i][e]);
                    }
                }
            }
            flush<VPT, false, VEC>(t, n, at, lanes, p.width, p.dgate_part + k * p.width,
                                  p.add_dgate != 0, nullptr);
        }
        if (p.post) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (n[i] <= 0) continue;
                float w[8];
                shared8<VEC>(w, gate + col[i], n[i], lanes);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sum_a[i][e] *= w[e];
                    if constexpr (LAYER) sum_b[i][e] *= w[e];
                }
            }
            const bool add = k != blockIdx.x;
            flush<VPT, false, VEC>(sum_a, n, at, lanes, p.width, my_sums + 2 * rows_of, add, nullptr);
            if constexpr (LAYER)
                flush<VPT, false, VEC>(sum_b, n, at, lanes, p.width, my_sums + 3 * rows_of, add, nullptr);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sum_a[i][e] = 0.0f;
                if constexpr (LAYER) sum_b[i][e] = 0.0f;
            }
    }
    flush<VPT, false, VEC>(dw_pre, n, at, lanes, p.width, my_sums, false, nullptr);
    if constexpr (LAYER) flush<VPT, false, VEC>(db_pre, n, at, lanes, p.width, my_sums + rows_of, false, nullptr);
    if (!p.gate) {
        flush<VPT, false, VEC>(sum_a, n, at, lanes, p.width, my_sums + 2 * rows_of, false, nullptr);
        if constexpr (LAYER)
            flush<VPT, false, VEC>(sum_b, n, at, lanes, p.width, my_sums + 3 * rows_of, false, nullptr);
    }
}

// The backward up to kFastWidth columns.  The rows come
// through a ring of shared-memory stages, filled by bulk copies one or
// two batches ahead (a batch is a row, or the eight rows of a CTA's warps:
// consecutive in memory, so four copies), because the column sums leave no
// registers to hold a row ahead.  8192 x 4096 bf16 with both norms and a gate
// per sequence: 67 us (6.0 TB/s) and 8 us for the sums' kernel; loads straight
// into registers took 146.  A stage is read piece by piece as the row
// needs it, and filled again once every thread is past its last read.  The layer
// norm's two more running sums spill over a CTA's rows (144 to 376 bytes at 128
// registers; up to 616 at other widths).
// VEC: rows in 16-byte pieces.  Others start anywhere: a copy takes the 16-byte
// pieces around them (cut at the tensor's end, whose last elements are then
// read from global memory), and a thread's columns are a row's threads apart.
struct BwdRing {
    int stages;
    uint32_t x_at, dxo_at, h_at, stage_bytes;   // dy at 0
    uint32_t sums_at;   // the post norm's running sums behind the stages, or 0: in dw_part
};

template <typename S, int VPT, bool WARP, bool VEC, bool LAYER, int THREADS, int HAS>
__global__ void __launch_bounds__(THREADS)
    norm_bwd_kernel(const __grid_constant__ NormBwd p, const __grid_constant__ BwdRing ring) {
    using row::f2;
    ptx::griddep_launch_dependents();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) float part[2][32];
    __shared__ float buf[WARP ? 8 * 512 : 1];
    __shared__ uint64_t full[8];
    __shared__ volatile uint32_t gave_up;
    constexpr int BATCH = WARP ? 8 : 1;   // rows
    constexpr bool ALL = (HAS & kHasAll) != 0;
    const bool has_dy = ALL || p.dy, has_dxo = ALL || p.dx_out, has_h = ALL || p.h;
    const bool has_dx = ALL || p.dx, has_dh = ALL || p.dh, has_w_pre = ALL || p.w_pre;
    const bool post = ALL ? (HAS & kHasPost) != 0 : p.post != 0;
    const bool has_w_post = ALL ? (HAS & kHasPost) != 0 : p.w_post != nullptr;
    const bool gated = ALL ? (HAS & kHasGate) != 0 : p.gate != nullptr;
    const int lanes = WARP ? 32 : static_cast<int>(blockDim.x);
    const int at = WARP ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
    const int own = WARP ? static_cast<int>(threadIdx.x >> 5) : 0;   // this thread's row of a batch
    if (threadIdx.x < 64) part[threadIdx.x >> 5][threadIdx.x & 31] = 0.0f;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ring.stages; ++i) ptx::mbar_init(&full[i], 1);
        gave_up = 0;
        ptx::fence_barrier_init();
    }
    __syncthreads();
    ptx::griddep_wait();

    const int chunks = static_cast<int>(p.groups * p.parts);
    const int parts = static_cast<int>(p.parts), in_group = static_cast<int>(p.rows / p.groups);
    // the CTA's batches in order: rows [r, end) of chunk k (no chunk is empty)
    struct Walk {
        int k, r, end;
    };
    auto enter = [&](Walk& w) {
        if (w.k >= chunks) return;
        const int g = w.k / parts, i = w.k - g * parts;
        w.r = g * in_group + static_cast<int>(static_cast<int64_t>(i) * in_group / parts);
        w.end = g * in_group + static_cast<int>(static_cast<int64_t>(i + 1) * in_group / parts);
    };
    auto next = [&](Walk& w) {
        w.r += BATCH;
        if (w.r >= w.end) {
            w.k += gridDim.x;
            enter(w);
        }
    };
    Walk ahead{static_cast<int>(blockIdx.x), 0, 0};
    uint32_t issued = 0;
    auto fill = [&]() {   // thread 0: copy the next batch of rows into its stage
        const uint32_t n = static_cast<uint32_t>(min(ahead.end - ahead.r, BATCH)) * static_cast<uint32_t>(p.width);
        uint8_t* to = smem + (issued % ring.stages) * ring.stage_bytes;
        uint64_t* bar = &full[issued % ring.stages];
        const int64_t first = static_cast<int64_t>(ahead.r) * p.width, all = p.rows * p.width;
        // the bytes of n elements of `size` from the first on, in whole pieces
        auto from = [&](uint32_t size) { return first * size & (VEC ? ~int64_t{0} : ~int64_t{15}); };
        auto bytes = [&](uint32_t size) -> uint32_t {
            if (VEC) return n * size;
            int64_t end = ((first + n) * size + 15) & ~int64_t{15};
            if (end > all * size) end = all * size & ~int64_t{15};
            return end > from(size) ? static_cast<uint32_t>(end - from(size)) : 0u;
        };
        const uint32_t b2 = bytes(2), bs = bytes(sizeof(S));
        ptx::mbar_arrive_expect_tx(bar, (has_dy ? b2 + bs : 0) + (has_dxo ? bs : 0) + (has_h ? b2 : 0));
        auto load = [&](uint32_t at, const void* t, uint32_t size, uint32_t count) {
            if (count) ptx::bulk_load(to + at, static_cast<const uint8_t*>(t) + from(size), count, bar);
        };
        if (has_dy) {
            load(0, p.dy, 2, b2);
            load(ring.x_at, p.x_out, sizeof(S), bs);
        }
        if (has_dxo) load(ring.dxo_at, p.dx_out, sizeof(S), bs);
        if (has_h) load(ring.h_at, p.h, 2, b2);
        ++issued;
        next(ahead);
    };
    if (threadIdx.x == 0) {
        enter(ahead);
        for (int i = 0; i < ring.stages && ahead.k < chunks; ++i) fill();
    }

    int turn = 0;
    auto sum = [&](float (&v)[2]) {
        if constexpr (WARP) {
            v[0] = row::warp_sum(v[0]);
            if constexpr (LAYER) v[1] = row::warp_sum(v[1]);
        } else if constexpr (LAYER) {
            row::block_sum16<2>(v, part[turn]);
        } else {
            float t[1] = {v[0]};
            row::block_sum16<1>(t, part[turn]);
            v[0] = t[0];
        }
        turn ^= 1;
    };
    const float inv_c = 1.0f / static_cast<float>(p.width);
    f2 dw_pre[VPT][4], sum_a[VPT][4];
    f2 db_pre[LAYER ? VPT : 1][4], sum_b[LAYER ? VPT : 1][4];
    int col[VPT], len[VPT];
    bool live[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        col[i] = piece_col<VEC>(at, i, lanes);
        len[i] = ALL && VEC ? 8 : piece_len<VEC>(col[i], lanes, p.width);
        live[i] = len[i] > 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dw_pre[i][e] = sum_a[i][e] = 0;
            if constexpr (LAYER) db_pre[i][e] = sum_b[i][e] = 0;
        }
    }
    // piece i of a vector that every row shares
    auto vec = [&](f2 (&v)[4], const auto* t, int i) {
        if constexpr (VEC) {
            row::shared_pairs(v, t + col[i]);
        } else {
            float x[8];
            load8<false>(x, t + col[i], len[i], lanes);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = row::mk2(x[2 * e], x[2 * e + 1]);
        }
    };
    // piece i of this thread's row of a batch: `part` is the batch's place in
    // the stage, `in` the row's first element there; elements from `safe` on
    // were not copied and come from `t`, the batch in global memory
    auto piece = [&](f2 (&v)[4], const auto* part, const auto* t, int in, int safe, int i) {
        using T = std::remove_cv_t<std::remove_pointer_t<decltype(part)>>;
        if constexpr (VEC) {
            row::Raw8<T> a;
            a.load_shared(part + in + col[i]);
            a.pairs(v);
        } else {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at_e = in + col[i] + e * lanes;
                x[e] = e >= len[i] ? 0.0f : static_cast<float>(at_e < safe ? part[at_e] : t[at_e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = row::mk2(x[2 * e], x[2 * e + 1]);
        }
    };
    auto put = [&](auto* t, const f2 (&v)[4], int i) {
        if constexpr (VEC) {
            row::store_pairs(t + col[i], v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < len[i]) store1(t + col[i] + e * lanes, e & 1 ? row::hi2(v[e / 2]) : row::lo2(v[e / 2]));
        }
    };
    auto out_sums = [&](const f2 (&acc)[VPT][4], float* out, bool add) {
        float v[VPT][8];
        int n[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            n[i] = len[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[i][2 * e] = row::lo2(acc[i][e]);
                v[i][2 * e + 1] = row::hi2(acc[i][e]);
            }
        }
        flush<VPT, WARP, VEC>(v, n, at, lanes, p.width, out, add, buf);
    };
    const int64_t rows_of = static_cast<int64_t>(gridDim.x) * p.width;
    float* const my_sums = p.dw_part + static_cast<int64_t>(blockIdx.x) * p.width;
    // where the chunks' shares of the post norm's sums meet: a CTA with many
    // chunks (a gate per token) adds them up in shared memory
    float* const post_w = ring.sums_at ? reinterpret_cast<float*>(smem + ring.sums_at) : my_sums + 2 * rows_of;
    float* const post_b = ring.sums_at ? post_w + p.width : my_sums + 3 * rows_of;
    // the end of a chunk: its part of dgate, and of the post norm's sums
    auto end_chunk = [&](const __nv_bfloat16* gate, int64_t k, bool first) {
        f2 t[VPT][4], w[4];
        if (p.dgate_part) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) t[i][e] = sum_a[i][e];
                if (!live[i] || !post) continue;
                if (has_w_post) {
                    vec(w, p.w_post, i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) t[i][e] = row::mul2(t[i][e], w[e]);
                }
                if constexpr (LAYER) {
                    if (p.b_post) {
                        vec(w, p.b_post, i);
#pragma unroll
                        for (int e = 0; e < 4; ++e) t[i][e] = row::fma2(sum_b[i][e], w[e], t[i][e]);
                    }
                }
            }
            out_sums(t, p.dgate_part + k * p.width, p.add_dgate != 0);
        }
        if (post) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (!live[i]) continue;
                vec(w, gate, i);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sum_a[i][e] = row::mul2(sum_a[i][e], w[e]);
                    if constexpr (LAYER) sum_b[i][e] = row::mul2(sum_b[i][e], w[e]);
                }
            }
            out_sums(sum_a, post_w, !first);
            if constexpr (LAYER) out_sums(sum_b, post_b, !first);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum_a[i][e] = 0;
                if constexpr (LAYER) sum_b[i][e] = 0;
            }
    };

    const f2 alpha = row::all2(p.alpha);
    Walk now{static_cast<int>(blockIdx.x), 0, 0};
    enter(now);
    // a row's statistics do not come through the ring: loaded a batch ahead
    float next_stat[4];
    auto load_stats = [&](const Walk& w) {
        next_stat[0] = next_stat[2] = 0.0f;
        next_stat[1] = next_stat[3] = 1.0f;
        const int64_t r = w.r + own;
        if (w.k >= chunks || r >= w.end || (!ALL && !p.stats)) return;
        if (post) {
            if constexpr (LAYER) next_stat[0] = p.stats[r];
            next_stat[1] = p.stats[p.rows + r];
        }
        if constexpr (LAYER) next_stat[2] = p.stats[2 * p.rows + r];
        next_stat[3] = p.stats[3 * p.rows + r];
    };
    load_stats(now);
    uint32_t stage = 0, phase = 0;
    while (now.k < chunks) {
        const __nv_bfloat16* gate = gated ? p.gate + now.k / parts * p.width : nullptr;
        const int k = now.k;
        for (; now.k == k; next(now)) {
            const int64_t r = now.r + own;
            const bool has_row = !WARP || r < now.end;
            const float m_post = next_stat[0], r_post = next_stat[1];
            const float m_pre = next_stat[2], r_pre = next_stat[3];
            Walk then = now;
            next(then);
            load_stats(then);
            ptx::mbar_wait(&full[stage], phase, &gave_up);
            const uint8_t* st = smem + stage * ring.stage_bytes;
            const int64_t base = r * p.width;
            const int in = own * static_cast<int>(p.width);
            // the batch in the stage and in global memory
            const int64_t batch = VEC ? 0 : static_cast<int64_t>(now.r) * p.width, all = p.rows * p.width;
            // elements of the batch before the tensor's last whole 16-byte piece ends
            auto copied = [&](int64_t piece_len16) {
                const int64_t n = (all & ~(piece_len16 - 1)) - batch;
                return n < INT_MAX ? static_cast<int>(n) : INT_MAX;
            };
            const int safe2 = VEC ? 0 : copied(8), safes = VEC ? 0 : copied(16 / sizeof(S));
            const int shift2 = VEC ? 0 : static_cast<int>(batch * 2 & 15);
            const int shifts = VEC ? 0 : static_cast<int>(batch * sizeof(S) & 15);
            const auto* s_dy = reinterpret_cast<const __nv_bfloat16*>(st + shift2);
            const auto* s_x = reinterpret_cast<const S*>(st + ring.x_at + shifts);
            const auto* s_dxo = reinterpret_cast<const S*>(st + ring.dxo_at + shifts);
            const auto* s_h = reinterpret_cast<const __nv_bfloat16*>(st + ring.h_at + shift2);
            const S* g_x = static_cast<const S*>(p.x_out) + batch;
            const S* g_dxo = static_cast<const S*>(p.dx_out) + batch;
            if (has_row) {
                f2 d[VPT][4], u[VPT][4];
                if (has_dy) {
                    f2 s0 = 0, s1 = 0;
                    const f2 rs = row::all2(r_pre), mr = row::all2(-m_pre * r_pre);
#pragma unroll
                    for (int i = 0; i < VPT; ++i) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) d[i][e] = u[i][e] = 0;
                        if (!live[i]) continue;
                        piece(d[i], s_dy, p.dy + batch, in, safe2, i);
                        piece(u[i], s_x, g_x, in, safes, i);
                        f2 w[4];
                        if (has_w_pre) vec(w, p.w_pre, i);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            u[i][e] = LAYER ? row::fma2(u[i][e], rs, mr) : row::mul2(u[i][e], rs);
                            dw_pre[i][e] = row::fma2(d[i][e], u[i][e], dw_pre[i][e]);
                            if constexpr (LAYER) db_pre[i][e] = row::add2(db_pre[i][e], d[i][e]);
                            if (has_w_pre) d[i][e] = row::mul2(d[i][e], w[e]);
                            s0 = row::fma2(d[i][e], u[i][e], s0);
                            if constexpr (LAYER) s1 = row::add2(s1, d[i][e]);
                        }
                    }
                    float s[2] = {row::lo2(s0) + row::hi2(s0), row::lo2(s1) + row::hi2(s1)};
                    sum(s);
                    // dX = dx' + r (g - mean(g) - u mean(g u))
                    const f2 cu = row::all2(-r_pre * (s[0] * inv_c));
                    const f2 cg = row::all2(-r_pre * (s[1] * inv_c));
#pragma unroll
                    for (int i = 0; i < VPT; ++i) {
                        if (!live[i]) continue;
                        f2 o[4];
                        if (has_dxo) {
                            piece(o, s_dxo, g_dxo, in, safes, i);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[e] = 0;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if constexpr (LAYER) o[e] = row::add2(o[e], cg);
                            d[i][e] = row::fma2(d[i][e], rs, row::fma2(u[i][e], cu, o[e]));
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < VPT; ++i) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) d[i][e] = 0;
                        if (!live[i] || !has_dxo) continue;
                        piece(d[i], s_dxo, g_dxo, in, safes, i);
                    }
                }
                // d is dX; u becomes the block's output, normed
                f2 s0 = 0, s1 = 0;
                const f2 rs = row::all2(r_post), mr = row::all2(-m_post * r_post);
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    if (!live[i]) continue;
                    if constexpr (!VEC) {   // elements past the row add to no sum
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            d[i][e] = row::mk2(2 * e < len[i] ? row::lo2(d[i][e]) : 0.0f,
                                               2 * e + 1 < len[i] ? row::hi2(d[i][e]) : 0.0f);
                    }
                    if (has_dx) {
                        f2 o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[e] = row::mul2(d[i][e], alpha);
                        put(static_cast<S*>(p.dx) + base, o, i);
                    }
                    if (!has_h) continue;
                    piece(u[i], s_h, p.h + batch, in, safe2, i);
                    f2 w[4];
                    if (post) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            u[i][e] = LAYER ? row::fma2(u[i][e], rs, mr) : row::mul2(u[i][e], rs);
                        if (has_w_post) vec(w, p.w_post, i);
                    }
                    if (gated) {
                        f2 gt[4];
                        vec(gt, gate, i);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sum_a[i][e] = row::fma2(d[i][e], u[i][e], sum_a[i][e]);
                            if constexpr (LAYER) sum_b[i][e] = row::add2(sum_b[i][e], d[i][e]);
                            d[i][e] = row::mul2(d[i][e], gt[e]);
                        }
                    } else if (post) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sum_a[i][e] = row::fma2(d[i][e], u[i][e], sum_a[i][e]);
                            if constexpr (LAYER) sum_b[i][e] = row::add2(sum_b[i][e], d[i][e]);
                        }
                    }
                    if (post) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (has_w_post) d[i][e] = row::mul2(d[i][e], w[e]);
                            s0 = row::fma2(d[i][e], u[i][e], s0);
                            if constexpr (LAYER) s1 = row::add2(s1, d[i][e]);
                        }
                    }
                }
                if (has_h) {
                    f2 ch = 0, cq = 0, scale = row::all2(1.0f);
                    if (post) {
                        float s[2] = {row::lo2(s0) + row::hi2(s0), row::lo2(s1) + row::hi2(s1)};
                        sum(s);
                        scale = rs;
                        ch = row::all2(-r_post * (s[0] * inv_c));
                        cq = row::all2(-r_post * (s[1] * inv_c));
                    }
                    if (has_dh) {
#pragma unroll
                        for (int i = 0; i < VPT; ++i) {
                            if (!live[i]) continue;
                            if (post) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const f2 t = LAYER ? row::fma2(u[i][e], ch, cq) : row::mul2(u[i][e], ch);
                                    d[i][e] = row::fma2(d[i][e], scale, t);
                                }
                            }
                            put(p.dh + base, d[i], i);
                        }
                    }
                }
            }
            if (++stage == static_cast<uint32_t>(ring.stages)) { stage = 0; phase ^= 1u; }
            // with a post norm over the CTA its sum's barrier is past the last read
            if (WARP || !(post && has_h)) __syncthreads();
            if (threadIdx.x == 0 && ahead.k < chunks) fill();
        }
        if (gated) end_chunk(gate, k, k == static_cast<int>(blockIdx.x));
    }
    out_sums(dw_pre, my_sums, false);
    if constexpr (LAYER) out_sums(db_pre, my_sums + rows_of, false);
    if (gated && post && ring.sums_at) {
        __syncthreads();
        for (int64_t c = threadIdx.x; c < p.width; c += blockDim.x) {
            my_sums[2 * rows_of + c] = post_w[c];
            if constexpr (LAYER) my_sums[3 * rows_of + c] = post_b[c];
        }
    }
    if (!gated) {
        out_sums(sum_a, my_sums + 2 * rows_of, false);
        if constexpr (LAYER) out_sums(sum_b, my_sums + 3 * rows_of, false);
    }
    if (threadIdx.x == 0 && gave_up) {
        // copies may still be on their way into this CTA's shared memory
        uint32_t never = 0;
        for (uint32_t i = 0; i < issued && i < static_cast<uint32_t>(ring.stages); ++i) {
            const uint32_t last = issued - 1 - i;   // the newest copy into each stage
            ptx::mbar_wait(&full[last % ring.stages], last / ring.stages & 1u, &never);
        }
        if (p.status) atomicOr(p.status, 1u);
    }
}

// Sums of partial rows: job j < dws adds the `ctas` rows of dw_part[which[j]],
// job dws + g the `parts` rows of group g of the gate.  A CTA takes 16 x V
// columns: 16 slices of the rows first, then the slices, in a fixed order.
// Small CTAs with eight loads in flight a thread: the kernel is latency.
struct NormSums {
    const float* dw_part;
    const float* dgate_part;
    float* out[4];
    float* dgate;
    int which[4];
    int dws;
    int64_t ctas, parts, width;
    int accumulate;
};

template <int V>
__global__ void __launch_bounds__(256) norm_sums_kernel(const __grid_constant__ NormSums p) {
    ptx::griddep_launch_dependents();
    __shared__ float part[16][16 * V + 1];
    ptx::griddep_wait();
    const int job = blockIdx.y, slice = threadIdx.x >> 4, lane = threadIdx.x & 15;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 16 * V + lane * V;
    const bool gate = job >= p.dws;
    const int64_t group = job - p.dws;
    const int64_t n = gate ? p.parts : p.ctas;
    const float* in = gate ? p.dgate_part + group * p.parts * p.width
                           : p.dw_part + p.which[job] * p.ctas * p.width;
    float s[V] = {};
    if (c < p.width) {   // with V = 4 the width is a multiple of 4
#pragma unroll 8
        for (int64_t i = slice; i < n; i += 16) {
            if constexpr (V == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(in + i * p.width + c));
                s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
            } else {
                s[0] += __ldcg(in + i * p.width + c);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) part[slice][lane * V + e] = s[e];
    __syncthreads();
    if (threadIdx.x < 16 * V) {
        const int64_t o = static_cast<int64_t>(blockIdx.x) * 16 * V + threadIdx.x;
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += part[i][threadIdx.x];
        if (o < p.width) {
            float* out = gate ? p.dgate + group * p.width : p.out[p.which[job]];
            out[o] = p.accumulate ? out[o] + t : t;
        }
    }
}

// Launches the jobs whose outputs are set; `groups`: of dgate.
void launch_sums(NormSums q, int64_t groups, cudaStream_t stream) {
    q.dws = 0;
    for (int j = 0; j < 4; ++j)
        if (q.out[j]) q.which[q.dws++] = j;
    const unsigned jobs = static_cast<unsigned>(q.dws + (q.dgate ? groups : 0));
    if (!jobs) return;
    // four columns a thread where that still makes a CTA for most SMs
    if (q.width % 4 == 0 && (q.width + 63) / 64 * jobs >= 128)
        launch_pdl(norm_sums_kernel<4>, dim3(static_cast<unsigned>((q.width + 63) / 64), jobs), dim3(256),
                   0, stream, q);
    else
        launch_pdl(norm_sums_kernel<1>, dim3(static_cast<unsigned>((q.width + 15) / 16), jobs), dim3(256),
                   0, stream, q);
}

// Shared memory for the ring of one CTA: what an SM has, less what L1 needs
// for the vectors (14 bytes a column at most), over the CTAs on it.
constexpr int kRingBytesPerSm = 160 * 1024;
constexpr uint32_t kRingMost = 208 * 1024;   // of one CTA, beside its static shared memory

template <typename S, int VPT, bool WARP, bool VEC, bool LAYER, int THREADS, int HAS>
int launch_bwd_ring(const NormBwd& p, const BwdPlan& b, cudaStream_t st) {
    BwdRing ring;
    const uint32_t n = static_cast<uint32_t>(p.width * (WARP ? 8 : 1));
    auto up = [](uint32_t v) { return (v + (VEC ? 0 : 32) + 127) / 128 * 128; };
    ring.x_at = up(n * 2);
    ring.dxo_at = ring.x_at + up(n * sizeof(S));
    ring.h_at = ring.dxo_at + up(n * sizeof(S));
    ring.stage_bytes = ring.h_at + up(n * 2);
    const uint32_t room = static_cast<uint32_t>(kRingBytesPerSm / b.per_sm);
    ring.stages = static_cast<int>(room / ring.stage_bytes);
    if (ring.stages > 4) ring.stages = 4;
    if (ring.stages < 2) ring.stages = 2;
    uint32_t bytes = ring.stages * ring.stage_bytes;
    ring.sums_at = 0;
    const uint32_t sums = static_cast<uint32_t>(p.width) * (LAYER ? 8 : 4);
    if (p.gate && p.post && b.groups * b.parts > b.ctas && bytes + sums <= kRingMost) {
        ring.sums_at = bytes;
        bytes += sums;
    }
    auto k = norm_bwd_kernel<S, VPT, WARP, VEC, LAYER, THREADS, HAS>;
    static host::SmemAllowance allowed;   // of this instance
    const int r = host::allow_smem(k, static_cast<int>(bytes), allowed);
    if (r != FP8_OK) return r;
    launch_pdl(k, dim3(b.ctas), dim3(b.threads), bytes, st, p, ring);
    return FP8_OK;
}

template <typename S, bool LAYER, bool VEC>
int launch_bwd_resident(const NormBwd& p, const BwdPlan& b, cudaStream_t st) {
    const bool all = p.dy && p.x_out && p.dx_out && p.h && p.dx && p.dh && p.w_pre && (!p.post || p.w_post);
    if (b.warp) {
        if constexpr (VEC) {
            if (all && !p.post && !p.gate && p.width == 256 * b.vpt)
                return b.vpt == 1 ? launch_bwd_ring<S, 1, true, true, LAYER, 256, kHasAll>(p, b, st)
                                  : launch_bwd_ring<S, 2, true, true, LAYER, 256, kHasAll>(p, b, st);
        }
        return b.vpt == 1 ? launch_bwd_ring<S, 1, true, VEC, LAYER, 256, 0>(p, b, st)
                          : launch_bwd_ring<S, 2, true, VEC, LAYER, 256, 0>(p, b, st);
    }
    if (all && (!VEC || p.width == 16 * b.threads)) {
        constexpr int A = kHasAll, P = kHasPost, G = kHasGate;
        if (p.post && p.gate) return launch_bwd_ring<S, 2, false, VEC, LAYER, 512, A | P | G>(p, b, st);
        if (!p.post && !p.gate) return launch_bwd_ring<S, 2, false, VEC, LAYER, 512, A>(p, b, st);
        if constexpr (VEC)
            return p.post ? launch_bwd_ring<S, 2, false, true, LAYER, 512, A | P>(p, b, st)
                          : launch_bwd_ring<S, 2, false, true, LAYER, 512, A | G>(p, b, st);
    }
    return launch_bwd_ring<S, 2, false, VEC, LAYER, 512, 0>(p, b, st);
}

template <typename S, bool LAYER>
int launch_bwd(const NormBwd& p, const BwdPlan& b, cudaStream_t st) {
    const bool vec = p.width % 8 == 0;
    if (p.width <= kFastWidth)
        return vec ? launch_bwd_resident<S, LAYER, true>(p, b, st) : launch_bwd_resident<S, LAYER, false>(p, b, st);
    const dim3 grid(b.ctas), block(b.threads);
    if (vec) launch_pdl(norm_bwd_any_kernel<S, true, LAYER>, grid, block, 0, st, p);
    else launch_pdl(norm_bwd_any_kernel<S, false, LAYER>, grid, block, 0, st, p);
    return FP8_OK;
}

}  // namespace

void launch_column_sums(const float* part, int64_t n, int64_t width, float* out, int accumulate,
                        cudaStream_t stream) {
    NormSums q{};
    q.dw_part = part;
    q.out[0] = out;
    q.ctas = n;
    q.width = width;
    q.accumulate = accumulate;
    launch_sums(q, 0, stream);
}

namespace {

// ------------------------------------------------------------------ host side


int check_shape(const char* what, int64_t rows, int64_t width, const void* gate, int64_t gate_rows,
                int kind, int type) {
    if (rows < 0 || width < 1 || rows > kMaxRows)
        return set_error(FP8_ERR_SHAPE, "%s: rows must be in 0..2^31-1025, width at least 1", what);
    if (width > kMaxWidth)
        return set_error(FP8_ERR_UNSUPPORTED, "%s: width %lld, built up to %lld", what,
                         static_cast<long long>(width), static_cast<long long>(kMaxWidth));
    if (gate ? (gate_rows < 1 || rows % gate_rows) : gate_rows != 0)
        return set_error(FP8_ERR_SHAPE, "%s: gate_rows must divide the rows (0 without a gate)", what);
    if (kind != FP8_NORM_RMS && kind != FP8_NORM_LAYER)
        return set_error(FP8_ERR_INVALID_ARG, "%s: unknown norm kind %d", what, kind);
    if (type != FP8_OUT_BF16 && type != FP8_OUT_F32)
        return set_error(FP8_ERR_INVALID_ARG, "%s: unknown stream type %d", what, type);
    return FP8_OK;
}

}  // namespace
}  // namespace fp8

using namespace fp8;
using namespace fp8::host;

extern "C" {

int fp8_norm_fwd(const fp8_norm_fwd_args_t* a, void* stream) {
    const char* what = "fp8_norm_fwd";
    if (!a) return set_error(FP8_ERR_INVALID_ARG, "%s: args is NULL", what);
    int st = check_shape(what, a->rows, a->width, a->gate, a->gate_rows, a->kind, a->stream_type);
    if (st != FP8_OK) return st;
    if (!(a->eps >= 0.0f)) return set_error(FP8_ERR_INVALID_ARG, "%s: eps must be >= 0", what);
    if (!a->x && !a->h && a->rows) return set_error(FP8_ERR_INVALID_ARG, "%s: x and h are NULL", what);
    if (!a->h && a->rows && (a->post_norm || a->gate))
        return set_error(FP8_ERR_INVALID_ARG, "%s: post_norm and gate need h", what);
    if (a->kind == FP8_NORM_RMS && (a->b_post || a->b_pre))
        return set_error(FP8_ERR_UNSUPPORTED, "%s: biases are built for the layer norm only", what);
    if (!a->post_norm && (a->w_post || a->b_post))
        return set_error(FP8_ERR_INVALID_ARG, "%s: w_post and b_post need post_norm", what);
    if (a->q) {
        if (a->q_format != FP8_E4M3 && a->q_format != FP8_E5M2)
            return set_error(FP8_ERR_INVALID_ARG, "%s: unknown FP8 format %d", what, a->q_format);
        if (a->q_granularity != FP8_GRAN_TENSOR && a->q_granularity != FP8_GRAN_ROW)
            return set_error(a->q_granularity == FP8_GRAN_1x128 || a->q_granularity == FP8_GRAN_128x128
                                 ? FP8_ERR_UNSUPPORTED : FP8_ERR_INVALID_ARG,
                             "%s: codes per tensor or per row, not granularity %d", what,
                             a->q_granularity);
        if (a->q_granularity == FP8_GRAN_TENSOR ? (!a->q_scale || a->q_scale_inv)
                                                : (a->q_scale || !a->q_scale_inv || a->amax))
            return set_error(FP8_ERR_INVALID_ARG, "%s: codes per tensor take q_scale (and amax), "
                                                  "codes per row q_scale_inv", what);
    } else if (a->rows && (a->q_scale || a->q_scale_inv || a->amax)) {
        return set_error(FP8_ERR_INVALID_ARG, "%s: q_scale, q_scale_inv and amax need q", what);
    }
    if (!a->x_out && !a->y && !a->q && !a->stats && a->rows)
        return set_error(FP8_ERR_INVALID_ARG, "%s: no output", what);
    for (const void* p : {a->x, a->h, a->gate, static_cast<const void*>(a->w_post),
                          static_cast<const void*>(a->b_post), static_cast<const void*>(a->w_pre),
                          static_cast<const void*>(a->b_pre), static_cast<const void*>(a->x_out),
                          static_cast<const void*>(a->y), static_cast<const void*>(a->q)})
        if (!aligned(p, 16))
            return set_error(FP8_ERR_ALIGN, "%s: tensors and vectors must be 16-byte aligned", what);
    for (const float* p : {a->q_scale, static_cast<const float*>(a->q_scale_inv),
                           static_cast<const float*>(a->amax), static_cast<const float*>(a->stats)})
        if (!aligned(p, 4))
            return set_error(FP8_ERR_ALIGN, "%s: scales and stats must be 4-byte aligned", what);
    if (a->amax) launch_zero_words(a->amax, 1, as_stream(stream));
    if (a->rows == 0) return launch_status(what);
    NormFwd p{};
    p.x = a->x;
    p.h = static_cast<const __nv_bfloat16*>(a->h);
    p.gate = static_cast<const __nv_bfloat16*>(a->gate);
    p.w_post = a->w_post; p.b_post = a->b_post; p.w_pre = a->w_pre; p.b_pre = a->b_pre;
    p.x_out = a->x_out;
    p.y = static_cast<__nv_bfloat16*>(a->y);
    p.q = a->q; p.q_scale = a->q_scale; p.q_scale_inv = a->q_scale_inv; p.amax = a->amax;
    p.stats = a->stats;
    p.rows = a->rows; p.width = a->width;
    p.rows_per_gate = a->gate ? a->rows / a->gate_rows : a->rows;
    p.alpha = a->alpha; p.eps = a->eps; p.post = a->post_norm != 0;
    p.q_fmt = a->q_format; p.q_rows = a->q_granularity == FP8_GRAN_ROW; p.pow2 = a->pow2 != 0;
    const bool layer = a->kind == FP8_NORM_LAYER;
    cudaStream_t s = as_stream(stream);
    if (a->stream_type == FP8_OUT_F32)
        layer ? launch_fwd<float, true>(p, s) : launch_fwd<float, false>(p, s);
    else
        layer ? launch_fwd<__nv_bfloat16, true>(p, s) : launch_fwd<__nv_bfloat16, false>(p, s);
    return launch_status(what);
}

size_t fp8_norm_bwd_workspace_size(int64_t rows, int64_t width, int64_t gate_rows) {
    if (rows < 0 || rows > kMaxRows || width < 1 || width > kMaxWidth || gate_rows < 0 ||
        (gate_rows > 0 && rows % gate_rows))
        return 0;
    const BwdPlan b = bwd_plan(rows, width, gate_rows);
    return 4 * (b.dw_floats + b.dgate_floats);
}

int fp8_norm_bwd(const fp8_norm_bwd_args_t* a, void* workspace, size_t workspace_bytes, void* stream) {
    const char* what = "fp8_norm_bwd";
    if (!a) return set_error(FP8_ERR_INVALID_ARG, "%s: args is NULL", what);
    int st = check_shape(what, a->rows, a->width, a->gate, a->gate_rows, a->kind, a->stream_type);
    if (st != FP8_OK) return st;
    if (!a->h && a->rows && (a->post_norm || a->gate || a->dh))
        return set_error(FP8_ERR_INVALID_ARG, "%s: post_norm, gate and dh need h", what);
    if (!a->post_norm && (a->w_post || a->b_post || a->dw_post || a->db_post))
        return set_error(FP8_ERR_INVALID_ARG, "%s: the post norm's vectors need post_norm", what);
    if (a->kind == FP8_NORM_RMS && (a->db_pre || a->db_post || a->b_post))
        return set_error(FP8_ERR_UNSUPPORTED, "%s: biases are built for the layer norm only", what);
    if (!a->gate && a->dgate) return set_error(FP8_ERR_INVALID_ARG, "%s: dgate needs gate", what);
    if (a->rows) {
        if (!a->dy && !a->dx_out)
            return set_error(FP8_ERR_INVALID_ARG, "%s: dy and dx_out are NULL", what);
        if (a->dy && !a->x_out) return set_error(FP8_ERR_INVALID_ARG, "%s: dy needs x_out", what);
        if ((a->dy || a->post_norm) && !a->stats)
            return set_error(FP8_ERR_INVALID_ARG, "%s: the norms need stats", what);
        if (!a->dy && (a->dw_pre || a->db_pre))
            return set_error(FP8_ERR_INVALID_ARG, "%s: dw_pre and db_pre need dy", what);
    }
    for (const void* p : {a->dy, a->x_out, a->dx_out, a->h, a->gate, static_cast<const void*>(a->w_post),
                          static_cast<const void*>(a->b_post), static_cast<const void*>(a->w_pre),
                          static_cast<const void*>(a->dx), static_cast<const void*>(a->dh),
                          static_cast<const void*>(a->dgate), static_cast<const void*>(workspace)})
        if (!aligned(p, 16))
            return set_error(FP8_ERR_ALIGN, "%s: tensors, vectors and workspace must be 16-byte aligned", what);
    for (const float* p : {a->stats, static_cast<const float*>(a->dw_pre), static_cast<const float*>(a->db_pre),
                           static_cast<const float*>(a->dw_post), static_cast<const float*>(a->db_post)})
        if (!aligned(p, 4)) return set_error(FP8_ERR_ALIGN, "%s: stats and sums must be 4-byte aligned", what);
    const BwdPlan b = bwd_plan(a->rows, a->width, a->gate ? a->gate_rows : 0);
    const size_t need = 4 * (b.dw_floats + b.dgate_floats);
    if (need && (!workspace || workspace_bytes < need))
        return set_error(FP8_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", what,
                         workspace ? workspace_bytes : size_t{0}, need);
    cudaStream_t s = as_stream(stream);
    if (a->rows == 0) {   // empty sums: zeros, or with accumulate what was there
        const size_t row_bytes = static_cast<size_t>(a->width) * 4;
        for (float* o : {a->dw_pre, a->db_pre, a->dw_post, a->db_post, a->dgate}) {
            if (!o || a->accumulate) continue;
            const cudaError_t e = cudaMemsetAsync(
                o, 0, o == a->dgate ? row_bytes * static_cast<size_t>(a->gate_rows) : row_bytes, s);
            if (e != cudaSuccess)
                return set_error(FP8_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
        }
        return FP8_OK;
    }
    NormBwd p{};
    p.dy = static_cast<const __nv_bfloat16*>(a->dy);
    p.x_out = a->x_out; p.dx_out = a->dx_out;
    p.h = static_cast<const __nv_bfloat16*>(a->h);
    p.gate = static_cast<const __nv_bfloat16*>(a->gate);
    p.w_post = a->w_post; p.b_post = a->b_post; p.w_pre = a->w_pre; p.stats = a->stats;
    p.dx = a->dx;
    p.dh = static_cast<__nv_bfloat16*>(a->dh);
    p.dw_part = static_cast<float*>(workspace);
    const bool direct = b.parts == 1;   // a chunk is a whole group: dgate itself
    p.dgate_part = !a->dgate ? nullptr : (direct ? a->dgate : p.dw_part + b.dw_floats);
    p.add_dgate = direct && a->accumulate;
    p.rows = a->rows; p.width = a->width; p.groups = b.groups; p.parts = b.parts;
    p.alpha = a->alpha; p.post = a->post_norm != 0;
    p.status = device_status_word();
    const bool layer = a->kind == FP8_NORM_LAYER;
    if (a->stream_type == FP8_OUT_F32)
        st = layer ? launch_bwd<float, true>(p, b, s) : launch_bwd<float, false>(p, b, s);
    else
        st = layer ? launch_bwd<__nv_bfloat16, true>(p, b, s) : launch_bwd<__nv_bfloat16, false>(p, b, s);
    if (st != FP8_OK) return st;
    NormSums q{};
    q.dw_part = p.dw_part;
    q.dgate_part = p.dw_part + b.dw_floats;
    q.out[0] = a->dw_pre; q.out[1] = a->db_pre; q.out[2] = a->dw_post; q.out[3] = a->db_post;
    q.dgate = direct ? nullptr : a->dgate;
    q.ctas = b.ctas; q.parts = b.parts; q.width = a->width;
    q.accumulate = a->accumulate != 0;
    launch_sums(q, b.groups, s);   // several parts a group: fewer groups than CTAs
    return launch_status(what);
}

}  // extern "C"

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
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/fp8linear.h"
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

// Eight elements from p; VEC: 16-byte pieces, all eight present.  Otherwise
// the first n, zeros after them.
template <bool VEC>
__device__ __forceinline__ void load8(float (&v)[8], const __nv_bfloat16* p, int n) {
    if constexpr (VEC) {
        row::unpack8(v, row::ld_stream(p));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? __bfloat162float(p[e]) : 0.0f;
    }
}

template <bool VEC>
__device__ __forceinline__ void load8(float (&v)[8], const float* p, int n) {
    if constexpr (VEC) {
        const uint4 a = row::ld_stream(p), b = row::ld_stream(p + 4);
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
        v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
        v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e] : 0.0f;
    }
}

// The same through L1, for the vectors that every row shares.
template <bool VEC>
__device__ __forceinline__ void shared8(float (&v)[8], const float* p, int n) {
    if constexpr (VEC) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p));
        const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        load8<false>(v, p, n);
    }
}

template <bool VEC>
__device__ __forceinline__ void shared8(float (&v)[8], const __nv_bfloat16* p, int n) {
    if constexpr (VEC)
        row::unpack8(v, __ldg(reinterpret_cast<const uint4*>(p)));
    else
        load8<false>(v, p, n);
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8], int n) {
    if constexpr (VEC) {
        *reinterpret_cast<uint4*>(p) = row::pack8(v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = __float2bfloat16_rn(v[e]);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(float* p, const float (&v)[8], int n) {
    if constexpr (VEC) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = v[e];
    }
}

// Mean (layer norm) and 1/sqrt(variance + eps) of the row whose pieces the
// threads hold; elements past the row are zero in v and left out of the sums.
template <int VPT, bool WARP, bool VEC, bool LAYER>
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
            if (VEC ? n[i] > 0 : e < n[i]) s[0] = fmaf(d, d, s[0]);
        }
    row_sum<WARP>(s, part, turn);
    rstd = 1.0f / sqrtf(s[0] * inv_c + eps);
}

// v = w (v - mean) rstd + b on one piece.
template <bool VEC>
__device__ __forceinline__ void apply_norm(float (&v)[8], const float* w, const float* b, int64_t c,
                                           int n, float mean, float rstd) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (v[e] - mean) * rstd;
    float s[8];
    if (w) {
        shared8<VEC>(s, w + c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= s[e];
    }
    if (b) {
        shared8<VEC>(s, b + c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += s[e];
    }
}

template <typename S, int VPT, bool WARP, bool VEC, bool LAYER, int THREADS>
__global__ void __launch_bounds__(THREADS)
    norm_fwd_kernel(const __grid_constant__ NormFwd p) {
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
        const int64_t c = 8 * static_cast<int64_t>(at + i * lanes);
        n[i] = static_cast<int>(p.width - c < 0 ? 0 : (p.width - c < 8 ? p.width - c : 8));
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = x[i][e] = 0.0f;
        if (n[i] > 0) {
            if (p.h) load8<VEC>(v[i], p.h + base + c, n[i]);
            if (xin) load8<VEC>(x[i], xin + base + c, n[i]);
        }
    }
    float mean_post = 0.0f, rstd_post = 0.0f, mean_pre = 0.0f, rstd_pre = 0.0f;
    if (p.post)
        row_stats<VPT, WARP, VEC, LAYER>(v, n, inv_c, p.eps, part, turn, mean_post, rstd_post);
    const __nv_bfloat16* gate =
        p.gate ? p.gate + (r / p.rows_per_gate) * p.width : nullptr;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t c = 8 * static_cast<int64_t>(at + i * lanes);
        if (n[i] <= 0) continue;
        if (p.post) apply_norm<VEC>(v[i], p.w_post, p.b_post, c, n[i], mean_post, rstd_post);
        if (gate) {
            float g[8];
            shared8<VEC>(g, gate + c, n[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[i][e] = VEC || e < n[i] ? fmaf(p.alpha, x[i][e], v[i][e]) : 0.0f;
        if (p.x_out) store8<VEC>(static_cast<S*>(p.x_out) + base + c, v[i], n[i]);
    }
    if (p.y || p.q || p.stats)
        row_stats<VPT, WARP, VEC, LAYER>(v, n, inv_c, p.eps, part, turn, mean_pre, rstd_pre);
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
        const int64_t c = 8 * static_cast<int64_t>(at + i * lanes);
        if (n[i] <= 0) continue;
        apply_norm<VEC>(v[i], p.w_pre, p.b_pre, c, n[i], mean_pre, rstd_pre);
        if (p.y) store8<VEC>(p.y + base + c, v[i], n[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (VEC || e < n[i]) top = max(top, row::abs_bits(v[i][e]));
    }
    if (!p.q) return;
    float s = 1.0f;
    if (p.q_rows || p.amax) top = row_max<WARP>(top, part, turn);
    if (p.q_rows) {
        // the per-row cast's rule: 1 for a row that is all zero or not finite
        const float a = __uint_as_float(top);
        if (a > 0.0f && a <= FLT_MAX) {
            s = __fdiv_rn(p.q_fmt == FP8_E4M3 ? 448.0f : 57344.0f, a);
            s = fminf(fmaxf(s, FLT_MIN), FLT_MAX);
            if (p.pow2) s = __uint_as_float(__float_as_uint(s) & 0xFF800000u);
        }
        if (at == 0) p.q_scale_inv[r] = __fdiv_rn(1.0f, s);
    } else {
        s = p.q_scale[0];
        if (p.amax && at == 0) row::raise_amax(p.amax, top);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t c = 8 * static_cast<int64_t>(at + i * lanes);
        if (n[i] <= 0) continue;
        const uint2 code = row::cvt8(p.q_fmt, v[i], s);
        if constexpr (VEC) {
            *reinterpret_cast<uint2*>(p.q + base + c) = code;
        } else {
            for (int e = 0; e < n[i]; ++e)
                p.q[base + c + e] = static_cast<uint8_t>((e < 4 ? code.x : code.y) >> (8 * (e & 3)));
        }
    }
}

template <typename S, bool VEC, bool LAYER>
void launch_fwd(const NormFwd& p, cudaStream_t st) {
    const int64_t pieces = (p.width + 7) / 8;
    // up to 1024 columns a warp holds a row: no CTA barrier, eight rows a CTA
    if (pieces <= 128) {
        const dim3 grid(static_cast<unsigned>((p.rows + 7) / 8));
        if (pieces <= 32)
            launch_pdl(norm_fwd_kernel<S, 1, true, VEC, LAYER, 256>, grid, dim3(256), 0, st, p);
        else if (pieces <= 64)
            launch_pdl(norm_fwd_kernel<S, 2, true, VEC, LAYER, 256>, grid, dim3(256), 0, st, p);
        else
            launch_pdl(norm_fwd_kernel<S, 4, true, VEC, LAYER, 256>, grid, dim3(256), 0, st, p);
        return;
    }
    const int threads = static_cast<int>(((pieces + 1) / 2 + 31) / 32 * 32);
    const dim3 grid(static_cast<unsigned>(p.rows));
    if (threads <= 512)
        launch_pdl(norm_fwd_kernel<S, 2, false, VEC, LAYER, 512>, grid, dim3(threads), 0, st, p);
    else
        launch_pdl(norm_fwd_kernel<S, 2, false, VEC, LAYER, 1024>, grid, dim3(threads), 0, st, p);
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
};

struct BwdPlan {
    bool warp;
    int vpt, threads, ctas;
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
    const int64_t per_sm = b.warp ? 2 : (b.threads >= 512 ? 1 : 512 / b.threads);
    const int64_t target = num_sms() * per_sm;
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
__device__ __forceinline__ void flush(float (&acc)[VPT][8], const int (&n)[VPT], int at, int lanes,
                                      int64_t width, float* out, bool add, float* buf) {
    if constexpr (WARP) {
        const int warp = threadIdx.x >> 5;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) buf[warp * 512 + 8 * (at + i * 32) + e] = acc[i][e];
        __syncthreads();
        for (int64_t c = threadIdx.x; c < width; c += blockDim.x) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) s += buf[w * 512 + c];
            out[c] = add ? out[c] + s : s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (n[i] <= 0) continue;
            float* o = out + 8 * static_cast<int64_t>(at + i * lanes);
            if (add) {
                for (int e = 0; e < n[i]; ++e) o[e] += acc[i][e];
            } else {
                store8<VEC>(o, acc[i], n[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
}

template <typename S, int VPT, bool WARP, bool VEC, bool LAYER, int THREADS>
__global__ void __launch_bounds__(THREADS)
    norm_bwd_kernel(const __grid_constant__ NormBwd p) {
    ptx::griddep_launch_dependents();
    __shared__ float part[128];
    __shared__ float buf[WARP ? 8 * 512 : 1];
    ptx::griddep_wait();
    const int lanes = WARP ? 32 : static_cast<int>(blockDim.x);
    const int at = WARP ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
    const int64_t first = WARP ? threadIdx.x >> 5 : 0;
    const int64_t step = WARP ? blockDim.x >> 5 : 1;
    const float inv_c = 1.0f / static_cast<float>(p.width);
    int turn = 0;

    float dw_pre[VPT][8], dw_post[VPT][8], dg[VPT][8];
    float db_pre[LAYER ? VPT : 1][8], db_post[LAYER ? VPT : 1][8];
    int n[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t c = 8 * static_cast<int64_t>(at + i * lanes);
        n[i] = static_cast<int>(p.width - c < 0 ? 0 : (p.width - c < 8 ? p.width - c : 8));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw_pre[i][e] = dw_post[i][e] = dg[i][e] = 0.0f;
            if constexpr (LAYER) db_pre[i][e] = db_post[i][e] = 0.0f;
        }
    }

    const int64_t chunks = p.groups * p.parts, in_group = p.rows / p.groups;
    for (int64_t k = blockIdx.x; k < chunks; k += gridDim.x) {
        const int64_t group = k / p.parts, part_no = k % p.parts;
        const int64_t begin = group * in_group + part_no * in_group / p.parts;
        const int64_t end = group * in_group + (part_no + 1) * in_group / p.parts;
        const __nv_bfloat16* gate = p.gate ? p.gate + group * p.width : nullptr;
        for (int64_t r = begin + first; r < end; r += step) {
            const int64_t base = r * p.width;
            float d[VPT][8], u[VPT][8], hv[VPT][8];
            float m_post = 0.0f, r_post = 1.0f;
            if (p.post) {
                m_post = LAYER ? p.stats[r] : 0.0f;
                r_post = p.stats[p.rows + r];
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int64_t c = 8 * static_cast<int64_t>(at + i * lanes);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[i][e] = hv[i][e] = 0.0f;
                if (n[i] > 0) {
                    if (p.dx_out) load8<VEC>(d[i], static_cast<const S*>(p.dx_out) + base + c, n[i]);
                    if (p.h) load8<VEC>(hv[i], p.h + base + c, n[i]);
                }
            }
            if (p.dy) {
                const float m_pre = LAYER ? p.stats[2 * p.rows + r] : 0.0f;
                const float r_pre = p.stats[3 * p.rows + r];
                float g[VPT][8], s[2] = {0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int64_t c = 8 * static_cast<int64_t>(at + i * lanes);
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[i][e] = u[i][e] = 0.0f;
                    if (n[i] <= 0) continue;
                    load8<VEC>(g[i], p.dy + base + c, n[i]);
                    load8<VEC>(u[i], static_cast<const S*>(p.x_out) + base + c, n[i]);
                    float w[8];
                    if (p.w_pre) shared8<VEC>(w, p.w_pre + c, n[i]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        u[i][e] = (u[i][e] - m_pre) * r_pre;
                        if (!VEC && e >= n[i]) u[i][e] = 0.0f;
                        dw_pre[i][e] = fmaf(g[i][e], u[i][e], dw_pre[i][e]);
                        if constexpr (LAYER) db_pre[i][e] += g[i][e];
                        if (p.w_pre) g[i][e] *= w[e];
                        s[0] = fmaf(g[i][e], u[i][e], s[0]);
                        s[1] += g[i][e];
                    }
                }
                if constexpr (LAYER) {
                    row_sum<WARP>(s, part, turn);
                } else {
                    float t[1] = {s[0]};
                    row_sum<WARP>(t, part, turn);
                    s[0] = t[0];
                    s[1] = 0.0f;
                }
                const float su = s[0] * inv_c, sg = s[1] * inv_c;
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        d[i][e] = fmaf(r_pre, g[i][e] - sg - u[i][e] * su, d[i][e]);
            }
            // from here d is dX; columns past the row hold values that no one uses
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int64_t c = 8 * static_cast<int64_t>(at + i * lanes);
                if (n[i] <= 0) continue;
                if (p.dx) {
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = p.alpha * d[i][e];
                    store8<VEC>(static_cast<S*>(p.dx) + base + c, o, n[i]);
                }
                if (!p.h) continue;
                float w[8];
                if (p.post) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) hv[i][e] = (hv[i][e] - m_post) * r_post;
                    if (p.w_post) shared8<VEC>(w, p.w_post + c, n[i]);
                }
                if (gate) {
                    float gt[8], pv[8];
                    shared8<VEC>(gt, gate + c, n[i]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) pv[e] = p.post && p.w_post ? hv[i][e] * w[e] : hv[i][e];
                    if (LAYER && p.post && p.b_post) {
                        float b[8];
                        shared8<VEC>(b, p.b_post + c, n[i]);
#pragma unroll
                        for (int e = 0; e < 8; ++e) pv[e] += b[e];
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dg[i][e] = fmaf(d[i][e], pv[e], dg[i][e]);
                        d[i][e] *= gt[e];
                    }
                }
                if (p.post) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (!VEC && e >= n[i]) {
                            d[i][e] = 0.0f;
                            continue;
                        }
                        dw_post[i][e] = fmaf(d[i][e], hv[i][e], dw_post[i][e]);
                        if constexpr (LAYER) db_post[i][e] += d[i][e];
                        if (p.w_post) d[i][e] *= w[e];
                        s[0] = fmaf(d[i][e], hv[i][e], s[0]);
                        s[1] += d[i][e];
                    }
                }
            }
            if (!p.h) continue;
            if (p.post) {
                if constexpr (LAYER) {
                    row_sum<WARP>(s, part, turn);
                } else {
                    float t[1] = {s[0]};
                    row_sum<WARP>(t, part, turn);
                    s[0] = t[0];
                    s[1] = 0.0f;
                }
            }
            const float sh = s[0] * inv_c, sq = s[1] * inv_c;
            if (p.dh) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int64_t c = 8 * static_cast<int64_t>(at + i * lanes);
                    if (n[i] <= 0) continue;
                    if (p.post) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            d[i][e] = r_post * (d[i][e] - sq - hv[i][e] * sh);
                    }
                    store8<VEC>(p.dh + base + c, d[i], n[i]);
                }
            }
        }
        if (gate && p.dgate_part)
            flush<VPT, WARP, VEC>(dg, n, at, lanes, p.width, p.dgate_part + k * p.width,
                                  p.add_dgate != 0, buf);
    }
    const int64_t rows_of = static_cast<int64_t>(gridDim.x) * p.width;
    float* out = p.dw_part + static_cast<int64_t>(blockIdx.x) * p.width;
    flush<VPT, WARP, VEC>(dw_pre, n, at, lanes, p.width, out, false, buf);
    flush<VPT, WARP, VEC>(dw_post, n, at, lanes, p.width, out + 2 * rows_of, false, buf);
    if constexpr (LAYER) {
        flush<VPT, WARP, VEC>(db_pre, n, at, lanes, p.width, out + rows_of, false, buf);
        flush<VPT, WARP, VEC>(db_post, n, at, lanes, p.width, out + 3 * rows_of, false, buf);
    }
}

// Sums of partial rows: job j < 4 adds dw_part[j][0 .. ctas), job 4 + g the
// `parts` rows of group g.  A CTA takes 32 columns: 32 slices of the rows
// first, then the slices, both in a fixed order.
struct NormSums {
    const float* dw_part;
    const float* dgate_part;
    float* out[4];
    float* dgate;
    int64_t ctas, parts, width;
    int accumulate;
};

__global__ void __launch_bounds__(1024) norm_sums_kernel(const __grid_constant__ NormSums p) {
    ptx::griddep_launch_dependents();
    __shared__ float part[32][33];
    ptx::griddep_wait();
    const int64_t job = blockIdx.y;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
    const int slice = threadIdx.x >> 5;
    float* out = job < 4 ? p.out[job] : p.dgate + (job - 4) * p.width;
    if (!out || (job >= 4 && !p.dgate)) return;
    const int64_t n = job < 4 ? p.ctas : p.parts;
    const float* in = job < 4 ? p.dw_part + job * p.ctas * p.width
                              : p.dgate_part + (job - 4) * p.parts * p.width;
    float s = 0.0f;
    if (c < p.width) {
#pragma unroll 4
        for (int64_t i = slice; i < n; i += 32) s += in[i * p.width + c];
    }
    part[slice][threadIdx.x & 31] = s;
    __syncthreads();
    if (slice == 0 && c < p.width) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += part[i][threadIdx.x];
        out[c] = p.accumulate ? out[c] + t : t;
    }
}

template <typename S, bool VEC, bool LAYER>
void launch_bwd(const NormBwd& p, const BwdPlan& b, cudaStream_t st) {
    const dim3 grid(b.ctas), block(b.threads);
    if (b.warp && b.vpt == 1) launch_pdl(norm_bwd_kernel<S, 1, true, VEC, LAYER, 256>, grid, block, 0, st, p);
    else if (b.warp) launch_pdl(norm_bwd_kernel<S, 2, true, VEC, LAYER, 256>, grid, block, 0, st, p);
    else if (b.threads <= 512)
        launch_pdl(norm_bwd_kernel<S, 2, false, VEC, LAYER, 512>, grid, block, 0, st, p);
    else
        launch_pdl(norm_bwd_kernel<S, 2, false, VEC, LAYER, 1024>, grid, block, 0, st, p);
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
    launch_pdl(norm_sums_kernel, dim3(static_cast<unsigned>((width + 31) / 32)), dim3(1024), 0,
               stream, q);
}

namespace {

// ------------------------------------------------------------------ host side

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

int launch_status(const char* what) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? FP8_OK : set_error(FP8_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int check_shape(const char* what, int64_t rows, int64_t width, const void* gate, int64_t gate_rows,
                int kind, int type) {
    if (rows < 0 || width < 1 || rows >= (int64_t{1} << 31))
        return set_error(FP8_ERR_SHAPE, "%s: rows must be in 0..2^31-1, width at least 1", what);
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
    p.rows_per_gate = a->gate ? a->rows / a->gate_rows : 1;
    p.alpha = a->alpha; p.eps = a->eps; p.post = a->post_norm != 0;
    p.q_fmt = a->q_format; p.q_rows = a->q_granularity == FP8_GRAN_ROW; p.pow2 = a->pow2 != 0;
    const bool vec = a->width % 8 == 0, layer = a->kind == FP8_NORM_LAYER;
    cudaStream_t s = as_stream(stream);
    if (a->stream_type == FP8_OUT_F32) {
        if (vec) layer ? launch_fwd<float, true, true>(p, s) : launch_fwd<float, true, false>(p, s);
        else layer ? launch_fwd<float, false, true>(p, s) : launch_fwd<float, false, false>(p, s);
    } else {
        if (vec) layer ? launch_fwd<__nv_bfloat16, true, true>(p, s) : launch_fwd<__nv_bfloat16, true, false>(p, s);
        else layer ? launch_fwd<__nv_bfloat16, false, true>(p, s) : launch_fwd<__nv_bfloat16, false, false>(p, s);
    }
    return launch_status(what);
}

size_t fp8_norm_bwd_workspace_size(int64_t rows, int64_t width, int64_t gate_rows) {
    if (rows < 0 || width < 1 || width > kMaxWidth || gate_rows < 0 ||
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
    const bool vec = a->width % 8 == 0, layer = a->kind == FP8_NORM_LAYER;
    if (a->stream_type == FP8_OUT_F32) {
        if (vec) layer ? launch_bwd<float, true, true>(p, b, s) : launch_bwd<float, true, false>(p, b, s);
        else layer ? launch_bwd<float, false, true>(p, b, s) : launch_bwd<float, false, false>(p, b, s);
    } else {
        if (vec) layer ? launch_bwd<__nv_bfloat16, true, true>(p, b, s) : launch_bwd<__nv_bfloat16, true, false>(p, b, s);
        else layer ? launch_bwd<__nv_bfloat16, false, true>(p, b, s) : launch_bwd<__nv_bfloat16, false, false>(p, b, s);
    }
    NormSums q{};
    q.dw_part = p.dw_part;
    q.dgate_part = p.dw_part + b.dw_floats;
    q.out[0] = a->dw_pre; q.out[1] = a->db_pre; q.out[2] = a->dw_post; q.out[3] = a->db_post;
    q.dgate = direct ? nullptr : a->dgate;
    q.ctas = b.ctas; q.parts = b.parts; q.width = a->width;
    q.accumulate = a->accumulate != 0;
    if (q.out[0] || q.out[1] || q.out[2] || q.out[3] || q.dgate) {
        // several parts a group: fewer groups than CTAs
        const unsigned jobs = static_cast<unsigned>(4 + (q.dgate ? b.groups : 0));
        launch_pdl(norm_sums_kernel, dim3(static_cast<unsigned>((a->width + 31) / 32), jobs),
                   dim3(1024), 0, s, q);
    }
    return launch_status(what);
}

}  // extern "C"

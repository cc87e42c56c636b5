// moe.cu -- tokens sorted by expert and back, around the experts' linears.
//
//   plan         a stable counting sort of the (token, slot) pairs by expert:
//                row(t, j) = offset[e] + #{pairs before (t, j) with expert e}
//   permute      xs[row] = x[token]                    (pad rows zero)
//   unpermute    y[t] = sum_j w[t, j] ys[row(t, j)]    (fp32, j ascending)
//   its gradient dys[row] = w[t, j] dy[t],  dw[t, j] = <dy[t], ys[row]>
//
// All of them move rows: the bound is HBM.  The copies go token by token, so
// that a token's row is read once for its k copies, and every sum runs in a
// fixed order, so that equal calls give equal bits.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/fp8linear.h"
#include "hostops.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowops.cuh"

namespace fp8 {
namespace {

constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32;
constexpr int kMaxExperts = 1024, kMaxSlots = 64;
constexpr int64_t kMost = int64_t{1} << 30;   // pairs and rows: 32-bit numbers and grids
// One CTA ranks up to this many pairs; past it the per-CTA histograms of a first
// launch cost less than the walk of one CTA over all of them (4000 pairs, 256
// experts: 13 us by one CTA, 6 by two launches; 32 pairs: 3.3 us by one CTA).
constexpr int kPlanOneCta = 2048;
constexpr int kPlanChunk = 512;    // pairs a CTA at least: one look of 32 a warp
constexpr int kPlanMaxCtas = 128;  // so that summing the CTAs' histograms stays short

struct PlanGrid {
    int ctas, chunk;
};

PlanGrid plan_grid(int64_t n) {
    if (n <= kPlanOneCta) return {1, static_cast<int>((n + 31) / 32 * 32)};
    int64_t chunk = (n + kPlanMaxCtas - 1) / kPlanMaxCtas;
    if (chunk < kPlanChunk) chunk = kPlanChunk;
    chunk = (chunk + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
    return {static_cast<int>((n + chunk - 1) / chunk), static_cast<int>(chunk)};
}

// hist[cta][e]: how many of the CTA's pairs go to expert e.
__global__ void __launch_bounds__(kPlanThreads)
    moe_hist_kernel(const int32_t* __restrict__ ids, int n, int experts, int chunk,
                    int32_t* __restrict__ hist) {
    ptx::griddep_launch_dependents();
    __shared__ int h[kMaxExperts];
    for (int e = threadIdx.x; e < experts; e += kPlanThreads) h[e] = 0;
    __syncthreads();
    ptx::griddep_wait();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * chunk;
    for (int i = threadIdx.x; i < chunk; i += 4 * kPlanThreads) {
        int e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {   // chunk is a multiple of kPlanThreads
            const int64_t at = first + i + k * kPlanThreads;
            e[k] = i + k * kPlanThreads < chunk && at < n ? ids[at] : -1;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (e[k] >= 0 && e[k] < experts) atomicAdd(&h[e[k]], 1);   // integers: any order
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += kPlanThreads)
        hist[static_cast<int64_t>(blockIdx.x) * experts + e] = h[e];
}

// Ranks and writes the CTA's chunk of pairs.  Each warp owns a contiguous
// part of the chunk: it counts its pairs per expert (lanes with the same
// expert find one another with a match), the counts become starting rows by
// a sum over the CTAs and warps before it, and a second walk hands the rows
// out in order.  Every CTA sums all CTAs' histograms itself (ctas x experts
// words from L2), which saves a launch.  65536 pairs to 64 experts: 7.6 us with
// the histograms' launch.
__global__ void __launch_bounds__(kPlanThreads)
    moe_place_kernel(const int32_t* __restrict__ ids, int n, int experts, int align, int chunk,
                     const int32_t* __restrict__ hist, int32_t* __restrict__ offsets,
                     int32_t* __restrict__ counts, int32_t* __restrict__ row_of,
                     int32_t* __restrict__ src, int rows) {
    ptx::griddep_launch_dependents();
    extern __shared__ int counters[];   // [warps][experts]: counts, then next rows
    __shared__ int total[kMaxExperts + 1], start[kMaxExperts + 1];
    __shared__ int warp_tot[kPlanWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto cnt = [&](int w, int e) -> int& { return counters[w * experts + e]; };
    for (int e = lane; e < experts; e += 32) cnt(warp, e) = 0;
    __syncwarp();
    ptx::griddep_wait();
    const int per_warp = (chunk + kPlanWarps * 32 - 1) / (kPlanWarps * 32) * 32;
    const int64_t cta_first = static_cast<int64_t>(blockIdx.x) * chunk;
    const int64_t cta_end = cta_first + chunk < n ? cta_first + chunk : n;
    const int64_t first = cta_first + static_cast<int64_t>(warp) * per_warp;
    const int64_t end = first + per_warp < cta_end ? first + per_warp : cta_end;
    const uint32_t below = (1u << lane) - 1u;

    constexpr int kAhead = 8;   // looks of 32 pairs loaded together
    int e[kAhead];
    auto load = [&](int64_t i) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t at = i + 32 * k + lane;
            e[k] = at < end ? ids[at] : -1;
            if (e[k] >= experts) e[k] = -1;
        }
    };
    for (int64_t i = first; i < end; i += 32 * kAhead) {
        load(i);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i + 32 * k >= end) break;
            const uint32_t same = __match_any_sync(row::kAll, e[k]);
            if (e[k] >= 0 && (same & below) == 0) cnt(warp, e[k]) += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // per expert: pairs in the CTAs before this one, and in all.  With few
    // experts several threads share one's column of the histograms.
    for (int x = threadIdx.x; x < experts; x += kPlanThreads) {
        int own = 0;
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) own += cnt(w, x);
        total[x] = hist ? 0 : own;
        start[x] = 0;
    }
    if (hist) {
        __syncthreads();
        const int ctas = static_cast<int>(gridDim.x);
        const int parts = experts < kPlanThreads ? kPlanThreads / experts : 1;
        for (int i = threadIdx.x; i < experts * parts; i += kPlanThreads) {
            const int x = i % experts, part = i / experts;
            int before = 0, all = 0;
#pragma unroll 8
            for (int b = part; b < ctas; b += parts) {
                const int h = hist[static_cast<int64_t>(b) * experts + x];
                all += h;
                before += b < static_cast<int>(blockIdx.x) ? h : 0;
            }
            atomicAdd(&total[x], all);      // integers: any order
            atomicAdd(&start[x], before);
        }
    }
    __syncthreads();
    // offsets: the exclusive sum of the padded totals, kPer experts a thread
    constexpr int kPer = kMaxExperts / kPlanThreads;
    int pad[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int x = static_cast<int>(threadIdx.x) * kPer + i;
        pad[i] = x < experts ? (total[x] + align - 1) / align * align : 0;
        sum += pad[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(row::kAll, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += warp_tot[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int x = static_cast<int>(threadIdx.x) * kPer + i;
        if (x < experts) {
            if (blockIdx.x == 0) {
                offsets[x] = run;
                counts[x] = total[x];
            }
            // pad rows of the experts that this CTA is dealt
            if (x % static_cast<int>(gridDim.x) == static_cast<int>(blockIdx.x))
                for (int r = run + total[x]; r < run + pad[i]; ++r) src[r] = -1;
            int next = run + start[x];
            for (int w = 0; w < kPlanWarps; ++w) {
                const int c = cnt(w, x);
                cnt(w, x) = next;
                next += c;
            }
        }
        run += pad[i];
        if (x == experts - 1) {
            start[experts] = run;
            if (blockIdx.x == 0) offsets[experts] = run;
        }
    }
    __syncthreads();
    for (int64_t r = start[experts] + static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
         r < rows; r += static_cast<int64_t>(gridDim.x) * kPlanThreads)
        src[r] = -1;
    for (int64_t i = first; i < end; i += 32 * kAhead) {
        if (end - first > 32 * kAhead) load(i);   // else still there from the count
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t at = i + 32 * k + lane;
            if (i + 32 * k >= end) break;
            const uint32_t same = __match_any_sync(row::kAll, e[k]);
            int r = -1;
            if (e[k] >= 0) r = cnt(warp, e[k]) + __popc(same & below);
            __syncwarp();
            if (e[k] >= 0 && (same & below) == 0) cnt(warp, e[k]) += __popc(same);
            __syncwarp();
            if (at < end) {
                row_of[at] = r;
                if (r >= 0) src[r] = static_cast<int32_t>(at);
            }
        }
    }
}

// ------------------------------------------------------------------ row copies

// How a CTA of 256 threads is dealt to rows: `lanes` threads a row (a power
// of two), 256 / lanes rows at a time.
constexpr int kRowThreads = 256;

int lanes_for(int64_t pieces) {
    int l = 8;
    while (l < kRowThreads && l < pieces) l <<= 1;
    return l;
}

// xs[row_of[t, j]] = x[t] for every slot j; V is the copied unit.  CTAs past
// the tokens' set the pad rows (src < 0) to zero.
template <typename V>
__global__ void __launch_bounds__(kRowThreads)
    moe_permute_kernel(const V* __restrict__ x, const float* __restrict__ scale, int64_t tokens,
                       int slots, int64_t units, const int32_t* __restrict__ row_of,
                       const int32_t* __restrict__ src, int64_t rows, V* __restrict__ xs,
                       float* __restrict__ scale_s, int lanes, int64_t token_ctas) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int sub = threadIdx.x / lanes, lane = threadIdx.x % lanes, per = kRowThreads / lanes;
    if (blockIdx.x < token_ctas) {
        const int64_t t = static_cast<int64_t>(blockIdx.x) * per + sub;
        if (t >= tokens) return;
        const int32_t* to = row_of + t * slots;
        for (int64_t u = lane; u < units; u += lanes) {
            const V v = x[t * units + u];
            for (int j = 0; j < slots; ++j) {
                const int64_t r = to[j];
                if (r >= 0 && r < rows) xs[r * units + u] = v;
            }
        }
        if (scale && lane == 0)
            for (int j = 0; j < slots; ++j)
                if (to[j] >= 0 && to[j] < rows) scale_s[to[j]] = scale[t];
    } else {
        const V zero{};
        for (int64_t r = (blockIdx.x - token_ctas) * per + sub; r < rows;
             r += (gridDim.x - token_ctas) * per) {
            if (src[r] >= 0) continue;
            for (int64_t u = lane; u < units; u += lanes) xs[r * units + u] = zero;
            if (scale && lane == 0) scale_s[r] = 0.0f;
        }
    }
}

// The same for rows that do not start on 16 bytes: a CTA brings a token's row
// into shared memory, each byte at its place modulo 16, and writes the copies
// in aligned 16-byte pieces put together from neighbouring words; single
// bytes only at a copy's two ends.
constexpr int kImageBytes = 32768;   // of a row at a time, at most

__global__ void __launch_bounds__(kRowThreads)
    moe_permute_bytes_kernel(const uint8_t* __restrict__ x, const float* __restrict__ scale,
                             int64_t tokens, int slots, int64_t row_bytes,
                             const int32_t* __restrict__ row_of, const int32_t* __restrict__ src,
                             int64_t rows, uint8_t* __restrict__ xs, float* __restrict__ scale_s) {
    ptx::griddep_launch_dependents();
    extern __shared__ __align__(16) uint8_t image[];   // the row's part, 64 bytes over
    __shared__ int to[kMaxSlots];
    ptx::griddep_wait();
    const int tid = threadIdx.x;
    const bool pad = blockIdx.x >= tokens;   // CTAs past the tokens: zeros into pad rows
    const int64_t t = blockIdx.x;
    if (!pad && tid < slots) {
        const int r = row_of[t * slots + tid];
        to[tid] = r >= 0 && r < rows ? r : -1;
        if (scale && to[tid] >= 0) scale_s[to[tid]] = scale[t];
    }
    // copies of `n` bytes, from image + at (pad: zeros), to `count` rows
    auto write = [&](int count, int64_t pad_row, int64_t first, int n, int at) {
        const int most = n / 16 + 1;   // aligned pieces, and one more turn for the ends
        for (int k = tid; k < count * (most + 1); k += kRowThreads) {
            const int j = k / (most + 1), i = k - j * (most + 1);
            const int64_t r = pad ? pad_row : to[j];
            if (r < 0) continue;
            uint8_t* out = xs + r * row_bytes + first;
            const int head = min(n, static_cast<int>(-reinterpret_cast<uintptr_t>(out) & 15));
            const int body = (n - head) / 16;
            if (i < body) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (!pad) {
                    const int b = at + head + 16 * i;
                    const uint32_t* q = reinterpret_cast<const uint32_t*>(image + (b & ~3));
                    const int s = 8 * (b & 3);
                    const uint32_t w0 = q[0], w1 = q[1], w2 = q[2], w3 = q[3], w4 = q[4];
                    v = make_uint4(__funnelshift_r(w0, w1, s), __funnelshift_r(w1, w2, s),
                                   __funnelshift_r(w2, w3, s), __funnelshift_r(w3, w4, s));
                }
                __stcs(reinterpret_cast<uint4*>(out + head + 16 * i), v);
            } else if (i == most - 1) {
                for (int e = 0; e < head; ++e) out[e] = pad ? uint8_t{0} : image[at + e];
            } else if (i == most) {
                for (int e = head + 16 * body; e < n; ++e) out[e] = pad ? uint8_t{0} : image[at + e];
            }
        }
    };
    auto part = [&](int64_t first) {
        return static_cast<int>(row_bytes - first < kImageBytes ? row_bytes - first : kImageBytes);
    };
    if (!pad) {
        for (int64_t first = 0; first < row_bytes; first += kImageBytes) {
            const int n = part(first);
            const uint8_t* in = x + t * row_bytes + first;
            const int at = static_cast<int>(reinterpret_cast<uintptr_t>(in) & 15);
            const int head = min(n, (16 - at) & 15), body = (n - head) / 16;
            __syncthreads();   // the image before this one has been read
            for (int i = tid; i < body; i += kRowThreads)
                *reinterpret_cast<uint4*>(image + at + head + 16 * i) = row::ld_stream(in + head + 16 * i);
            const int tail = n - head - 16 * body;
            if (tid < head) image[at + tid] = in[tid];
            else if (tid >= 32 && tid - 32 < tail)
                image[at + head + 16 * body + tid - 32] = in[head + 16 * body + tid - 32];
            __syncthreads();
            write(slots, 0, first, n, at);
        }
    } else {
        for (int64_t r = blockIdx.x - tokens; r < rows; r += gridDim.x - tokens) {
            if (src[r] >= 0) continue;
            for (int64_t first = 0; first < row_bytes; first += kImageBytes) write(1, r, first, part(first), 0);
            if (scale && tid == 0) scale_s[r] = 0.0f;
        }
    }
}

// The same for rows of at least 1 KB in 16-byte units, by bulk copies alone:
// a warp takes a token's row (or a piece of a long one) into a slot of shared
// memory and each lane sends it to one of the slots' rows; no register or
// load unit touches the data.  Two slots a warp: one filled while the other
// is sent (8192 tokens to 8 of 64 experts, rows of 8 KB: 117 us with two, 122
// with three or four).  The copies run at 5.8 TB/s, a write of one stream of
// the same size at 7.5: the scattered rows are the bound, not the copy engine
// (through registers they took 10% longer).
constexpr int kBulkSlots = 2;
constexpr int kBulkSlotBytes = 16384;        // at most; longer rows go in pieces
constexpr int kBulkSmem = 200 * 1024;

struct BulkRows {
    const uint8_t* x;
    const float* scale;
    const int32_t* row_of;
    const int32_t* src;
    uint8_t* xs;
    float* scale_s;
    unsigned* status;
    int64_t tokens, rows, row_bytes;
    int slots, slot_bytes, pieces;           // pieces a row
};

__global__ void __launch_bounds__(256)
    moe_permute_bulk_kernel(const __grid_constant__ BulkRows p) {
    ptx::griddep_launch_dependents();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[8 * kBulkSlots];
    __shared__ volatile uint32_t gave_up;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    uint8_t* zeros = smem + nw * kBulkSlots * p.slot_bytes;
    uint8_t* mine = smem + warp * kBulkSlots * p.slot_bytes;
    uint64_t* bar = full + warp * kBulkSlots;
    if (lane == 0)
        for (int i = 0; i < kBulkSlots; ++i) ptx::mbar_init(&bar[i], 1);
    if (threadIdx.x == 0) gave_up = 0;
    ptx::fence_barrier_init();
    for (int i = threadIdx.x * 16; i < p.slot_bytes; i += blockDim.x * 16)
        *reinterpret_cast<uint4*>(zeros + i) = make_uint4(0, 0, 0, 0);
    ptx::fence_proxy_async_smem();   // the zeros are read by bulk copies
    __syncthreads();
    ptx::griddep_wait();
    const int64_t step = static_cast<int64_t>(gridDim.x) * nw;
    const int64_t first = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
    const int64_t items = p.tokens * p.pieces;
    auto bytes_of = [&](int64_t piece) {
        const int64_t left = p.row_bytes - piece * p.slot_bytes;
        return static_cast<uint32_t>(left < p.slot_bytes ? left : p.slot_bytes);
    };
    uint32_t issued = 0;
    auto fill = [&](int64_t item) {   // lane 0
        const int64_t t = item / p.pieces, piece = item - t * p.pieces;
        uint64_t* b = &bar[issued % kBulkSlots];
        ptx::mbar_arrive_expect_tx(b, bytes_of(piece));
        ptx::bulk_load(mine + issued % kBulkSlots * p.slot_bytes,
                       p.x + t * p.row_bytes + piece * p.slot_bytes, bytes_of(piece), b);
    };
    // the first rows on their way, and the first token's destinations
    for (int i = 0; i < kBulkSlots - 1; ++i) {
        if (first + i * step >= items) break;
        if (lane == 0) fill(first + i * step);
        ++issued;
    }
    auto dest = [&](int64_t item, int j) -> int64_t {
        if (item >= items || j >= p.slots) return -1;
        const int64_t r = p.row_of[item / p.pieces * p.slots + j];
        return r < p.rows ? r : -1;
    };
    int64_t to0 = dest(first, lane), to1 = dest(first, lane + 32);
    uint32_t done = 0;
    bool ok = true;
    for (int64_t item = first; item < items; item += step) {
        const int64_t r0 = to0, r1 = to1;
        to0 = dest(item + step, lane);
        to1 = dest(item + step, lane + 32);
        const int64_t t = item / p.pieces, piece = item - t * p.pieces;
        const uint32_t n = bytes_of(piece);
        ok = ptx::mbar_wait(&bar[done % kBulkSlots], done / kBulkSlots & 1u, &gave_up);
        ok = __all_sync(row::kAll, ok);
        if (!ok) break;
        const uint8_t* from = mine + done % kBulkSlots * p.slot_bytes;
        if (r0 >= 0) ptx::bulk_store(p.xs + r0 * p.row_bytes + piece * p.slot_bytes, from, n);
        if (r1 >= 0) ptx::bulk_store(p.xs + r1 * p.row_bytes + piece * p.slot_bytes, from, n);
        ptx::bulk_commit_group();
        if (p.scale && piece == 0) {
            if (r0 >= 0) p.scale_s[r0] = p.scale[t];
            if (r1 >= 0) p.scale_s[r1] = p.scale[t];
        }
        ++done;
        // the next fill takes the slot of the item before this one
        const int64_t next = item + (kBulkSlots - 1) * step;
        if (next < items) {
            ptx::bulk_wait_group_read<1>();
            __syncwarp();
            if (lane == 0) fill(next);
            ++issued;
        }
    }
    if (ok) {
        // pad rows, up to 32 at a look: with few rows they spread over the warps
        const int64_t share = (p.rows + step - 1) / step;
        const int look = static_cast<int>(share < 32 ? share : 32);
        for (int64_t r0 = first * look; r0 < p.rows; r0 += step * look) {
            const int64_t r = r0 + lane;
            if (lane < look && r < p.rows && p.src[r] < 0) {
                for (int64_t piece = 0; piece < p.pieces; ++piece)
                    ptx::bulk_store(p.xs + r * p.row_bytes + piece * p.slot_bytes, zeros, bytes_of(piece));
                if (p.scale) p.scale_s[r] = 0.0f;
            }
        }
        ptx::bulk_commit_group();
    } else if (lane == 0) {
        // fills may still be on their way into this CTA's shared memory
        uint32_t never = 0;
        for (; done < issued; ++done) ptx::mbar_wait(&bar[done % kBulkSlots], done / kBulkSlots & 1u, &never);
        if (p.status) atomicOr(p.status, 1u);
    }
    ptx::bulk_wait_group_all();
}

// Elements of type T (bf16 or fp32) as fp32, N at a time.  Stores leave L2
// first: 384 -> 372 us for the gradient of 8191 tokens' 8 rows of 14 KB.
template <typename T, int N>
struct Piece;
template <>
struct Piece<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ Raw raw(const __nv_bfloat16* p) { return row::ld_stream(p); }
    static __device__ __forceinline__ void open(float (&v)[8], const uint4& w) { row::unpack8(v, w); }
    static __device__ __forceinline__ void load(float (&v)[8], const __nv_bfloat16* p) {
        row::unpack8(v, row::ld_stream(p));
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
        __stcs(reinterpret_cast<uint4*>(p), row::pack8(v));
    }
};
template <>
struct Piece<float, 4> {
    using Raw = uint4;
    static __device__ __forceinline__ Raw raw(const float* p) { return row::ld_stream(p); }
    static __device__ __forceinline__ void open(float (&v)[4], const uint4& w) {
        v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y);
        v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ void load(float (&v)[4], const float* p) {
        open(v, row::ld_stream(p));
    }
    static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    }
};
template <>
struct Piece<__nv_bfloat16, 1> {
    using Raw = uint16_t;
    static __device__ __forceinline__ Raw raw(const __nv_bfloat16* p) {
        return __ldg(reinterpret_cast<const uint16_t*>(p));
    }
    static __device__ __forceinline__ void open(float (&v)[1], Raw w) { v[0] = row::bf_lo(w); }
    static __device__ __forceinline__ void load(float (&v)[1], const __nv_bfloat16* p) {
        v[0] = __bfloat162float(*p);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[1]) {
        *p = __float2bfloat16_rn(v[0]);
    }
};
template <>
struct Piece<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ Raw raw(const float* p) { return __ldg(p); }
    static __device__ __forceinline__ void open(float (&v)[1], Raw w) { v[0] = w; }
    static __device__ __forceinline__ void load(float (&v)[1], const float* p) { v[0] = *p; }
    static __device__ __forceinline__ void store(float* p, const float (&v)[1]) { *p = v[0]; }
};

// y[t] = sum_j w[t, j] ys[row_of[t, j]] (w null: 1), fp32 in the order of j,
// rounded once.  A CTA takes 256 / lanes tokens; their rows and weights first,
// in shared memory (a dropped slot as -1), then the pieces of eight slots at
// a time, so that a thread has eight loads in flight: 8192 tokens' 8 rows of
// 8 KB in 90 us (6.7 TB/s; four loads behind tests took 160).
template <typename T, int N>
__global__ void __launch_bounds__(kRowThreads)
    moe_unpermute_kernel(const T* __restrict__ ys, const int32_t* __restrict__ row_of,
                         const float* __restrict__ w, int64_t tokens, int slots, int64_t width,
                         int64_t rows, T* __restrict__ y, int lanes) {
    ptx::griddep_launch_dependents();
    __shared__ int from[kRowThreads / 8 * kMaxSlots];
    __shared__ float wt[kRowThreads / 8 * kMaxSlots];
    ptx::griddep_wait();
    const int sub = threadIdx.x / lanes, lane = threadIdx.x % lanes, per = kRowThreads / lanes;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * per, t = t0 + sub;
    for (int i = threadIdx.x; i < per * slots && t0 * slots + i < tokens * slots; i += kRowThreads) {
        const int r = row_of[t0 * slots + i];
        from[i] = r >= 0 && r < rows ? r : -1;
        wt[i] = w ? w[t0 * slots + i] : 1.0f;
    }
    __syncthreads();
    if (t >= tokens) return;
    for (int64_t c = static_cast<int64_t>(lane) * N; c < width; c += static_cast<int64_t>(lanes) * N) {
        float acc[N] = {};
        for (int j = 0; j < slots; j += 8) {
            typename Piece<T, N>::Raw v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = j + i < slots ? from[sub * slots + j + i] : -1;
                v[i] = r >= 0 ? Piece<T, N>::raw(ys + static_cast<int64_t>(r) * width + c)
                              : typename Piece<T, N>::Raw{};
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (j + i >= slots || from[sub * slots + j + i] < 0) continue;
                float x[N];
                Piece<T, N>::open(x, v[i]);
                const float f = wt[sub * slots + j + i];
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] = fmaf(f, x[e], acc[e]);
            }
        }
        Piece<T, N>::store(y + t * width + c, acc);
    }
}

// The gradient of the weighted sum, token by token: dys[row] = w dy[t] and
// dw[t, j] = <dy[t], ys[row]>, so dy is read once for its k rows.  A CTA is a
// token; CTAs past the tokens set the pad rows to zero.
template <typename T, int N>
__global__ void __launch_bounds__(kRowThreads)
    moe_unpermute_bwd_kernel(const T* __restrict__ dy, const T* __restrict__ ys,
                             const int32_t* __restrict__ row_of, const int32_t* __restrict__ src,
                             const float* __restrict__ w, int64_t tokens, int slots, int64_t width,
                             int64_t rows, T* __restrict__ dys, float* __restrict__ dw) {
    ptx::griddep_launch_dependents();
    __shared__ float part[kRowThreads / 32][kMaxSlots];
    ptx::griddep_wait();
    if (blockIdx.x >= tokens) {
        const float zero[N] = {};
        for (int64_t r = blockIdx.x - tokens; r < rows; r += gridDim.x - tokens) {
            if (src[r] >= 0) continue;
            for (int64_t c = static_cast<int64_t>(threadIdx.x) * N; c < width; c += kRowThreads * N)
                Piece<T, N>::store(dys + r * width + c, zero);
        }
        return;
    }
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t* to = row_of + t * slots;
    for (int j = 0; j < slots; ++j) {
        const int64_t r = to[j];
        const float f = w ? w[t * slots + j] : 1.0f;
        float dot = 0.0f;
        if (r >= 0 && r < rows) {
            for (int64_t c = static_cast<int64_t>(threadIdx.x) * N; c < width; c += kRowThreads * N) {
                float g[N], v[N], o[N];
                Piece<T, N>::load(g, dy + t * width + c);
                Piece<T, N>::load(v, ys + r * width + c);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    dot = fmaf(g[e], v[e], dot);
                    o[e] = f * g[e];
                }
                Piece<T, N>::store(dys + r * width + c, o);
            }
        }
        dot = row::warp_sum(dot);
        if (lane == 0) part[warp][j] = dot;
    }
    __syncthreads();
    if (dw && static_cast<int>(threadIdx.x) < slots) {
        float s = 0.0f;
        for (int i = 0; i < kRowThreads / 32; ++i) s += part[i][threadIdx.x];
        dw[t * slots + threadIdx.x] = s;
    }
}

// The same for rows that the CTA's registers hold (VPT pieces a thread): dy is
// read once, and the next slot's piece of ys is loaded while this one's is
// used.  8191 tokens' 8 rows of 14 KB: 364 us (5.8 TB/s; 446 reading dy again
// for each slot, most of it from HBM).  Two and four pieces are held to 64
// registers, for four CTAs an SM (373 us with three, although four bf16 pieces
// then spill 48 bytes), one piece to 32, for eight (8192 tokens' 8 rows of
// 2 KB: 52 us, 62 with five).
template <typename T, int N, int VPT>
__global__ void __launch_bounds__(kRowThreads, VPT == 1 ? 8 : 4)
    moe_unpermute_bwd_held_kernel(const T* __restrict__ dy, const T* __restrict__ ys,
                                  const int32_t* __restrict__ row_of, const int32_t* __restrict__ src,
                                  const float* __restrict__ w, int64_t tokens, int slots,
                                  int64_t width, int64_t rows, T* __restrict__ dys,
                                  float* __restrict__ dw) {
    ptx::griddep_launch_dependents();
    __shared__ float part[kRowThreads / 32][kMaxSlots];
    __shared__ int to[kMaxSlots];
    __shared__ float wt[kMaxSlots];
    ptx::griddep_wait();
    const int threads = static_cast<int>(blockDim.x);
    if (blockIdx.x >= tokens) {
        const float zero[N] = {};
        for (int64_t r = blockIdx.x - tokens; r < rows; r += gridDim.x - tokens) {
            if (src[r] >= 0) continue;
            for (int64_t c = static_cast<int64_t>(threadIdx.x) * N; c < width; c += threads * N)
                Piece<T, N>::store(dys + r * width + c, zero);
        }
        return;
    }
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int j = threadIdx.x; j < slots; j += threads) {
        const int r = row_of[t * slots + j];
        to[j] = r >= 0 && r < rows ? r : -1;
        wt[j] = w ? w[t * slots + j] : 1.0f;
    }
    bool live[VPT];
    uint4 g[VPT], a[VPT], b[VPT];   // dy; ys of this slot and of the next
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t c = static_cast<int64_t>(threadIdx.x + i * threads) * N;
        live[i] = c < width;
        g[i] = live[i] ? row::ld_stream(dy + t * width + c) : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    auto fetch = [&](uint4 (&v)[VPT], int j) {
        const int64_t r = j < slots ? to[j] : -1;
        if (r < 0) return;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i])
                v[i] = row::ld_stream(ys + r * width + static_cast<int64_t>(threadIdx.x + i * threads) * N);
    };
    fetch(b, 0);
    for (int j = 0; j < slots; ++j) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) a[i] = b[i];
        fetch(b, j + 1);
        const int64_t r = to[j];
        float dot = 0.0f;
        if (r >= 0) {
            const float f = wt[j];
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (!live[i]) continue;
                float x[N], y[N], o[N];
                Piece<T, N>::open(x, g[i]);
                Piece<T, N>::open(y, a[i]);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    dot = fmaf(x[e], y[e], dot);
                    o[e] = f * x[e];
                }
                Piece<T, N>::store(dys + r * width + static_cast<int64_t>(threadIdx.x + i * threads) * N, o);
            }
        }
        dot = row::warp_sum(dot);
        if (lane == 0) part[warp][j] = dot;
    }
    if (!dw) return;
    __syncthreads();
    for (int j = threadIdx.x; j < slots; j += threads) {
        float s = 0.0f;
        for (int i = 0; i < threads / 32; ++i) s += part[i][j];
        dw[t * slots + j] = s;
    }
}

// ------------------------------------------------------------------ host side


int check_routing(const char* what, int64_t tokens, int slots, int64_t rows) {
    if (tokens < 0 || slots < 1 || slots > kMaxSlots || rows < 0)
        return set_error(FP8_ERR_SHAPE, "%s: tokens and rows must be >= 0, slots in 1..%d", what,
                         kMaxSlots);
    if (tokens > kMost || tokens * slots > kMost || rows > kMost)
        return set_error(FP8_ERR_SHAPE, "%s: tokens x slots and rows must be at most 2^30", what);
    return FP8_OK;
}

template <typename V>
void launch_permute(const void* x, const float* scale, int64_t tokens, int slots, int64_t row_bytes,
                    const int32_t* row_of, const int32_t* src, int64_t rows, void* xs,
                    float* scale_s, cudaStream_t st) {
    const int64_t units = row_bytes / static_cast<int64_t>(sizeof(V));
    const int lanes = lanes_for(units), per = kRowThreads / lanes;
    const int64_t token_ctas = (tokens + per - 1) / per;
    const int64_t want = (rows + per * 16 - 1) / (per * 16);
    const int64_t pad_ctas = want < 1 ? 1 : (want > 8 * num_sms() ? 8 * num_sms() : want);
    launch_pdl(moe_permute_kernel<V>, dim3(static_cast<unsigned>(token_ctas + pad_ctas)),
               dim3(kRowThreads), 0, st, static_cast<const V*>(x), scale, tokens, slots, units,
               row_of, src, rows, static_cast<V*>(xs), scale_s, lanes, token_ctas);
}

void launch_permute_bytes(const void* x, const float* scale, int64_t tokens, int slots,
                          int64_t row_bytes, const int32_t* row_of, const int32_t* src, int64_t rows,
                          void* xs, float* scale_s, cudaStream_t st) {
    const int64_t want = (rows + 15) / 16;
    const int64_t pad_ctas = want > 8 * num_sms() ? 8 * num_sms() : want;
    launch_pdl(moe_permute_bytes_kernel, dim3(static_cast<unsigned>(tokens + pad_ctas)),
               dim3(kRowThreads), 64 + (row_bytes < kImageBytes ? (row_bytes + 15) / 16 * 16 : kImageBytes),
               st, static_cast<const uint8_t*>(x), scale, tokens, slots, row_bytes, row_of, src, rows,
               static_cast<uint8_t*>(xs), scale_s);
}

int launch_permute_bulk(const void* x, const float* scale, int64_t tokens, int slots,
                        int64_t row_bytes, const int32_t* row_of, const int32_t* src, int64_t rows,
                        void* xs, float* scale_s, cudaStream_t st) {
    BulkRows p{};
    p.x = static_cast<const uint8_t*>(x); p.scale = scale; p.row_of = row_of; p.src = src;
    p.xs = static_cast<uint8_t*>(xs); p.scale_s = scale_s; p.status = device_status_word();
    p.tokens = tokens; p.rows = rows; p.row_bytes = row_bytes; p.slots = slots;
    p.slot_bytes = static_cast<int>(row_bytes < kBulkSlotBytes ? (row_bytes + 127) / 128 * 128 : kBulkSlotBytes);
    p.pieces = static_cast<int>((row_bytes + p.slot_bytes - 1) / p.slot_bytes);
    int warps = (kBulkSmem - p.slot_bytes) / (kBulkSlots * p.slot_bytes);
    if (warps > 8) warps = 8;
    static host::SmemAllowance allowed;
    const int r = host::allow_smem(moe_permute_bulk_kernel, kBulkSmem, allowed);
    if (r != FP8_OK) return r;
    const int smem = (warps * kBulkSlots + 1) * p.slot_bytes;
    // small rows leave room for more CTAs on an SM
    int per_sm = kBulkSmem / smem;
    if (per_sm > 8) per_sm = 8;
    const int64_t work = tokens * p.pieces + rows / 8 + 1;
    const int64_t most = static_cast<int64_t>(num_sms()) * per_sm;
    launch_pdl(moe_permute_bulk_kernel, dim3(static_cast<unsigned>(work < most ? work : most)),
               dim3(warps * 32), smem, st, p);
    return FP8_OK;
}

template <typename T, int N>
void launch_unpermute(const void* ys, const int32_t* row_of, const float* w, int64_t tokens,
                      int slots, int64_t width, int64_t rows, void* y, cudaStream_t st) {
    const int lanes = lanes_for((width + N - 1) / N), per = kRowThreads / lanes;
    launch_pdl(moe_unpermute_kernel<T, N>, dim3(static_cast<unsigned>((tokens + per - 1) / per)),
               dim3(kRowThreads), 0, st, static_cast<const T*>(ys), row_of, w, tokens, slots, width, rows,
               static_cast<T*>(y), lanes);
}

template <typename T, int N>
void launch_unpermute_bwd(const void* dy, const void* ys, const int32_t* row_of, const int32_t* src,
                          const float* w, int64_t tokens, int slots, int64_t width, int64_t rows,
                          void* dys, float* dw, cudaStream_t st) {
    const int64_t want = (rows + 15) / 16;
    const int64_t pad_ctas = want < 1 ? 1 : (want > 8 * num_sms() ? 8 * num_sms() : want);
    const dim3 grid(static_cast<unsigned>(tokens + pad_ctas));
    auto go = [&](auto kernel, int threads) {
        launch_pdl(kernel, grid, dim3(threads), 0, st, static_cast<const T*>(dy),
                   static_cast<const T*>(ys), row_of, src, w, tokens, slots, width, rows,
                   static_cast<T*>(dys), dw);
    };
    if constexpr (N > 1) {
        const int64_t pieces = width / N;
        if (pieces <= kRowThreads)   // a width of 0 still writes dw
            return go(moe_unpermute_bwd_held_kernel<T, N, 1>,
                      pieces < 32 ? 32 : static_cast<int>((pieces + 31) / 32 * 32));
        if (pieces <= 2 * kRowThreads) return go(moe_unpermute_bwd_held_kernel<T, N, 2>, kRowThreads);
        if (pieces <= 4 * kRowThreads) return go(moe_unpermute_bwd_held_kernel<T, N, 4>, kRowThreads);
    }
    go(moe_unpermute_bwd_kernel<T, N>, kRowThreads);
}

}  // namespace
}  // namespace fp8

using namespace fp8;
using namespace fp8::host;

extern "C" {

int64_t fp8_moe_rows(int64_t tokens, int slots, int experts, int align) {
    if (tokens < 0 || slots < 1 || slots > kMaxSlots || experts < 1 || experts > kMaxExperts ||
        align < 1 || align > 4096 || tokens > kMost || tokens * slots > kMost)
        return -1;
    const int64_t n = tokens * slots;
    return n + (n < experts ? n : experts) * (align - 1);
}

size_t fp8_moe_workspace_size(int64_t tokens, int slots, int experts) {
    if (fp8_moe_rows(tokens, slots, experts, 1) < 0) return 0;
    const PlanGrid g = plan_grid(tokens * slots);
    return g.ctas > 1 ? static_cast<size_t>(g.ctas) * experts * sizeof(int32_t) : 0;
}

int fp8_moe_plan(const int32_t* ids, int64_t tokens, int slots, int experts, int align,
                 int32_t* offsets, int32_t* counts, int32_t* row_of, int32_t* src, int64_t rows,
                 void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_routing("fp8_moe_plan", tokens, slots, rows);
    if (st != FP8_OK) return st;
    if (experts < 1 || experts > kMaxExperts)
        return set_error(FP8_ERR_SHAPE, "fp8_moe_plan: experts %d outside 1..%d", experts, kMaxExperts);
    if (align < 1 || align > 4096)
        return set_error(FP8_ERR_SHAPE, "fp8_moe_plan: align %d outside 1..4096", align);
    const int64_t need_rows = fp8_moe_rows(tokens, slots, experts, align);
    if (need_rows < 0 || need_rows > kMost || rows < need_rows)
        return set_error(FP8_ERR_SHAPE, "fp8_moe_plan: %lld rows, %lld needed (fp8_moe_rows)",
                         static_cast<long long>(rows), static_cast<long long>(need_rows));
    if (!offsets || !counts || ((!ids || !row_of) && tokens) || (!src && rows))
        return set_error(FP8_ERR_INVALID_ARG, "fp8_moe_plan: NULL pointer");
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(row_of, 4) ||
        !aligned(src, 4) || !aligned(workspace, 4))
        return set_error(FP8_ERR_ALIGN, "fp8_moe_plan: pointers must be 4-byte aligned");
    const int n = static_cast<int>(tokens * slots);
    const PlanGrid g = plan_grid(n);
    const size_t need = fp8_moe_workspace_size(tokens, slots, experts);
    if (need && (!workspace || workspace_bytes < need))
        return set_error(FP8_ERR_INVALID_ARG, "fp8_moe_plan: workspace of %zu bytes, %zu needed",
                         workspace ? workspace_bytes : size_t{0}, need);
    int32_t* hist = nullptr;
    if (g.ctas > 1) {
        hist = static_cast<int32_t*>(workspace);
        launch_pdl(moe_hist_kernel, dim3(g.ctas), dim3(kPlanThreads), 0, as_stream(stream), ids, n,
                   experts, g.chunk, hist);
    }
    static host::SmemAllowance allowed;
    const int smem = kPlanWarps * experts * static_cast<int>(sizeof(int));
    const int r = smem > 32768 ? host::allow_smem(moe_place_kernel, smem, allowed) : FP8_OK;
    if (r != FP8_OK) return r;
    launch_pdl(moe_place_kernel, dim3(g.ctas), dim3(kPlanThreads), smem, as_stream(stream), ids, n,
               experts, align, g.chunk, static_cast<const int32_t*>(hist), offsets, counts, row_of,
               src, static_cast<int>(rows));
    return launch_status("fp8_moe_plan");
}

int fp8_moe_permute(const void* x, const float* scale, int64_t tokens, int slots, int64_t row_bytes,
                    const int32_t* row_of, const int32_t* src, int64_t rows, void* xs,
                    float* scale_s, void* stream) {
    const int st = check_routing("fp8_moe_permute", tokens, slots, rows);
    if (st != FP8_OK) return st;
    if (row_bytes < 1 || row_bytes > (int64_t{1} << 24))
        return set_error(FP8_ERR_SHAPE, "fp8_moe_permute: row of %lld bytes outside 1..2^24",
                         static_cast<long long>(row_bytes));
    if (((!x || !row_of) && tokens) || ((!xs || !src) && rows))
        return set_error(FP8_ERR_INVALID_ARG, "fp8_moe_permute: NULL pointer");
    if ((scale != nullptr) != (scale_s != nullptr) && tokens && rows)
        return set_error(FP8_ERR_INVALID_ARG, "fp8_moe_permute: scale and scale_s go together");
    if (!aligned(x, 16) || !aligned(xs, 16) || !aligned(row_of, 4) || !aligned(src, 4) ||
        !aligned(scale, 4) || !aligned(scale_s, 4))
        return set_error(FP8_ERR_ALIGN,
                         "fp8_moe_permute: x and xs must be 16-byte aligned, the rest 4-byte");
    if (!rows) return FP8_OK;
    // Rows of whole 16-byte pieces: in bulk copies, short ones (where a copy's
    // fixed cost shows) through registers.  Others: put together from shared
    // memory, short ones in the widest unit that every row starts on.
    if (row_bytes % 16 == 0 && row_bytes >= 1024) {
        const int r = launch_permute_bulk(x, scale, tokens, slots, row_bytes, row_of, src, rows, xs,
                                          scale_s, as_stream(stream));
        if (r != FP8_OK) return r;
    } else if (row_bytes % 16 == 0)
        launch_permute<uint4>(x, scale, tokens, slots, row_bytes, row_of, src, rows, xs, scale_s, as_stream(stream));
    else if (row_bytes >= 512)
        launch_permute_bytes(x, scale, tokens, slots, row_bytes, row_of, src, rows, xs, scale_s, as_stream(stream));
    else if (row_bytes % 4 == 0)
        launch_permute<uint32_t>(x, scale, tokens, slots, row_bytes, row_of, src, rows, xs, scale_s, as_stream(stream));
    else if (row_bytes % 2 == 0)
        launch_permute<uint16_t>(x, scale, tokens, slots, row_bytes, row_of, src, rows, xs, scale_s, as_stream(stream));
    else
        launch_permute<uint8_t>(x, scale, tokens, slots, row_bytes, row_of, src, rows, xs, scale_s, as_stream(stream));
    return launch_status("fp8_moe_permute");
}

int fp8_moe_unpermute(const void* ys, int type, const int32_t* row_of, const float* weights,
                      int64_t tokens, int slots, int64_t width, int64_t rows, void* y, void* stream) {
    const int st = check_routing("fp8_moe_unpermute", tokens, slots, rows);
    if (st != FP8_OK) return st;
    if (type != FP8_OUT_BF16 && type != FP8_OUT_F32)
        return set_error(FP8_ERR_INVALID_ARG, "fp8_moe_unpermute: unknown type %d", type);
    if (width < 0 || width > (int64_t{1} << 22))
        return set_error(FP8_ERR_SHAPE, "fp8_moe_unpermute: width outside 0..2^22");
    if ((!row_of || (!y && width)) && tokens)
        return set_error(FP8_ERR_INVALID_ARG, "fp8_moe_unpermute: NULL pointer");
    if (!ys && tokens && rows && width)
        return set_error(FP8_ERR_INVALID_ARG, "fp8_moe_unpermute: NULL pointer");
    if (!aligned(ys, 16) || !aligned(y, 16) || !aligned(row_of, 4) || !aligned(weights, 4))
        return set_error(FP8_ERR_ALIGN,
                         "fp8_moe_unpermute: ys and y must be 16-byte aligned, the rest 4-byte");
    if (!tokens || !width) return FP8_OK;
    if (type == FP8_OUT_BF16) {
        if (width % 8 == 0)
            launch_unpermute<__nv_bfloat16, 8>(ys, row_of, weights, tokens, slots, width, rows, y, as_stream(stream));
        else
            launch_unpermute<__nv_bfloat16, 1>(ys, row_of, weights, tokens, slots, width, rows, y, as_stream(stream));
    } else if (width % 4 == 0) {
        launch_unpermute<float, 4>(ys, row_of, weights, tokens, slots, width, rows, y, as_stream(stream));
    } else {
        launch_unpermute<float, 1>(ys, row_of, weights, tokens, slots, width, rows, y, as_stream(stream));
    }
    return launch_status("fp8_moe_unpermute");
}

int fp8_moe_unpermute_bwd(const void* dy, const void* ys, int type, const int32_t* row_of,
                          const int32_t* src, const float* weights, int64_t tokens, int slots,
                          int64_t width, int64_t rows, void* dys, float* dweights, void* stream) {
    const int st = check_routing("fp8_moe_unpermute_bwd", tokens, slots, rows);
    if (st != FP8_OK) return st;
    if (type != FP8_OUT_BF16 && type != FP8_OUT_F32)
        return set_error(FP8_ERR_INVALID_ARG, "fp8_moe_unpermute_bwd: unknown type %d", type);
    if (width < 0 || width > (int64_t{1} << 22))
        return set_error(FP8_ERR_SHAPE, "fp8_moe_unpermute_bwd: width outside 0..2^22");
    if (((!dy && width) || !row_of) && tokens)
        return set_error(FP8_ERR_INVALID_ARG, "fp8_moe_unpermute_bwd: NULL pointer");
    if ((!src || ((!ys || !dys) && width)) && rows)
        return set_error(FP8_ERR_INVALID_ARG, "fp8_moe_unpermute_bwd: NULL pointer");
    if (!aligned(dy, 16) || !aligned(ys, 16) || !aligned(dys, 16) || !aligned(row_of, 4) ||
        !aligned(src, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
        return set_error(FP8_ERR_ALIGN, "fp8_moe_unpermute_bwd: dy, ys and dys must be 16-byte "
                                        "aligned, the rest 4-byte");
    if (!tokens && !rows) return FP8_OK;
    if (type == FP8_OUT_BF16) {
        if (width % 8 == 0)
            launch_unpermute_bwd<__nv_bfloat16, 8>(dy, ys, row_of, src, weights, tokens, slots, width, rows, dys, dweights, as_stream(stream));
        else
            launch_unpermute_bwd<__nv_bfloat16, 1>(dy, ys, row_of, src, weights, tokens, slots, width, rows, dys, dweights, as_stream(stream));
    } else if (width % 4 == 0) {
        launch_unpermute_bwd<float, 4>(dy, ys, row_of, src, weights, tokens, slots, width, rows, dys, dweights, as_stream(stream));
    } else {
        launch_unpermute_bwd<float, 1>(dy, ys, row_of, src, weights, tokens, slots, width, rows, dys, dweights, as_stream(stream));
    }
    return launch_status("fp8_moe_unpermute_bwd");
}

}  // extern "C"

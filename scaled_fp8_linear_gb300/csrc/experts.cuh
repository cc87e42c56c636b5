// experts.cuh -- the rows of each expert's product, read from the offsets on the
// device, and the units of work that they are cut into.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "rowops.cuh"

namespace fp8 {
namespace {

constexpr int kMaxGemmExperts = 256;

// A launch's share of each product's rows.  A product whose last 256-row block
// is at most half full can leave that remainder to a second launch in 128-row
// tiles, which starts on the SMs as the first launch's CTAs run out of tiles.
enum { kAllRows = 0, kWholeBlocks = 1, kRemainder = 2 };

// The products' rows and tiles, in shared memory: product e has rows begin[e]
// .. end[e] and units first[e] .. first[e + 1].  One product without offsets.
struct Units {
    int begin[kMaxGemmExperts], end[kMaxGemmExperts];
    int first[kMaxGemmExperts + 1];
};

// Fills `u` (every thread of the CTA; ends with a barrier).  Offsets are held
// to 0 .. M and made never to fall, so whatever they are no unit reaches
// outside and there are no more units than the rows allow.
__device__ __forceinline__ void make_units(Units* u, int M, const int32_t* offsets, int experts, int num_n,
                                           int part, int rows_per_tile) {
    const int t = static_cast<int>(threadIdx.x);
    if (t < 32) {   // one warp, 32 products at a time
        int run = 0, high = offsets ? min(max(offsets[0], 0), M) : 0;
        for (int base = 0; base < experts; base += 32) {
            const int e = base + t;
            const bool on = e < experts;
            // the row after this product's last: the largest offset up to its own
            int end = high;
            if (on) end = max(high, offsets ? min(max(offsets[e + 1], 0), M) : M);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int w = __shfl_up_sync(row::kAll, end, o);
                if (t >= o) end = max(end, w);
            }
            int begin = __shfl_up_sync(row::kAll, end, 1);
            if (t == 0) begin = high;
            high = __shfl_sync(row::kAll, end, 31);
            const int rest = (end - begin) % 256;
            const int left = rest <= 128 ? rest : 0;   // what a second launch takes
            if (part == kWholeBlocks) end -= left;
            if (part == kRemainder) begin = end - left;
            const int n = on ? (end - begin + rows_per_tile - 1) / rows_per_tile * num_n : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int w = __shfl_up_sync(row::kAll, incl, o);
                if (t >= o) incl += w;
            }
            if (on) {
                u->begin[e] = begin;
                u->end[e] = end;
                u->first[e] = run + incl - n;
            }
            run += __shfl_sync(row::kAll, incl, 31);
        }
        if (t == 0) u->first[experts] = run;
    }
    __syncthreads();
}

// The product that a unit belongs to: the last that starts at or before it.
__device__ __forceinline__ int expert_of(int unit, const Units* u, int experts) {
    int lo = 0, hi = experts;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (u->first[mid] <= unit) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace
}  // namespace fp8

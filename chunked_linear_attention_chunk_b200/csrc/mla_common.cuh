// mla_common.cuh -- what the latent-attention kernels share: sizes, packed-sequence lookup.
#pragma once

#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace mla {

constexpr int kDN = 128, kDR = 64, kDV = 128;  // expanded form: key part, shared rotated part, value
constexpr int kDQ = kDN + kDR;                 // query row of a head
constexpr int kDKV = kDN + kDV;                // kv row of a head
constexpr int kDL = 512;                       // absorbed form: latent part of a cached row
constexpr int kDC = kDL + kDR;                 // a cached row

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The packed offsets of one axis are usable: cu[0] = 0, non-decreasing, cu[N] <= T.  All threads
// of the CTA call it (it ends in a barrier).
template <int kThreads>
__device__ __forceinline__ bool offsets_ok(const int32_t *__restrict__ cu, int N, int T)
{
    int bad = 0;
    for (int i = threadIdx.x; i <= N; i += kThreads) {
        const int x = cu[i];
        bad |= x < 0 || x > T || (i == 0 ? x != 0 : x < cu[i - 1]);
    }
    return __syncthreads_or(bad) == 0;
}

// Work item x of the list that has count(0) items for sequence 0, then count(1) for sequence 1,
// and so on: its sequence and its place among that sequence's items.  False past the end.  All
// threads of the CTA call it; `sh` is 36 ints of shared memory.
struct Item {
    int seq, k;
};
template <int kThreads, class Count>
__device__ __forceinline__ bool find_item(int N, int64_t x, Count count, Item &it, int *sh)
{
    static_assert(kThreads % 32 == 0 && kThreads <= 1024, "whole warps");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t base = 0;
    for (int s0 = 0; s0 < N; s0 += kThreads) {
        const int s = s0 + tid;
        const int c = s < N ? count(s) : 0;
        int inc = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, d);
            inc += lane >= d ? y : 0;
        }
        if (lane == 31)
            sh[warp] = inc;
        __syncthreads();
        int before = 0, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            before += w < warp ? sh[w] : 0;
            total += sh[w];
        }
        const int64_t rel = x - base - before - (inc - c);
        if (rel >= 0 && rel < c) {
            sh[33] = s;
            sh[34] = (int)rel;
        }
        __syncthreads();
        base += total;
        if (x < base) {
            it.seq = sh[33];
            it.k = sh[34];
            return true;
        }
    }
    return false;
}

}  // namespace mla
}  // namespace kda

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

// A sum over the CTA; all threads call it.  `sh` is 40 int64 of shared memory.
template <int kThreads>
__device__ __forceinline__ int64_t cta_sum(int64_t x, int64_t *sh)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, d);
    if ((threadIdx.x & 31) == 0)
        sh[threadIdx.x >> 5] = x;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kThreads / 32; ++w)
        total += sh[w];
    __syncthreads();
    return total;
}

// Work item x of the list that has count(0) items for sequence 0, then count(1) for sequence 1,
// and so on: its sequence and its place among that sequence's items.  False past the end.  All
// threads of the CTA call it; `sh` is 40 int64 of shared memory.
struct Item {
    int seq, k;
};
template <int kThreads, class Count>
__device__ __forceinline__ bool find_item(int N, int64_t x, Count count, Item &it, int64_t *sh)
{
    static_assert(kThreads % 32 == 0 && kThreads <= 1024, "whole warps");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t base = 0;
    for (int s0 = 0; s0 < N; s0 += kThreads) {
        const int s = s0 + tid;
        const int64_t c = s < N ? count(s) : 0;
        int64_t inc = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, d);
            inc += lane >= d ? y : 0;
        }
        if (lane == 31)
            sh[warp] = inc;
        __syncthreads();
        int64_t before = 0, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            before += w < warp ? sh[w] : 0;
            total += sh[w];
        }
        const int64_t rel = x - base - before - (inc - c);
        if (rel >= 0 && rel < c) {
            sh[33] = s;
            sh[34] = rel;
        }
        __syncthreads();
        base += total;
        if (x < base) {
            it.seq = (int)sh[33];
            it.k = (int)sh[34];
            return true;
        }
    }
    return false;
}

// 2^x by the hardware's approximation (2 ulp; results below the normal range flush to 0).
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace mla
}  // namespace kda

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
// and so on: its sequence and its place among that sequence's items, or seq = -1 past the end.
// `count` sees every sequence and sets `bad` for what is not to be used; the whole CTA learns of
// it.  Up to 64 sequences one warp goes through the list, beyond that all threads share it (every
// warp by itself would cost the CTA more than the barriers do).  Any 32 counts of usable offsets
// add up to less than 2^31.  All threads call; `sh` is 40 int64 of shared memory.
struct Item {
    int seq, k;
    bool bad;
};
template <int kThreads, class Count>
__device__ __forceinline__ Item find_item(int N, int64_t x, Count count, int64_t *sh)
{
    static_assert(kThreads % 32 == 0 && kThreads <= 1024, "whole warps");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto scan = [&](int c) {  // inclusive sum over the lanes
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, c, d);
            c += lane >= d ? y : 0;
        }
        return c;
    };
    bool bad = false;
    int64_t base = 0;
    if (tid == 0)
        sh[33] = -1;
    __syncwarp();
    if (N <= 64) {
        if (warp == 0) {
            for (int s0 = 0; s0 < N; s0 += 32) {
                const int c = s0 + lane < N ? count(s0 + lane, bad) : 0, inc = scan(c);
                const int64_t rel = x - base - (inc - c);
                if (rel >= 0 && rel < c) {
                    sh[33] = s0 + lane;
                    sh[34] = rel;
                }
                base += __shfl_sync(0xffffffffu, inc, 31);
                __syncwarp();
            }
        }
    } else {
        for (int s0 = 0; s0 < N; s0 += kThreads) {
            const int s = s0 + tid, c = s < N ? count(s, bad) : 0, inc = scan(c);
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
            base += total;
            if (s0 + kThreads < N)
                __syncthreads();
        }
    }
    Item it;
    it.bad = __syncthreads_or(bad) != 0;
    it.seq = (int)sh[33];
    it.k = (int)sh[34];
    return it;
}

// Sequence n's rows [lo, hi) of a packed axis of T; bad unless 0 = cu[0] <= cu[1] <= .. <= T.
struct Span {
    int lo, hi;
    __device__ __forceinline__ int len() const { return hi - lo; }
};
__device__ __forceinline__ Span span_of(const int32_t *__restrict__ cu, int n, int T, bool &bad)
{
    Span s{cu[n], cu[n + 1]};
    bad |= s.lo < 0 || s.hi < s.lo || s.hi > T || (n == 0 && s.lo != 0);
    return s;
}

// Debug builds: whether a CTA's rows [row, row + rows) of a sequence of `len` rows that starts at
// `first` lie in the sequence and on its packed axis of T.  (Offsets, lengths and pages that come from
// device arrays are checked in every build.)
__device__ __forceinline__ bool rows_in(int64_t row, int64_t rows, int64_t len, int64_t first, int64_t T)
{
    return !kDebugChecks || (row >= 0 && rows > 0 && row + rows <= len && first >= 0 && first + len <= T);
}

// 2^x by the hardware's approximation (2 ulp; results below the normal range flush to 0).
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bits [lo, hi) of a word (bounds may lie outside 0 .. 32).
__device__ __forceinline__ uint32_t bit_span(int lo, int hi)
{
    const uint32_t below = hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : (1u << hi) - 1;
    const uint32_t skip = lo >= 32 ? 0xffffffffu : lo <= 0 ? 0u : (1u << lo) - 1;
    return below & ~skip;
}

}  // namespace mla
}  // namespace kda

// mla_tc.cuh -- tensor-core and barrier pieces that the latent-attention kernels share.
#pragma once

#include <cudaTypedefs.h>

#include "mla_common.cuh"
#include "tcgen05.cuh"

namespace kda {
namespace mla {

// Bounded waits of one role.  A try suspends the thread for some microseconds while the barrier is
// not ready, so the limit is of the order of seconds (some 3 us and 3 s measured).  After the first wait
// that runs out the role waits no more, so a broken pipeline ends soon; `finish` records it in the
// status word, once, at the kernel's end (a few instructions a wait matter: the roles' loops share the
// instruction cache).
// The lanes of a warp may disagree about a wait that ran out as its barrier completed, so a role whose
// lanes act together (elect) runs its loop to the end, with nothing to wait for, and what must not
// follow such a wait (a copy) asks for `dead` behind the election.  (Leaving the loop by a vote of the
// lanes cost the issuing warps 1 % of the forward and the backward.)
constexpr uint32_t kWaitTries = 1u << 20;
constexpr unsigned long long kDrainNs = 10000000ull;
struct Waits {
    bool dead;
    uint32_t tries = kWaitTries;
    __device__ __forceinline__ void operator()(uint64_t *bar, uint32_t parity)
    {
        const uint32_t a = smem_u32(bar);
        if (dead)
            return;
#pragma unroll 1
        for (uint32_t n = 0; !mbar_try_wait(a, parity); ++n)
            if (n == tries) {
                dead = true;
                break;
            }
    }
    // Three barriers at once.  A ready wait takes some 300 cycles while copies and products keep
    // shared memory busy; the three tests are in flight together.
    __device__ __forceinline__ void operator()(uint64_t *x, uint32_t px, uint64_t *y, uint32_t py, uint64_t *z, uint32_t pz)
    {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p, q, r;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 r, [%5], %6;\n\t"
            "and.pred p, p, q;\n\t"
            "and.pred p, p, r;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(x)), "r"(px), "r"(smem_u32(y)), "r"(py), "r"(smem_u32(z)), "r"(pz)
            : "memory");
        if (!ok) {
            (*this)(x, px);
            (*this)(y, py);
            (*this)(z, pz);
        }
    }
    // The CTA's roles are over: all threads call.  Where one gave up, copies and products may still be
    // on their way into shared and tensor memory, which go with the CTA: they get some milliseconds.
    __device__ __forceinline__ void finish(unsigned int *status) const
    {
        if (dead)
            report_device_error(status, KDA_ERR_DEVICE_TIMEOUT);
        tc::fence_before_sync();
        if (__syncthreads_or(dead))
            for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < kDrainNs;)
                __nanosleep(1000);
        tc::fence_after_sync();
    }
};

// One lane of a converged warp, the same one every time.  Roles that issue copies or products run
// with all lanes and let the elected one issue: descriptors then stay in uniform registers, which
// measured 30 cycles a 64 x 32 x 16 product against 48 behind `if (lane == 0)`.
__device__ __forceinline__ bool elect()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// Shared-memory descriptors as a constant upper word (strides, swizzle) and a lower word that
// steps with the address (`lo` + bytes / 16).
struct Desc {
    uint32_t lo, hi;
    __device__ __forceinline__ Desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, tc::Swizzle sw)
    {
        const uint64_t d = tc::smem_desc(saddr, lbo, sbo, sw);
        lo = (uint32_t)d;
        hi = (uint32_t)(d >> 32);
    }
    __device__ __forceinline__ uint64_t at(uint32_t bytes) const { return ((uint64_t)hi << 32) | (lo + (bytes >> 4)); }
};

// A place in a ring of kN stages, and the parity of its current round.
template <int kN>
struct Ring {
    uint32_t slot = 0, round = 0;
    __device__ __forceinline__ void step()
    {
        if (++slot == kN) {
            slot = 0;
            ++round;
        }
    }
};

__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Four bytes global -> shared, and an arrival on `bar` (one of its count) once this thread's copies
// so far have landed.
__device__ __forceinline__ void cp_async_4(void *smem, const void *gmem)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A barrier and a vote of one group of four softmax warps.
__device__ __forceinline__ void softmax_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ bool softmax_or(int group, bool x)
{
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 128, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((int)x), "r"(1 + group)
        : "memory");
    return r != 0;
}

// P^T of the decode, MN-major with the swizzle of its row length: [64 rows][NC columns] bfloat16, or
// three terms of [64 rows][NC columns] e5m2 one behind the other (16 columns: side by side in rows of
// 64 bytes).
template <int NC, bool k8>
constexpr uint32_t kPRow = k8 ? (NC == 16 ? 64 : NC) : 2 * NC;  // bytes of a row
template <int NC, bool k8>
__device__ __forceinline__ uint32_t p_off(int row, int col, int term)
{
    if (k8) {
        if (NC == 16)
            return row * 64 + ((term ^ (row >> 1 & 3)) << 4) + col;
        return (term * 64 + row) * NC + (((col >> 4) ^ (NC == 64 ? row >> 1 & 3 : row >> 2 & 1)) << 4) + (col & 15);
    }
    if (NC == 16)
        return row * 32 + (((col >> 3) ^ (row >> 2 & 1)) << 4) + (col & 7) * 2;
    return NC == 64 ? tc::mnmaj_sw128(row, col, 64) : tc::mnmaj_sw64(row, col);
}
template <int NC, bool k8>
__device__ __forceinline__ Desc p_desc(uint32_t base)
{
    if (k8 && NC == 32)  // the terms are the next 32-column atoms of one operand
        return Desc(base, 64 * 32, 256, tc::kSw32);
    if (k8)
        return Desc(base, 0, 512, tc::kSw64);
    return NC == 64 ? Desc(base, 64 * 128, 1024, tc::kSw128)
                    : NC == 32 ? Desc(base, 0, 512, tc::kSw64) : Desc(base, 0, 256, tc::kSw32);
}

// 8, 16 or 32 columns of an M = 64 accumulator in fragment order (see ld_16x256b_x1).
template <int kCols>
__device__ __forceinline__ void load_s(uint32_t taddr, float (&s)[kCols / 8][4])
{
    uint32_t r[kCols / 2];
    if constexpr (kCols == 32)
        tc::ld_16x256b_x4(taddr, r);
    else if constexpr (kCols == 16)
        tc::ld_16x256b_x2(taddr, r);
    else
        tc::ld_16x256b_x1(taddr, r);
    tc::wait_ld();
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i)
        s[i / 4][i % 4] = __uint_as_float(r[i]);
}

// A row of q is t (q1 + q2 / kTerm2) in e4m3 terms.
constexpr float kTerm2 = 32.0f;

// The same and the columns `apart` further on, divided by kTerm2: the two terms' sum.
template <int kCols>
__device__ __forceinline__ void load_s2(uint32_t taddr, uint32_t apart, float (&s)[kCols / 8][4])
{
    float t[kCols / 8][4];
    load_s<kCols>(taddr, s);
    load_s<kCols>(taddr + apart, t);
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i)
        s[i / 4][i % 4] = fmaf(t[i / 4][i % 4], 1.0f / kTerm2, s[i / 4][i % 4]);
}

// 8 or 16 columns of this thread's lane.
template <int kCols>
__device__ __forceinline__ void load_row(uint32_t taddr, uint32_t (&r)[kCols])
{
    if constexpr (kCols == 16)
        tc::ld_32x32b_x16(taddr, r);
    else
        tc::ld_32x32b_x8(taddr, r);
}
template <int kCols>
__device__ __forceinline__ void store_row(uint32_t taddr, const uint32_t (&r)[kCols])
{
    if constexpr (kCols == 16)
        tc::st_32x32b_x16(taddr, r);
    else
        tc::st_32x32b_x8(taddr, r);
}

// A kernel's tensor map (a __grid_constant__ argument) into the descriptor cache.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// cuTensorMapEncodeTiled, reached through the runtime (the library does not link the driver).
inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// A tensor of 2-byte (bfloat16) or 1-byte elements with up to five axes, innermost first: their
// extents, the byte strides of all but the innermost (in any order: an axis may step inside
// another's row), and the box of one copy.  A box row of 128 or 64 bytes is swizzled by that
// length; what lies outside the tensor reads as zeros.
inline cudaError_t make_map(CUtensorMap *m, const void *base, int elem, int rank, const int64_t *extent,
                            const int64_t *stride, const int *box)
{
    const PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
    if (!enc)
        return cudaErrorNotSupported;
    cuuint64_t dims[5], strides[4];
    cuuint32_t b[5], estr[5];
    for (int i = 0; i < rank; ++i) {
        dims[i] = (cuuint64_t)extent[i];
        b[i] = (cuuint32_t)box[i];
        estr[i] = 1;
        if (i > 0)
            strides[i - 1] = (cuuint64_t)stride[i - 1];
    }
    const CUresult r = enc(m, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, rank,
                           const_cast<void *>(base), dims, strides, b, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           box[0] * elem == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Rows of `numbers` bfloat16 for each of H heads ([rows, H, numbers]; H = 0: [rows, numbers]) as
// [block of 64 numbers][head][row][64] (or [row][64]), boxes of box_rows rows and `blocks` blocks
// of one head.
inline cudaError_t make_rows_map(CUtensorMap *m, const void *base, int numbers, int H, int64_t rows, int box_rows,
                                 int blocks)
{
    const int64_t nb = (int64_t)numbers * 2;
    if (H == 0) {
        const int64_t extent[2] = {numbers, rows}, stride[1] = {nb};
        const int box[2] = {64, box_rows};
        return make_map(m, base, 2, 2, extent, stride, box);
    }
    const int64_t extent[4] = {64, rows, H, numbers / 64}, stride[3] = {H * nb, nb, 128};
    const int box[4] = {64, box_rows, 1, blocks};
    return make_map(m, base, 2, 4, extent, stride, box);
}

}  // namespace mla
}  // namespace kda

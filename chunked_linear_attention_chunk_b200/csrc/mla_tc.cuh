// mla_tc.cuh -- tensor-core and barrier pieces that the latent-attention kernels share.
#pragma once

#include <cudaTypedefs.h>

#include "mla_common.cuh"
#include "tcgen05.cuh"

namespace kda {
namespace mla {

// Bounded waits of one role: after the first one that runs out (recorded in the status word) the
// role waits no more, so a broken pipeline ends soon instead of at every barrier's limit.
struct Waits {
    unsigned int *status;
    bool dead;
    __device__ __forceinline__ void operator()(uint64_t *bar, uint32_t parity)
    {
        if (!dead && !mbar_wait_bounded(bar, parity, status))
            dead = true;
    }
};

__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A barrier and a vote of the four softmax warps.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool softmax_or(bool x)
{
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 128, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((int)x)
        : "memory");
    return r != 0;
}

// P^T of the decode: [64 rows][NC columns] bfloat16, MN-major with the swizzle of its row length.
template <int NC>
__device__ __forceinline__ uint32_t p_off(int row, int col)
{
    return NC == 64 ? tc::mnmaj_sw128(row, col, 64) : tc::mnmaj_sw64(row, col);
}
template <int NC>
__device__ __forceinline__ uint64_t p_desc(uint32_t base, int ks)
{
    return NC == 64 ? tc::smem_desc(base + ks * 2048, 64 * 128, 1024, tc::kSw128)
                    : tc::smem_desc(base + ks * 1024, 0, 512, tc::kSw64);
}

// A 64 x NC accumulator of an M = 64 product in fragment order (see ld_16x256b_x4).
template <int NC>
__device__ __forceinline__ void load_s(uint32_t taddr, float (&s)[NC / 8][4])
{
    uint32_t r[NC / 2];
    if constexpr (NC == 64)
        tc::ld_16x256b_x8(taddr, r);
    else
        tc::ld_16x256b_x4(taddr, r);
    tc::wait_ld();
#pragma unroll
    for (int i = 0; i < NC / 2; ++i)
        s[i / 4][i % 4] = __uint_as_float(r[i]);
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

// A 3-D tensor of 2-byte (bfloat16) or 1-byte elements, innermost extent first, with the byte
// strides of the outer two; boxes whose rows are 128 or 64 bytes, swizzled by that length, zeros
// outside the tensor.
inline cudaError_t make_map_3d(CUtensorMap *m, const void *base, int elem, int64_t d0, int64_t d1, int64_t d2,
                               int64_t s1, int64_t s2, int b0, int b1, int b2)
{
    const PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
    if (!enc)
        return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
    const cuuint64_t strides[2] = {(cuuint64_t)s1, (cuuint64_t)s2};
    const cuuint32_t box[3] = {(cuuint32_t)b0, (cuuint32_t)b1, (cuuint32_t)b2};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r =
        enc(m, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            b0 * elem == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace mla
}  // namespace kda

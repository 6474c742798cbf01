// api_checks.h -- argument-check helpers shared by the extern "C" entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>
#include <initializer_list>

#include "../../include/kda.h"

namespace kda {

constexpr int64_t kMaxElems = (int64_t)1 << 40;
constexpr int kMaxPackedTokens = 0x7fffffff - 64;  // packed axis; cu_seqlens are int32

struct Range {
    uintptr_t lo = 0, hi = 0;  // [lo, hi)
    Range() = default;
    Range(const void *p, int64_t bytes) : lo((uintptr_t)p), hi((uintptr_t)p + (uintptr_t)(bytes > 0 ? bytes : 0)) {}
    bool empty() const { return lo == 0 || hi <= lo; }
};

inline bool overlaps(const Range &x, const Range &y)
{
    if (x.empty() || y.empty())
        return false;
    return x.lo < y.hi && y.lo < x.hi;
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// beta is read one element at a time: its natural alignment is enough.
inline bool beta_aligned(const void *beta, int es) { return ((uintptr_t)beta % (uintptr_t)es) == 0; }

inline int elem_size(kda_dtype dt) { return dt == KDA_BF16 ? 2 : 4; }

inline bool dtype_ok(kda_dtype dt) { return dt == KDA_BF16 || dt == KDA_F32; }

inline kda_status check_gmin(float g_min)
{
    if (!std::isfinite(g_min) || !(g_min < 0.0f))
        return KDA_ERR_INVALID_ARG;
    if (g_min < KDA_G_MIN_LOWEST)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

inline kda_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// Product of non-negative ints with an overflow bound; -1 when it exceeds kMaxElems.
inline int64_t safe_prod(std::initializer_list<int64_t> xs)
{
    int64_t p = 1;
    for (int64_t x : xs) {
        if (x < 0)
            return -1;
        if (x != 0 && p > kMaxElems / x)
            return -1;
        p *= x;
    }
    return p;
}

// The pointers that are not null are 16-byte aligned.
inline bool all_aligned(std::initializer_list<const void *> ps)
{
    for (const void *p : ps)
        if (p && !aligned16(p))
            return false;
    return true;
}

}  // namespace kda

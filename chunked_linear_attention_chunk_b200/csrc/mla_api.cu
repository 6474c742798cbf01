// mla_api.cu -- the extern "C" boundary of the latent-attention operators: argument and
// aliasing checks, workspace sizing and dispatch.  See include/kda.h for their contract.
#include "api_checks.h"
#include "kda_common.cuh"
#include "kda_internal.h"

using namespace kda;

namespace {

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

struct Tensor {
    const void *p;
    int64_t bytes;
    bool out;
};

// No output overlaps another output or an input.
bool any_alias(std::initializer_list<Tensor> ts)
{
    for (const Tensor *x = ts.begin(); x != ts.end(); ++x)
        for (const Tensor *y = x + 1; y != ts.end(); ++y)
            if ((x->out || y->out) && overlaps(Range(x->p, x->bytes), Range(y->p, y->bytes)))
                return true;
    return false;
}

kda_status check_expanded(int N, int Tq, int Tk, int H, int dn, int dr, int dv, kda_dtype dtype, float scale)
{
    if (N < 1 || Tq < 0 || Tk < 0 || H < 1 || dn < 1 || dr < 1 || dv < 1 || !dtype_ok(dtype))
        return KDA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f))
        return KDA_ERR_INVALID_ARG;
    if (N > 65535 || H > 65535 || Tq > kMaxPackedTokens || Tk > kMaxPackedTokens || dn != 128 || dr != 64 ||
        dv != 128 || dtype != KDA_BF16)
        return KDA_ERR_UNSUPPORTED;
    if (safe_prod({Tq, H, dn + dr}) < 0 || safe_prod({Tk, H, dn + dv}) < 0)
        return KDA_ERR_INVALID_ARG;
    if (((int64_t)(Tq > Tk ? Tq : Tk) / 128 + N) * H > 0x7fffffff)  // blocks of a launch
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

bool page_size_ok(int ps) { return ps == 16 || ps == 32 || (ps >= 64 && ps % 64 == 0 && ps <= 65536); }

kda_status check_cache(int N, int G, int dl, int dr, kda_dtype dtype, kda_dtype cache_dtype, const void *cache,
                       const float *cache_scale, int num_pages, int page_size, const int32_t *block_table,
                       int max_pages, const int32_t *kv_lens)
{
    if (N < 1 || G < 1 || dl < 1 || dr < 1 || !dtype_ok(dtype) || num_pages < 1 || page_size < 1 || max_pages < 1)
        return KDA_ERR_INVALID_ARG;
    if (cache_dtype != KDA_BF16 && cache_dtype != KDA_E4M3 && cache_dtype != KDA_F32)
        return KDA_ERR_INVALID_ARG;
    if (dl != 512 || dr != 64 || dtype != KDA_BF16 || cache_dtype == KDA_F32 || !page_size_ok(page_size) || N > 65535 ||
        G > 1024)
        return KDA_ERR_UNSUPPORTED;
    // rows of the pool and of a sequence are 32-bit, the latter up to the end of its last 64-row tile
    if (safe_prod({num_pages, page_size, G}) < 0 || (int64_t)num_pages * page_size * G > 0x7fffffff ||
        (int64_t)max_pages * page_size > 0x7fffffc0 / G || safe_prod({num_pages, page_size, G, dl + dr}) < 0)
        return KDA_ERR_UNSUPPORTED;
    if (!cache || !block_table || !kv_lens || (cache_dtype == KDA_E4M3) != (cache_scale != nullptr))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(cache) || !aligned4(cache_scale) || !aligned4(block_table) || !aligned4(kv_lens))
        return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}

kda_status append(uint32_t late_us, int N, const int32_t *cu_new, int T_new, int G, int dl, int dr, kda_dtype dtype,
                  const void *kv_new, const int32_t *kv_lens, const int32_t *block_table, int max_pages,
                  kda_dtype cache_dtype, void *cache, float *cache_scale, int num_pages, int page_size,
                  kda_stream_t stream)
{
    if (T_new < 0 || !cu_new)
        return KDA_ERR_INVALID_ARG;
    const kda_status st = check_cache(N, G, dl, dr, dtype, cache_dtype, cache, cache_scale, num_pages, page_size,
                                      block_table, max_pages, kv_lens);
    if (st != KDA_OK)
        return st;
    if (T_new > kMaxPackedTokens || safe_prod({T_new, G, dl + dr}) < 0)
        return KDA_ERR_UNSUPPORTED;
    if (T_new == 0)
        return KDA_OK;
    if (!kv_new)
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(kv_new) || !aligned4(cu_new))
        return KDA_ERR_ALIGNMENT;
    const int64_t row = (dl + dr) * (cache_dtype == KDA_BF16 ? 2 : 1);
    if (any_alias({{kv_new, (int64_t)T_new * G * (dl + dr) * 2, false},
                   {cu_new, (N + 1) * 4ll, false},
                   {block_table, (int64_t)N * max_pages * 4, false},
                   {kv_lens, N * 4ll, false},
                   {cache, (int64_t)num_pages * page_size * G * row, true},
                   {cache_scale, cache_scale ? (int64_t)num_pages * G * 4 : 0, true}}))
        return KDA_ERR_ALIAS;
    return from_cuda(launch_mla_append(N, cu_new, T_new, G, kv_new, kv_lens, block_table, max_pages,
                                       cache_dtype == KDA_E4M3, cache, cache_scale, num_pages, page_size, late_us,
                                       (cudaStream_t)stream));
}

}  // namespace

extern "C" {

kda_status kda_mla_fwd(int N, const int32_t *cu_q, const int32_t *cu_k, int Tq, int Tk, int H, int dn, int dr, int dv,
                       kda_dtype dtype, int causal, float scale, const void *q, const void *kv, const void *k_rope,
                       void *o, float *lse, kda_stream_t stream)
{
    const kda_status st = check_expanded(N, Tq, Tk, H, dn, dr, dv, dtype, scale);
    if (st != KDA_OK)
        return st;
    if (!cu_q || !cu_k)
        return KDA_ERR_INVALID_ARG;
    if (Tq == 0)
        return KDA_OK;
    if (!q || !o || (Tk > 0 && (!kv || !k_rope)))
        return KDA_ERR_INVALID_ARG;
    if (!all_aligned({q, kv, k_rope, o}) || !aligned4(lse) || !aligned4(cu_q) || !aligned4(cu_k))
        return KDA_ERR_ALIGNMENT;
    const int64_t nq = (int64_t)Tq * H, nk = (int64_t)Tk * H;
    if (any_alias({{q, nq * (dn + dr) * 2, false},
                   {kv, nk * (dn + dv) * 2, false},
                   {k_rope, (int64_t)Tk * dr * 2, false},
                   {cu_q, (N + 1) * 4ll, false},
                   {cu_k, (N + 1) * 4ll, false},
                   {o, nq * dv * 2, true},
                   {lse, lse ? nq * 4 : 0, true}}))
        return KDA_ERR_ALIAS;
    return from_cuda(launch_mla_fwd(N, cu_q, cu_k, Tq, Tk, H, causal != 0, scale, q, kv, k_rope, o, lse,
                                    (cudaStream_t)stream));
}

size_t kda_mla_bwd_workspace(int Tq, int Tk, int H, int dn, int dr, int dv, kda_dtype dtype)
{
    if (check_expanded(1, Tq, Tk, H, dn, dr, dv, dtype, 1.0f) != KDA_OK)
        return 0;
    return mla_bwd_workspace(Tq, Tk, H);
}

kda_status kda_mla_bwd(int N, const int32_t *cu_q, const int32_t *cu_k, int Tq, int Tk, int H, int dn, int dr, int dv,
                       kda_dtype dtype, int causal, float scale, const void *q, const void *kv, const void *k_rope,
                       const void *o, const float *lse, const void *dO, void *dq, void *dkv, void *dk_rope,
                       void *workspace, size_t ws_bytes, kda_stream_t stream)
{
    const kda_status st = check_expanded(N, Tq, Tk, H, dn, dr, dv, dtype, scale);
    if (st != KDA_OK)
        return st;
    if (!cu_q || !cu_k)
        return KDA_ERR_INVALID_ARG;
    if (Tq == 0 && Tk == 0)
        return KDA_OK;
    if (Tq > 0 && (!q || !o || !lse || !dO || !dq))
        return KDA_ERR_INVALID_ARG;
    if (Tk > 0 && (!kv || !k_rope || !dkv || !dk_rope))
        return KDA_ERR_INVALID_ARG;
    if (!all_aligned({q, kv, k_rope, o, dO, dq, dkv, dk_rope, workspace}) || !aligned4(lse) || !aligned4(cu_q) ||
        !aligned4(cu_k))
        return KDA_ERR_ALIGNMENT;
    const size_t need = mla_bwd_workspace(Tq, Tk, H);
    if (!workspace || ws_bytes < need)
        return KDA_ERR_WORKSPACE;
    const int64_t nq = (int64_t)Tq * H, nk = (int64_t)Tk * H;
    if (any_alias({{q, nq * (dn + dr) * 2, false},
                   {kv, nk * (dn + dv) * 2, false},
                   {k_rope, (int64_t)Tk * dr * 2, false},
                   {o, nq * dv * 2, false},
                   {lse, nq * 4, false},
                   {dO, nq * dv * 2, false},
                   {cu_q, (N + 1) * 4ll, false},
                   {cu_k, (N + 1) * 4ll, false},
                   {dq, nq * (dn + dr) * 2, true},
                   {dkv, nk * (dn + dv) * 2, true},
                   {dk_rope, (int64_t)Tk * dr * 2, true},
                   {workspace, (int64_t)need, true}}))
        return KDA_ERR_ALIAS;
    return from_cuda(launch_mla_bwd(N, cu_q, cu_k, Tq, Tk, H, causal != 0, scale, q, kv, k_rope, o, lse, dO, dq, dkv,
                                    dk_rope, workspace, (cudaStream_t)stream));
}

size_t kda_mla_decode_workspace(int N, int Sq, int H, int G, int dl, int dr)
{
    if (N < 1 || Sq < 1 || H < 1 || G < 1 || H % G != 0 || dl != 512 || dr != 64 || N > 65535 || G > 1024 ||
        safe_prod({N, Sq, H, dl + dr}) < 0)
        return 0;
    return mla_decode_workspace(N, Sq, H, G);
}

kda_status kda_mla_decode(int N, int Sq, int H, int G, int dl, int dr, kda_dtype dtype, float scale, const void *q,
                          kda_dtype cache_dtype, const void *cache, const float *cache_scale, int num_pages,
                          int page_size, const int32_t *block_table, int max_pages, const int32_t *kv_lens, void *o,
                          float *lse, void *workspace, size_t ws_bytes, kda_stream_t stream)
{
    if (Sq < 1 || H < 1 || !std::isfinite(scale) || !(scale > 0.0f))
        return KDA_ERR_INVALID_ARG;
    const kda_status st = check_cache(N, G, dl, dr, dtype, cache_dtype, cache, cache_scale, num_pages, page_size,
                                      block_table, max_pages, kv_lens);
    if (st != KDA_OK)
        return st;
    if (H % G != 0 || !q || !o)
        return KDA_ERR_INVALID_ARG;
    const int64_t rows = safe_prod({N, Sq, H}), nq = safe_prod({N, Sq, H, dl + dr});
    if (rows < 0 || nq < 0 || rows > 0x7fffffff)
        return KDA_ERR_UNSUPPORTED;
    if (!all_aligned({q, o, workspace}) || !aligned4(lse))
        return KDA_ERR_ALIGNMENT;
    const size_t need = mla_decode_workspace(N, Sq, H, G);
    if (need > 0 && (!workspace || ws_bytes < need))
        return KDA_ERR_WORKSPACE;
    const int64_t row = (dl + dr) * (cache_dtype == KDA_BF16 ? 2 : 1);
    if (any_alias({{q, nq * 2, false},
                   {cache, (int64_t)num_pages * page_size * G * row, false},
                   {cache_scale, cache_scale ? (int64_t)num_pages * G * 4 : 0, false},
                   {block_table, (int64_t)N * max_pages * 4, false},
                   {kv_lens, N * 4ll, false},
                   {o, rows * dl * 2, true},
                   {lse, lse ? rows * 4 : 0, true},
                   {workspace, (int64_t)need, true}}))
        return KDA_ERR_ALIAS;
    return from_cuda(launch_mla_decode(N, Sq, H, G, scale, q, cache_dtype == KDA_E4M3, cache, cache_scale, num_pages,
                                       page_size, block_table, max_pages, kv_lens, o, lse, workspace,
                                       (cudaStream_t)stream));
}

kda_status kda_mla_cache_append(int N, const int32_t *cu_new, int T_new, int G, int dl, int dr, kda_dtype dtype,
                                const void *kv_new, const int32_t *kv_lens, const int32_t *block_table, int max_pages,
                                kda_dtype cache_dtype, void *cache, float *cache_scale, int num_pages, int page_size,
                                kda_stream_t stream)
{
    return append(0, N, cu_new, T_new, G, dl, dr, dtype, kv_new, kv_lens, block_table, max_pages, cache_dtype, cache,
                  cache_scale, num_pages, page_size, stream);
}

kda_status kda_selftest_append_timeout(uint32_t limit_us, int N, const int32_t *cu_new, int T_new, int G, int dl, int dr,
                                       kda_dtype dtype, const void *kv_new, const int32_t *kv_lens,
                                       const int32_t *block_table, int max_pages, kda_dtype cache_dtype, void *cache,
                                       float *cache_scale, int num_pages, int page_size, kda_stream_t stream)
{
    if (limit_us < 1 || limit_us > 2000000u)
        return KDA_ERR_INVALID_ARG;
    return append(limit_us, N, cu_new, T_new, G, dl, dr, dtype, kv_new, kv_lens, block_table, max_pages, cache_dtype,
                  cache, cache_scale, num_pages, page_size, stream);
}

}  // extern "C"

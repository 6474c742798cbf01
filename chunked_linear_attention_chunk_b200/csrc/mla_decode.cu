// mla_decode.cu -- absorbed latent attention of a few new tokens over a paged cache.
//
//   s_j = scale q . c_j,  o = sum_j softmax_j(s) c_j[0:512]
// One warp per (sequence, token, head); its lanes hold the query row and o.
#include <cuda_fp8.h>

#include "mla_common.cuh"

namespace kda {

namespace {

using namespace mla;

constexpr int kThreads = 256;

struct DecArgs {
    int N, Sq, H, G, num_pages, page_size, max_pages;
    float scale;
    const __nv_bfloat16 *q;
    const void *cache;
    const float *cache_scale;
    const int32_t *block_table, *kv_lens;
    __nv_bfloat16 *o;
    float *lse;
    unsigned int *status;
};

template <bool kE4M3>
__device__ __forceinline__ float element(const void *p, int64_t i)
{
    if constexpr (kE4M3)
        return float(static_cast<const __nv_fp8_e4m3 *>(p)[i]);
    else
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

template <bool kE4M3>
__global__ void __launch_bounds__(kThreads) mla_decode_kernel(DecArgs a)
{
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (unit >= (int64_t)a.N * a.Sq * a.H)
        return;
    const int n = (int)(unit / ((int64_t)a.Sq * a.H)), i = (int)(unit / a.H % a.Sq), h = (int)(unit % a.H);
    const int g = h / (a.H / a.G), len = a.kv_lens[n];
    if (len < 0 || len > (int64_t)a.max_pages * a.page_size) {
        report_device_error(a.status, KDA_ERR_INVALID_ARG);
        return;
    }
    const int last = max(0, len - a.Sq + 1 + i);
    float qf[18], acc[16] = {}, m = -INFINITY, l = 0.0f;
    for (int c = 0; c < 18; ++c)
        qf[c] = __bfloat162float(a.q[unit * kDC + c * 32 + lane]) * a.scale;
    for (int j = 0; j < last; ++j) {
        const int page = a.block_table[(int64_t)n * a.max_pages + j / a.page_size];
        if (page < 0 || page >= a.num_pages) {
            report_device_error(a.status, KDA_ERR_INVALID_ARG);
            return;
        }
        const int64_t row = (((int64_t)page * a.page_size + j % a.page_size) * a.G + g) * kDC;
        const float sc = kE4M3 ? a.cache_scale[(int64_t)page * a.G + g] : 1.0f;
        float x[18], s = 0.0f;
        for (int c = 0; c < 18; ++c) {
            x[c] = element<kE4M3>(a.cache, row + c * 32 + lane) * sc;
            s += qf[c] * x[c];
        }
        s = warp_sum(s);
        const float mn = fmaxf(m, s), r = expf(m - mn), p = expf(s - mn);
        l = l * r + p;
        m = mn;
        for (int c = 0; c < 16; ++c)
            acc[c] = acc[c] * r + p * x[c];
    }
    for (int c = 0; c < 16; ++c)
        a.o[unit * kDL + c * 32 + lane] = __float2bfloat16(last > 0 ? acc[c] / l : 0.0f);
    if (a.lse && lane == 0)
        a.lse[unit] = last > 0 ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t mla_decode_workspace(int, int, int, int) { return 256; }

cudaError_t launch_mla_decode(int N, int Sq, int H, int G, float scale, const void *q, bool e4m3, const void *cache,
                              const float *cache_scale, int num_pages, int page_size, const int32_t *block_table,
                              int max_pages, const int32_t *kv_lens, void *o, float *lse, void *, cudaStream_t s)
{
    DecArgs a{N, Sq, H, G, num_pages, page_size, max_pages, scale, static_cast<const __nv_bfloat16 *>(q), cache,
              cache_scale, block_table, kv_lens, static_cast<__nv_bfloat16 *>(o), lse, device_status_ptr()};
    if (!a.status)
        return cudaErrorInvalidDevice;
    const int64_t units = (int64_t)N * Sq * H;
    (e4m3 ? mla_decode_kernel<true> : mla_decode_kernel<false>)<<<(unsigned)((units + 7) / 8), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kda

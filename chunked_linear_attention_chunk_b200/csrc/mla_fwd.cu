// mla_fwd.cu -- expanded latent attention over packed sequences, forward.
//
//   s_ij = scale (q_i . [k_j, k_rope_j]),  o_i = sum_j e^{s_ij - lse_i} v_j
// with the running maximum and sum of the softmax in float32.  One warp per (query, head): its
// lanes hold the query row, walk the visible keys and keep o in registers.
#include "mla_common.cuh"

namespace kda {

namespace {

using namespace mla;

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
    mla_fwd_kernel(int N, const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, int Tq, int Tk, int H,
                   bool causal, float scale, const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ kv,
                   const __nv_bfloat16 *__restrict__ kr, __nv_bfloat16 *__restrict__ o, float *__restrict__ lse,
                   unsigned int *status)
{
    const bool okq = offsets_ok<kThreads>(cu_q, N, Tq), okk = offsets_ok<kThreads>(cu_k, N, Tk);
    if (!okq || !okk) {
        if (threadIdx.x == 0)
            report_device_error(status, KDA_ERR_INVALID_ARG);
        return;
    }
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t row = unit / H;
    const int h = (int)(unit % H);
    if (row >= cu_q[N])
        return;
    int lo = 0, hi = N;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu_q[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    const int lq = cu_q[lo + 1] - cu_q[lo], lk = cu_k[lo + 1] - cu_k[lo], i = (int)(row - cu_q[lo]);
    const int last = causal ? min(lk, max(0, i + lk - lq + 1)) : lk;
    float qf[6], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.0f;
    for (int c = 0; c < 6; ++c)
        qf[c] = __bfloat162float(q[(row * H + h) * kDQ + c * 32 + lane]) * scale;
    for (int j = 0; j < last; ++j) {
        const int64_t t = cu_k[lo] + j;
        const __nv_bfloat16 *kvr = kv + (t * H + h) * kDKV;
        float s = 0.0f;
        for (int c = 0; c < 4; ++c)
            s += qf[c] * __bfloat162float(kvr[c * 32 + lane]);
        for (int c = 0; c < 2; ++c)
            s += qf[4 + c] * __bfloat162float(kr[t * kDR + c * 32 + lane]);
        s = warp_sum(s);
        const float mn = fmaxf(m, s), r = expf(m - mn), p = expf(s - mn);
        l = l * r + p;
        m = mn;
        for (int c = 0; c < 4; ++c)
            acc[c] = acc[c] * r + p * __bfloat162float(kvr[kDN + c * 32 + lane]);
    }
    for (int c = 0; c < 4; ++c)
        o[(row * H + h) * kDV + c * 32 + lane] = __float2bfloat16(last > 0 ? acc[c] / l : 0.0f);
    if (lse && lane == 0)
        lse[row * H + h] = last > 0 ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_mla_fwd(int N, const int32_t *cu_q, const int32_t *cu_k, int Tq, int Tk, int H, bool causal,
                           float scale, const void *q, const void *kv, const void *k_rope, void *o, float *lse,
                           cudaStream_t s)
{
    unsigned int *status = device_status_ptr();
    if (!status)
        return cudaErrorInvalidDevice;
    const int64_t units = (int64_t)Tq * H, grid = (units + kThreads / 32 - 1) / (kThreads / 32);
    mla_fwd_kernel<<<(unsigned)grid, kThreads, 0, s>>>(
        N, cu_q, cu_k, Tq, Tk, H, causal, scale, static_cast<const __nv_bfloat16 *>(q),
        static_cast<const __nv_bfloat16 *>(kv), static_cast<const __nv_bfloat16 *>(k_rope),
        static_cast<__nv_bfloat16 *>(o), lse, status);
    return cudaGetLastError();
}

}  // namespace kda

// mla_bwd.cu -- gradients of the expanded latent attention over packed sequences.
//
//   p_ij = e^{s_ij - lse_i},  dS_ij = scale p_ij (dO_i . v_j - D_i),  D_i = dO_i . o_i
// One warp per (query, head) sums dq over its keys; one per (key, head) sums dk, dv and its
// head's part of dk_rope over its queries; the parts are then added over the heads in order.
#include "mla_common.cuh"

namespace kda {

namespace {

using namespace mla;

constexpr int kThreads = 256;

__device__ __forceinline__ int seq_of(const int32_t *__restrict__ cu, int N, int64_t row)
{
    int lo = 0, hi = N;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ float at(const __nv_bfloat16 *p, int64_t i) { return __bfloat162float(p[i]); }

struct BwdArgs {
    int N, Tq, Tk, H;
    bool causal;
    float scale;
    const int32_t *cu_q, *cu_k;
    const __nv_bfloat16 *q, *kv, *kr, *o, *dO;
    const float *lse;
    __nv_bfloat16 *dq, *dkv, *dkr;
    float *delta, *part;
    unsigned int *status;
};

__device__ __forceinline__ bool axes_ok(const BwdArgs &a)
{
    const bool okq = offsets_ok<kThreads>(a.cu_q, a.N, a.Tq), okk = offsets_ok<kThreads>(a.cu_k, a.N, a.Tk);
    if (!okq || !okk) {
        if (threadIdx.x == 0)
            report_device_error(a.status, KDA_ERR_INVALID_ARG);
        return false;
    }
    return true;
}

__global__ void __launch_bounds__(kThreads) mla_dq_kernel(BwdArgs a)
{
    if (!axes_ok(a))
        return;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, h = (int)(unit % a.H);
    const int64_t row = unit / a.H;
    if (row >= a.cu_q[a.N])
        return;
    const int n = seq_of(a.cu_q, a.N, row);
    const int lq = a.cu_q[n + 1] - a.cu_q[n], lk = a.cu_k[n + 1] - a.cu_k[n], i = (int)(row - a.cu_q[n]);
    const int last = a.causal ? min(lk, max(0, i + lk - lq + 1)) : lk;
    const int64_t r = row * a.H + h;
    float qf[6], dof[4], dq[6] = {}, delta = 0.0f;
    for (int c = 0; c < 6; ++c)
        qf[c] = at(a.q, r * kDQ + c * 32 + lane) * a.scale;
    for (int c = 0; c < 4; ++c) {
        dof[c] = at(a.dO, r * kDV + c * 32 + lane);
        delta += dof[c] * at(a.o, r * kDV + c * 32 + lane);
    }
    delta = warp_sum(delta);
    if (lane == 0)
        a.delta[r] = delta;
    const float lse = a.lse[r];
    for (int j = 0; j < last; ++j) {
        const int64_t t = a.cu_k[n] + j, kvr = (t * a.H + h) * kDKV;
        float kf[6], s = 0.0f, dp = 0.0f;
        for (int c = 0; c < 6; ++c) {
            kf[c] = c < 4 ? at(a.kv, kvr + c * 32 + lane) : at(a.kr, t * kDR + (c - 4) * 32 + lane);
            s += qf[c] * kf[c];
        }
        for (int c = 0; c < 4; ++c)
            dp += dof[c] * at(a.kv, kvr + kDN + c * 32 + lane);
        const float ds = a.scale * expf(warp_sum(s) - lse) * (warp_sum(dp) - delta);
        for (int c = 0; c < 6; ++c)
            dq[c] += ds * kf[c];
    }
    for (int c = 0; c < 6; ++c)
        a.dq[r * kDQ + c * 32 + lane] = __float2bfloat16(dq[c]);
}

__global__ void __launch_bounds__(kThreads) mla_dkv_kernel(BwdArgs a)
{
    if (!axes_ok(a))
        return;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, h = (int)(unit % a.H);
    const int64_t t = unit / a.H;
    if (t >= a.cu_k[a.N])
        return;
    const int n = seq_of(a.cu_k, a.N, t);
    const int lq = a.cu_q[n + 1] - a.cu_q[n], lk = a.cu_k[n + 1] - a.cu_k[n], j = (int)(t - a.cu_k[n]);
    const int first = a.causal ? max(0, j - (lk - lq)) : 0;
    const int64_t kvr = (t * a.H + h) * kDKV;
    float kf[6], vf[4], dk[6] = {}, dv[4] = {};
    for (int c = 0; c < 6; ++c)
        kf[c] = (c < 4 ? at(a.kv, kvr + c * 32 + lane) : at(a.kr, t * kDR + (c - 4) * 32 + lane)) * a.scale;
    for (int c = 0; c < 4; ++c)
        vf[c] = at(a.kv, kvr + kDN + c * 32 + lane);
    for (int i = first; i < lq; ++i) {
        const int64_t r = (int64_t)(a.cu_q[n] + i) * a.H + h;
        float qf[6], dof[4], s = 0.0f, dp = 0.0f;
        for (int c = 0; c < 6; ++c) {
            qf[c] = at(a.q, r * kDQ + c * 32 + lane);
            s += qf[c] * kf[c];
        }
        for (int c = 0; c < 4; ++c) {
            dof[c] = at(a.dO, r * kDV + c * 32 + lane);
            dp += dof[c] * vf[c];
        }
        const float p = expf(warp_sum(s) - a.lse[r]);
        const float ds = a.scale * p * (warp_sum(dp) - a.delta[r]);
        for (int c = 0; c < 6; ++c)
            dk[c] += ds * qf[c];
        for (int c = 0; c < 4; ++c)
            dv[c] += p * dof[c];
    }
    for (int c = 0; c < 4; ++c) {
        a.dkv[kvr + c * 32 + lane] = __float2bfloat16(dk[c]);
        a.dkv[kvr + kDN + c * 32 + lane] = __float2bfloat16(dv[c]);
    }
    for (int c = 0; c < 2; ++c)
        a.part[(t * a.H + h) * kDR + c * 32 + lane] = dk[4 + c];
}

__global__ void __launch_bounds__(kThreads) mla_dkr_kernel(BwdArgs a)
{
    if (!axes_ok(a))
        return;
    const int64_t x = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t t = x / kDR;
    if (t >= a.cu_k[a.N])
        return;
    float sum = 0.0f;
    for (int h = 0; h < a.H; ++h)
        sum += a.part[(t * a.H + h) * kDR + x % kDR];
    a.dkr[x] = __float2bfloat16(sum);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t mla_bwd_workspace(int Tq, int Tk, int H)
{
    return round256((size_t)Tq * H * 4) + round256((size_t)Tk * H * kDR * 4) + 256;
}

cudaError_t launch_mla_bwd(int N, const int32_t *cu_q, const int32_t *cu_k, int Tq, int Tk, int H, bool causal,
                           float scale, const void *q, const void *kv, const void *k_rope, const void *o,
                           const float *lse, const void *dO, void *dq, void *dkv, void *dk_rope, void *workspace,
                           cudaStream_t s)
{
    typedef const __nv_bfloat16 *In;
    typedef __nv_bfloat16 *Out;
    BwdArgs a{N, Tq, Tk, H, causal, scale, cu_q, cu_k, In(q), In(kv), In(k_rope), In(o), In(dO), lse,
              Out(dq), Out(dkv), Out(dk_rope), static_cast<float *>(workspace),
              reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + round256((size_t)Tq * H * 4)),
              device_status_ptr()};
    if (!a.status)
        return cudaErrorInvalidDevice;
    const int W = kThreads / 32;
    if (Tq > 0)
        mla_dq_kernel<<<(unsigned)(((int64_t)Tq * H + W - 1) / W), kThreads, 0, s>>>(a);
    if (Tk > 0) {
        mla_dkv_kernel<<<(unsigned)(((int64_t)Tk * H + W - 1) / W), kThreads, 0, s>>>(a);
        mla_dkr_kernel<<<(unsigned)(((int64_t)Tk * kDR + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace kda

// mla_cache.cu -- writing new rows into the paged latent cache (bfloat16, or e4m3 with a
// power-of-two scale for each page and latent group).
//
// Bound by bytes: a new row is read once (1152 B) and written once (1152 or 576 B); a page that
// held earlier rows and whose scale grows is read and written once more.  One CTA takes one
// (page that receives rows, group): the page is where the scale lives, so one CTA sees all that
// decides it and no two CTAs write the same page.  Up to 64 new rows at a time come to shared memory
// by bulk copies.  bfloat16 rows leave it the same way.  For codes they are read there twice, for
// the maximum and for the rounding; longer pages read the rest from global memory, the second time
// from L2.  Three CTAs an SM (more for smaller pages), so that some wait for rows while others round
// theirs; nine warps each (eighteen: 33 us for the 27 below; rows held in registers, two CTAs an SM: 37).
// Measured: 16 prompts of 500 to 8000 rows into an 8-bit cache 27.5 us (4.7 TB/s; a page is 8 us of
// lookups, rows, maximum and stores; 39 us with pages of 16), into a bfloat16 one 32 us (5.4 TB/s);
// one row for each of 256 sequences 6 us, most of it the launch.
#include <cuda_fp8.h>

#include "mla_common.cuh"

namespace kda {

namespace {

using namespace mla;

constexpr int kVecs = kDC / 8;  // 16-byte vectors of a bfloat16 row
constexpr int kPass = 4;        // rows the CTA takes at once
constexpr int kThreads = kPass * kVecs;
constexpr int kCopyThreads = 96;  // of a CTA that only looks up and copies (bfloat16)
constexpr int kStaged = 64;     // rows in shared memory
constexpr int kBatch = 6;       // passes of earlier rows in flight

struct AppendArgs {
    int N, T_new, G, max_pages, num_pages, page_size;
    const int32_t *cu, *kv_lens, *block_table;
    const __nv_bfloat16 *x;
    void *cache;
    float *cache_scale;
    unsigned int *status;
    unsigned long long limit_ns;  // kLate: how long a wait for rows lasts
};

// The larger of m and the eight |x|, two halves of a word each, compared as integers: NaN is above
// infinity, which is above all.
__device__ __forceinline__ uint32_t amax8(uint32_t m, uint4 v)
{
    constexpr uint32_t k = 0x7fff7fffu;
    return __vimax3_s16x2(__vimax3_s16x2(m, v.x & k, v.y & k), v.z & k, v.w & k);
}

// Two floats to two e4m3 codes, to nearest even (saturating; the caller's scale leaves |x| <= 448).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint2 quantise8(uint4 v, float inv)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16x2(w[i]);
        c[i] = e4m3x2(f.x * inv, f.y * inv);
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Four codes times f, rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f)
{
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 x = __half22float2(__half2(a)), y = __half22float2(__half2(b));
    return e4m3x2(x.x * f, x.y * f) | (e4m3x2(y.x * f, y.y * f) << 16);
}

// The smallest power of two s >= 2^-100 with amax <= 448 s, for the bits of amax; NaN for an
// infinite or NaN one.
__device__ __forceinline__ float scale_for(uint32_t b)
{
    if (b >= 0x7f800000u)
        return __uint_as_float(0x7fc00000u);
    // amax = 1.f 2^(E - 127); 448 = 1.75 2^8
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}

// kLate: the self-test of what follows when rows do not land in time (their copies are left out).
// Nothing may be written then: the scale and the earlier rows of the page are not this call's alone.
template <bool kE4M3, bool kLate>
__global__ void __launch_bounds__(kE4M3 ? kThreads : kCopyThreads, 4) mla_append_kernel(AppendArgs a)
{
    const unsigned long long limit = kLate ? a.limit_ns : kWaitLimitNs;
    extern __shared__ __align__(16) unsigned char staged_rows[];
    __shared__ int64_t sh[40];
    __shared__ uint32_t s_max[kThreads / 32];
    __shared__ uint64_t landed;
    const int tid = threadIdx.x, ps = a.page_size;
    if (tid == 0) {
        mbar_init(&landed, 1);
        fence_mbar_init_cluster();
    }
    // sequence n touches the pages of its places [len, len + new rows)
    const Item it = find_item<kE4M3 ? kThreads : kCopyThreads>(
        a.N, blockIdx.x,
        [&](int n, bool &bad) {
            const int m = span_of(a.cu, n, a.T_new, bad).len(), len = a.kv_lens[n];
            // a refused length stands for one page, whose CTA reports it
            return m <= 0 ? 0 : len < 0 ? 1 : (len % ps + m - 1) / ps + 1;
        },
        sh);
    if (it.bad && tid == 0)
        report_device_error(a.status, KDA_ERR_INVALID_ARG);
    if (it.bad || it.seq < 0)
        return;
    const int n = it.seq, g = blockIdx.y, len = a.kv_lens[n], m = a.cu[n + 1] - a.cu[n];
    const int64_t p_idx = len < 0 ? -1 : (int64_t)len / ps + it.k;
    const int page = p_idx >= 0 && p_idx < a.max_pages ? a.block_table[(int64_t)n * a.max_pages + p_idx] : -1;
    if (page < 0 || page >= a.num_pages) {
        if (tid == 0)
            report_device_error(a.status, KDA_ERR_INVALID_ARG);
        return;
    }
    const int slot0 = it.k == 0 ? len % ps : 0;                         // first slot written
    const int64_t first = it.k == 0 ? 0 : (int64_t)it.k * ps - len % ps;  // its row among the sequence's
    const int rows = (int)min((int64_t)(ps - slot0), m - first);
    if (!rows_in(slot0, rows, ps, (int64_t)page * ps, (int64_t)a.num_pages * ps) ||
        !rows_in(first, rows, m, a.cu[n], a.T_new)) {
        report_device_error(a.status, KDA_ERR_DEVICE_BOUNDS);
        return;
    }
    const int r0 = tid / kVecs, vec = tid % kVecs;  // this thread's first row and its vector
    const uint4 *src = reinterpret_cast<const uint4 *>(a.x + ((a.cu[n] + first + r0) * a.G + g) * kDC) + vec;
    const int64_t step = (int64_t)kPass * a.G * kVecs;  // vectors from a pass to the next
    const int64_t row0 = ((int64_t)page * ps + slot0 + r0) * a.G + g;
    // rows [r, r + count) of the new ones to shared memory, by the first warp
    const __nv_bfloat16 *x = a.x + ((a.cu[n] + first) * a.G + g) * kDC;
    auto fetch = [&](int r, int count) {
        if (tid == 0)
            mbar_arrive_expect_tx(&landed, count * kDC * 2);
        __syncwarp();
        if (kLate)
            return;
        if (a.G == 1) {
            if (tid == 0)
                bulk_g2s(staged_rows, x + (int64_t)r * kDC, count * kDC * 2, &landed);
        } else {
            for (int i = tid; i < count; i += 32)
                bulk_g2s(staged_rows + i * kDC * 2, x + (int64_t)(r + i) * a.G * kDC, kDC * 2, &landed);
        }
    };
    if constexpr (!kE4M3) {  // and from there to the cache
        if (tid >= 32)
            return;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.cache) + (((int64_t)page * ps + slot0) * a.G + g) * kDC;
        for (int r = 0, k = 0; r < rows; r += kStaged, ++k) {
            const int count = min(rows - r, kStaged);
            fetch(r, count);
            if (__any_sync(0xffffffffu, !mbar_wait_bounded(&landed, k & 1, a.status, limit))) {
                mbar_wait_bounded(&landed, k & 1, a.status, limit);  // copies on their way, before the CTA ends
                return;
            }
            if (a.G == 1) {
                if (tid == 0)
                    bulk_s2g(dst + (int64_t)r * kDC, staged_rows, count * kDC * 2);
            } else {
                for (int i = tid; i < count; i += 32)
                    bulk_s2g(dst + (int64_t)(r + i) * a.G * kDC, staged_rows + i * kDC * 2, kDC * 2);
            }
            bulk_commit();
            bulk_wait_all();  // also before the CTA's shared memory goes
            __syncwarp();
        }
        return;
    }
    const int staged = min(rows, kStaged);
    if (tid < 32)
        fetch(0, staged);
    float *sp = a.cache_scale + (int64_t)page * a.G + g;
    const float old = slot0 > 0 ? *sp : 0.0f;  // read by all before one thread writes it (barrier between)
    uint32_t mx = 0;
    for (int r = kStaged + r0; r < rows; r += kPass)
        mx = amax8(mx, src[(int64_t)(r - r0) * a.G * kVecs]);
    const bool late = !mbar_wait_bounded(&landed, 0, a.status, limit);
    const uint4 *held_new = reinterpret_cast<const uint4 *>(staged_rows) + tid;
#pragma unroll 4
    for (int i = 0; i * kPass + r0 < staged; ++i)
        mx = amax8(mx, held_new[i * kThreads]);
    mx = max(mx & 0xffffu, mx >> 16) << 16;  // the bits of a float32
    mx = __reduce_max_sync(0xffffffffu, mx);
    if ((tid & 31) == 0)
        s_max[tid >> 5] = mx;
    if (__syncthreads_or(late)) {
        mbar_wait_bounded(&landed, 0, a.status, limit);  // copies on their way, before the CTA ends
        return;
    }
    mx = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
        mx = max(mx, s_max[w]);
    const float need = scale_for(mx);
    // a NaN scale (new or held) stays NaN
    const float now = slot0 > 0 ? (need != need || old != old ? __uint_as_float(0x7fc00000u) : fmaxf(need, old)) : need;
    if (tid == 0)
        *sp = now;
    unsigned char *codes = static_cast<unsigned char *>(a.cache);
    if (slot0 > 0 && !(now == old)) {  // earlier rows of the page, at the larger scale
        const float f = old / now;
        unsigned char *held = codes + (((int64_t)page * ps + r0) * a.G + g) * kDC + vec * 8;
        for (int i0 = 0; i0 * kPass + r0 < slot0; i0 += kBatch) {
            uint2 u[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if ((i0 + i) * kPass + r0 < slot0)
                    u[i] = *reinterpret_cast<const uint2 *>(held + (i0 + i) * step * 8);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if ((i0 + i) * kPass + r0 < slot0)
                    *reinterpret_cast<uint2 *>(held + (i0 + i) * step * 8) = make_uint2(rescale4(u[i].x, f), rescale4(u[i].y, f));
        }
    }
    const float inv = 1.0f / now;  // exact: a power of two from 2^-100 to 2^120
    unsigned char *dst = codes + row0 * kDC + vec * 8;
#pragma unroll 4
    for (int i = 0; i * kPass + r0 < staged; ++i)
        *reinterpret_cast<uint2 *>(dst + i * step * 8) = quantise8(held_new[i * kThreads], inv);
    for (int r = kStaged + r0; r < rows; r += kPass) {
        const int64_t at = (int64_t)(r - r0) * a.G * kVecs;
        *reinterpret_cast<uint2 *>(dst + at * 8) = quantise8(src[at], inv);
    }
}

}  // namespace

cudaError_t launch_mla_append(int N, const int32_t *cu_new, int T_new, int G, const void *kv_new,
                              const int32_t *kv_lens, const int32_t *block_table, int max_pages, bool e4m3, void *cache,
                              float *cache_scale, int num_pages, int page_size, uint32_t late_us, cudaStream_t s)
{
    AppendArgs a{N, T_new, G, max_pages, num_pages, page_size, cu_new, kv_lens, block_table,
                 static_cast<const __nv_bfloat16 *>(kv_new), cache, cache_scale, device_status_ptr(), late_us * 1000ull};
    if (!a.status)
        return cudaErrorInvalidDevice;
    // a sequence of m > 0 rows touches at most (m - 1) / page_size + 2 pages, and no more than m
    const int64_t most = (int64_t)T_new / page_size + 2 * (int64_t)N;
    const dim3 grid((unsigned)(most < T_new ? most : T_new), G);
    auto kernel = late_us > 0 ? (e4m3 ? mla_append_kernel<true, true> : mla_append_kernel<false, true>)
                              : (e4m3 ? mla_append_kernel<true, false> : mla_append_kernel<false, false>);
    const int smem = (page_size < kStaged ? page_size : kStaged) * kDC * 2;
    // (the limit is the kernel's, shared by all host threads: the same one whatever this call's pages)
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStaged * kDC * 2);
    if (e != cudaSuccess)
        return e;
    kernel<<<grid, e4m3 ? kThreads : kCopyThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kda

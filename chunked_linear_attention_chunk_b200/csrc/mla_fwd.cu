// mla_fwd.cu -- expanded latent attention over packed sequences, forward.
//
//   s_ij = scale (q_i . [k_j, k_rope_j]),  o_i = sum_j e^{s_ij - lse_i} v_j
// with the running maximum and sum of the softmax in float32, in base 2 (scale log2(e) is folded
// into the exponent's multiply-add).  Bound by the tensor cores: 640 flops a (query, key) pair and
// head against 2 x 256 B of K and V a key that 256 queries share.
//
// One CTA takes 256 queries of one head as two tiles of 128, so that one tile's softmax runs
// while the tensor cores work for the other, and walks the keys 80 at a time:
//   S = Q K^T        (M = 128, N = 80, K = 192; K and the heads' shared k_rope side by side)
//   O += P V         (M = 128, N = 128, K = 80; P in tensor memory, V read MN-major)
// Tensor memory holds two O tiles, and 128 columns a tile for S and P.  80 keys are the most whose S
// (80) and P (40) fit there side by side, so that S of the next step is taken as soon as the threads
// have read this one's; with 96 keys P has to overwrite S and S waits for P V: 320 us against 297
// (16 heads, 8192 tokens, causal; one warp issuing all products 375, since a warp feeds nothing to
// the tensor cores in the 150 cycles that a ready barrier takes).  A 128 x 80 x 16 product takes 52
// cycles (its operands' 6.5 KB of shared memory) against 40 ideal, so a step is 1890 cycles of
// products at least; it measured 2100.  8192 tokens, 16 heads, causal: 305 us (1.13 PFLOP/s) in a loop,
// where the 1000 W limit holds the clock near 1.56 GHz; 272 us (1.26) by itself.
//
// Warps: 0-3 and 4-7 softmax of tile 0 and 1, one row a thread, no exchange between threads; O is
// rescaled only when a row's maximum grows by more than 2^8 (float32 sums and a bfloat16 weight
// hold as well); 8 copies (TMA); 9 issues S, 10 issues O.
#include "mla_common.cuh"
#include "mla_tc.cuh"

namespace kda {

namespace {

using namespace mla;

constexpr int kThreads = 352;
constexpr int kRows = 128;               // queries a tile
constexpr int kTiles = 2;                // tiles a CTA
constexpr int kKeys = 80;                // keys a step
constexpr int kV = 3;                    // stages of V
constexpr uint32_t kP = kKeys;           // columns from S to P
constexpr uint32_t kQBlk = kRows * 128;  // 64 numbers of 128 rows
constexpr uint32_t kKBlk = kKeys * 128;
constexpr float kGrow = 8.0f;            // log2 by which a maximum may grow without rescaling

struct FwdArgs {
    int N, Tq, Tk, H;
    bool causal;
    float scale_log2;
    const int32_t *cu_q, *cu_k;
    __nv_bfloat16 *o;
    float *lse;
    unsigned int *status;
};

// q, kv and k_rope as [block of 64 numbers][head][row][64]; a box is all blocks of an operand.
struct FwdMaps {
    CUtensorMap q, kv, kr;
};

struct FwdSmem {
    alignas(1024) unsigned char q[kTiles][3 * kQBlk];
    alignas(1024) unsigned char k[2][3 * kKBlk];
    alignas(1024) unsigned char v[kV][2 * kKBlk];
    uint64_t q_full, k_full[2], k_empty[2], v_full[kV], v_empty[kV], v_tail;
    uint64_t s_full[kTiles], s_read[kTiles], p_full[kTiles], pv_done[kTiles];
    uint32_t tmem_slot;
    int64_t find[40];
};

// Keys [0, last] are visible to query i of a sequence.
__device__ __forceinline__ int last_key(int i, int lq, int lk, bool causal)
{
    return causal ? min(lk - 1, i + lk - lq) : lk - 1;
}

__global__ void __launch_bounds__(kThreads, 1)
    mla_fwd_kernel(const __grid_constant__ FwdMaps maps, FwdArgs a)
{
    extern __shared__ unsigned char raw[];
    FwdSmem &sm = *reinterpret_cast<FwdSmem *>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x % a.H;
    if (tid == 0) {
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.v_tail, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
        }
        for (int i = 0; i < kV; ++i) {
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(&sm.s_full[t], 1);
            mbar_init(&sm.s_read[t], 4);
            mbar_init(&sm.p_full[t], 4);
            mbar_init(&sm.pv_done[t], 1);
        }
        fence_mbar_init_cluster();
    }
    const Item it = find_item<kThreads>(
        a.N, blockIdx.x / a.H,
        [&](int n, bool &bad) {
            span_of(a.cu_k, n, a.Tk, bad);
            return (span_of(a.cu_q, n, a.Tq, bad).len() + kTiles * kRows - 1) / (kTiles * kRows);
        },
        sm.find);
    if (it.bad && tid == 0)
        report_device_error(a.status, KDA_ERR_INVALID_ARG);
    if (it.bad || it.seq < 0)
        return;
    const int q0 = a.cu_q[it.seq], k0 = a.cu_k[it.seq], lq = a.cu_q[it.seq + 1] - q0, lk = a.cu_k[it.seq + 1] - k0;
    // with a causal mask the last queries see the most keys: they go first
    const int i0 = ((lq + kTiles * kRows - 1) / (kTiles * kRows) - 1 - it.k) * kTiles * kRows;
    if (!rows_in(i0, min(kTiles * kRows, lq - i0), lq, q0, a.Tq) || (kDebugChecks && (k0 < 0 || k0 + lk > a.Tk))) {
        report_device_error(a.status, KDA_ERR_DEVICE_BOUNDS);
        return;
    }
    int steps[kTiles], n_steps = 0;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const int first = i0 + t * kRows, last = min(lq, first + kRows) - 1;
        steps[t] = first < lq ? max(0, last_key(last, lq, lk, a.causal) + kKeys) / kKeys : 0;
        n_steps = max(n_steps, steps[t]);
    }

    if (warp == 8)
        tc::tmem_alloc(&sm.tmem_slot, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem_slot;
    Waits wait{false};

    if (warp == 8) {
        // ---------------- copies
        if (n_steps > 0) {
            if (elect()) {
                mbar_arrive_expect_tx(&sm.q_full, ((steps[0] > 0) + (steps[1] > 0)) * 3 * kQBlk);
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
                    if (steps[t] > 0)
                        tma_load_4d(sm.q[t], &maps.q, 0, q0 + i0 + t * kRows, h, 0, &sm.q_full);
            }
            Ring<kV> rv;
            for (int j = 0; j < n_steps; ++j, rv.step()) {
                const int s = j & 1, key = k0 + j * kKeys, live = lk - j * kKeys;
                if (j >= 2)
                    wait(&sm.k_empty[s], (j / 2 - 1) & 1);
                if (elect() && !wait.dead) {
                    mbar_arrive_expect_tx(&sm.k_full[s], 3 * kKBlk);
                    tma_load_4d(sm.k[s], &maps.kv, 0, key, h, 0, &sm.k_full[s]);
                    tma_load_2d(sm.k[s] + 2 * kKBlk, &maps.kr, 0, key, &sm.k_full[s]);
                }
                if (rv.round > 0)
                    wait(&sm.v_empty[rv.slot], (rv.round - 1) & 1);
                uint64_t *bar = live < kKeys ? &sm.v_tail : &sm.v_full[rv.slot];
                if (elect() && !wait.dead) {
                    mbar_arrive_expect_tx(bar, 2 * kKBlk);
                    tma_load_4d(sm.v[rv.slot], &maps.kv, 0, key, h, 2, bar);
                }
                if (live < kKeys) {
                    // rows behind the sequence's end may hold anything (0 * NaN): zeros for O
                    wait(&sm.v_tail, 0);
                    for (int i = lane; i < (kKeys - live) * 16; i += 32)
                        *reinterpret_cast<uint4 *>(sm.v[rv.slot] + (i & 8 ? kKBlk : 0) + (live + i / 16) * 128 + (i & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (elect())
                        mbar_arrive(&sm.v_full[rv.slot]);
                }
            }
        }
    } else if (warp == 9) {
        // ---------------- S, as soon as the tile's threads have read the one before
        constexpr uint32_t id = tc::idesc_bf16(kRows, kKeys, false, false);
        const Desc qd(smem_u32(sm.q[0]), 16, 1024, tc::kSw128), kd(smem_u32(sm.k[0]), 16, 1024, tc::kSw128);
        if (n_steps > 0)
            wait(&sm.q_full, 0);
        for (int j = 0; j < n_steps; ++j) {
            wait(&sm.k_full[j & 1], (j / 2) & 1);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                if (j >= steps[t])
                    continue;
                if (j > 0)
                    wait(&sm.s_read[t], (j - 1) & 1);
                tc::fence_after_sync();
                if (elect()) {
#pragma unroll
                    for (int ks = 0; ks < kDQ / 16; ++ks)
                        tc::mma_bf16(tmem + t * 128, qd.at(t * 3 * kQBlk + (ks >> 2) * kQBlk + (ks & 3) * 32),
                                     kd.at((j & 1) * 3 * kKBlk + (ks >> 2) * kKBlk + (ks & 3) * 32), id, ks > 0 ? 1u : 0u);
                    tc::commit(&sm.s_full[t]);
                }
            }
            if (elect())
                tc::commit(&sm.k_empty[j & 1]);
        }
    } else if (warp == 10) {
        // ---------------- O
        constexpr uint32_t id = tc::idesc_bf16(kRows, kDV, false, true);
        const Desc vd(smem_u32(sm.v[0]), kKBlk, 1024, tc::kSw128);
        Ring<kV> rv;
        for (int j = 0; j < n_steps; ++j, rv.step()) {
            wait(&sm.v_full[rv.slot], rv.round & 1);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                if (j >= steps[t])
                    continue;
                wait(&sm.p_full[t], j & 1);
                tc::fence_after_sync();
                if (elect()) {
#pragma unroll
                    for (int ks = 0; ks < kKeys / 16; ++ks)
                        tc::mma_bf16_ts(tmem + 256 + t * 128, tmem + t * 128 + kP + ks * 8,
                                        vd.at(rv.slot * 2 * kKBlk + ks * 2048), id, j > 0 || ks > 0 ? 1u : 0u);
                    tc::commit(&sm.pv_done[t]);
                }
            }
            if (elect())
                tc::commit(&sm.v_empty[rv.slot]);
        }
    } else {
        // ---------------- softmax: one row a thread
        const int t = warp >> 2, row = i0 + t * kRows + (warp & 3) * 32 + lane;
        const int last = last_key(row, lq, lk, a.causal);
        const int last_0 = last_key(i0 + t * kRows, lq, lk, a.causal);  // the tile's first row sees the fewest keys
        const uint32_t s_addr = tc::taddr(tmem, (uint32_t)(warp & 3) * 32, t * 128), o_addr = s_addr + 256;
        const int n = t == 0 ? steps[0] : steps[1];
        float m = -INFINITY, l = 0.0f;
        for (int j = 0; j < n; ++j) {
            wait(&sm.s_full[t], j & 1);
            tc::fence_after_sync();
            uint32_t x[kKeys];
            tc::ld_32x32b_x32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(x));
            tc::ld_32x32b_x32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
            tc::ld_32x32b_x16(s_addr + 64, *reinterpret_cast<uint32_t(*)[16]>(x + 64));
            tc::wait_ld();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.s_read[t]);
            if ((j + 1) * kKeys - 1 > last_0) {
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) {
                    const uint32_t seen = bit_span(0, last + 1 - j * kKeys - c);
#pragma unroll
                    for (int i = 0; i < 32 && c + i < kKeys; ++i)
                        x[c + i] = seen >> i & 1 ? x[c + i] : __float_as_uint(-INFINITY);
                }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < kKeys; ++i)
                mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(x[i]));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
            const bool grow = top > m + kGrow;
            if (__any_sync(0xffffffffu, grow)) {
                const float mn = grow ? top : m, f = grow ? ex2(m - mn) : 1.0f;
                m = mn;
                l *= f;
                if (j > 0) {
                    wait(&sm.pv_done[t], (j - 1) & 1);
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t y[32];
                        tc::ld_32x32b_x32(o_addr + c * 32, y);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                        tc::st_32x32b_x32(o_addr + c * 32, y);
                    }
                }
            }
            const float sub = m == -INFINITY ? 0.0f : m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t p[kKeys / 2];
#pragma unroll
            for (int i = 0; i < kKeys; i += 2) {
                const float e0 = ex2(fmaf(__uint_as_float(x[i]), a.scale_log2, -sub));
                const float e1 = ex2(fmaf(__uint_as_float(x[i + 1]), a.scale_log2, -sub));
                sum[i & 2] += e0;
                sum[(i & 2) + 1] += e1;
                p[i / 2] = pack_bf16x2(e0, e1);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            if (j > 0) {
                wait(&sm.pv_done[t], (j - 1) & 1);  // P's place has been read
                tc::fence_after_sync();
            }
            tc::st_32x32b_x32(s_addr + kP, *reinterpret_cast<const uint32_t(*)[32]>(p));
            tc::st_32x32b_x8(s_addr + kP + 32, *reinterpret_cast<const uint32_t(*)[8]>(p + 32));
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.p_full[t]);
        }
        // ---- the rows' results, through the place of the tile's Q (read for the last time before
        // the last O), so that the writes are whole rows
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t r = (int64_t)(q0 + row) * a.H + h;
        if (n > 0) {
            wait(&sm.pv_done[t], (n - 1) & 1);
            tc::fence_after_sync();
        }
        const int tr = tid & (kRows - 1);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            uint32_t y[32];
            if (n > 0) {
                tc::ld_32x32b_x32(o_addr + c * 32, y);
                tc::wait_ld();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = l == 0.0f ? 0u
                                     : pack_bf16x2(__uint_as_float(y[8 * i + 2 * k]) * inv,
                                                   __uint_as_float(y[8 * i + 2 * k + 1]) * inv);
                *reinterpret_cast<uint4 *>(sm.q[t] + tr * 256 + (((c * 4 + i) ^ (tr & 7)) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
        for (int v = tr; v < kRows * 16; v += kRows) {
            const int vr = v >> 4, c = v & 15, i = i0 + t * kRows + vr;
            if (i < lq)
                *reinterpret_cast<uint4 *>(a.o + ((int64_t)(q0 + i) * a.H + h) * kDV + c * 8) =
                    *reinterpret_cast<const uint4 *>(sm.q[t] + vr * 256 + ((c ^ (vr & 7)) << 4));
        }
        if (a.lse && row < lq)
            a.lse[r] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
    wait.finish(a.status);
    if (warp == 8)
        tc::tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_mla_fwd(int N, const int32_t *cu_q, const int32_t *cu_k, int Tq, int Tk, int H, bool causal,
                           float scale, const void *q, const void *kv, const void *k_rope, void *o, float *lse,
                           cudaStream_t s)
{
    FwdArgs a{N, Tq, Tk, H, causal, scale * kLog2e, cu_q, cu_k, static_cast<__nv_bfloat16 *>(o), lse, device_status_ptr()};
    if (!a.status)
        return cudaErrorInvalidDevice;
    FwdMaps maps{};
    cudaError_t e = make_rows_map(&maps.q, q, kDQ, H, Tq, kRows, 3);
    if (e == cudaSuccess && Tk > 0)
        e = make_rows_map(&maps.kv, kv, kDKV, H, Tk, kKeys, 2);
    if (e == cudaSuccess && Tk > 0)
        e = make_rows_map(&maps.kr, k_rope, kDR, 0, Tk, kKeys, 1);
    const size_t smem = sizeof(FwdSmem) + 1024;
    static_assert(sizeof(FwdSmem) + 1024 <= 232448, "shared memory of one CTA");
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(mla_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    const int64_t items = (int64_t)Tq / (kTiles * kRows) + N;  // at least the tile pairs of any N sequences
    mla_fwd_kernel<<<(unsigned)(items * H), kThreads, smem, s>>>(maps, a);
    return cudaGetLastError();
}

}  // namespace kda

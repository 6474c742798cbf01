// mla_bwd.cu -- gradients of the expanded latent attention over packed sequences.
//
//   p_ij = e^{s_ij - lse_i},  D_i = dO_i . o_i,  e_ij = p_ij (dO_i . v_j - D_i)
//   dq_i = scale sum_j e_ij [k_j, k_rope_j];  dk_j = scale sum_i e_ij q_i;  dv_j = sum_i p_ij dO_i
// Bound by the tensor cores.  Sums over queries and sums over keys are taken by two launches of
// one kernel, each keeping its sums in tensor memory: a single pass would have to add dq across
// CTAs with atomics (an order of its own every time) and needs 128 + 192 + 192 accumulator columns
// beside S and dP, more than there are.  The price is S and dP twice: 1152 multiply-adds a pair
// for the 832 of the formulas.
//
// Both launches hold a 128-row tile (X: queries for dq, keys for dk and dv) and step through the
// other side (Y) 96 rows at a time:
//   S = X1 Y1^T (K = 192),  dP = X2 Y2^T (K = 128),  acc1 += e Y1 (N = 192),
//   keys only: acc2 += p Y2 (N = 128)
// with X1, Y1 the q and [k, k_rope] rows and X2, Y2 the dO and v rows.  A Y tile serves as K-major
// operand of the first two products and MN-major operand of the last two; p and e go back to
// tensor memory as their A operands, over the S and dP they came from.  The products are issued
//   acc2(i), S(i + 1), acc1(i), dP(i + 1)
// so that the threads always have two products' time for p(i + 1) and two for e(i), without a
// second S or dP buffer.
//
// Warps: 0-11 elementwise (row = tensor-memory lane; four warps for each 32 columns: with two
// groups of 48 the threads, not the products, set the pace); 12 copies (TMA); 13 issues the products.  The launch for dq computes D first and leaves D and lse
// in base 2, head by head, for the other.  dk_rope's parts are added over the heads, in order, by
// a third launch.
#include "mla_common.cuh"
#include "mla_tc.cuh"

namespace kda {

namespace {

using namespace mla;

constexpr int kGroups = 3;               // elementwise warpgroups, each a third of the columns
constexpr int kElem = kGroups * 128;     // their threads
constexpr int kThreads = kElem + 64;
constexpr int kRows = 128;               // X rows of a CTA
constexpr int kStep = 96;                // Y rows a step
constexpr int kPart = kStep / kGroups;   // columns of a group
constexpr int kY1 = 3, kY2 = 1;          // stages
constexpr uint32_t kXBlk = kRows * 128;  // 64 numbers of the rows
constexpr uint32_t kYBlk = kStep * 128;
constexpr uint32_t kColS = 0, kColP = kStep, kCol2 = 2 * kStep, kCol1 = kCol2 + 128;  // tensor memory columns
static_assert(kCol1 + kDQ <= 512, "tensor memory");

struct BwdArgs {
    int N, Tq, Tk, H;
    bool causal;
    float scale;
    const int32_t *cu_q, *cu_k;
    const __nv_bfloat16 *o, *dO;
    const float *lse;
    __nv_bfloat16 *dq, *dkv, *dkr;
    float *delta, *lse2;  // [H][Tq]
    float *part;          // [H][Tk][64]
    unsigned int *status;
};

// x1, x2: boxes of kRows rows; y1, y2: of kStep rows.  The key side is two maps (kv and k_rope).
struct BwdMaps {
    CUtensorMap x1, x1r, x2, y1, y1r, y2;
};

struct BwdSmem {
    alignas(1024) unsigned char x1[3 * kXBlk];
    alignas(1024) unsigned char x2[2 * kXBlk];
    alignas(1024) unsigned char y1[kY1][3 * kYBlk];
    alignas(1024) unsigned char y2[kY2][2 * kYBlk];
    float col[kY1][2][kStep];  // keys: lse in base 2 and D of a step's queries
    float dsum[2][kRows];      // queries: halves of D
    uint64_t x_full, y1_full[kY1], y1_empty[kY1], y2_full[kY2], y2_empty[kY2], tail;
    uint64_t s_full, p_full, dp_full, e_full, done;
    uint32_t tmem_slot;
    int64_t find[40];
};

__device__ __forceinline__ void elem_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kElem) : "memory"); }

// kPart columns of this thread's lane as bfloat16 pairs.
__device__ __forceinline__ void store_part(uint32_t taddr, const float (&x)[kPart])
{
    uint32_t w[kPart / 2];
#pragma unroll
    for (int i = 0; i < kPart / 2; ++i)
        w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    tc::st_32x32b_x16(taddr, w);
    tc::wait_st();
}

__device__ __forceinline__ void load_part(uint32_t taddr, float (&x)[kPart])
{
    uint32_t a[kPart];
    tc::ld_32x32b_x32(taddr, a);
    tc::wait_ld();
#pragma unroll
    for (int i = 0; i < kPart; ++i)
        x[i] = __uint_as_float(a[i]);
}

// 32 columns of this thread's lane, times f, as bfloat16 into vectors [v0, v0 + 4) of its row of
// `vecs` 16-byte vectors (swizzled: neighbouring rows start in different banks).
__device__ __forceinline__ void stage_bf16(unsigned char *rows, int vecs, int r, int v0, uint32_t taddr, float f)
{
    float x[32];
    load_part(taddr, x);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(rows + r * vecs * 16 + (((v0 + i) ^ (r & 7)) << 4)) =
            make_uint4(pack_bf16x2(x[8 * i] * f, x[8 * i + 1] * f), pack_bf16x2(x[8 * i + 2] * f, x[8 * i + 3] * f),
                       pack_bf16x2(x[8 * i + 4] * f, x[8 * i + 5] * f), pack_bf16x2(x[8 * i + 6] * f, x[8 * i + 7] * f));
}

template <bool kKeys>  // X rows are keys (dk, dv), else queries (dq)
__global__ void __launch_bounds__(kThreads, 1)
    mla_bwd_kernel(const __grid_constant__ BwdMaps maps, BwdArgs a)
{
    extern __shared__ unsigned char raw[];
    BwdSmem &sm = *reinterpret_cast<BwdSmem *>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x % a.H;
    const Item it = find_item<kThreads>(
        a.N, blockIdx.x / a.H,
        [&](int n, bool &bad) {
            const Span q = span_of(a.cu_q, n, a.Tq, bad), k = span_of(a.cu_k, n, a.Tk, bad);
            return ((kKeys ? k : q).len() + kRows - 1) / kRows;
        },
        sm.find);
    if (it.bad && tid == 0)
        report_device_error(a.status, KDA_ERR_INVALID_ARG);
    if (it.bad || it.seq < 0)
        return;
    const int q0 = a.cu_q[it.seq], k0 = a.cu_k[it.seq], lq = a.cu_q[it.seq + 1] - q0, lk = a.cu_k[it.seq + 1] - k0;
    const int lx = kKeys ? lk : lq, ly = kKeys ? lq : lk;
    // with a causal mask the first keys and the last queries have the most to do: they go first
    const int r0 = (kKeys ? it.k : (lx + kRows - 1) / kRows - 1 - it.k) * kRows, rows = min(kRows, lx - r0);
    const int off = lk - lq;  // causal: key j is visible to query i from i = j - off on
    // Y rows [y_first, y_end)
    const int y_first = kKeys && a.causal ? max(0, r0 - off) : 0;
    const int y_end = !kKeys && a.causal ? min(ly, r0 + rows + off) : ly;
    const int steps = y_first < y_end ? (y_end - y_first + kStep - 1) / kStep : 0;

    if (tid == 0) {
        mbar_init(&sm.x_full, 1);
        mbar_init(&sm.tail, 1);
        for (int i = 0; i < kY1; ++i) {
            mbar_init(&sm.y1_full[i], kKeys ? 33 : 1);
            mbar_init(&sm.y1_empty[i], 1);
        }
        for (int i = 0; i < kY2; ++i) {
            mbar_init(&sm.y2_full[i], 1);
            mbar_init(&sm.y2_empty[i], 1);
        }
        mbar_init(&sm.s_full, 1);
        mbar_init(&sm.dp_full, 1);
        mbar_init(&sm.p_full, kElem / 32);
        mbar_init(&sm.e_full, kElem / 32);
        mbar_init(&sm.done, 1);
        fence_mbar_init_cluster();
    }
    if (warp == kElem / 32)
        tc::tmem_alloc(&sm.tmem_slot, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem_slot;
    Waits wait{a.status, false};

    if (warp == kElem / 32) {
        // ---------------- copies
        if (steps > 0 && elect()) {
            mbar_arrive_expect_tx(&sm.x_full, 5 * kXBlk);
            const int x = (kKeys ? k0 : q0) + r0;
            tma_load_4d(sm.x1, &maps.x1, 0, x, h, 0, &sm.x_full);
            if (kKeys)
                tma_load_2d(sm.x1 + 2 * kXBlk, &maps.x1r, 0, x, &sm.x_full);
            tma_load_4d(sm.x2, &maps.x2, 0, x, h, kKeys ? 2 : 0, &sm.x_full);
        }
        __syncwarp();
        Ring<kY1> r1;
        Ring<kY2> r2;
        uint32_t tails = 0;
        // rows behind the sequence's end may hold anything (0 * NaN): zeros
        auto zero_tail = [&](unsigned char *p, int blocks, int live, uint64_t *full) {
            wait(&sm.tail, tails++ & 1);
            for (int i = lane; i < (kStep - live) * 8 * blocks; i += 32)
                *reinterpret_cast<uint4 *>(p + i % blocks * kYBlk + (live + i / (8 * blocks)) * 128 +
                                           i / blocks % 8 * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (elect())
                mbar_arrive(full);
        };
        for (int i = 0; i < steps && !wait.dead; ++i, r1.step(), r2.step()) {
            const int first = y_first + i * kStep, live = ly - first, y = (kKeys ? q0 : k0) + first;
            float cl[kStep / 32], cd[kStep / 32];
            if (kKeys)
#pragma unroll
                for (int c = 0; c < kStep / 32; ++c) {
                    const bool in = c * 32 + lane < live;
                    cl[c] = in ? a.lse2[(int64_t)h * a.Tq + y + c * 32 + lane] : INFINITY;
                    cd[c] = in ? a.delta[(int64_t)h * a.Tq + y + c * 32 + lane] : 0.0f;
                }
            if (r1.round > 0)
                wait(&sm.y1_empty[r1.slot], (r1.round - 1) & 1);
            if (wait.dead)
                break;
            uint64_t *bar = live < kStep ? &sm.tail : &sm.y1_full[r1.slot];
            if (elect()) {
                mbar_arrive_expect_tx(bar, 3 * kYBlk);
                tma_load_4d(sm.y1[r1.slot], &maps.y1, 0, y, h, 0, bar);
                if (!kKeys)
                    tma_load_2d(sm.y1[r1.slot] + 2 * kYBlk, &maps.y1r, 0, y, bar);
            }
            __syncwarp();
            if (kKeys) {
#pragma unroll
                for (int c = 0; c < kStep / 32; ++c) {
                    sm.col[r1.slot][0][c * 32 + lane] = cl[c];
                    sm.col[r1.slot][1][c * 32 + lane] = cd[c];
                }
                mbar_arrive(&sm.y1_full[r1.slot]);
            }
            if (live < kStep)
                zero_tail(sm.y1[r1.slot], 3, live, &sm.y1_full[r1.slot]);
            if (r2.round > 0)
                wait(&sm.y2_empty[r2.slot], (r2.round - 1) & 1);
            if (wait.dead)
                break;
            bar = live < kStep ? &sm.tail : &sm.y2_full[r2.slot];
            if (elect()) {
                mbar_arrive_expect_tx(bar, 2 * kYBlk);
                tma_load_4d(sm.y2[r2.slot], &maps.y2, 0, y, h, kKeys ? 0 : 2, bar);
            }
            __syncwarp();
            if (live < kStep)
                zero_tail(sm.y2[r2.slot], 2, live, &sm.y2_full[r2.slot]);
        }
    } else if (warp == kElem / 32 + 1) {
        // ---------------- products
        constexpr uint32_t id_s = tc::idesc_bf16(kRows, kStep, false, false), id_1 = tc::idesc_bf16(kRows, kDQ, false, true),
                           id_2 = tc::idesc_bf16(kRows, kDV, false, true);
        const Desc x1(smem_u32(sm.x1), 16, 1024, tc::kSw128), x2(smem_u32(sm.x2), 16, 1024, tc::kSw128),
            y1(smem_u32(sm.y1[0]), 16, 1024, tc::kSw128), y2(smem_u32(sm.y2[0]), 16, 1024, tc::kSw128),
            t1(smem_u32(sm.y1[0]), kYBlk, 1024, tc::kSw128), t2(smem_u32(sm.y2[0]), kYBlk, 1024, tc::kSw128);
        // tensor-memory column of the 16 Y rows ks of p or e: each group's at its own start
        auto a_col = [](uint32_t base, int ks) { return base + (ks >> 1) * kPart + (ks & 1) * 8; };
        static_assert(kPart == 32, "two 16-row steps a group");
        auto scores = [&](uint32_t slot) {
            if (elect()) {
#pragma unroll
                for (int ks = 0; ks < kDQ / 16; ++ks)
                    tc::mma_bf16(tmem + kColS, x1.at((ks >> 2) * kXBlk + (ks & 3) * 32),
                                 y1.at(slot * 3 * kYBlk + (ks >> 2) * kYBlk + (ks & 3) * 32), id_s, ks > 0 ? 1u : 0u);
                tc::commit(&sm.s_full);
            }
        };
        auto dps = [&](uint32_t slot) {
            if (elect()) {
#pragma unroll
                for (int ks = 0; ks < kDV / 16; ++ks)
                    tc::mma_bf16(tmem + kColP, x2.at((ks >> 2) * kXBlk + (ks & 3) * 32),
                                 y2.at(slot * 2 * kYBlk + (ks >> 2) * kYBlk + (ks & 3) * 32), id_s, ks > 0 ? 1u : 0u);
                tc::commit(&sm.dp_full);
                if (!kKeys)
                    tc::commit(&sm.y2_empty[slot]);
            }
        };
        Ring<kY1> r1;  // of step i + 1
        Ring<kY2> r2;
        uint32_t now1 = 0, now2 = 0;
        if (steps > 0) {
            wait(&sm.x_full, 0);
            wait(&sm.y1_full[0], 0);
            tc::fence_after_sync();
            scores(0);
            wait(&sm.y2_full[0], 0);
            tc::fence_after_sync();
            dps(0);
            r1.step();
            r2.step();
        }
        for (int i = 0; i < steps && !wait.dead; ++i, r1.step(), r2.step()) {
            wait(&sm.p_full, i & 1);  // p(i) written, or at least S(i) read
            tc::fence_after_sync();
            if (kKeys && elect()) {
#pragma unroll
                for (int ks = 0; ks < kStep / 16; ++ks)
                    tc::mma_bf16_ts(tmem + kCol2, tmem + a_col(kColS, ks), t2.at(now2 * 2 * kYBlk + ks * 2048), id_2,
                                    i > 0 || ks > 0 ? 1u : 0u);
                tc::commit(&sm.y2_empty[now2]);
            }
            if (i + 1 < steps) {
                wait(&sm.y1_full[r1.slot], r1.round & 1);
                tc::fence_after_sync();
                scores(r1.slot);
            }
            wait(&sm.e_full, i & 1);
            tc::fence_after_sync();
            if (elect()) {
#pragma unroll
                for (int ks = 0; ks < kStep / 16; ++ks)
                    tc::mma_bf16_ts(tmem + kCol1, tmem + a_col(kColP, ks), t1.at(now1 * 3 * kYBlk + ks * 2048), id_1,
                                    i > 0 || ks > 0 ? 1u : 0u);
                tc::commit(&sm.y1_empty[now1]);
                if (i + 1 == steps)
                    tc::commit(&sm.done);
            }
            if (i + 1 < steps) {
                wait(&sm.y2_full[r2.slot], r2.round & 1);
                tc::fence_after_sync();
                dps(r2.slot);
            }
            now1 = r1.slot;
            now2 = r2.slot;
        }
    } else {
        // ---------------- elementwise: row r0 + r, columns group * 32 ..
        const int r = (warp & 3) * 32 + lane, group = warp >> 2;
        const bool live = r < rows;
        const uint32_t addr = tc::taddr(tmem, (uint32_t)(warp & 3) * 32, group * kPart);
        const float sl2 = a.scale * kLog2e;
        float lse2 = INFINITY, delta = 0.0f;
        if constexpr (!kKeys) {
            const int64_t row = (int64_t)(q0 + r0 + r) * a.H + h;
            if (live && group < 2) {  // half a row each
                const uint4 *x = reinterpret_cast<const uint4 *>(a.o + row * kDV + group * 64);
                const uint4 *y = reinterpret_cast<const uint4 *>(a.dO + row * kDV + group * 64);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 u = x[c], v = y[c];
                    const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = unpack_bf16x2(uw[k]), g = unpack_bf16x2(vw[k]);
                        delta += f.x * g.x + f.y * g.y;
                    }
                }
            }
            if (group < 2)
                sm.dsum[group][r] = delta;
            const float l = live ? a.lse[row] : -INFINITY;
            lse2 = l == -INFINITY ? INFINITY : l * kLog2e;  // a row that sees no key: weights 0
            elem_sync();
            delta = sm.dsum[0][r] + sm.dsum[1][r];
            if (live && group == 0) {
                a.delta[(int64_t)h * a.Tq + q0 + r0 + r] = delta;
                a.lse2[(int64_t)h * a.Tq + q0 + r0 + r] = lse2;
            }
        }
        Ring<kY1> r1;
        for (int i = 0; i < steps; ++i, r1.step()) {
            const int y = y_first + i * kStep + group * kPart;  // place of the first column
            // columns lo .. hi - 1 are visible to the row
            int lo = 0, hi = kPart;
            bool edge;
            if (kKeys) {
                edge = i + 1 == steps || (a.causal && r0 + kRows - 1 > y_first + i * kStep + off);
                hi = ly - y;
                lo = a.causal ? r0 + r - off - y : 0;
            } else {
                edge = (i + 1) * kStep > (a.causal ? min(ly, r0 + off + 1) : ly);
                hi = (a.causal ? min(ly, r0 + r + off + 1) : ly) - y;
            }
            float p[kPart], x[kPart];
            wait(&sm.s_full, i & 1);
            tc::fence_after_sync();
            load_part(addr + kColS, p);
            if (kKeys) {
                wait(&sm.y1_full[r1.slot], r1.round & 1);  // the step's lse and D
                const float4 *l = reinterpret_cast<const float4 *>(sm.col[r1.slot][0] + group * kPart);
#pragma unroll
                for (int c = 0; c < kPart / 4; ++c) {
                    const float4 v = l[c];
                    p[4 * c] = ex2(fmaf(p[4 * c], sl2, -v.x));
                    p[4 * c + 1] = ex2(fmaf(p[4 * c + 1], sl2, -v.y));
                    p[4 * c + 2] = ex2(fmaf(p[4 * c + 2], sl2, -v.z));
                    p[4 * c + 3] = ex2(fmaf(p[4 * c + 3], sl2, -v.w));
                }
            } else {
#pragma unroll
                for (int c = 0; c < kPart; ++c)
                    p[c] = ex2(fmaf(p[c], sl2, -lse2));
            }
            if (edge) {
#pragma unroll
                for (int c = 0; c < kPart; ++c)
                    if (c < lo || c >= hi)
                        p[c] = 0.0f;
            }
            if (kKeys)
                store_part(addr + kColS, p);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.p_full);
            wait(&sm.dp_full, i & 1);
            tc::fence_after_sync();
            load_part(addr + kColP, x);
            if (kKeys) {
                const float4 *d = reinterpret_cast<const float4 *>(sm.col[r1.slot][1] + group * kPart);
#pragma unroll
                for (int c = 0; c < kPart / 4; ++c) {
                    const float4 v = d[c];
                    x[4 * c] = p[4 * c] * (x[4 * c] - v.x);
                    x[4 * c + 1] = p[4 * c + 1] * (x[4 * c + 1] - v.y);
                    x[4 * c + 2] = p[4 * c + 2] * (x[4 * c + 2] - v.z);
                    x[4 * c + 3] = p[4 * c + 3] * (x[4 * c + 3] - v.w);
                }
            } else {
#pragma unroll
                for (int c = 0; c < kPart; ++c)
                    x[c] = p[c] * (x[c] - delta);
            }
            if (edge) {  // a hidden pair's dP may be anything
#pragma unroll
                for (int c = 0; c < kPart; ++c)
                    if (c < lo || c >= hi)
                        x[c] = 0.0f;
            }
            store_part(addr + kColP, x);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.e_full);
        }
        // ---- the sums, through shared memory (nothing reads the tiles any more), so that the
        // writes are whole rows
        if (steps > 0) {
            wait(&sm.done, 0);
            tc::fence_after_sync();
        }
        const uint32_t base = tc::taddr(tmem, (uint32_t)(warp & 3) * 32, 0);
        constexpr int kVecs = (kKeys ? kDKV : kDQ) / 8;  // 16-byte vectors of a row of dkv or dq
        unsigned char *rowbuf = sm.x1;                   // x1 and x2: 80 KB
        float *part = reinterpret_cast<float *>(sm.y1[0]);
        static_assert(kRows * kDKV * 2 <= 5 * kXBlk && kRows * kDR * 4 <= kY1 * 3 * kYBlk, "room for the sums");
        if (steps > 0) {
            if (kKeys) {
                // dk (4 x 32 columns), dv (4 x 32), the rope part of dk (2 x 32), a group every third
#pragma unroll 1
                for (int c = group; c < 8; c += kGroups)
                    stage_bf16(rowbuf, kVecs, r, c * 4, base + (c < 4 ? kCol1 + c * 32 : kCol2 + (c - 4) * 32),
                               c < 4 ? a.scale : 1.0f);
                if (group > 0) {
                    float x[32];
                    load_part(base + kCol1 + kDN + (group - 1) * 32, x);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4 *>(part + r * kDR + ((((group - 1) * 8 + i) ^ (r & 7)) << 2)) =
                            make_float4(x[4 * i] * a.scale, x[4 * i + 1] * a.scale, x[4 * i + 2] * a.scale,
                                        x[4 * i + 3] * a.scale);
                }
            } else {
#pragma unroll 1
                for (int c = group; c < 6; c += kGroups)
                    stage_bf16(rowbuf, kVecs, r, c * 4, base + kCol1 + c * 32, a.scale);
            }
        }
        elem_sync();
        const uint4 zero = make_uint4(0, 0, 0, 0);
        __nv_bfloat16 *dst = kKeys ? a.dkv + ((int64_t)(k0 + r0) * a.H + h) * kDKV : a.dq + ((int64_t)(q0 + r0) * a.H + h) * kDQ;
        const int64_t pitch = (int64_t)a.H * (kKeys ? kDKV : kDQ);
        for (int v = tid; v < rows * kVecs; v += kElem) {
            const int vr = v / kVecs, c = v % kVecs;
            *reinterpret_cast<uint4 *>(dst + vr * pitch + c * 8) =
                steps > 0 ? *reinterpret_cast<const uint4 *>(rowbuf + vr * kVecs * 16 + ((c ^ (vr & 7)) << 4)) : zero;
        }
        if (kKeys) {
            float4 *out = reinterpret_cast<float4 *>(a.part + ((int64_t)h * a.Tk + k0 + r0) * kDR);
            for (int v = tid; v < rows * (kDR / 4); v += kElem) {
                const int vr = v / (kDR / 4), c = v % (kDR / 4);
                out[v] = steps > 0 ? *reinterpret_cast<const float4 *>(part + vr * kDR + ((c ^ (vr & 7)) << 2))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kElem / 32)
        tc::tmem_dealloc(tmem, 512);
}

// dk_rope: its heads' parts in order, four numbers a thread.
__global__ void __launch_bounds__(256) mla_dkr_kernel(BwdArgs a)
{
    bool bad = false;
    for (int n = threadIdx.x; n < a.N; n += 256) {
        span_of(a.cu_q, n, a.Tq, bad);
        span_of(a.cu_k, n, a.Tk, bad);
    }
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (__syncthreads_or(bad) || x >= (int64_t)a.cu_k[a.N] * (kDR / 4))
        return;
    const float4 *p = reinterpret_cast<const float4 *>(a.part) + x;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int h = 0; h < a.H; ++h) {
        const float4 v = p[(int64_t)h * a.Tk * (kDR / 4)];
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
    }
    reinterpret_cast<uint2 *>(a.dkr)[x] = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

template <bool kKeys>
cudaError_t launch_side(const BwdMaps &maps, const BwdArgs &a, cudaStream_t s)
{
    const size_t smem = sizeof(BwdSmem) + 1024;
    static_assert(sizeof(BwdSmem) + 1024 <= 232448, "shared memory of one CTA");
    const cudaError_t e =
        cudaFuncSetAttribute(mla_bwd_kernel<kKeys>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    const int64_t grid = ((int64_t)(kKeys ? a.Tk : a.Tq) / kRows + a.N) * a.H;  // at least the tiles of any N sequences
    if (grid > 0x7fffffff)
        return cudaErrorInvalidValue;
    mla_bwd_kernel<kKeys><<<(unsigned)grid, kThreads, smem, s>>>(maps, a);
    return cudaGetLastError();
}

}  // namespace

size_t mla_bwd_workspace(int Tq, int Tk, int H)
{
    return 2 * round256((size_t)Tq * H * 4) + round256((size_t)Tk * H * kDR * 4) + 256;
}

cudaError_t launch_mla_bwd(int N, const int32_t *cu_q, const int32_t *cu_k, int Tq, int Tk, int H, bool causal,
                           float scale, const void *q, const void *kv, const void *k_rope, const void *o,
                           const float *lse, const void *dO, void *dq, void *dkv, void *dk_rope, void *workspace,
                           cudaStream_t s)
{
    const size_t rows = round256((size_t)Tq * H * 4);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    BwdArgs a{N, Tq, Tk, H, causal, scale, cu_q, cu_k, static_cast<const __nv_bfloat16 *>(o),
              static_cast<const __nv_bfloat16 *>(dO), lse, static_cast<__nv_bfloat16 *>(dq),
              static_cast<__nv_bfloat16 *>(dkv), static_cast<__nv_bfloat16 *>(dk_rope), reinterpret_cast<float *>(ws),
              reinterpret_cast<float *>(ws + rows), reinterpret_cast<float *>(ws + 2 * rows), device_status_ptr()};
    if (!a.status)
        return cudaErrorInvalidDevice;
    cudaError_t e = cudaSuccess;
    auto map = [&](CUtensorMap *m, const void *p, int numbers, int heads, int64_t n, int box, int blocks) {
        if (e == cudaSuccess && n > 0)
            e = make_rows_map(m, p, numbers, heads, n, box, blocks);
    };
    if (Tq > 0) {
        BwdMaps m{};
        map(&m.x1, q, kDQ, H, Tq, kRows, 3);
        map(&m.x2, dO, kDV, H, Tq, kRows, 2);
        map(&m.y1, kv, kDKV, H, Tk, kStep, 2);
        map(&m.y1r, k_rope, kDR, 0, Tk, kStep, 1);
        map(&m.y2, kv, kDKV, H, Tk, kStep, 2);
        if (e == cudaSuccess)
            e = launch_side<false>(m, a, s);
    }
    if (Tk > 0) {
        BwdMaps m{};
        map(&m.x1, kv, kDKV, H, Tk, kRows, 2);
        map(&m.x1r, k_rope, kDR, 0, Tk, kRows, 1);
        map(&m.x2, kv, kDKV, H, Tk, kRows, 2);
        map(&m.y1, q, kDQ, H, Tq, kStep, 3);
        map(&m.y2, dO, kDV, H, Tq, kStep, 2);
        if (e == cudaSuccess)
            e = launch_side<true>(m, a, s);
        if (e != cudaSuccess)
            return e;
        mla_dkr_kernel<<<(unsigned)(((int64_t)Tk * (kDR / 4) + 255) / 256), 256, 0, s>>>(a);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace kda

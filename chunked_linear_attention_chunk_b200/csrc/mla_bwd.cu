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
// other side (Y) 64 rows at a time:
//   S = X1 Y1^T (K = 192),  dP = X2 Y2^T (K = 128),  acc1 += e Y1 (N = 192),
//   keys only: acc2 += p Y2 (N = 128)
// with X1, Y1 the q and [k, k_rope] rows and X2, Y2 the dO and v rows.  A Y tile serves as K-major
// operand of the first two products and MN-major operand of the last two.
//
// A 128 x 64 x 16 product takes 52 cycles with both operands in shared memory and 32 with X in
// tensor memory, so X lives there as far as it fits beside the sums: all of it for dq (160 + 192
// columns), dO's partner v for dk and dv (64 + 320; k stays in shared memory).  That leaves one S
// and one dP of 64 columns, which the threads read at once; p and e go to the sums through shared
// memory, so that S and dP never wait for the sums.
//
// Three warps issue the products, one S, one dP, one the sums: a warp that finds its barriers ready
// still spends some 150 cycles on each, in which it feeds nothing to the tensor cores, and a 128 x
// 64 x 16 product takes about as long to issue as to run.  Two sets of eight warps take steps in
// turn, a thread half of a row.  The launch for dq computes D first and leaves D and lse in base 2,
// head by head, for the other.  dk_rope's parts are added over the heads, in order, by a third
// launch.
//
// Measured: 16 heads, 8192 tokens, causal: 414 us for dq and 547 us for dk and dv by themselves, 1120-1140
// us a call in a loop, where the 1000 W limit holds the clock near 1.5 GHz: 0.79 PFLOP/s of the formulas'
// 832 multiply-adds a pair, 1.1 of those taken; the tensor pipe is active 74 and 68 % of the time.  Six
// packed documents of 100 to 1500 tokens: 215-219 us; there a CTA's first 250 KB (2 to 3 us) and its last
// stores weigh as much as its ten steps (0.82 and 1.09 us each).
//
// Warps: 0-15 elementwise; 16 copies (TMA) of X and Y1; 17 S; 18 the sums; 19 dP and copies of Y2.
#include "mla_common.cuh"
#include "mla_tc.cuh"

namespace kda {

namespace {

using namespace mla;

constexpr int kElemWarps = 16;
constexpr int kElem = kElemWarps * 32;   // elementwise threads: two sets, two threads a row
constexpr int kThreads = kElem + 128;    // 20 warps: one more on a scheduler would cost 16 registers a thread
constexpr int kRows = 128;               // X rows of a CTA
constexpr int kStep = 64;                // Y rows a step
constexpr uint32_t kXBlk = kRows * 128;  // 64 numbers of the rows
constexpr uint32_t kYBlk = kStep * 128;

// Tensor-memory columns.
template <bool kKeys>
struct Cols {
    static constexpr uint32_t X1 = 0, X2 = kKeys ? 0 : 96;  // X1: queries only
    static constexpr uint32_t S = kKeys ? 64 : 160, P = S + kStep;
    static constexpr uint32_t Acc2 = P + kStep, Acc1 = kKeys ? Acc2 + 128 : Acc2;  // Acc2: keys only
    static_assert(Acc1 + kDQ <= 512, "tensor memory");
};

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

template <bool kKeys>
struct BwdSmem {
    // stages; with three of Y1 the keys' S waits for copies (its stage is held until acc1)
    static constexpr int kY1 = kKeys ? 4 : 5, kY2 = kKeys ? 2 : 4;
    alignas(1024) unsigned char x1[kKeys ? 3 * kXBlk : 16];
    // queries: the last two stages hold x1 on its way to tensor memory
    alignas(1024) unsigned char y1[kY1][3 * kYBlk];
    alignas(1024) unsigned char y2[kY2][2 * kYBlk];
    // e, p [128 rows][64 numbers]; before the first step x2 on its way to tensor memory
    alignas(1024) unsigned char e[kXBlk], p[kXBlk];
    alignas(16) float col[kKeys ? kY1 : 1][2][kStep];  // keys: lse in base 2 and D of a step's queries
    float delta[kRows];                    // queries: D
    uint64_t x_landed, x_full, y1_full[kY1], y1_empty[kY1], y2_full[kY2], y2_empty[kY2], tail[2];
    uint64_t s_full[2], dp_full[2], p_full[2], e_full[2], acc1_done[2], acc2_done[2];  // by step parity
    uint64_t s_read, dp_read, done;
    uint32_t tmem_slot;
    int64_t find[40];
};

// A warp clears the rows from `live` on of `blocks` blocks and passes the stage on: rows behind a
// sequence's end may hold anything, and 0 * NaN is NaN.
__device__ __forceinline__ void zero_tail(unsigned char *p, int blocks, int live, uint64_t *full)
{
    for (int i = threadIdx.x & 31; i < (kStep - live) * 8 * blocks; i += 32)
        *reinterpret_cast<uint4 *>(p + i % blocks * kYBlk + (live + i / (8 * blocks)) * 128 + i / blocks % 8 * 16) =
            make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
    if (elect())
        mbar_arrive(full);
}

__device__ __forceinline__ void elem_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kElem) : "memory"); }

// 32 columns of this thread's lane.
__device__ __forceinline__ void load_32(uint32_t taddr, float (&x)[32])
{
    uint32_t a[32];
    tc::ld_32x32b_x32(taddr, a);
    tc::wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i)
        x[i] = __uint_as_float(a[i]);
}

// 32 numbers of row r as bfloat16 into vectors [v0, v0 + 4) of its 128-byte row (swizzled).
__device__ __forceinline__ void store_32(unsigned char *rows, int r, int v0, const float (&x)[32])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(rows + r * 128 + (((v0 + i) ^ (r & 7)) << 4)) =
            make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                       pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
}

// Row r of a block of 64 numbers (swizzled) to 32 columns of this thread's lane.
__device__ __forceinline__ void keep_64(uint32_t taddr, const unsigned char *rows, int r)
{
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint4 v = *reinterpret_cast<const uint4 *>(rows + r * 128 + ((i ^ (r & 7)) << 4));
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
    }
    tc::st_32x32b_x32(taddr, w);
}

// 32 columns of this thread's lane, times f, as bfloat16 into vectors [v0, v0 + 4) of its row of
// `vecs` 16-byte vectors (swizzled: neighbouring rows start in different banks).
__device__ __forceinline__ void stage_bf16(unsigned char *rows, int vecs, int r, int v0, uint32_t taddr, float f)
{
    float x[32];
    load_32(taddr, x);
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
    using SM = BwdSmem<kKeys>;
    using C = Cols<kKeys>;
    SM &sm = *reinterpret_cast<SM *>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x % a.H;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the next launch may set up meanwhile
    if (warp == kElemWarps)
        tc::tmem_alloc(&sm.tmem_slot, 512);
    if (tid == 0) {
        mbar_init(&sm.x_landed, 1);
        mbar_init(&sm.x_full, kKeys ? 8 : kElemWarps);
        mbar_init(&sm.tail[0], 1);
        mbar_init(&sm.tail[1], 1);
        for (int i = 0; i < SM::kY1; ++i) {
            mbar_init(&sm.y1_full[i], kKeys ? 33 : 1);
            mbar_init(&sm.y1_empty[i], 1);
        }
        for (int i = 0; i < SM::kY2; ++i) {
            mbar_init(&sm.y2_full[i], 1);
            mbar_init(&sm.y2_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.dp_full[i], 1);
            mbar_init(&sm.p_full[i], 8);
            mbar_init(&sm.e_full[i], 8);
            mbar_init(&sm.acc1_done[i], 1);
            mbar_init(&sm.acc2_done[i], 1);
        }
        mbar_init(&sm.s_read, 8);
        mbar_init(&sm.dp_read, 8);
        mbar_init(&sm.done, 1);
        fence_mbar_init_cluster();
        prefetch_map(&maps.x1);
        prefetch_map(&maps.x2);
        prefetch_map(&maps.y1);
        prefetch_map(&maps.y2);
        prefetch_map(kKeys ? &maps.x1r : &maps.y1r);
    }
    const Item it = find_item<kThreads>(
        a.N, blockIdx.x / a.H,
        [&](int n, bool &bad) {
            const Span q = span_of(a.cu_q, n, a.Tq, bad), k = span_of(a.cu_k, n, a.Tk, bad);
            return ((kKeys ? k : q).len() + kRows - 1) / kRows;
        },
        sm.find);
    if (it.bad && tid == 0)
        report_device_error(a.status, KDA_ERR_INVALID_ARG);
    if (it.bad || it.seq < 0) {
        if (warp == kElemWarps) {
            tc::tmem_dealloc(sm.tmem_slot, 512);
            asm volatile("griddepcontrol.wait;" ::: "memory");  // no launch ends before the one it follows
        }
        return;
    }
    const int q0 = a.cu_q[it.seq], k0 = a.cu_k[it.seq], lq = a.cu_q[it.seq + 1] - q0, lk = a.cu_k[it.seq + 1] - k0;
    const int lx = kKeys ? lk : lq, ly = kKeys ? lq : lk;
    // with a causal mask the first keys and the last queries have the most to do: they go first
    const int r0 = (kKeys ? it.k : (lx + kRows - 1) / kRows - 1 - it.k) * kRows;
    int rows = min(kRows, lx - r0);
    const int off = lk - lq;  // causal: key j is visible to query i from i = j - off on
    // Y rows [y_first, y_end)
    const int y_first = kKeys && a.causal ? max(0, r0 - off) : 0;
    const int y_end = !kKeys && a.causal ? min(ly, r0 + rows + off) : ly;
    int steps = y_first < y_end ? (y_end - y_first + kStep - 1) / kStep : 0;
    if (!rows_in(r0, rows, lx, kKeys ? k0 : q0, kKeys ? a.Tk : a.Tq) ||
        (steps > 0 && !rows_in(y_first, y_end - y_first, ly, kKeys ? q0 : k0, kKeys ? a.Tq : a.Tk))) {
        report_device_error(a.status, KDA_ERR_DEVICE_BOUNDS);
        rows = steps = 0;
    }

    if (warp == kElemWarps && steps > 0 && elect()) {
        const int x = (kKeys ? k0 : q0) + r0;
        mbar_arrive_expect_tx(&sm.x_landed, 5 * kXBlk);
        unsigned char *x1 = kKeys ? sm.x1 : sm.y1[SM::kY1 - 2];
        tma_load_4d(x1, &maps.x1, 0, x, h, 0, &sm.x_landed);
        if (kKeys)
            tma_load_2d(x1 + 2 * kXBlk, &maps.x1r, 0, x, &sm.x_landed);
        tma_load_4d(sm.e, &maps.x2, 0, x, h, kKeys ? 2 : 0, &sm.x_landed);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem_slot;
    Waits wait{false};

    if (warp == kElemWarps) {
        // ---------------- copies of Y1
        asm volatile("griddepcontrol.wait;" ::: "memory");  // keys: the launch that writes D and lse
        Ring<SM::kY1> r1;
        for (int i = 0; i < steps; ++i, r1.step()) {
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
            else if (!kKeys && r1.slot == SM::kY1 - 2)
                wait(&sm.x_full, 0);
            uint64_t *bar = live < kStep ? &sm.tail[0] : &sm.y1_full[r1.slot];
            if (elect() && !wait.dead) {
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
            if (live < kStep) {
                wait(&sm.tail[0], 0);
                zero_tail(sm.y1[r1.slot], 3, live, &sm.y1_full[r1.slot]);
            }
        }
    } else if (warp == kElemWarps + 1) {
        // ---------------- S, as soon as the threads have read the one before
        constexpr uint32_t id = tc::idesc_bf16(kRows, kStep, false, false);
        const Desc x1(smem_u32(sm.x1), 16, 1024, tc::kSw128), y1(smem_u32(sm.y1[0]), 16, 1024, tc::kSw128);
        Ring<SM::kY1> r1;
        if (steps > 0)
            wait(kKeys ? &sm.x_landed : &sm.x_full, 0);
        for (int i = 0; i < steps; ++i, r1.step()) {
            wait(&sm.y1_full[r1.slot], r1.round & 1);
            if (i > 0)
                wait(&sm.s_read, (i - 1) & 1);
            tc::fence_after_sync();
            if (elect()) {
                const uint32_t y0 = r1.slot * 3 * kYBlk;
#pragma unroll
                for (int ks = 0; ks < kDQ / 16; ++ks) {
                    const uint64_t b = y1.at(y0 + (ks >> 2) * kYBlk + (ks & 3) * 32);
                    if (kKeys)
                        tc::mma_bf16(tmem + C::S, x1.at((ks >> 2) * kXBlk + (ks & 3) * 32), b, id, ks > 0 ? 1u : 0u);
                    else
                        tc::mma_bf16_ts(tmem + C::S, tmem + C::X1 + ks * 8, b, id, ks > 0 ? 1u : 0u);
                }
                tc::commit(&sm.s_full[i & 1]);
            }
        }
    } else if (warp == kElemWarps + 3) {
        // ---------------- dP, likewise, and the copies of Y2
        constexpr uint32_t id = tc::idesc_bf16(kRows, kStep, false, false);
        const Desc y2(smem_u32(sm.y2[0]), 16, 1024, tc::kSw128);
        auto fetch = [&](int i, int slot) {
            const int first = y_first + i * kStep, live = ly - first;
            uint64_t *bar = live < kStep ? &sm.tail[1] : &sm.y2_full[slot];
            if (elect() && !wait.dead) {
                mbar_arrive_expect_tx(bar, 2 * kYBlk);
                tma_load_4d(sm.y2[slot], &maps.y2, 0, (kKeys ? q0 : k0) + first, h, kKeys ? 0 : 2, bar);
            }
            __syncwarp();
            if (live < kStep) {
                wait(&sm.tail[1], 0);
                zero_tail(sm.y2[slot], 2, live, &sm.y2_full[slot]);
            }
        };
        for (int i = 0; i < SM::kY2 && i < steps; ++i)
            fetch(i, i);
        Ring<SM::kY2> r2, rf;
        if (steps > 0)
            wait(&sm.x_full, 0);
        for (int i = 0; i < steps; ++i, r2.step()) {
            wait(&sm.y2_full[r2.slot], r2.round & 1);
            if (i > 0)
                wait(&sm.dp_read, (i - 1) & 1);
            tc::fence_after_sync();
            if (elect()) {
                const uint32_t y0 = r2.slot * 2 * kYBlk;
#pragma unroll
                for (int ks = 0; ks < kDV / 16; ++ks)
                    tc::mma_bf16_ts(tmem + C::P, tmem + C::X2 + ks * 8, y2.at(y0 + (ks >> 2) * kYBlk + (ks & 3) * 32), id,
                                    ks > 0 ? 1u : 0u);
                tc::commit(&sm.dp_full[i & 1]);
            }
            // dP(i - 1) has been read; once acc2(i - 1) is over its Y2 makes room
            if (i > 0) {
                if (i - 1 + SM::kY2 < steps) {
                    if (kKeys)
                        wait(&sm.y2_empty[rf.slot], rf.round & 1);
                    fetch(i - 1 + SM::kY2, rf.slot);
                }
                rf.step();
            }
        }
    } else if (warp == kElemWarps + 2) {
        // ---------------- the sums
        constexpr uint32_t id_1 = tc::idesc_bf16(kRows, kDQ, false, true), id_2 = tc::idesc_bf16(kRows, kDV, false, true);
        const Desc t1(smem_u32(sm.y1[0]), kYBlk, 1024, tc::kSw128), t2(smem_u32(sm.y2[0]), kYBlk, 1024, tc::kSw128),
            ed(smem_u32(sm.e), 16, 1024, tc::kSw128), pd(smem_u32(sm.p), 16, 1024, tc::kSw128);
        Ring<SM::kY1> r1;
        Ring<SM::kY2> r2;
        for (int i = 0; i < steps; ++i, r1.step(), r2.step()) {
            const uint32_t buf = i & 1, par = (i >> 1) & 1;
            if (kKeys) {
                wait(&sm.y2_full[r2.slot], r2.round & 1);
                wait(&sm.p_full[buf], par);
                tc::fence_after_sync();
                if (elect()) {
#pragma unroll
                    for (int ks = 0; ks < kStep / 16; ++ks)
                        tc::mma_bf16(tmem + C::Acc2, pd.at(ks * 32), t2.at(r2.slot * 2 * kYBlk + ks * 2048), id_2,
                                     i > 0 || ks > 0 ? 1u : 0u);
                    tc::commit(&sm.acc2_done[buf]);
                    tc::commit(&sm.y2_empty[r2.slot]);
                }
            }
            wait(&sm.e_full[buf], par);
            tc::fence_after_sync();
            if (elect()) {
#pragma unroll
                for (int ks = 0; ks < kStep / 16; ++ks)
                    tc::mma_bf16(tmem + C::Acc1, ed.at(ks * 32), t1.at(r1.slot * 3 * kYBlk + ks * 2048), id_1,
                                 i > 0 || ks > 0 ? 1u : 0u);
                tc::commit(&sm.acc1_done[buf]);
                tc::commit(&sm.y1_empty[r1.slot]);
                if (i + 1 == steps)
                    tc::commit(&sm.done);
            }
        }
    } else {
        // ---------------- elementwise: half a row a thread, every other step
        const int r = (warp & 3) * 32 + lane, quarter = warp >> 2, half = quarter & 1, set = quarter >> 1;
        const bool live = r < rows;
        const uint32_t base = tc::taddr(tmem, (uint32_t)(warp & 3) * 32, 0);
        const float sl2 = a.scale * kLog2e;
        float lse2 = INFINITY, delta = 0.0f;
        auto arrive = [&](uint64_t *bar) {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar);
        };
        // for D = dO . o, 16 lanes a row: loaded first, all at once (dO from the tile that comes with X
        // instead measured 219 us against 210 for six packed documents)
        constexpr int kDRows = kKeys ? 1 : kRows / kElemWarps / 2;
        uint4 od[kDRows][2];
        float l = 0.0f;
        const int d0 = warp * (kRows / kElemWarps) + (lane >> 4);
        if constexpr (!kKeys) {
            l = live ? a.lse[(int64_t)(q0 + r0 + r) * a.H + h] : -INFINITY;
#pragma unroll
            for (int k = 0; k < kDRows; ++k) {
                const int64_t at = ((int64_t)(q0 + r0 + d0 + 2 * k) * a.H + h) * kDV + (lane & 15) * 8;
                const bool in = d0 + 2 * k < rows;
                od[k][0] = in ? *reinterpret_cast<const uint4 *>(a.o + at) : make_uint4(0, 0, 0, 0);
                od[k][1] = in ? *reinterpret_cast<const uint4 *>(a.dO + at) : make_uint4(0, 0, 0, 0);
            }
        }
        // X to tensor memory (a row a lane), 64 numbers a warp at a time
        if (steps > 0 && (!kKeys || quarter < 2)) {
            wait(&sm.x_landed, 0);
            if (!kKeys && quarter < 3)
                keep_64(base + C::X1 + quarter * 32, sm.y1[SM::kY1 - 2] + quarter * kXBlk, r);
            else if (kKeys)
                keep_64(base + C::X2 + quarter * 32, sm.e + quarter * kXBlk, r);
            else
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    keep_64(base + C::X2 + b * 32, sm.e + b * kXBlk, r);
            tc::wait_st();
            tc::fence_before_sync();
            arrive(&sm.x_full);
        }
        if constexpr (!kKeys) {
#pragma unroll
            for (int k = 0; k < kDRows; ++k) {
                const uint4 u = od[k][0], v = od[k][1];
                const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
                float d = 0.0f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 f = unpack_bf16x2(uw[c]), g = unpack_bf16x2(vw[c]);
                    d += f.x * g.x + f.y * g.y;
                }
#pragma unroll
                for (int c = 8; c > 0; c >>= 1)
                    d += __shfl_xor_sync(0xffffffffu, d, c);
                if ((lane & 15) == 0)
                    sm.delta[d0 + 2 * k] = d;
            }
            lse2 = l == -INFINITY ? INFINITY : l * kLog2e;  // a row that sees no key: weights 0
            elem_sync();
            delta = sm.delta[r];
            if (live && quarter == 0) {
                a.delta[(int64_t)h * a.Tq + q0 + r0 + r] = delta;
                a.lse2[(int64_t)h * a.Tq + q0 + r0 + r] = lse2;
            }
        }
        // the first step's p goes where v lands: not before the warps that take v from there have their
        // rows (S is issued without them; the later steps wait for the sum of the one before)
        if (kKeys && set == 0 && steps > 0)
            wait(&sm.x_full, 0);
        for (int i = set; i < steps; i += 2) {
            const int y = y_first + i * kStep;  // place of the step's first column
            const uint32_t par = (i >> 1) & 1;
            const int slot = i % SM::kY1, round = i / SM::kY1;
            // columns lo .. hi - 1 are visible to the row
            int lo = 0, hi;
            bool edge;
            if (kKeys) {
                edge = y + kStep > ly || (a.causal && r0 + kRows - 1 > y + off);
                hi = ly - y;
                lo = a.causal ? r0 + r - off - y : 0;
            } else {
                edge = y + kStep > (a.causal ? min(ly, r0 + off + 1) : ly);
                hi = (a.causal ? min(ly, r0 + r + off + 1) : ly) - y;
            }
            const uint32_t seen = edge ? bit_span(lo - half * 32, hi - half * 32) : 0xffffffffu;
            float p[32], x[32];
            wait(&sm.s_full[set], par);
            tc::fence_after_sync();
            load_32(base + C::S + half * 32, p);
            tc::fence_before_sync();
            arrive(&sm.s_read);
            if (kKeys) {
                wait(&sm.y1_full[slot], round & 1);  // the step's lse and D
                const float4 *l = reinterpret_cast<const float4 *>(sm.col[slot][0] + half * 32);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float4 v = l[k];
                    p[4 * k] = ex2(fmaf(p[4 * k], sl2, -v.x));
                    p[4 * k + 1] = ex2(fmaf(p[4 * k + 1], sl2, -v.y));
                    p[4 * k + 2] = ex2(fmaf(p[4 * k + 2], sl2, -v.z));
                    p[4 * k + 3] = ex2(fmaf(p[4 * k + 3], sl2, -v.w));
                }
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    p[k] = ex2(fmaf(p[k], sl2, -lse2));
            }
            if (edge) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    p[k] = seen >> k & 1 ? p[k] : 0.0f;
            }
            if (kKeys) {
                if (i > 0)
                    wait(&sm.acc2_done[set ^ 1], ((i - 1) >> 1) & 1);
                store_32(sm.p, r, half * 4, p);
                fence_proxy_async_smem();
                arrive(&sm.p_full[set]);
            }
            wait(&sm.dp_full[set], par);
            tc::fence_after_sync();
            load_32(base + C::P + half * 32, x);
            tc::fence_before_sync();
            arrive(&sm.dp_read);
            if (kKeys) {
                const float4 *d = reinterpret_cast<const float4 *>(sm.col[slot][1] + half * 32);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float4 v = d[k];
                    x[4 * k] = p[4 * k] * (x[4 * k] - v.x);
                    x[4 * k + 1] = p[4 * k + 1] * (x[4 * k + 1] - v.y);
                    x[4 * k + 2] = p[4 * k + 2] * (x[4 * k + 2] - v.z);
                    x[4 * k + 3] = p[4 * k + 3] * (x[4 * k + 3] - v.w);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    x[k] = p[k] * (x[k] - delta);
            }
            if (edge) {  // a hidden pair's dP may be anything
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    x[k] = seen >> k & 1 ? x[k] : 0.0f;
            }
            if (i > 0)
                wait(&sm.acc1_done[set ^ 1], ((i - 1) >> 1) & 1);
            store_32(sm.e, r, half * 4, x);
            fence_proxy_async_smem();
            arrive(&sm.e_full[set]);
        }
        // ---- the sums, through shared memory (nothing reads the tiles any more), so that the
        // writes are whole rows
        if (steps > 0) {
            wait(&sm.done, 0);
            tc::fence_after_sync();
        }
        constexpr int kVecs = (kKeys ? kDKV : kDQ) / 8;  // 16-byte vectors of a row of dkv or dq
        unsigned char *rowbuf = sm.y1[0];
        float *part = reinterpret_cast<float *>(sm.e);
        static_assert(sizeof(sm.y1) >= kRows * kVecs * 16 && 2 * kXBlk >= kRows * kDR * 4, "room for the sums");
        if (steps > 0) {
            if (kKeys) {
                // dk (4 x 32 columns), dv (4 x 32), the rope part of dk (2 x 32), shared out to the groups
#pragma unroll 1
                for (int c = quarter; c < 10; c += 4) {
                    if (c < 8) {
                        stage_bf16(rowbuf, kVecs, r, c * 4, base + (c < 4 ? C::Acc1 + c * 32 : C::Acc2 + (c - 4) * 32),
                                   c < 4 ? a.scale : 1.0f);
                        continue;
                    }
                    float x[32];
                    load_32(base + C::Acc1 + kDN + (c - 8) * 32, x);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4 *>(part + r * kDR + ((((c - 8) * 8 + i) ^ (r & 7)) << 2)) =
                            make_float4(x[4 * i] * a.scale, x[4 * i + 1] * a.scale, x[4 * i + 2] * a.scale,
                                        x[4 * i + 3] * a.scale);
                }
            } else {
#pragma unroll 1
                for (int c = quarter; c < 6; c += 4)
                    stage_bf16(rowbuf, kVecs, r, c * 4, base + C::Acc1 + c * 32, a.scale);
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
    wait.finish(a.status);
    if (warp == kElemWarps)
        tc::tmem_dealloc(tmem, 512);
}

// dk_rope: its heads' parts in order, four numbers a thread.
__global__ void __launch_bounds__(256) mla_dkr_kernel(BwdArgs a)
{
    bool bad = false;
    asm volatile("griddepcontrol.wait;" ::: "memory");
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

// A launch that may set up while the one before it in the stream ends (`early`; it waits on the
// device before it reads what that one writes).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t s, bool early,
                         const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool kKeys>
cudaError_t launch_side(const BwdMaps &maps, const BwdArgs &a, cudaStream_t s)
{
    const size_t smem = sizeof(BwdSmem<kKeys>) + 1024;
    static_assert(sizeof(BwdSmem<kKeys>) + 1024 <= 232448, "shared memory of one CTA");
    const cudaError_t e =
        cudaFuncSetAttribute(mla_bwd_kernel<kKeys>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    const int64_t grid = ((int64_t)(kKeys ? a.Tk : a.Tq) / kRows + a.N) * a.H;  // at least the tiles of any N sequences
    return launch_after(mla_bwd_kernel<kKeys>, (unsigned)grid, kThreads, smem, s, kKeys && a.Tq > 0, maps, a);
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
        e = launch_after(mla_dkr_kernel, (unsigned)(((int64_t)Tk * (kDR / 4) + 255) / 256), 256, 0, s, true, a);
    }
    return e;
}

}  // namespace kda

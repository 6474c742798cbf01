// mla_decode.cu -- absorbed latent attention of a few new tokens over a paged cache.
//
//   s_j = scale q . c_j,  o = sum_j softmax_j(s) c_j[0:512]
// Every query head of a latent group reads the same cached rows (1152 B each in bfloat16), so a
// row is brought in once for up to 64 (token, head) columns and the kernel is bound by the cache's
// bytes: at 32 columns it has 2 (576 + 512) 32 / 1152 = 60 flops a byte, a quarter of what the
// tensor cores could take.
//
// Roles are swapped so that the tensor cores' M is the cached rows, not the few heads, and
// nothing is padded:
//   S^T [64 rows x NC columns] = C Q^T          (M = 64, K = 576; C as the copy laid it down)
//   O^T [512 x NC] += C[:, 0:512]^T P^T         (M = 128 four times, K = 64; C read MN-major)
// The same shared-memory tile is the A operand of both; only P^T (64 x NC) is written by threads.
//
// One persistent CTA per SM takes an equal share of all 64-row tiles of all (sequence, group)
// units in order, so a batch of any lengths is balanced without the host knowing them.  A unit
// inside one CTA's share is finished there; the others leave normalised partial results with
// their log-sum-exp in the workspace, which a second launch joins in order (equal calls give
// equal bits; the shares depend on the lengths and the SM count alone).
//
// Warps: 0-3 softmax (S^T in the 16-lane M = 64 layout, running maximum per column, O^T in
// tensor memory rescaled only when a column's maximum grows by more than 2^8, which float32 sums
// and a bfloat16 weight hold exactly as well); 4 copies (TMA, 16 KB pairs of 64 x 64 blocks through
// a ring); 5 issues S^T block by block as it arrives; 6 issues O^T and frees the ring; 7 loads Q.
#include <cudaTypedefs.h>
#include <cuda_fp8.h>

#include "mla_common.cuh"
#include "mla_tc.cuh"

namespace kda {

namespace {

using namespace mla;

constexpr int kConv = 8;  // warps that turn codes into bfloat16 rows
template <bool kE4M3>
constexpr int kThreads = kE4M3 ? 256 + kConv * 32 : 256;
constexpr int kTok = 64;                    // cached rows a tile
constexpr uint32_t kBlk = kTok * 128;       // 64 rows x 64 numbers, 128-byte swizzle
constexpr uint32_t kPair = 2 * kBlk;        // 128 latent numbers: the M of one O^T product
constexpr int kPairs = kDL / 128;           // pairs a tile
constexpr float kGrow = 8.0f;               // log2 by which a maximum may grow without rescaling

struct DecArgs {
    int N, Sq, H, G, num_pages, page_size, max_pages, CT, shares;
    float scale_log2;
    const __nv_bfloat16 *q;
    const float *cache_scale;
    const int32_t *block_table, *kv_lens;
    __nv_bfloat16 *o;
    float *lse;
    float *part_o, *part_lse;  // [CTA][2][NC][512], [CTA][2][NC]
    int2 *meta;                // [unit][CT]: first share, 2 * shares + (the first starts inside its share)
    unsigned int *status;
};

// The cache as [block of 64 numbers][pool row][group][64], so that one copy brings a pair of
// blocks (or the rope block) of up to 64 rows as the products read them; and q as [block][row][64].
struct DecMaps {
    CUtensorMap pair, rope, q;
    int rows;    // pool rows a copy: min(page_size, 64)
    int q_rows;  // rows of q a copy
};

// Tiles of a sequence; 0 for a length that is refused.
__device__ __forceinline__ int tiles_of(const DecArgs &a, int n)
{
    const int len = a.kv_lens[n];
    return len > 0 && len <= (int64_t)a.max_pages * a.page_size ? (len + kTok - 1) / kTok : 0;
}

// One CTA's share of the tiles, piece by piece; a piece is a run of tiles of one unit.
struct Pieces {
    int n, g, t, tiles, take;  // current piece: sequence, group, first tile, the unit's tiles, tiles taken
    int64_t left, pos;         // tiles left behind the current piece; place of the piece's first tile
    __device__ __forceinline__ void settle(const DecArgs &a)
    {
        while (n < a.N && (tiles = tiles_of(a, n)) == 0) {
            ++n;
            g = 0;
        }
        take = (int)min((int64_t)(tiles - t), left);
        left -= take;
    }
    __device__ __forceinline__ void next(const DecArgs &a)
    {
        pos += take;
        t = 0;
        if (++g == a.G) {
            g = 0;
            ++n;
        }
        settle(a);
    }
};

template <int NC, bool kE4M3>
struct DecSmem {
    // pairs and rope blocks of bfloat16 rows held, and pairs of blocks of codes in flight
    static constexpr int kRing = kE4M3 ? (NC == 64 ? 5 : 7) : (NC == 64 ? 8 : 10);
    static constexpr int kRopes = kE4M3 ? 1 : (NC == 64 ? 2 : 3);
    static constexpr int kStage = kE4M3 ? (NC == 64 ? 6 : 8) : 1;
    alignas(1024) unsigned char pair[kRing][kPair];
    alignas(1024) unsigned char rope[kRopes][kBlk];
    alignas(1024) unsigned char q[kDC / 64][NC * 128];
    alignas(1024) unsigned char p[kTok * NC * 2];
    alignas(1024) unsigned char stage[kStage][kE4M3 ? kBlk : 16];
    float red[4][NC];  // per warp: column maxima, then column sums
    float fac[NC];     // per column: rescaling factor, then 1 / sum
    uint64_t full_pair[kRing], empty_pair[kRing], full_rope[kRopes], empty_rope[kRopes];
    uint64_t full_stage[kStage], empty_stage[kStage];
    uint64_t s_full[2], s_empty[2], p_full, pv_done, q_full, q_empty;
    uint32_t tmem_slot;
    int64_t find[40];
    int64_t share[3];  // begin, end of the CTA's share; tiles a share
    int first[3];      // n, g, t of its first tile
};

// Four e4m3 codes as bfloat16 pairs: exact, NaN codes stay NaN.
__device__ __forceinline__ uint2 decode4(uint32_t w)
{
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 x = __half22float2(__half2(a)), y = __half22float2(__half2(b));
    return make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(y.x, y.y));
}

template <int NC, bool kE4M3>
__global__ void __launch_bounds__(kThreads<kE4M3>, 1)
    mla_decode_kernel(const __grid_constant__ DecMaps maps, DecArgs a)
{
    extern __shared__ unsigned char raw[];
    using SM = DecSmem<NC, kE4M3>;
    constexpr int kT = kThreads<kE4M3>;
    SM &sm = *reinterpret_cast<SM *>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int share = blockIdx.x / a.CT, ct = blockIdx.x % a.CT, Hg = a.H / a.G, cols = a.Sq * Hg;
    constexpr uint32_t kTmemCols = NC == 64 ? 512 : 256;

    if (tid == 0) {
        for (int i = 0; i < SM::kRing; ++i) {
            mbar_init(&sm.full_pair[i], kE4M3 ? kConv * 32 : 1);
            mbar_init(&sm.empty_pair[i], 1);
        }
        for (int i = 0; i < SM::kRopes; ++i) {
            mbar_init(&sm.full_rope[i], kE4M3 ? kConv * 32 : 1);
            mbar_init(&sm.empty_rope[i], 1);
        }
        for (int i = 0; i < SM::kStage; ++i) {
            mbar_init(&sm.full_stage[i], 1);
            mbar_init(&sm.empty_stage[i], kConv);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_empty[i], 4);
        }
        mbar_init(&sm.p_full, 128);
        mbar_init(&sm.pv_done, 1);
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        fence_mbar_init_cluster();
    }
    if (warp == 4)
        tc::tmem_alloc(&sm.tmem_slot, kTmemCols);
    // this CTA's share: all tiles, then the unit that its first one falls in
    {
        int64_t mine = 0;
        bool bad = false;
        for (int n = tid; n < a.N; n += kT) {
            const int t = tiles_of(a, n);
            mine += t;
            bad |= t == 0 && a.kv_lens[n] != 0;
            if (t == 0 && n % a.shares == share)  // nobody's piece: the join writes its (empty) result
                for (int g = 0; g < a.G; ++g)
                    a.meta[((int64_t)n * a.G + g) * a.CT + ct] = make_int2(0, 0);
        }
        if (bad)
            report_device_error(a.status, KDA_ERR_INVALID_ARG);
        const int64_t all = cta_sum<kT>(mine, sm.find);
        const int64_t total = all * a.G, per = (total + a.shares - 1) / a.shares;
        const int64_t begin = min(total, share * per), end = min(total, begin + per);
        Item it{0, 0};
        if (begin < end)
            find_item<kT>(a.N, begin, [&](int n) { return tiles_of(a, n) * a.G; }, it, sm.find);
        if (tid == 0) {
            sm.share[0] = begin;
            sm.share[1] = end;
            sm.share[2] = per;
            const int tiles = begin < end ? tiles_of(a, it.seq) : 1;
            sm.first[0] = it.seq;
            sm.first[1] = it.k / tiles;
            sm.first[2] = it.k % tiles;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem_slot;
    const int64_t begin = sm.share[0], end = sm.share[1], per = sm.share[2];
    Pieces w;
    w.n = sm.first[0], w.g = sm.first[1], w.t = sm.first[2];
    w.pos = begin;
    w.left = end - begin;
    w.take = 0;
    if (begin < end)
        w.settle(a);
    Waits wait{a.status, false};

    if (warp == 4) {
        // ---------------- copies
        const int ppt = kTok / maps.rows;  // copies a block
        int batch_n = -1, batch_0 = 0, ids = 0;
        Ring<SM::kRing> rp;
        Ring<SM::kRopes> rr;
        Ring<SM::kStage> rst;
        for (; w.take > 0 && !wait.dead; w.next(a)) {
            const int len = a.kv_lens[w.n], pages = (len + a.page_size - 1) / a.page_size;
            const int32_t *row = a.block_table + (int64_t)w.n * a.max_pages;
            int e = w.t * kTok / a.page_size, off = w.t * kTok % a.page_size;  // page entry, slot in it
            for (int t = w.t; t < w.t + w.take && !wait.dead; ++t) {
                // the pool rows of the tile's copies, from the table 32 entries at a time
                int at[4], live = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    at[b] = -1;
                    if (b < ppt && e < pages) {
                        if (w.n != batch_n || e < batch_0 || e >= batch_0 + 32) {
                            batch_n = w.n;
                            batch_0 = e;
                            ids = e + lane < pages ? row[e + lane] : 0;
                        }
                        const int page = __shfl_sync(0xffffffffu, ids, e - batch_0);
                        if (page >= 0 && page < a.num_pages) {
                            at[b] = page * a.page_size + off;
                            ++live;
                        } else if (lane == 0) {
                            report_device_error(a.status, KDA_ERR_INVALID_ARG);
                        }
                        off += maps.rows;
                        if (off >= a.page_size) {
                            off = 0;
                            ++e;
                        }
                    }
                }
                constexpr uint32_t kRow = kE4M3 ? 64 : 128;  // bytes of a block's row
                const uint32_t bytes = (uint32_t)(live * maps.rows) * kRow;
                // n blocks from `block` on; pages of 64 rows and more take one copy
                auto copy = [&](unsigned char *dst, int block, int n, uint64_t *bar) {
                    mbar_arrive_expect_tx(bar, n * bytes);
                    if (ppt == 1) {
                        if (at[0] >= 0)
                            tma_load_4d(dst, n == 2 ? &maps.pair : &maps.rope, 0, w.g, at[0], block, bar);
                        return;
                    }
                    for (int i = 0; i < n; ++i)
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (at[b] >= 0)
                                tma_load_4d(dst + i * kTok * kRow + b * maps.rows * kRow, &maps.rope, 0, w.g, at[b],
                                            block + i, bar);
                };
                if constexpr (kE4M3) {
#pragma unroll
                    for (int j = 0; j <= kPairs; ++j, rst.step()) {
                        if (rst.round > 0)
                            wait(&sm.empty_stage[rst.slot], (rst.round - 1) & 1);
                        if (!wait.dead && elect())
                            copy(sm.stage[rst.slot], j == 0 ? 2 * kPairs : 2 * (j - 1), j == 0 ? 1 : 2,
                                 &sm.full_stage[rst.slot]);
                    }
                } else {
                    if (rr.round > 0)
                        wait(&sm.empty_rope[rr.slot], (rr.round - 1) & 1);
                    if (!wait.dead && elect())
                        copy(sm.rope[rr.slot], 2 * kPairs, 1, &sm.full_rope[rr.slot]);
                    rr.step();
#pragma unroll
                    for (int j = 0; j < kPairs; ++j, rp.step()) {
                        if (rp.round > 0)
                            wait(&sm.empty_pair[rp.slot], (rp.round - 1) & 1);
                        if (!wait.dead && elect())
                            copy(sm.pair[rp.slot], 2 * j, 2, &sm.full_pair[rp.slot]);
                    }
                }
                wait.dead = __any_sync(0xffffffffu, wait.dead);
            }
        }
    } else if (warp == 5) {
        // ---------------- S^T = C Q^T, block by block as the tile arrives (rope first)
        constexpr uint32_t id = tc::idesc_bf16(64, NC, false, false);
        const Desc rope(smem_u32(sm.rope[0]), 16, 1024, tc::kSw128), pair(smem_u32(sm.pair[0]), 16, 1024, tc::kSw128),
            qd(smem_u32(sm.q[0]), 16, 1024, tc::kSw128);
        Ring<SM::kRing> rp;
        Ring<SM::kRopes> rr;
        Ring<2> rs;
        uint32_t nq = 0;
        for (; w.take > 0 && !wait.dead; w.next(a), ++nq) {
            wait(&sm.q_full, nq & 1);
            for (int t = 0; t < w.take && !wait.dead; ++t, rs.step()) {
                if (rs.round > 0)
                    wait(&sm.s_empty[rs.slot], (rs.round - 1) & 1);
                const uint32_t d = tmem + rs.slot * NC;
                wait(&sm.full_rope[rr.slot], rr.round & 1);
                tc::fence_after_sync();
                if (elect()) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc::mma_bf16(d, rope.at(rr.slot * kBlk + ks * 32), qd.at((kDC / 64 - 1) * NC * 128 + ks * 32), id,
                                     ks > 0 ? 1u : 0u);
                    tc::commit(&sm.empty_rope[rr.slot]);
                }
                rr.step();
#pragma unroll
                for (int j = 0; j < kPairs; ++j, rp.step()) {
                    wait(&sm.full_pair[rp.slot], rp.round & 1);
                    tc::fence_after_sync();
                    if (elect()) {
                        const uint32_t c0 = rp.slot * kPair;
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            tc::mma_bf16(d, pair.at(c0 + (ks >> 2) * kBlk + (ks & 3) * 32),
                                         qd.at((2 * j + (ks >> 2)) * NC * 128 + (ks & 3) * 32), id, 1u);
                    }
                }
                if (elect())
                    tc::commit(&sm.s_full[rs.slot]);
            }
            if (elect())
                tc::commit(&sm.q_empty);
        }
    } else if (warp == 6) {
        // ---------------- O^T += C^T P^T, 128 latent numbers at a time
        constexpr uint32_t id = tc::idesc_bf16(128, NC, true, true);
        const Desc pair(smem_u32(sm.pair[0]), kBlk, 1024, tc::kSw128), pd = p_desc<NC>(smem_u32(sm.p));
        Ring<SM::kRing> rp;
        uint32_t nt = 0;
        for (; w.take > 0 && !wait.dead; w.next(a))
            for (int t = 0; t < w.take && !wait.dead; ++t, ++nt) {
                wait(&sm.p_full, nt & 1);
                tc::fence_after_sync();
#pragma unroll
                for (int j = 0; j < kPairs; ++j, rp.step())
                    if (elect()) {
                        const uint32_t c0 = rp.slot * kPair;
#pragma unroll
                        for (int ks = 0; ks < kTok / 16; ++ks)
                            tc::mma_bf16(tmem + (2 + j) * NC, pair.at(c0 + ks * 2048), pd.at(ks * kPStep<NC>), id,
                                         t > 0 || ks > 0 ? 1u : 0u);
                        tc::commit(&sm.empty_pair[rp.slot]);
                        if (j == kPairs - 1)
                            tc::commit(&sm.pv_done);
                    }
            }
    } else if (warp == 7) {
        // ---------------- Q of each piece: NC columns (token, head) x 576, K-major blocks of 64.
        // Columns behind the last hold other rows of q or nothing; they stay columns of their own.
        uint32_t nq = 0;
        for (; w.take > 0 && !wait.dead; w.next(a), ++nq) {
            if (nq > 0)
                wait(&sm.q_empty, (nq - 1) & 1);
            if (wait.dead)
                break;
            const int left = cols - ct * NC;
            if (maps.q_rows == NC) {  // one group: a sequence's columns are rows in order
                if (elect()) {
                    mbar_arrive_expect_tx(&sm.q_full, kDC / 64 * NC * 128);
                    tma_load_3d(sm.q[0], &maps.q, 0, w.n * cols + ct * NC, 0, &sm.q_full);
                }
            } else {
                const int n = (min(left, NC) + maps.q_rows - 1) / maps.q_rows;  // runs of q_rows heads
                if (elect())
                    mbar_arrive_expect_tx(&sm.q_full, (uint32_t)(n * maps.q_rows) * kDC * 2);
                __syncwarp();
                for (int i = lane; i < n * (kDC / 64); i += 32) {
                    const int c = i / (kDC / 64) * maps.q_rows, blk = i % (kDC / 64), cg = ct * NC + c;
                    const int r = (w.n * a.Sq + cg / Hg) * a.H + w.g * Hg + cg % Hg;
                    tma_load_3d(sm.q[blk] + c * 128, &maps.q, 0, r, blk, &sm.q_full);
                }
                __syncwarp();
            }
        }
    } else if (kE4M3 && warp >= 8) {
        // ---------------- codes to bfloat16 rows: 8 rows x 4 vectors of 16 codes a warp, so that
        // both the swizzled reads and the swizzled writes touch every bank once
        static_assert(kConv * 8 == kTok, "one pass of the warps covers a block's rows");
        const int chunk = lane >> 3;
        Ring<SM::kRing> rp;
        Ring<SM::kRopes> rr;
        Ring<SM::kStage> rst;
        for (; w.take > 0 && !wait.dead; w.next(a)) {
            const int len = a.kv_lens[w.n];
            for (int t = w.t; t < w.t + w.take && !wait.dead; ++t) {
                const int rows = len - t * kTok;
#pragma unroll
                for (int j = 0; j <= kPairs; ++j, rst.step()) {  // the rope block, then the pairs
                    unsigned char *dst = j == 0 ? sm.rope[rr.slot] : sm.pair[rp.slot];
                    if (j == 0 && rr.round > 0)
                        wait(&sm.empty_rope[rr.slot], (rr.round - 1) & 1);
                    if (j > 0 && rp.round > 0)
                        wait(&sm.empty_pair[rp.slot], (rp.round - 1) & 1);
                    wait(&sm.full_stage[rst.slot], rst.round & 1);
                    uint4 c[2];
#pragma unroll
                    for (int i = 0; i < (j == 0 ? 1 : 2); ++i) {
                        const int row = (warp - 8) * 8 + (lane & 7);
                        c[i] = *reinterpret_cast<const uint4 *>(sm.stage[rst.slot] + i * kBlk / 2 + row * 64 +
                                                                ((chunk ^ ((row >> 1) & 3)) << 4));
                        if (row >= rows)  // behind the sequence's end: anything may be there
                            c[i] = make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < (j == 0 ? 1 : 2); ++i) {
                        const int row = (warp - 8) * 8 + (lane & 7);
                        const uint2 x = decode4(c[i].x), y = decode4(c[i].y), z = decode4(c[i].z), u = decode4(c[i].w);
                        unsigned char *p = dst + i * kBlk + row * 128;
                        *reinterpret_cast<uint4 *>(p + (((2 * chunk) ^ (row & 7)) << 4)) = make_uint4(x.x, x.y, y.x, y.y);
                        *reinterpret_cast<uint4 *>(p + (((2 * chunk + 1) ^ (row & 7)) << 4)) = make_uint4(z.x, z.y, u.x, u.y);
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sm.empty_stage[rst.slot]);
                    fence_proxy_async_smem();
                    mbar_arrive(j == 0 ? &sm.full_rope[rr.slot] : &sm.full_pair[rp.slot]);
                    if (j == 0)
                        rr.step();
                    else
                        rp.step();
                }
            }
        }
    } else {
        // ---------------- softmax: rows 16 warp + lane / 4 (+ 8), columns 8 j + 2 (lane % 4) (+ 1)
        constexpr int J = NC / 8;
        const int r0 = warp * 16 + (lane >> 2);
        const uint32_t lane_base = tc::taddr(tmem, (uint32_t)warp * 32, 0);
        uint32_t nt = 0, np = 0;
        for (; w.take > 0; w.next(a)) {
            const int len = a.kv_lens[w.n];
            float m[2 * J], l[2 * J];
#pragma unroll
            for (int i = 0; i < 2 * J; ++i) {
                // columns behind the last: weights 0, and no say in when to rescale
                m[i] = ct * NC + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1) < cols ? -INFINITY : INFINITY;
                l[i] = 0.0f;
            }
            for (int t = w.t; t < w.t + w.take; ++t, ++nt, np += kPairs) {
                const uint32_t sb = nt & 1;
                float page_scale = 1.0f;  // of this warp's 16 rows, which lie in one page
                if constexpr (kE4M3) {
                    const int p0 = t * kTok + warp * 16;
                    if (p0 < len) {
                        const int page = a.block_table[(int64_t)w.n * a.max_pages + p0 / a.page_size];
                        if (page >= 0 && page < a.num_pages)
                            page_scale = a.cache_scale[(int64_t)page * a.G + w.g];
                    }
                }
                wait(&sm.s_full[sb], (nt / 2) & 1);
                tc::fence_after_sync();
                float s[J][4];
                load_s<NC>(lane_base + sb * NC, s);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.s_empty[sb]);
                bool grow = false;
                const bool edge = (t + 1) * kTok > len - a.Sq + 1;  // some column's last row is in this tile
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x = s[j][i] * (kE4M3 ? a.scale_log2 * page_scale : a.scale_log2);
                        if (edge) {
                            const int cg = ct * NC + 8 * j + 2 * (lane & 3) + (i & 1);
                            const int last = len - a.Sq + min(cg / Hg, a.Sq - 1);
                            if (t * kTok + r0 + (i >> 1) * 8 > last)
                                x = -INFINITY;
                        }
                        s[j][i] = x;
                        grow |= x > m[2 * j + (i & 1)] + kGrow;
                    }
                if (softmax_or(grow)) {
                    // new column maxima over the tile's 64 rows
                    float f[2 * J];
#pragma unroll
                    for (int i = 0; i < 2 * J; ++i) {
                        float x = fmaxf(s[i >> 1][i & 1], s[i >> 1][2 + (i & 1)]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1)
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        if (lane < 4)
                            sm.red[warp][8 * (i >> 1) + 2 * lane + (i & 1)] = x;
                    }
                    softmax_sync();
#pragma unroll
                    for (int i = 0; i < 2 * J; ++i) {
                        const int c = 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
                        const float mn = fmaxf(fmaxf(fmaxf(sm.red[0][c], sm.red[1][c]), fmaxf(sm.red[2][c], sm.red[3][c])),
                                               m[i]);
                        f[i] = m[i] == mn ? 1.0f : ex2(m[i] - mn);
                        m[i] = mn;
                        l[i] *= f[i];
                        if (warp == 0 && lane < 4)
                            sm.fac[c] = f[i];
                    }
                    softmax_sync();
                    if (t > w.t) {
                        wait(&sm.pv_done, (nt - 1) & 1);  // O^T of the tiles so far is complete
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int b = 0; b < kPairs * NC / 16; ++b) {
                            uint32_t y[16];
                            tc::ld_32x32b_x16(lane_base + 2 * NC + b * 16, y);
                            tc::wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                y[i] = __float_as_uint(__uint_as_float(y[i]) * sm.fac[b * 16 % NC + i]);
                            tc::st_32x32b_x16(lane_base + 2 * NC + b * 16, y);
                        }
                        tc::wait_st();
                    }
                }
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float mm = m[2 * j + (i & 1)];
                        s[j][i] = ex2(s[j][i] - (mm == -INFINITY ? 0.0f : mm));
                        l[2 * j + (i & 1)] += s[j][i];
                    }
                if (nt > 0)
                    wait(&sm.pv_done, (nt - 1) & 1);  // P^T has been read
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int c = 8 * j + 2 * (lane & 3);
                    *reinterpret_cast<uint32_t *>(sm.p + p_off<NC>(r0, c)) =
                        pack_bf16x2(s[j][0] * page_scale, s[j][1] * page_scale);
                    *reinterpret_cast<uint32_t *>(sm.p + p_off<NC>(r0 + 8, c)) =
                        pack_bf16x2(s[j][2] * page_scale, s[j][3] * page_scale);
                }
                // rows behind the sequence's end may hold anything (0 * NaN): zeros for O^T
                const int rows = len - t * kTok;
                if (!kE4M3 && rows < kTok) {
#pragma unroll
                    for (int j = 0; j < kPairs; ++j) {
                        const uint32_t sl = (np + j) % SM::kRing;
                        wait(&sm.full_pair[sl], ((np + j) / SM::kRing) & 1);
                        for (int v = tid; v < (kTok - rows) * 16; v += 128)
                            *reinterpret_cast<uint4 *>(sm.pair[sl] + (v & 8 ? kBlk : 0) + (rows + v / 16) * 128 +
                                                       (v & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc::fence_before_sync();
                mbar_arrive(&sm.p_full);
            }
            // ---- the piece's sums, and its result
#pragma unroll
            for (int i = 0; i < 2 * J; ++i) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
                if (lane < 4)
                    sm.red[warp][8 * (i >> 1) + 2 * lane + (i & 1)] = l[i];
            }
            softmax_sync();
            const bool whole = w.take == w.tiles;
            const int64_t unit = (int64_t)w.n * a.G + w.g, start = w.pos - w.t;  // place of the unit's first tile
            const int64_t slot = (int64_t)blockIdx.x * 2 + (start <= begin ? 0 : 1);
            if (warp == 0 && lane < 4) {
#pragma unroll
                for (int i = 0; i < 2 * J; ++i) {
                    const int c = 8 * (i >> 1) + 2 * lane + (i & 1), cg = ct * NC + c;
                    const float sum = sm.red[0][c] + sm.red[1][c] + sm.red[2][c] + sm.red[3][c];
                    const float lse2 = sum == 0.0f ? -INFINITY : m[i] + log2f(sum);
                    sm.fac[c] = sum == 0.0f ? 0.0f : 1.0f / sum;
                    if (!whole)
                        a.part_lse[slot * NC + c] = lse2;
                    else if (a.lse && cg < cols)
                        a.lse[((int64_t)w.n * a.Sq + cg / Hg) * a.H + w.g * Hg + cg % Hg] = lse2 * kLn2;
                }
            }
            if (tid == 0 && w.t == 0)
                a.meta[unit * a.CT + ct] =
                    make_int2((int)(start / per),
                              2 * (int)((start + w.tiles - 1) / per - start / per + 1) + (start % per != 0 ? 1 : 0));
            softmax_sync();
            wait(&sm.pv_done, (nt - 1) & 1);
            tc::fence_after_sync();
            const int dim = warp * 32 + lane;
#pragma unroll 1
            for (int b = 0; b < kPairs * NC / 16; ++b) {
                uint32_t y[16];
                tc::ld_32x32b_x16(lane_base + 2 * NC + b * 16, y);
                tc::wait_ld();
                const int d = b * 16 / NC * 128 + dim, c0 = b * 16 % NC;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int c = c0 + i, cg = ct * NC + c;
                    if (cg >= cols)
                        break;
                    const float x = sm.fac[c] == 0.0f ? 0.0f : __uint_as_float(y[i]) * sm.fac[c];
                    if (whole)
                        a.o[(((int64_t)w.n * a.Sq + cg / Hg) * a.H + w.g * Hg + cg % Hg) * kDL + d] = __float2bfloat16(x);
                    else
                        a.part_o[(slot * NC + c) * kDL + d] = x;
                }
            }
            softmax_sync();  // sm.fac and sm.red are free again
            tc::fence_before_sync();
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 4)
        tc::tmem_dealloc(tmem, kTmemCols);
}

// Joins the partial results of the units that several shares cover, and writes the empty result
// of the units that none does.  One warp per (unit, column); 16 of the 512 numbers a lane.
template <int NC>
__global__ void __launch_bounds__(256) mla_decode_join_kernel(DecArgs a)
{
    const int lane = threadIdx.x & 31, c = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int64_t uc = blockIdx.x;  // unit * CT + ct
    const int ct = (int)(uc % a.CT), Hg = a.H / a.G, cg = ct * NC + c;
    const int64_t unit = uc / a.CT;
    const int2 mt = a.meta[uc];
    const int count = mt.y >> 1;
    if (count == 1 || cg >= a.Sq * Hg)
        return;
    const int64_t r = (unit / a.G * a.Sq + cg / Hg) * a.H + unit % a.G * Hg + cg % Hg;
    float mx = -INFINITY;
    auto slot_of = [&](int i) { return ((int64_t)(mt.x + i) * a.CT + ct) * 2 + (i == 0 ? mt.y & 1 : 0); };
    for (int i = 0; i < count; ++i) {
        const float x = a.part_lse[slot_of(i) * NC + c];
        mx = x > mx || x != x ? x : mx;
    }
    float acc[16] = {}, sum = 0.0f;
    for (int i = 0; i < count; ++i) {
        const int64_t s = slot_of(i) * NC + c;
        const float x = a.part_lse[s], wgt = x == -INFINITY ? 0.0f : ex2(x - mx);
        sum += wgt;
        const float4 *p = reinterpret_cast<const float4 *>(a.part_o + s * kDL) + lane;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 v = p[k * 32];
            acc[4 * k] += wgt * v.x;
            acc[4 * k + 1] += wgt * v.y;
            acc[4 * k + 2] += wgt * v.z;
            acc[4 * k + 3] += wgt * v.w;
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint2 *dst = reinterpret_cast<uint2 *>(a.o + r * kDL) + lane;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        dst[k * 32] = make_uint2(pack_bf16x2(acc[4 * k] * inv, acc[4 * k + 1] * inv),
                                 pack_bf16x2(acc[4 * k + 2] * inv, acc[4 * k + 3] * inv));
    if (a.lse && lane == 0)
        a.lse[r] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

int columns(int Sq, int H, int G) { return Sq * (H / G) <= 32 ? 32 : 64; }

struct DecPlan {
    int nc, ct, shares;
    size_t part_lse, part_o, total;
};

DecPlan plan(int N, int Sq, int H, int G)
{
    DecPlan p;
    p.nc = columns(Sq, H, G);
    p.ct = (Sq * (H / G) + p.nc - 1) / p.nc;
    p.shares = num_sms() / p.ct > 0 ? num_sms() / p.ct : 1;
    const size_t slots = (size_t)p.shares * p.ct * 2;
    p.part_lse = ((size_t)N * G * p.ct * sizeof(int2) + 255) / 256 * 256;
    p.part_o = p.part_lse + (slots * p.nc * 4 + 255) / 256 * 256;
    p.total = p.part_o + slots * p.nc * kDL * 4;
    return p;
}

template <int NC, bool kE4M3>
cudaError_t launch_nc(DecMaps &maps, const DecArgs &a, cudaStream_t s)
{
    const size_t smem = sizeof(DecSmem<NC, kE4M3>) + 1024;
    static_assert(sizeof(DecSmem<NC, kE4M3>) + 1024 <= 232448, "shared memory of one CTA");
    auto kernel = mla_decode_kernel<NC, kE4M3>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    // q: runs of columns that are consecutive rows
    const int Hg = a.H / a.G;
    maps.q_rows = a.G == 1 ? NC : Hg % 8 == 0 ? 8 : 1;
    const int64_t extent[3] = {64, (int64_t)a.N * a.Sq * a.H, kDC / 64}, stride[2] = {kDC * 2, 128};
    const int box[3] = {64, maps.q_rows, maps.q_rows == NC ? kDC / 64 : 1};
    if ((e = make_map(&maps.q, a.q, 2, 3, extent, stride, box)) != cudaSuccess)
        return e;
    kernel<<<a.shares * a.CT, kThreads<kE4M3>, smem, s>>>(maps, a);
    mla_decode_join_kernel<NC><<<dim3(a.N * a.G * a.CT, NC / 8), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t mla_decode_workspace(int N, int Sq, int H, int G) { return plan(N, Sq, H, G).total; }

cudaError_t launch_mla_decode(int N, int Sq, int H, int G, float scale, const void *q, bool e4m3, const void *cache,
                              const float *cache_scale, int num_pages, int page_size, const int32_t *block_table,
                              int max_pages, const int32_t *kv_lens, void *o, float *lse, void *workspace,
                              cudaStream_t s)
{
    const DecPlan p = plan(N, Sq, H, G);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    DecArgs a{N, Sq, H, G, num_pages, page_size, max_pages, p.ct, p.shares, scale * kLog2e,
              static_cast<const __nv_bfloat16 *>(q), cache_scale, block_table, kv_lens,
              static_cast<__nv_bfloat16 *>(o), lse, reinterpret_cast<float *>(ws + p.part_o),
              reinterpret_cast<float *>(ws + p.part_lse), reinterpret_cast<int2 *>(ws), device_status_ptr()};
    if (!a.status)
        return cudaErrorInvalidDevice;
    DecMaps maps;
    maps.rows = page_size < kTok ? page_size : kTok;
    const int64_t es = e4m3 ? 1 : 2;
    const int64_t extent[4] = {64, G, (int64_t)num_pages * page_size, kDC / 64};
    const int64_t stride[3] = {kDC * es, G * kDC * es, 64 * es};
    const int pair_box[4] = {64, 1, maps.rows, 2}, rope_box[4] = {64, 1, maps.rows, 1};
    cudaError_t e = make_map(&maps.pair, cache, (int)es, 4, extent, stride, pair_box);
    if (e == cudaSuccess)
        e = make_map(&maps.rope, cache, (int)es, 4, extent, stride, rope_box);
    if (e != cudaSuccess)
        return e;
    if (e4m3)
        return p.nc == 32 ? launch_nc<32, true>(maps, a, s) : launch_nc<64, true>(maps, a, s);
    return p.nc == 32 ? launch_nc<32, false>(maps, a, s) : launch_nc<64, false>(maps, a, s);
}

}  // namespace kda

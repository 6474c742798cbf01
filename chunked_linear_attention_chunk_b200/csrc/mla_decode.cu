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

template <bool kE4M3>
constexpr int kThreads = kE4M3 ? 384 : 256;
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
    // pairs and rope blocks of bfloat16 rows held, and blocks of codes in flight
    static constexpr int kRing = kE4M3 ? (NC == 64 ? 7 : 8) : (NC == 64 ? 8 : 10);
    static constexpr int kRopes = kE4M3 ? (NC == 64 ? 1 : 2) : (NC == 64 ? 2 : 3);
    static constexpr int kStage = kE4M3 ? (NC == 64 ? 6 : 10) : 1;
    alignas(1024) unsigned char pair[kRing][kPair];
    alignas(1024) unsigned char rope[kRopes][kBlk];
    alignas(1024) unsigned char q[kDC / 64][NC * 128];
    alignas(1024) unsigned char p[kTok * NC * 2];
    alignas(1024) unsigned char stage[kStage][kE4M3 ? kBlk / 2 : 16];
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

// Four e4m3 codes as bfloat16 pairs (exact).  A code's exponent and mantissa, moved to the top of
// a bfloat16's mantissa and the foot of its exponent, are the value times 2^-120 (subnormals
// included); the product with 2^120 is exact.  NaN codes are the caller's business.
__device__ __forceinline__ void decode4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const __nv_bfloat162 up = __halves2bfloat162(__ushort_as_bfloat16(0x7b80), __ushort_as_bfloat16(0x7b80));
    const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
    const uint32_t x = ((a >> 4) & 0x07f007f0u) | (a & 0x80008000u), y = ((b >> 4) & 0x07f007f0u) | (b & 0x80008000u);
    const __nv_bfloat162 u = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&x), up);
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&y), up);
    lo = *reinterpret_cast<const uint32_t *>(&u);
    hi = *reinterpret_cast<const uint32_t *>(&v);
}

// Sixteen codes to bfloat16; a NaN code (0x7f, 0xff) becomes NaN.
__device__ __forceinline__ void decode16(uint4 c, uint4 &lo, uint4 &hi)
{
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t r[8], nan = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        decode4(w[i], r[2 * i], r[2 * i + 1]);
        nan |= (w[i] & 0x7f7f7f7fu) + 0x01010101u;
    }
    if (nan & 0x80808080u) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (((w[i >> 2] >> (i & 3) * 8) & 0x7f) == 0x7f)
                r[i >> 1] |= 0x7fffu << (i & 1) * 16;
    }
    lo = make_uint4(r[0], r[1], r[2], r[3]);
    hi = make_uint4(r[4], r[5], r[6], r[7]);
}

template <int NC, bool kE4M3>
__global__ void __launch_bounds__(kThreads<kE4M3>, 1)
    mla_decode_kernel(const __grid_constant__ CUtensorMap cache_map, DecArgs a, int box_rows)
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
            mbar_init(&sm.full_pair[i], kE4M3 ? 128 : 1);
            mbar_init(&sm.empty_pair[i], 1);
        }
        for (int i = 0; i < SM::kRopes; ++i) {
            mbar_init(&sm.full_rope[i], kE4M3 ? 128 : 1);
            mbar_init(&sm.empty_rope[i], 1);
        }
        for (int i = 0; i < SM::kStage; ++i) {
            mbar_init(&sm.full_stage[i], 1);
            mbar_init(&sm.empty_stage[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_empty[i], 4);
        }
        mbar_init(&sm.p_full, 128);
        mbar_init(&sm.pv_done, 1);
        mbar_init(&sm.q_full, 32);
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
        const int ppt = kTok / box_rows;  // boxes a block
        int batch_n = -1, batch_0 = 0, ids = 0;
        uint32_t np = 0, nr = 0;  // pairs and ropes so far
        for (; w.take > 0 && !wait.dead; w.next(a)) {
            const int len = a.kv_lens[w.n], pages = (len + a.page_size - 1) / a.page_size;
            const int32_t *row = a.block_table + (int64_t)w.n * a.max_pages;
            for (int t = w.t; t < w.t + w.take && !wait.dead; ++t) {
                // the token rows of the tile's boxes (at most four), from the table 32 entries at a time
                int at[4], live = 0;
                for (int b = 0; b < ppt; ++b) {
                    const int p0 = t * kTok + b * box_rows;
                    at[b] = -1;
                    if (p0 >= len)
                        continue;
                    const int e = p0 / a.page_size;
                    if (w.n != batch_n || e < batch_0 || e >= batch_0 + 32) {
                        batch_n = w.n;
                        batch_0 = e;
                        ids = e + lane < pages ? row[e + lane] : 0;
                    }
                    const int page = __shfl_sync(0xffffffffu, ids, e - batch_0);
                    if (page < 0 || page >= a.num_pages) {
                        if (lane == 0)
                            report_device_error(a.status, KDA_ERR_INVALID_ARG);
                        continue;
                    }
                    at[b] = page * a.page_size + p0 % a.page_size;
                    ++live;
                }
                if (lane == 0) {
                    // 64 numbers of each live box's rows
                    auto block = [&](unsigned char *dst, int x, uint64_t *bar) {
                        for (int b = 0; b < ppt; ++b)
                            if (at[b] >= 0)
                                tma_load_3d(dst + b * box_rows * (kE4M3 ? 64 : 128), &cache_map, x, w.g, at[b], bar);
                    };
                    const uint32_t bytes = (uint32_t)live * box_rows * (kE4M3 ? 64u : 128u);
                    if constexpr (kE4M3) {
                        for (int j = 0; j < kDC / 64; ++j, ++np) {
                            const uint32_t s = np % SM::kStage;
                            if (np >= SM::kStage)
                                wait(&sm.empty_stage[s], (np / SM::kStage - 1) & 1);
                            if (wait.dead)
                                break;
                            mbar_arrive_expect_tx(&sm.full_stage[s], bytes);
                            block(sm.stage[s], j == 0 ? kDL : (j - 1) * 64, &sm.full_stage[s]);
                        }
                    } else {
                        const uint32_t r = nr % SM::kRopes;
                        if (nr >= SM::kRopes)
                            wait(&sm.empty_rope[r], (nr / SM::kRopes - 1) & 1);
                        ++nr;
                        if (!wait.dead) {
                            mbar_arrive_expect_tx(&sm.full_rope[r], bytes);
                            block(sm.rope[r], kDL, &sm.full_rope[r]);
                        }
                        for (int j = 0; j < kPairs; ++j, ++np) {
                            const uint32_t s = np % SM::kRing;
                            if (np >= SM::kRing)
                                wait(&sm.empty_pair[s], (np / SM::kRing - 1) & 1);
                            if (wait.dead)
                                break;
                            mbar_arrive_expect_tx(&sm.full_pair[s], 2 * bytes);
                            block(sm.pair[s], j * 128, &sm.full_pair[s]);
                            block(sm.pair[s] + kBlk, j * 128 + 64, &sm.full_pair[s]);
                        }
                    }
                }
                wait.dead = __shfl_sync(0xffffffffu, (int)wait.dead, 0) != 0;
            }
        }
    } else if (warp == 5) {
        // ---------------- S^T = C Q^T, block by block as the tile arrives (rope first)
        if (lane == 0) {
            const uint32_t id = tc::idesc_bf16(64, NC, false, false);
            uint32_t np = 0, nr = 0, nt = 0, nq = 0;
            for (; w.take > 0 && !wait.dead; w.next(a), ++nq) {
                wait(&sm.q_full, nq & 1);
                for (int t = 0; t < w.take && !wait.dead; ++t, ++nt) {
                    const uint32_t sb = nt & 1;
                    if (nt >= 2)
                        wait(&sm.s_empty[sb], (nt / 2 - 1) & 1);
                    tc::fence_after_sync();
                    const uint32_t d = tmem + sb * NC;
                    auto block = [&](const unsigned char *c, const unsigned char *qb, bool first) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            tc::mma_bf16(d, tc::smem_desc(smem_u32(c) + ks * 32, 16, 1024, tc::kSw128),
                                         tc::smem_desc(smem_u32(qb) + ks * 32, 16, 1024, tc::kSw128), id,
                                         first && ks == 0 ? 0u : 1u);
                    };
                    const uint32_t rs = nr % SM::kRopes;
                    wait(&sm.full_rope[rs], (nr / SM::kRopes) & 1);
                    block(sm.rope[rs], sm.q[kDC / 64 - 1], true);
                    tc::commit(&sm.empty_rope[rs]);
                    ++nr;
                    for (int j = 0; j < kPairs; ++j, ++np) {
                        const uint32_t s = np % SM::kRing;
                        wait(&sm.full_pair[s], (np / SM::kRing) & 1);
                        block(sm.pair[s], sm.q[2 * j], false);
                        block(sm.pair[s] + kBlk, sm.q[2 * j + 1], false);
                    }
                    tc::commit(&sm.s_full[sb]);
                }
                tc::commit(&sm.q_empty);
            }
        }
        __syncwarp();
    } else if (warp == 6) {
        // ---------------- O^T += C^T P^T, 128 latent numbers at a time
        if (lane == 0) {
            const uint32_t id = tc::idesc_bf16(128, NC, true, true);
            uint32_t np = 0, nt = 0;
            for (; w.take > 0 && !wait.dead; w.next(a))
                for (int t = 0; t < w.take && !wait.dead; ++t, ++nt) {
                    wait(&sm.p_full, nt & 1);
                    tc::fence_after_sync();
                    for (int j = 0; j < kPairs; ++j, ++np) {
                        const uint32_t s = np % SM::kRing;
#pragma unroll
                        for (int ks = 0; ks < kTok / 16; ++ks)
                            tc::mma_bf16(tmem + (2 + j) * NC,
                                         tc::smem_desc(smem_u32(sm.pair[s]) + ks * 2048, kBlk, 1024, tc::kSw128),
                                         p_desc<NC>(smem_u32(sm.p), ks), id, t > 0 || ks > 0 ? 1u : 0u);
                        tc::commit(&sm.empty_pair[s]);
                    }
                    tc::commit(&sm.pv_done);
                }
        }
        __syncwarp();
    } else if (warp == 7) {
        // ---------------- Q of each piece: NC columns (token, head) x 576, K-major blocks of 64
        uint32_t nq = 0;
        for (; w.take > 0 && !wait.dead; w.next(a), ++nq) {
            if (nq > 0)
                wait(&sm.q_empty, (nq - 1) & 1);
            for (int c = 0; c < NC; ++c) {
                const int cg = ct * NC + c;
                const bool live = cg < cols;
                const int64_t r = live ? ((int64_t)w.n * a.Sq + cg / Hg) * a.H + w.g * Hg + cg % Hg : 0;
                const __nv_bfloat16 *src = a.q + r * kDC;
                for (int v = lane; v < kDC / 8; v += 32)
                    cp_async_16_zfill(sm.q[v >> 3] + c * 128 + (((v & 7) ^ (c & 7)) << 4), src + v * 8, live);
            }
            cp_async_commit();
            cp_async_wait<0>();
            fence_proxy_async_smem();
            mbar_arrive(&sm.q_full);
        }
    } else if (kE4M3 && warp >= 8) {
        // ---------------- codes to bfloat16 rows: 8 rows x 4 vectors of 16 codes a warp, so that
        // both the swizzled reads and the swizzled writes touch every bank once
        const int chunk = lane >> 3;
        uint32_t nb = 0, np = 0, nr = 0;
        for (; w.take > 0 && !wait.dead; w.next(a)) {
            const int len = a.kv_lens[w.n];
            for (int t = w.t; t < w.t + w.take && !wait.dead; ++t) {
                const int rows = len - t * kTok;
                for (int j = 0; j < kDC / 64; ++j, ++nb) {
                    const uint32_t st = nb % SM::kStage;
                    unsigned char *dst;
                    uint64_t *full;
                    if (j == 0) {
                        const uint32_t r = nr % SM::kRopes;
                        if (nr >= SM::kRopes)
                            wait(&sm.empty_rope[r], (nr / SM::kRopes - 1) & 1);
                        dst = sm.rope[r];
                        full = &sm.full_rope[r];
                        ++nr;
                    } else {
                        const uint32_t s = np % SM::kRing;
                        if (np >= SM::kRing)
                            wait(&sm.empty_pair[s], (np / SM::kRing - 1) & 1);
                        dst = sm.pair[s] + (j & 1 ? 0 : kBlk);
                        full = &sm.full_pair[s];
                        np += (j & 1) ^ 1;
                    }
                    wait(&sm.full_stage[st], (nb / SM::kStage) & 1);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int row = (i * 4 + warp - 8) * 8 + (lane & 7);
                        const uint4 c = *reinterpret_cast<const uint4 *>(sm.stage[st] + row * 64 +
                                                                         ((chunk ^ ((row >> 1) & 3)) << 4));
                        uint4 lo, hi;
                        decode16(c, lo, hi);
                        if (row >= rows)  // behind the sequence's end: anything may be there
                            lo = hi = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(dst + row * 128 + (((2 * chunk) ^ (row & 7)) << 4)) = lo;
                        *reinterpret_cast<uint4 *>(dst + row * 128 + (((2 * chunk + 1) ^ (row & 7)) << 4)) = hi;
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sm.empty_stage[st]);
                    fence_proxy_async_smem();
                    if (!(j & 1))  // the rope block, or a pair's second block
                        mbar_arrive(full);
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
            for (int i = 0; i < 2 * J; ++i)
                m[i] = -INFINITY, l[i] = 0.0f;
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
cudaError_t launch_nc(const CUtensorMap &map, const DecArgs &a, int box_rows, cudaStream_t s)
{
    const size_t smem = sizeof(DecSmem<NC, kE4M3>) + 1024;
    static_assert(sizeof(DecSmem<NC, kE4M3>) + 1024 <= 232448, "shared memory of one CTA");
    auto kernel = mla_decode_kernel<NC, kE4M3>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    kernel<<<a.shares * a.CT, kThreads<kE4M3>, smem, s>>>(map, a, box_rows);
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
    const int box_rows = page_size < kTok ? page_size : kTok;
    // [576 numbers][G groups][token rows of the pool], boxes of 64 numbers of one group's rows
    CUtensorMap map;
    const int64_t rows = (int64_t)num_pages * page_size;
    const int es = e4m3 ? 1 : 2;
    const cudaError_t e =
        make_map_3d(&map, cache, es, kDC, G, rows, (int64_t)kDC * es, (int64_t)G * kDC * es, 64, 1, box_rows);
    if (e != cudaSuccess)
        return e;
    if (e4m3)
        return p.nc == 32 ? launch_nc<32, true>(map, a, box_rows, s) : launch_nc<64, true>(map, a, box_rows, s);
    return p.nc == 32 ? launch_nc<32, false>(map, a, box_rows, s) : launch_nc<64, false>(map, a, box_rows, s);
}

}  // namespace kda

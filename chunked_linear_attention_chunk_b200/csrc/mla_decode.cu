// mla_decode.cu -- absorbed latent attention of a few new tokens over a paged cache.
//
//   s_j = scale q . c_j,  o = sum_j softmax_j(s) c_j[0:512]
// Every query head of a latent group reads the same cached rows (1152 B each in bfloat16, 576 B in
// e4m3), so a row is brought in once for up to 64 (token, head) columns and the kernel is bound by
// the cache's bytes: at 32 columns it has 2 (576 + 512) 32 / 1152 = 60 flops a byte, a quarter of
// what the tensor cores could take.
//
// Roles are swapped so that the tensor cores' M is the cached rows, not the few heads, and nothing
// is padded:
//   S^T [64 rows x NC columns] = C Q^T          (M = 64, K = 576; C as the copy laid it down)
//   O^T [512 x NC] += C[:, 0:512]^T P^T         (M = 128 four times, K = 64; C read MN-major)
// The same shared-memory tile is the A operand of both; only P^T (64 x NC) is written by threads.
//
// e4m3 rows: both products are taken on the codes as they lie in the cache (kind::f8f6f4), and
// what is exact in bfloat16 becomes several 8-bit terms of the other operand.
// Q is split into two e4m3 terms at a power-of-two scale of its own for each row, q = t (q1 + q2 /
// 32) with the row's largest in [128 t, 256 t): q1 keeps four bits and q2 the next four, which is all
// a bfloat16 has, so the terms are further columns of the product and S^T stays as exact as float32
// sums are.  32 is the most that q1's rounding (up to 8 t) allows: 8 * 32 < 448.  e4m3's smallest
// step, 2^-9, is then 2^-14 t of q, so a number keeps its eight bits from 2^-7 t up (2^-14 of the
// row's largest at least) and is off by 2^-15 t below that (2^-22 of the largest at most).
// A weight times its page's scale is brought into range by a running maximum of its own for each
// column, over score + log2(scale) (2^11 to 2^15 at the maximum), and split into three e5m2 terms of
// three bits each at one common scale: nine bits (a bfloat16 weight has eight) down to 2^-19 of the
// maximum, and 2^-28 of it at worst.  Up to 32 columns the terms are three times as many columns of
// one product, added up at the end; at 64, where tensor memory has no room for that, three products into one sum.
// Turning the codes into f16 rows in shared memory instead costs its bandwidth: 64 KB written and
// read again a tile, 190 us where this took 165 (256 sequences of 3000 to 5000 rows, 32 heads).
//
// One persistent CTA per SM takes an equal share of all 64-row tiles of all (sequence, group)
// units in order, so a batch of any lengths is balanced without the host knowing them.  A unit
// inside one CTA's share is finished there; the others leave normalised partial results with
// their log-sum-exp in the workspace, which a second launch joins in order (equal calls give
// equal bits; the shares depend on the lengths and the SM count alone).
//
// Measured (one launch and its join, inputs larger than L2): 256 sequences of 3000 to 5000 rows, 32
// heads: bfloat16 217-220 us, 5.5 TB/s; e4m3 147-157 us, 4.0 TB/s.  A tile of 64 e4m3 rows takes
// 1450 cycles: 666 of S^T and 464 of O^T products (both bound by shared memory), the softmax's chain
// of waits and stores next to them; in a loop the 1000 W limit holds the clock near 1.45 GHz, and
// alone the launch takes 122 us.  23 ragged sequences up to 40000 rows, 2 tokens each: 131-133 us.
// Also measured, and slower: prefetching tiles into L2 ahead of the copies (249 and 203 us for the
// two batches), fetching the next S^T while the weights are stored (220 and 155, ragged 135), half
// tiles of codes as places, nine for the eight there are (154.7 for 152.4).
//
// Warps: 0-3 and 8-11 softmax, half the columns each (S^T in the 16-lane M = 64 layout, running
// maximum per column, O^T in tensor memory rescaled only when a column's maximum grows by more than
// 2^8, which float32 sums and a bfloat16 weight hold exactly as well); 4 and 7 copies, every other
// tile each (TMA: half a tile of bfloat16 rows or a whole one of codes at a time); 5 loads Q and
// issues S^T; 6 issues O^T and frees the rows.
#include <cudaTypedefs.h>
#include <cuda_fp8.h>

#include "mla_common.cuh"
#include "mla_tc.cuh"

namespace kda {

namespace {

using namespace mla;

constexpr int kThreads = 384;
constexpr int kTok = 64;                    // cached rows a tile
constexpr uint32_t kBlk = kTok * 128;       // 64 rows x 128 bytes, 128-byte swizzle
constexpr int kPairs = kDL / 128;           // 128 latent numbers: the M of one O^T product
constexpr float kGrow = 8.0f;               // log2 by which a maximum may grow without rescaling
// e4m3: log2 of a weight (times its page's scale) at its maximum, and by how much that may grow: up
// to 2^15 in all, below e5m2's largest.  A weight's last place is 2^-27 of the maximum, so a
// million of them in one CTA's share are off by 2^-8 of it together; 13 and 2 rescale O^T so often
// that the 8-bit batch above takes 159 us for 151, and 7 and 8 lose long tails of small weights.
constexpr float kLift = 11.0f, kGrowO = 4.0f;

struct DecArgs {
    int N, Sq, H, G, num_pages, page_size, max_pages, CT, shares;
    float scale_log2;
    const __nv_bfloat16 *q;
    const float *cache_scale;
    const int32_t *block_table, *kv_lens;
    __nv_bfloat16 *o;
    float *lse;
    float *part_o, *part_lse;  // [CTA][2][4][NC / 4][128][4] (pair, column / 4, number, column % 4), [CTA][2][NC]
    int4 *meta;                // [share][CT]: the unit that starts in the share and goes on behind it, as
                               // sequence, group, shares covered (0: there is none), which of the two slots
    // e4m3: q's terms [2][rows of q][576] and row scales
    unsigned char *q_terms;
    float *q_scale;
    unsigned int *status;
};

// bfloat16: the cache as [block of 64 numbers][pool row][group][64], so that one copy brings half a
// tile (or the rope block) as the products read it; e4m3: [block of 128 codes][pool row][group]
// [128], and the rope part.  q as [block][row][64], or its terms as [block][term][row][128] and
// [term][row][64].
struct DecMaps {
    CUtensorMap latent, rope, q, q_rope;
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
    int64_t left;              // tiles left behind the current piece
    bool inside;               // the piece's unit starts inside the share
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
        t = 0;
        inside = true;
        if (++g == a.G) {
            g = 0;
            ++n;
        }
        settle(a);
    }
    __device__ __forceinline__ bool whole() const { return take == tiles; }
};

template <int NC, bool kE4M3>
struct DecSmem {
    // bfloat16: half tiles and rope blocks in flight; e4m3: tiles of codes
    static constexpr int kRing = kE4M3 ? 1 : (NC == 64 ? 4 : 5);
    static constexpr int kRopes = kE4M3 || NC == 64 ? 1 : 2;
    static constexpr int kStage = kE4M3 ? (NC == 64 ? 3 : NC == 32 ? 4 : 5) : 1;
    static constexpr uint32_t kSlot = kE4M3 ? 16 : 4 * kBlk;
    static_assert(kRing <= 4 * kRopes, "a warp that waits for a rope place knows the round before the last consumed");
    static constexpr uint32_t kCodes = 4 * kBlk + kBlk / 2;  // a tile of codes: 4 x 128, then 64
    static constexpr int kSW = kE4M3 ? 2 * NC : NC;          // columns of S^T
    static constexpr int kPB = NC == 64 && !kE4M3 ? 1 : 2;   // buffers of P^T (one where a second is 1 KB too much)
    static constexpr uint32_t kP = kTok * kPRow<NC, kE4M3> * (kE4M3 && NC > 16 ? 3 : 1);  // bytes of one
    // parts of O^T: a weight's three terms side by side where tensor memory has the room, one sum of
    // their three products where it has not
    static constexpr int kParts = kE4M3 && NC <= 32 ? 3 : 1;
    alignas(1024) unsigned char ring[kRing][kSlot];
    alignas(1024) unsigned char rope[kRopes][kE4M3 ? 16 : kBlk];
    // bfloat16: [9 blocks][NC rows][128 B]; e4m3: [4 blocks][2 NC rows][128 B], [2 NC rows][64 B]
    alignas(1024) unsigned char q[kE4M3 ? 2 * NC * kDC : NC * kDC * 2];
    alignas(1024) unsigned char p[kPB][kP];
    alignas(1024) unsigned char stage[kStage][kE4M3 ? kCodes : 16];
    alignas(16) float red[4][NC];  // per warp: column maxima, then column sums
    float page_lg[2][4];  // e4m3: log2 of the warps' page scales
    float fac[NC], top[NC], ahead[NC];  // per column: rescaling factor, then 1 / sum; the maximum; e4m3: see there
    float scale[kStage][4];  // of a tile's boxes: their pages' scales
    int row[NC];            // output row of a column, less the sequence's and group's first
    uint64_t full[kRing], empty[kRing], full_rope[kRopes], empty_rope[kRopes];
    uint64_t full_stage[kStage], empty_stage[kStage], full_scale[kStage];
    uint64_t s_full[2], s_empty[2], p_full[kPB], pv_done[kPB], q_full, q_empty;
    uint32_t tmem_slot;
    int64_t find[40];
    int64_t share[3];  // first tile and tiles of the CTA's share, tiles of a full one
    int first[4];      // n, g, t of its first tile; whether that is the unit's first
};

// Two numbers as e4m3 codes of their first (lo 16 bits) and second term.
__device__ __forceinline__ uint32_t terms2(float2 x)
{
    const __nv_fp8x2_storage_t a = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(a, __NV_E4M3)));
    const __nv_fp8x2_storage_t b =
        __nv_cvt_float2_to_fp8x2(make_float2((x.x - f.x) * kTerm2, (x.y - f.y) * kTerm2), __NV_SATFINITE, __NV_E4M3);
    return (uint32_t)a | ((uint32_t)b << 16);
}

// q's two terms, a warp a row: t = 2^e with max|q| < 256 t, and t and 1 / t normal numbers; a row
// with an infinity or a NaN gets a NaN for its scale.
__global__ void __launch_bounds__(256) mla_split_q_kernel(DecArgs a, int64_t rows)
{
    // the launches before this one are over; the next one may start (it reads what they wrote, and
    // waits before it reads the terms)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (r >= rows)
        return;
    uint4 x[3];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int v = lane + 32 * i;
        x[i] = v < kDC / 8 ? reinterpret_cast<const uint4 *>(a.q + r * kDC)[v] : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mx = max(mx, max(u[k] << 16 & 0x7fffffffu, u[k] & 0x7fff0000u));
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    const int e = max((int)(mx >> 23) - 127 - 7, -100);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    if (lane == 0)
        a.q_scale[r] = __uint_as_float(mx >= 0x7f800000u ? 0x7fc00000u : (uint32_t)(127 + e) << 23);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int v = lane + 32 * i;
        if (v >= kDC / 8)
            break;
        const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t t[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = unpack_bf16x2(u[k]);
            t[k] = terms2(make_float2(f.x * inv, f.y * inv));
        }
        *reinterpret_cast<uint2 *>(a.q_terms + r * kDC + v * 8) =
            make_uint2(__byte_perm(t[0], t[1], 0x5410), __byte_perm(t[2], t[3], 0x5410));
        *reinterpret_cast<uint2 *>(a.q_terms + (rows + r) * kDC + v * 8) =
            make_uint2(__byte_perm(t[0], t[1], 0x7632), __byte_perm(t[2], t[3], 0x7632));
    }
}

template <int NC, bool kE4M3>
__global__ void __launch_bounds__(kThreads, 1)
    mla_decode_kernel(const __grid_constant__ DecMaps maps, DecArgs a)
{
    extern __shared__ unsigned char raw[];
    using SM = DecSmem<NC, kE4M3>;
    SM &sm = *reinterpret_cast<SM *>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int share = blockIdx.x / a.CT, ct = blockIdx.x % a.CT, Hg = a.H / a.G, cols = a.Sq * Hg;
    constexpr uint32_t kTmemCols = 2 * SM::kSW + kPairs * SM::kParts * NC <= 256 ? 256 : 512;
    constexpr uint32_t kColO = 2 * SM::kSW;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be set up meanwhile
    if (tid == 0) {
        prefetch_map(&maps.latent);
        prefetch_map(&maps.rope);
        prefetch_map(&maps.q);
        if (kE4M3)
            prefetch_map(&maps.q_rope);
        for (int i = 0; i < SM::kRing; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < SM::kRopes; ++i) {
            mbar_init(&sm.full_rope[i], 1);
            mbar_init(&sm.empty_rope[i], 1);
        }
        for (int i = 0; i < SM::kStage; ++i) {
            mbar_init(&sm.full_stage[i], 1);
            mbar_init(&sm.empty_stage[i], 1);
            mbar_init(&sm.full_scale[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_empty[i], 8);
        }
        for (int i = 0; i < SM::kPB; ++i) {
            mbar_init(&sm.p_full[i], 8);
            mbar_init(&sm.pv_done[i], 1);
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        fence_mbar_init_cluster();
    }
    if (warp == 4)
        tc::tmem_alloc(&sm.tmem_slot, kTmemCols);
    if (tid >= 160 && tid < 160 + NC) {
        const int c = tid - 160, cg = ct * NC + c;
        sm.row[c] = cg / Hg * a.H + cg % Hg;
    }
    if (!kE4M3)  // the launches before this one are over (e4m3: they were before the terms' launch went on)
        asm volatile("griddepcontrol.wait;" ::: "memory");
    // this CTA's share: all tiles, then the unit that its first one falls in
    {
        int64_t mine = 0;
        bool bad = false, none = false;
        for (int n = tid; n < a.N; n += kThreads) {
            const int t = tiles_of(a, n);
            mine += t;
            bad |= t == 0 && a.kv_lens[n] != 0;
            none |= t == 0 && n % a.shares == share;
        }
        if (bad)
            report_device_error(a.status, KDA_ERR_INVALID_ARG);
        const int64_t total = cta_sum<kThreads>(mine, sm.find) * a.G;
        const int64_t per = total < 0x7fffffff - a.shares ? (uint32_t)(total + a.shares - 1) / (uint32_t)a.shares
                                                          : (total + a.shares - 1) / a.shares;
        const int64_t begin = min(total, share * per), end = min(total, begin + per);
        const Item it = find_item<kThreads>(a.N, begin, [&](int n, bool &) { return tiles_of(a, n) * a.G; }, sm.find);
        if (tid == 0) {
            const int tiles = begin < end ? tiles_of(a, it.seq) : 1;
            sm.share[0] = begin;
            sm.share[1] = end - begin;
            sm.share[2] = per;
            sm.first[0] = it.seq;
            sm.first[1] = it.k / tiles;
            sm.first[2] = it.k % tiles;
        }
        // sequences that are nobody's piece are dealt out for their (empty) results
        tc::fence_before_sync();
        if (__syncthreads_or(none))
            for (int n = share; n < a.N; n += a.shares)
                if (tiles_of(a, n) == 0)
                    for (int i = warp; i < a.G * min(NC, cols - ct * NC); i += kThreads / 32) {
                        const int64_t row = (int64_t)n * a.Sq * a.H + i % a.G * Hg + sm.row[i / a.G];
                        for (int v = lane; v < kDL / 8; v += 32)
                            reinterpret_cast<uint4 *>(a.o + row * kDL)[v] = make_uint4(0, 0, 0, 0);
                        if (lane == 0 && a.lse)
                            a.lse[row] = -INFINITY;
                    }
        tc::fence_after_sync();
    }
    const uint32_t tmem = sm.tmem_slot;
    Pieces w;
    w.n = sm.first[0], w.g = sm.first[1], w.t = sm.first[2];
    w.left = sm.share[1];
    w.take = 0;
    w.inside = false;
    if (w.left > 0)
        w.settle(a);
    if (w.take > 0 && (!rows_in(w.t, w.take, w.tiles, 0, w.tiles) || !rows_in(w.n, 1, a.N, 0, a.N) ||
                       !rows_in(w.g, 1, a.G, 0, a.G))) {
        report_device_error(a.status, KDA_ERR_DEVICE_BOUNDS);
        w.take = 0;
    }
    Waits wait{false};

    if (warp == 4 || warp == 7) {
        // ---------------- copies: every other tile each (a tile's lookups, waits and copies take a warp
        // longer than the tensor cores need for it).  Waiting for a place that the other warp filled
        // last is sound: a warp's previous tile had all but the last round of that place consumed.
        const uint32_t me = warp == 4 ? 0 : 1;
        uint32_t nt = 0;
        const int ppt = kTok / maps.rows;  // copies a block
        int batch_n = -1, batch_0 = 0, ids = 0;
        Ring<SM::kRing> rp;
        Ring<SM::kRopes> rr;
        Ring<SM::kStage> rst;
        for (; w.take > 0 && !wait.dead; w.next(a)) {
            const int len = a.kv_lens[w.n], pages = (len + a.page_size - 1) / a.page_size;
            const int32_t *row = a.block_table + (int64_t)w.n * a.max_pages;
            for (int t = w.t; t < w.t + w.take && !wait.dead; ++t, ++nt, rp.step(), rp.step(), rr.step(), rst.step()) {
                if ((nt & 1) != me)
                    continue;
                int e = t * kTok / a.page_size, off = t * kTok % a.page_size;  // page entry, slot in it
                // the pool rows of the tile's copies, from the table 32 entries at a time
                int at[4], live = 0, my_page = -1;  // my_page: of box `lane`
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
                            if (lane == b)
                                my_page = page;
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
                const uint32_t bytes = (uint32_t)(live * maps.rows) * 128u;
                // four blocks from `block` on; pages of 64 rows and more take one copy
                auto half = [&](unsigned char *dst, int block, uint64_t *bar) {
                    if (ppt == 1) {
                        if (at[0] >= 0)
                            tma_load_4d(dst, &maps.latent, 0, w.g, at[0], block, bar);
                        return;
                    }
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (at[b] >= 0)
                                tma_load_4d(dst + i * kBlk + b * maps.rows * 128, &maps.latent, 0, w.g, at[b], block + i,
                                            bar);
                };
                auto rope = [&](unsigned char *dst, int row_bytes, uint64_t *bar) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        if (at[b] >= 0)
                            tma_load_3d(dst + b * maps.rows * row_bytes, &maps.rope, 0, w.g, at[b], bar);
                };
                if constexpr (kE4M3) {
                    if (rst.round > 0)
                        wait(&sm.empty_stage[rst.slot], (rst.round - 1) & 1);
                    if (elect() && !wait.dead) {
                        mbar_arrive_expect_tx(&sm.full_stage[rst.slot], 4 * bytes + bytes / 2);
                        rope(sm.stage[rst.slot] + 4 * kBlk, 64, &sm.full_stage[rst.slot]);
                        half(sm.stage[rst.slot], 0, &sm.full_stage[rst.slot]);
                    }
                    // the page scales come on their own (a place is free once its tile's P^T has been used)
                    if (!wait.dead && lane < 4) {
                        float *dst = &sm.scale[rst.slot][lane];
                        if (my_page >= 0) {
                            cp_async_4(dst, a.cache_scale + (int64_t)my_page * a.G + w.g);
                            cp_async_arrive(&sm.full_scale[rst.slot]);
                        } else {  // no page there: a plain store, which a plain arrival follows
                            *dst = 1.0f;
                            mbar_arrive(&sm.full_scale[rst.slot]);
                        }
                    }
                    __syncwarp();
                } else {
                    Ring<SM::kRing> rh = rp;
                    if (rh.round > 0)  // (first: then the rope place is a round behind at most)
                        wait(&sm.empty[rh.slot], (rh.round - 1) & 1);
                    if (rr.round > 0)
                        wait(&sm.empty_rope[rr.slot], (rr.round - 1) & 1);
                    if (elect() && !wait.dead) {
                        mbar_arrive_expect_tx(&sm.full_rope[rr.slot], bytes);
                        rope(sm.rope[rr.slot], 128, &sm.full_rope[rr.slot]);
                        mbar_arrive_expect_tx(&sm.full[rh.slot], 4 * bytes);
                        half(sm.ring[rh.slot], 0, &sm.full[rh.slot]);
                    }
                    rh.step();
                    if (rh.round > 0)
                        wait(&sm.empty[rh.slot], (rh.round - 1) & 1);
                    if (elect() && !wait.dead) {
                        mbar_arrive_expect_tx(&sm.full[rh.slot], 4 * bytes);
                        half(sm.ring[rh.slot], 4, &sm.full[rh.slot]);
                    }
                }
                wait.dead = __any_sync(0xffffffffu, wait.dead);
            }
        }
    } else if (warp == 5) {
        // ---------------- S^T = C Q^T.  Q of each piece: NC columns (token, head) x 576, K-major; e4m3: its
        // terms, the second behind the first.  Columns behind the last hold other rows of q or
        // nothing; they stay columns of their own.
        if constexpr (kE4M3)
            asm volatile("griddepcontrol.wait;" ::: "memory");  // the launch that writes the terms
        constexpr uint32_t kBytes = kE4M3 ? 2 * kDC : kDC * 2;  // of a column
        Ring<SM::kRing> rp;
        Ring<SM::kRopes> rr;
        Ring<SM::kStage> rst;
        Ring<2> rs;
        uint32_t nq = 0;
        for (; w.take > 0; w.next(a), ++nq) {
            if (nq > 0)
                wait(&sm.q_empty, (nq - 1) & 1);
            if (maps.q_rows == NC) {  // one group: a sequence's columns are rows in order
                if (elect() && !wait.dead) {
                    const int r = w.n * cols + ct * NC;
                    mbar_arrive_expect_tx(&sm.q_full, NC * kBytes);
                    if constexpr (kE4M3) {
                        tma_load_4d(sm.q, &maps.q, 0, r, 0, 0, &sm.q_full);
                        tma_load_3d(sm.q + 4 * SM::kSW * 128, &maps.q_rope, 0, r, 0, &sm.q_full);
                    } else {
                        tma_load_3d(sm.q, &maps.q, 0, r, 0, &sm.q_full);
                    }
                }
            } else {
                const int n = (min(cols - ct * NC, NC) + maps.q_rows - 1) / maps.q_rows;  // runs of q_rows heads
                const int row0 = w.n * a.Sq * a.H + w.g * Hg;
                // a copy's destination is a multiple of 128 bytes: single rope rows of codes (64 bytes)
                // are moved by the lanes instead
                const bool by_hand = kE4M3 && maps.q_rows == 1;
                if (by_hand) {
                    for (int i = lane; i < 2 * n; i += 32) {
                        const int c = i >> 1, k = i & 1, r = k * NC + c;
                        const uint4 *src = reinterpret_cast<const uint4 *>(
                            a.q_terms + ((int64_t)k * a.N * a.Sq * a.H + row0 + sm.row[c]) * kDC + kDL);
                        unsigned char *dst = sm.q + 4 * SM::kSW * 128 + r * 64;
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            *reinterpret_cast<uint4 *>(dst + ((v ^ ((r >> 1) & 3)) << 4)) = src[v];
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                const int copies = kE4M3 ? (by_hand ? 8 : 10) : kDC / 64;
                if (elect() && !wait.dead)
                    mbar_arrive_expect_tx(&sm.q_full,
                                          (uint32_t)(n * maps.q_rows) * (by_hand ? kBytes - 2 * kDR : kBytes));
                __syncwarp();
                for (int i = lane; i < n * copies && !wait.dead; i += 32) {
                    const int c = i / copies * maps.q_rows, blk = i % copies;
                    const int r = row0 + sm.row[c];
                    if (!kE4M3)
                        tma_load_3d(sm.q + blk * NC * 128 + c * 128, &maps.q, 0, r, blk, &sm.q_full);
                    else if (blk < 8)
                        tma_load_4d(sm.q + (blk >> 1) * SM::kSW * 128 + ((blk & 1) * NC + c) * 128, &maps.q, 0, r, blk & 1,
                                    blk >> 1, &sm.q_full);
                    else
                        tma_load_3d(sm.q + 4 * SM::kSW * 128 + ((blk & 1) * NC + c) * 64, &maps.q_rope, 0, r, blk & 1,
                                    &sm.q_full);
                }
                __syncwarp();
            }
            wait(&sm.q_full, nq & 1);
            for (int t = 0; t < w.take; ++t, rs.step()) {
                if (rs.round > 0)
                    wait(&sm.s_empty[rs.slot], (rs.round - 1) & 1);
                const uint32_t d = tmem + rs.slot * SM::kSW;
                if constexpr (kE4M3) {
                    constexpr uint32_t id = tc::idesc_e4m3(64, SM::kSW);
                    const Desc cd(smem_u32(sm.stage[0]), 16, 1024, tc::kSw128), qd(smem_u32(sm.q), 16, 1024, tc::kSw128),
                        cr(smem_u32(sm.stage[0]), 16, 512, tc::kSw64), qr(smem_u32(sm.q), 16, 512, tc::kSw64);
                    wait(&sm.full_stage[rst.slot], rst.round & 1);
                    tc::fence_after_sync();
                    if (elect()) {
                        const uint32_t c0 = rst.slot * SM::kCodes;
#pragma unroll
                        for (int ks = 0; ks < 16; ++ks)
                            tc::mma_f8(d, cd.at(c0 + (ks >> 2) * kBlk + (ks & 3) * 32),
                                       qd.at((ks >> 2) * SM::kSW * 128 + (ks & 3) * 32), id, ks > 0 ? 1u : 0u);
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks)
                            tc::mma_f8(d, cr.at(c0 + 4 * kBlk + ks * 32), qr.at(4 * SM::kSW * 128 + ks * 32), id, 1u);
                        tc::commit(&sm.s_full[rs.slot]);
                    }
                    rst.step();
                } else {
                    constexpr uint32_t id = tc::idesc_bf16(64, NC, false, false);
                    const Desc rope(smem_u32(sm.rope[0]), 16, 1024, tc::kSw128),
                        cd(smem_u32(sm.ring[0]), 16, 1024, tc::kSw128), qd(smem_u32(sm.q), 16, 1024, tc::kSw128);
                    wait(&sm.full_rope[rr.slot], rr.round & 1);
                    tc::fence_after_sync();
                    if (elect()) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            tc::mma_bf16(d, rope.at(rr.slot * kBlk + ks * 32),
                                         qd.at((kDC / 64 - 1) * NC * 128 + ks * 32), id, ks > 0 ? 1u : 0u);
                        tc::commit(&sm.empty_rope[rr.slot]);
                    }
                    rr.step();
#pragma unroll
                    for (int j = 0; j < 2; ++j, rp.step()) {
                        wait(&sm.full[rp.slot], rp.round & 1);
                        tc::fence_after_sync();
                        if (elect()) {
                            const uint32_t c0 = rp.slot * SM::kSlot;
#pragma unroll
                            for (int ks = 0; ks < 16; ++ks)
                                tc::mma_bf16(d, cd.at(c0 + (ks >> 2) * kBlk + (ks & 3) * 32),
                                             qd.at((4 * j + (ks >> 2)) * NC * 128 + (ks & 3) * 32), id, 1u);
                            if (j == 1)
                                tc::commit(&sm.s_full[rs.slot]);
                        }
                    }
                }
            }
            if (elect())
                tc::commit(&sm.q_empty);
        }
    } else if (warp == 6) {
        // ---------------- O^T += C^T P^T, 128 latent numbers at a time
        const Desc pd = p_desc<NC, kE4M3>(smem_u32(sm.p[0]));
        Ring<SM::kRing> rp;
        Ring<SM::kStage> rst;
        Ring<SM::kPB> rb;
        for (; w.take > 0; w.next(a))
            for (int t = 0; t < w.take; ++t, rb.step()) {
                wait(&sm.p_full[rb.slot], rb.round & 1);
                tc::fence_after_sync();
                const uint32_t p0 = rb.slot * SM::kP;
                if constexpr (kE4M3) {
                    constexpr uint32_t id = tc::idesc_e4m3_e5m2_mn(128, SM::kParts * NC);
                    constexpr int kTurns = 3 / SM::kParts;  // products of a term each, or one of all
                    const Desc cd(smem_u32(sm.stage[0]), kBlk, 1024, tc::kSw128);
                    if (elect()) {
                        const uint32_t c0 = rst.slot * SM::kCodes;
#pragma unroll
                        for (int j = 0; j < kPairs; ++j)
#pragma unroll
                            for (int k = 0; k < 2 * kTurns; ++k)
                                tc::mma_f8(tmem + kColO + j * SM::kParts * NC, cd.at(c0 + j * kBlk + (k & 1) * 4096),
                                           pd.at(p0 + (k >> 1) * kTok * NC + (k & 1) * 32 * kPRow<NC, true>), id,
                                           t > 0 || k > 0 ? 1u : 0u);
                        tc::commit(&sm.empty_stage[rst.slot]);
                        tc::commit(&sm.pv_done[rb.slot]);
                    }
                    rst.step();
                } else {
                    constexpr uint32_t id = tc::idesc_bf16(128, NC, true, true);
                    const Desc cd(smem_u32(sm.ring[0]), kBlk, 1024, tc::kSw128);
#pragma unroll
                    for (int j = 0; j < 2; ++j, rp.step())
                        if (elect()) {
                            const uint32_t c0 = rp.slot * SM::kSlot;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                tc::mma_bf16(tmem + kColO + (2 * j + (k >> 2)) * NC,
                                             cd.at(c0 + (k >> 2) * 2 * kBlk + (k & 3) * 2048),
                                             pd.at(p0 + (k & 3) * 32 * NC), id, t > 0 || (k & 3) > 0 ? 1u : 0u);
                            tc::commit(&sm.empty[rp.slot]);
                            if (j == 1)
                                tc::commit(&sm.pv_done[rb.slot]);
                        }
                }
            }
    } else {
        // ---------------- softmax: a group of four warps half the columns each; a thread rows
        // 16 (warp % 4) + lane / 4 (+ 8), the group's columns 8 j + 2 (lane % 4) (+ 1)
        if (kE4M3)  // q's row scales
            asm volatile("griddepcontrol.wait;" ::: "memory");
        constexpr int kCols = NC / 2, J = kCols / 8, kCh = kCols < 16 ? kCols : 16;  // kCh: columns of O^T at once
        const int group = warp >> 3, quarter = warp & 3, gtid = quarter * 32 + lane, r0 = quarter * 16 + (lane >> 2);
        const uint32_t lane_base = tc::taddr(tmem, (uint32_t)quarter * 32, 0) + group * kCols;
        auto col = [&](int i) { return group * kCols + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1); };
        uint32_t nt = 0;
        bool go_on = false;  // a unit goes on behind the share that it starts in
        Ring<SM::kRing> rp;
        Ring<SM::kStage> rst;
        // P^T and O^T of tile n: which buffer and round
        auto pv_wait = [&](uint32_t n) { wait(&sm.pv_done[n % SM::kPB], n / SM::kPB & 1); };
        Pieces next = w;
        for (; w.take > 0; w = next) {
            const int len = a.kv_lens[w.n];
            // e4m3: the maximum of score + log2(page scale) is m + ahead (kept apart, for scores whose last
            // place is above 1), and a weight's share of O^T is p scale base, in units of 2^(m + ahead - kLift)
            float m[2 * J], l[2 * J], qs[kE4M3 ? 2 * J : 1], ahead[kE4M3 ? 2 * J : 1], base[kE4M3 ? 2 * J : 1];
#pragma unroll
            for (int i = 0; i < 2 * J; ++i) {
                // columns behind the last: weights 0, and no say in when to rescale
                m[i] = ct * NC + col(i) < cols ? -INFINITY : INFINITY;
                l[i] = 0.0f;
                if (kE4M3) {
                    const int c = col(i);
                    ahead[i] = 0.0f;
                    base[i] = 0.0f;
                    qs[i] = ct * NC + c < cols
                                ? a.q_scale[(int64_t)w.n * a.Sq * a.H + w.g * Hg + sm.row[c]] * a.scale_log2 : 0.0f;
                }
            }
            for (int t = w.t; t < w.t + w.take; ++t, ++nt, rst.step()) {
                const uint32_t sb = nt & 1;
                // S^T, the page scales, and (where there are two buffers) that P^T's has been read
                uint64_t *s_bar = &sm.s_full[sb];
                const uint32_t s_par = nt / 2 & 1;
                const bool old = SM::kPB == 2 && nt >= 2;
                wait(s_bar, s_par, old ? &sm.pv_done[sb] : s_bar, old ? s_par ^ 1 : s_par,
                     kE4M3 ? &sm.full_scale[rst.slot] : s_bar, kE4M3 ? rst.round & 1 : s_par);
                tc::fence_after_sync();
                float page_scale = 1.0f;  // of this warp's 16 rows, which lie in one page
                if constexpr (kE4M3)
                    page_scale = sm.scale[rst.slot][quarter * 16 / maps.rows];
                float s[J][4];
                if constexpr (kE4M3)
                    load_s2<kCols>(lane_base + sb * SM::kSW, NC, s);
                else
                    load_s<kCols>(lane_base + sb * SM::kSW, s);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.s_empty[sb]);
                const float lg = kE4M3 ? log2f(page_scale) : 0.0f;
                bool grow = false;
                const bool edge = (t + 1) * kTok > len - a.Sq + 1;  // some column's last row is in this tile
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int k = 2 * j + i;
                        const float f = kE4M3 ? qs[k] * page_scale : a.scale_log2;
                        s[j][i] *= f;
                        s[j][2 + i] *= f;
                        if (edge) {
                            const int cg = ct * NC + col(k);
                            const int last = len - a.Sq + (a.Sq == 1 ? 0 : min(cg / Hg, a.Sq - 1));
                            if (t * kTok + r0 > last)
                                s[j][i] = -INFINITY;
                            if (t * kTok + r0 + 8 > last)
                                s[j][2 + i] = -INFINITY;
                        }
                        // (rounded down: what passes is no further above m, wherever m is)
                        const float most = kE4M3 ? __fadd_rd(m[k], fminf(kGrow, ahead[k] - lg + kGrowO)) : m[k] + kGrow;
                        grow |= s[j][i] > most || s[j][2 + i] > most;
                    }
                if (softmax_or(group, grow)) {
                    // new column maxima over the tile's 64 rows
                    float f[2 * J];
#pragma unroll
                    for (int i = 0; i < 2 * J; ++i) {
                        float x = fmaxf(s[i >> 1][i & 1], s[i >> 1][2 + (i & 1)]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1)
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        if (lane < 4)
                            sm.red[quarter][col(i)] = x;
                    }
                    if (kE4M3 && lane == 0)
                        sm.page_lg[group][quarter] = lg;
                    softmax_sync(group);
#pragma unroll
                    for (int i = 0; i < 2 * J; ++i) {
                        const int c = col(i);
                        const float mn = fmaxf(fmaxf(fmaxf(sm.red[0][c], sm.red[1][c]), fmaxf(sm.red[2][c], sm.red[3][c])),
                                               m[i]);
                        f[i] = m[i] == mn ? 1.0f : ex2(m[i] - mn);
                        l[i] *= f[i];
                        if (kE4M3) {
                            const float held = m[i] == -INFINITY ? -INFINITY : m[i] == mn ? ahead[i] : m[i] - mn + ahead[i];
                            float most = held;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                most = fmaxf(most, sm.red[k][c] - (mn == -INFINITY ? 0.0f : mn) + sm.page_lg[group][k]);
                            ahead[i] = most == -INFINITY ? 0.0f : most;
                            f[i] = ex2(held - ahead[i]);
                            base[i] = ex2(kLift - ahead[i]);
                        }
                        m[i] = mn;
                        if (quarter == 0 && lane < 4)
                            sm.fac[c] = f[i];
                    }
                    softmax_sync(group);
                    if (t > w.t) {
                        pv_wait(nt - 1);  // O^T of the tiles so far is complete
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int b = 0; b < kPairs * SM::kParts * kCols / kCh; ++b) {
                            const int c0 = b * kCh % kCols;
                            const uint32_t at = lane_base + kColO + b * kCh / kCols * NC + c0;
                            uint32_t y[kCh];
                            load_row<kCh>(at, y);
                            tc::wait_ld();
#pragma unroll
                            for (int i = 0; i < kCh; ++i)
                                y[i] = __float_as_uint(__uint_as_float(y[i]) * sm.fac[group * kCols + c0 + i]);
                            store_row<kCh>(at, y);
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
                if (SM::kPB == 1 && nt > 0)
                    pv_wait(nt - 1);  // P^T's one buffer has been read
                // base is at most 2^111 (a page of zeros has a scale of 2^-100): of a page scale above 2^16 the
                // rest goes to the weights, or its product with base would pass float32's range
                if (kE4M3 && page_scale > 65536.0f) {
                    const float part = page_scale * (1.0f / 65536.0f);
                    page_scale = 65536.0f;
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[j][i] *= part;
                }
                unsigned char *pt = sm.p[nt % SM::kPB];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int c = col(2 * j);
                    if constexpr (kE4M3) {
                        // rounded to f16, then the leading three bits of what is left at a time, the last rounded
                        const float g[2] = {page_scale * base[2 * j], page_scale * base[2 * j + 1]};
                        __half2 h[2] = {__floats2half2_rn(s[j][0] * g[0], s[j][1] * g[1]),
                                        __floats2half2_rn(s[j][2] * g[0], s[j][3] * g[1])};
#pragma unroll
                        for (int k = 0; k < 3; ++k) {
                            uint32_t u[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t x = *reinterpret_cast<const uint32_t *>(&h[i]);
                                u[i] = (k < 2 ? x : x + 0x00800080u) & 0xff00ff00u;
                                h[i] = __hsub2(h[i], *reinterpret_cast<const __half2 *>(&u[i]));
                            }
                            const uint32_t v = __byte_perm(u[0], u[1], 0x7531);
                            *reinterpret_cast<uint16_t *>(pt + p_off<NC, true>(r0, c, k)) = (uint16_t)v;
                            *reinterpret_cast<uint16_t *>(pt + p_off<NC, true>(r0 + 8, c, k)) = (uint16_t)(v >> 16);
                        }
                    } else {
                        *reinterpret_cast<uint32_t *>(pt + p_off<NC, false>(r0, c, 0)) = pack_bf16x2(s[j][0], s[j][1]);
                        *reinterpret_cast<uint32_t *>(pt + p_off<NC, false>(r0 + 8, c, 0)) = pack_bf16x2(s[j][2], s[j][3]);
                    }
                }
                // rows behind the sequence's end may hold anything (0 * NaN): zeros for O^T
                const int rows = len - t * kTok;
                if constexpr (kE4M3) {
                    if (rows < kTok) {
                        wait(&sm.full_stage[rst.slot], rst.round & 1);
                        for (int v = group * 128 + gtid; v < (kTok - rows) * 32; v += 256)
                            *reinterpret_cast<uint4 *>(sm.stage[rst.slot] + (v >> 3 & 3) * kBlk + (rows + v / 32) * 128 +
                                                       (v & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                } else {
                    if (rows < kTok) {
                        Ring<SM::kRing> rz = rp;
#pragma unroll
                        for (int j = 0; j < 2; ++j, rz.step()) {
                            wait(&sm.full[rz.slot], rz.round & 1);
                            for (int v = group * 128 + gtid; v < (kTok - rows) * 32; v += 256)
                                *reinterpret_cast<uint4 *>(sm.ring[rz.slot] + (v >> 3 & 3) * kBlk + (rows + v / 32) * 128 +
                                                           (v & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    rp.step();
                    rp.step();
                }
                fence_proxy_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.p_full[nt % SM::kPB]);
            }
            // ---- the piece's sums, and its result (the next one is looked up while the last products run)
            next.next(a);
#pragma unroll
            for (int i = 0; i < 2 * J; ++i) {
                const int c = col(i);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
                if (lane < 4) {
                    sm.red[quarter][c] = l[i];
                    if (quarter == 0) {
                        sm.top[c] = m[i];
                        if (kE4M3)
                            sm.ahead[c] = ahead[i];
                    }
                }
            }
            softmax_sync(group);
            const bool whole = w.whole();
            const int64_t slot = (int64_t)blockIdx.x * 2 + (w.inside ? 1 : 0);
            const int64_t row0 = (int64_t)w.n * a.Sq * a.H + w.g * Hg;
            if (gtid < kCols) {
                const int c = group * kCols + gtid;
                const float sum = sm.red[0][c] + sm.red[1][c] + sm.red[2][c] + sm.red[3][c];
                const float lse2 = sum == 0.0f ? -INFINITY : sm.top[c] + log2f(sum);
                const float unit = kE4M3 ? ex2(sm.ahead[c] - kLift) : 1.0f;
                sm.fac[c] = sum == 0.0f ? 0.0f : unit / sum;
                if (!whole)
                    a.part_lse[slot * NC + c] = lse2;
                else if (a.lse && ct * NC + c < cols)
                    a.lse[row0 + sm.row[c]] = lse2 * kLn2;
            }
            if (w.t == 0 && !whole) {
                go_on = true;
                if (tid == 0)
                    a.meta[blockIdx.x] = make_int4(w.n, w.g, 1 + (int)((w.tiles - w.take + sm.share[2] - 1) / sm.share[2]),
                                                   w.inside ? 1 : 0);
            }
            softmax_sync(group);
            pv_wait(nt - 1);
            tc::fence_after_sync();
            const int dim = gtid, live = cols - ct * NC;
#pragma unroll 1
            for (int b = 0; b < kPairs * kCols / kCh; ++b) {
                const int pair = b * kCh / kCols, c0 = group * kCols + b * kCh % kCols;
                const uint32_t at = lane_base + kColO + pair * SM::kParts * NC + b * kCh % kCols;
                uint32_t y[SM::kParts][kCh];
#pragma unroll
                for (int i = 0; i < SM::kParts; ++i)
                    load_row<kCh>(at + i * NC, y[i]);
                float f[kCh];
#pragma unroll
                for (int i = 0; i < kCh; i += 4)
                    *reinterpret_cast<float4 *>(f + i) = *reinterpret_cast<const float4 *>(sm.fac + c0 + i);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < kCh; ++i)
                {
                    float x = __uint_as_float(y[0][i]);
#pragma unroll
                    for (int k = 1; k < SM::kParts; ++k)
                        x += __uint_as_float(y[k][i]);
                    f[i] = f[i] == 0.0f ? 0.0f : x * f[i];
                }
                if (!whole) {
                    float *dst = a.part_o + ((slot * kPairs + pair) * (NC / 4) + c0 / 4) * 512 + dim * 4;
#pragma unroll
                    for (int i = 0; i < kCh; i += 4)
                        *reinterpret_cast<float4 *>(dst + i * 128) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
                } else {
                    // a lane and its neighbour trade columns, so that each writes two numbers at once
                    __nv_bfloat16 *dst = a.o + row0 * kDL + pair * 128 + (dim & ~1);
#pragma unroll
                    for (int i = 0; i < kCh; i += 2) {
                        const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? f[i] : f[i + 1], 1);
                        const uint32_t v = lane & 1 ? pack_bf16x2(got, f[i + 1]) : pack_bf16x2(f[i], got);
                        const int c = c0 + i + (lane & 1);
                        if (c < live)
                            *reinterpret_cast<uint32_t *>(dst + (int64_t)sm.row[c] * kDL) = v;
                    }
                }
            }
            softmax_sync(group);  // sm.fac and sm.red are free again
            tc::fence_before_sync();
        }
        if (tid == 0 && !go_on)
            a.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    wait.finish(a.status);
    if (warp == 4)
        tc::tmem_dealloc(tmem, kTmemCols);
}

// Joins the partial results of the unit that starts in share x and goes on behind it.  128 threads,
// one latent number each, take four columns of kP pairs; the shares' weights are formed once, by the
// first threads.
constexpr int kJoinShares = 64;  // weights held at once

template <int NC, int kP>
__global__ void __launch_bounds__(128) mla_decode_join_kernel(DecArgs a)
{
    __shared__ __align__(16) float wgt[kJoinShares][4];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, c0 = blockIdx.y * 4, pair0 = blockIdx.z * kP;
    const int4 mt = a.meta[blockIdx.x];
    const int count = mt.z, ct = blockIdx.x % a.CT, Hg = a.H / a.G, left = a.Sq * Hg - ct * NC - c0;
    if (count == 0 || left <= 0)
        return;
    const int64_t row0 = (int64_t)mt.x * a.Sq * a.H + mt.y * Hg;
    auto slot_of = [&](int i) { return ((int64_t)blockIdx.x + (int64_t)i * a.CT) * 2 + (i == 0 ? mt.w : 0); };
    // warp c: column c's largest lse and the sum of weights
    const int lane = tid & 31, c = tid >> 5;
    float top = -INFINITY;
    for (int i = lane; i < count; i += 32) {
        const float x = a.part_lse[slot_of(i) * NC + c0 + c];
        top = x > top || x != x ? x : top;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, top, d);
        top = x > top || x != x ? x : top;
    }
    float sum = 0.0f, acc[kP][4] = {};
    for (int i0 = 0; i0 < count; i0 += kJoinShares) {
        const int n = min(kJoinShares, count - i0);
        for (int i = lane; i < n; i += 32) {
            const float x = a.part_lse[slot_of(i0 + i) * NC + c0 + c], v = x == -INFINITY ? 0.0f : ex2(x - top);
            wgt[i][c] = v;
            sum += v;
        }
        __syncthreads();
#pragma unroll(kP == 1 ? 4 : 2)
        for (int i = 0; i < n; ++i) {
            const float4 *part = reinterpret_cast<const float4 *>(a.part_o) +
                                 ((slot_of(i0 + i) * kPairs + pair0) * (NC / 4) + c0 / 4) * 128 + tid;
            const float4 f = *reinterpret_cast<const float4 *>(wgt[i]);
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const float4 v = part[p * (NC / 4) * 128];
                acc[p][0] += f.x * v.x;
                acc[p][1] += f.y * v.y;
                acc[p][2] += f.z * v.z;
                acc[p][3] += f.w * v.w;
            }
        }
        __syncthreads();
    }
    sum = warp_sum(sum);
    if (lane == 0)
        wgt[0][c] = sum;
    const int cg = ct * NC + c0 + c;
    if (pair0 == 0 && a.lse && lane == 0 && c < left)
        a.lse[row0 + cg / Hg * a.H + cg % Hg] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int kg = ct * NC + c0 + k;
        const float s = wgt[0][k];
        if (k < left)
#pragma unroll
            for (int p = 0; p < kP; ++p)
                a.o[(row0 + kg / Hg * a.H + kg % Hg) * kDL + (pair0 + p) * 128 + tid] =
                    __float2bfloat16(s == 0.0f ? 0.0f : acc[p][k] / s);
    }
}

// Columns of a CTA.  Half as many cost less than half as much (products of 32 columns take 45 cycles
// and of 16 about as long), but leave room for more rows in flight and shorten the softmax: 16
// heads in 16 columns 124 us for 145 in 32 over the 8-bit batch, 205 for 214 over the bfloat16 one.
int columns(int Sq, int H, int G)
{
    const int n = Sq * (H / G);
    return n <= 16 ? 16 : n <= 32 ? 32 : 64;
}

struct DecPlan {
    int nc, ct, shares;
    size_t part_lse, part_o, q_scale, q_terms, total;
};

DecPlan plan(int N, int Sq, int H, int G)
{
    DecPlan p;
    p.nc = columns(Sq, H, G);
    p.ct = (Sq * (H / G) + p.nc - 1) / p.nc;
    p.shares = num_sms() / p.ct > 0 ? num_sms() / p.ct : 1;
    const size_t slots = (size_t)p.shares * p.ct * 2;
    p.part_lse = ((size_t)p.shares * p.ct * sizeof(int4) + 255) / 256 * 256;
    p.part_o = p.part_lse + (slots * p.nc * 4 + 255) / 256 * 256;
    const size_t rows = (size_t)N * Sq * H;
    p.q_scale = p.part_o + slots * p.nc * kDL * 4;
    p.q_terms = p.q_scale + (rows * 4 + 255) / 256 * 256;
    p.total = p.q_terms + 2 * rows * kDC;
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
    const int64_t rows = (int64_t)a.N * a.Sq * a.H;
    maps.q_rows = a.G == 1 ? NC : Hg % 8 == 0 ? 8 : 1;
    const bool all = maps.q_rows == NC;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;  // every launch sets up while the one before it ends, and waits for it on the device
    if constexpr (kE4M3) {
        const int64_t extent[4] = {128, rows, 2, 4}, stride[3] = {kDC, rows * kDC, 128};
        const int box[4] = {128, maps.q_rows, all ? 2 : 1, all ? 4 : 1};
        const int64_t rope[3] = {kDR, rows, 2};
        const int rope_box[3] = {kDR, maps.q_rows, all ? 2 : 1};
        if ((e = make_map(&maps.q, a.q_terms, 1, 4, extent, stride, box)) != cudaSuccess ||
            (e = make_map(&maps.q_rope, a.q_terms + kDL, 1, 3, rope, stride, rope_box)) != cudaSuccess)
            return e;
        cfg.gridDim = dim3((unsigned)((rows + 7) / 8));
        cfg.blockDim = dim3(256);
        if ((e = cudaLaunchKernelEx(&cfg, mla_split_q_kernel, a, rows)) != cudaSuccess)
            return e;
    } else {
        const int64_t extent[3] = {64, rows, kDC / 64}, stride[2] = {kDC * 2, 128};
        const int box[3] = {64, maps.q_rows, all ? kDC / 64 : 1};
        if ((e = make_map(&maps.q, a.q, 2, 3, extent, stride, box)) != cudaSuccess)
            return e;
    }
    cfg.gridDim = dim3(a.shares * a.CT);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, maps, a)) != cudaSuccess)
        return e;
    // (few units: each is cut into many shares, and a thread takes one pair of blocks of them)
    const bool few = (int64_t)a.N * a.G * 16 <= a.shares;
    cfg.gridDim = dim3(a.shares * a.CT, NC / 4, few ? kPairs : 1);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return few ? cudaLaunchKernelEx(&cfg, mla_decode_join_kernel<NC, 1>, a)
               : cudaLaunchKernelEx(&cfg, mla_decode_join_kernel<NC, kPairs>, a);
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
              reinterpret_cast<float *>(ws + p.part_lse), reinterpret_cast<int4 *>(ws), ws + p.q_terms,
              reinterpret_cast<float *>(ws + p.q_scale), device_status_ptr()};
    if (!a.status)
        return cudaErrorInvalidDevice;
    DecMaps maps{};
    maps.rows = page_size < kTok ? page_size : kTok;
    const int es = e4m3 ? 1 : 2, block = 128 / es;  // numbers of a 128-byte row
    const int64_t extent[4] = {block, G, (int64_t)num_pages * page_size, kDL / block};
    const int64_t stride[3] = {kDC * es, (int64_t)G * kDC * es, 128};
    const int box[4] = {block, 1, maps.rows, maps.rows == kTok ? 4 : 1};
    cudaError_t e = make_map(&maps.latent, cache, es, 4, extent, stride, box);
    if (e == cudaSuccess) {
        const int64_t rope[3] = {kDR, G, (int64_t)num_pages * page_size};
        const int rope_box[3] = {kDR, 1, maps.rows};
        e = make_map(&maps.rope, static_cast<const unsigned char *>(cache) + kDL * es, es, 3, rope, stride, rope_box);
    }
    if (e != cudaSuccess)
        return e;
    if (e4m3)
        return p.nc == 16   ? launch_nc<16, true>(maps, a, s)
               : p.nc == 32 ? launch_nc<32, true>(maps, a, s)
                            : launch_nc<64, true>(maps, a, s);
    return p.nc == 16   ? launch_nc<16, false>(maps, a, s)
           : p.nc == 32 ? launch_nc<32, false>(maps, a, s)
                        : launch_nc<64, false>(maps, a, s);
}

}  // namespace kda

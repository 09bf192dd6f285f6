// cg_int4_weigh: the attention weight that every token of the 4-bit cache gets, sum over a
// request's new tokens i and the query heads g of a KV head of p_igj = 2^(z_igj - m_ig) / l_ig,
// z the scores in powers of two.
//
// The maximum m and the sum l of a row are over all of its tokens, so a first kernel goes over K
// for m and l of every row (a running maximum and sum, pieces joined by k_weigh_join), and a second one sums
// over the rows of every token: from the scores, which the first one left in the workspace (k_weigh_apply),
// or, where there is no room for them, from K again (k_weigh_sums). Requests with more than kTileRows rows of
// a KV head go to tcgen05 (cachegen_weigh_many.cu), those with fewer come here:
//   1 .. 8 rows    k_weigh_few. K is read once at 80 bytes a token and head of 128 channels in groups of 32, and
//                  what bounds it is the work on a blob of 16 tokens, some 700 instructions a warp: 64 requests
//                  of up to 8192 tokens, 4 rows: 59 us for 278 MB, with join 5 and apply 20 88 us in all; a
//                  floor of 42 at the copy rate. (mma.sync: 16 tokens by 8 rows is all that there are.)
//   9 .. 64 rows   k_weigh_stats, 16 or 32 rows at a time, which read K again for each 32.
// Sums go by rows in a fixed order, 256 or so to a partial sum, so the same call gives the same bits.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cg_weigh.h"

namespace {

constexpr int kRing = 8;           // blobs in a warp's ring
constexpr int kItemTokens = 64;    // of a block in the second pass, a blob to a warp; or,
// from so many rows on, a blob to a block, whose warps share the rows. (Without stored scores and without room
// for the sums of kTileRows' kernel: a prompt of 32768 tokens, say, or a chunk of 8192 under a table for 131072.)
constexpr int kManyRows = 512;
constexpr int kMaxBlocks = 640;    // of the first pass

// ------------------------------------------------------------------- scores

// With mid = lo + 8 s and m = n - 8 in [-8, 7], q.k^ = sum_g s_g (q.m)_g + mid_g (sum q)_g. Where a
// few channels of a group are large, s and lo follow those and the others' codes lie near 8:
// q.n and lo (sum q) would be large and cancel (an error of 1.3e-5 in the weights, of 3e-8 so). The
// products of bf16 pairs are exact, everything else is fp32.

// The queries of 8 rows of a KV head, from row0 on. qf: the second factor of the instruction, column
// g is the row row0 + g times a power of two that brings it below 2^-7 (so that no s (q.m) overflows
// whose score does not). Of rows 2t and 2t + 1, rho: scale2 over that power; sq: scale2 times the sum
// of q in each group.
template <typename B>
struct Queries {
    uint32_t qf[B::kWords][4];
    float2 rho, sq[B::kGroups];
};

template <typename B>
__device__ __forceinline__ void load_rows(const AttnArgs &p, const AttnRequest &rq, int h, int row0, Queries<B> *to)
{
    constexpr int NW = B::kWords, NG = B::kGroups, WPG = NW / NG;
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3, row = row0 + g;
    const bool there = row < rq.rows;
    const int qt = there ? row / p.ratio : 0, qh = h * p.ratio + (there ? row - qt * p.ratio : 0);
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.a.q) +
                             (int64_t)(rq.row0 + qt) * p.a.q_token_stride + qh * p.a.q_head_stride;
    uint4 v[NW];
    uint32_t top = 0;        // largest |q| of the row (as bf16 bits, in both halves)
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        v[w] = there ? *reinterpret_cast<const uint4 *>(q + 32 * w + 8 * t) : make_uint4(0, 0, 0, 0);
        top = __vmaxu2(__vmaxu2(top, v[w].x & 0x7FFF7FFFu), v[w].y & 0x7FFF7FFFu);
        top = __vmaxu2(__vmaxu2(top, v[w].z & 0x7FFF7FFFu), v[w].w & 0x7FFF7FFFu);
    }
    top = max(top & 0xFFFFu, top >> 16);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    // exact, but for what is 2^-110 of the row's largest
    const int e = max((int)(top >> 7) - 127, -118);
    const float up = pow2((-8 - e) >> 1), up2 = pow2((-7 - e) >> 1);
    const float rho = p.scale2 * pow2((8 + e) >> 1) * pow2((9 + e) >> 1);
    float sum[NG] = {};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const uint4 c = v[w];
        // channels i and i + 4 side by side, as the codes of a word come
        to->qf[w][0] = pack_bf16(par_s(c.x) * up * up2, par_s(c.z) * up * up2);
        to->qf[w][1] = pack_bf16(par_lo(c.x) * up * up2, par_lo(c.z) * up * up2);
        to->qf[w][2] = pack_bf16(par_s(c.y) * up * up2, par_s(c.w) * up * up2);
        to->qf[w][3] = pack_bf16(par_lo(c.y) * up * up2, par_lo(c.w) * up * up2);
        sum[w / WPG] += ((par_s(c.x) + par_lo(c.x)) + (par_s(c.y) + par_lo(c.y))) +
                        ((par_s(c.z) + par_lo(c.z)) + (par_s(c.w) + par_lo(c.w)));
    }
    to->rho = make_float2(__shfl_sync(0xFFFFFFFFu, rho, 8 * t), __shfl_sync(0xFFFFFFFFu, rho, 8 * t + 4));
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 2);
        const float mine = p.scale2 * sum[i];
        to->sq[i] = make_float2(__shfl_sync(0xFFFFFFFFu, mine, 8 * t), __shfl_sync(0xFFFFFFFFu, mine, 8 * t + 4));
    }
}

// The keys of a blob as the first factor, tokens g and g + 8.
template <typename B>
struct Keys {
    uint32_t a[B::kWords][8];            // per word, codes 0 .. 3 of token g and of g + 8 by turns
    float s[2][B::kGroups], mid[2][B::kGroups];
};

template <typename B>
__device__ __forceinline__ void load_keys(const uint8_t *blob, int lane, Keys<B> *to)
{
    constexpr int D = B::kD, NW = B::kWords, NG = B::kGroups;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t k[NW], par[NG];
        load_words(k, blob + B::kKCodes + (g + 8 * j) * (D / 2) + t * (D / 8));
        load_words(par, blob + B::kKParams + (g + 8 * j) * 4 * NG);
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                to->a[w][2 * i + j] = centred(k[w], i);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            to->s[j][i] = par_s(par[i]);
            to->mid[j][i] = fmaf(8.0f, par_s(par[i]), par_lo(par[i]));
        }
    }
}

// A product of the instruction that the compiler may move among others.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t *a, uint32_t b0, uint32_t b1, const float *c)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// Scores in powers of two, less m, of a row tile: z[j] are token g + 8 j with rows 2t and 2t + 1.
template <typename B>
__device__ __forceinline__ void scores_of(const Keys<B> &k, const Queries<B> &q, float2 m, float2 (&z)[2])
{
    constexpr int NW = B::kWords, NG = B::kGroups, WPG = NW / NG;
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float2 y[2];
#pragma unroll
    for (int gi = 0; gi < NG; ++gi) {
        float acc[4];
#pragma unroll
        for (int w = gi * WPG; w < (gi + 1) * WPG; ++w)
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                mma(acc, &k.a[w][2 * i], q.qf[w][i], q.qf[w][i + 1], w == gi * WPG && i == 0 ? zero : acc);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 s = make_float2(k.s[j][gi], k.s[j][gi]), mid = make_float2(k.mid[j][gi], k.mid[j][gi]);
            const float2 x = make_float2(acc[2 * j], acc[2 * j + 1]);
            y[j] = gi ? fma2(s, x, y[j]) : mul2(s, x);
            z[j] = fma2(mid, q.sq[gi], gi ? z[j] : make_float2(-m.x, -m.y));
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
        z[j] = fma2(y[j], q.rho, z[j]);
}

// Where not every token is seen by every row: -inf for those that are not. x: positions of the rows.
__device__ __forceinline__ void hide(const AttnArgs &p, int tok, int g, const int (&x)[2], int window, float2 (&z)[2])
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int at = tok + g + 8 * j;
        if (at > x[0] || (x[0] - at >= window && at >= p.a.sinks))
            z[j].x = -INFINITY;
        if (at > x[1] || (x[1] - at >= window && at >= p.a.sinks))
            z[j].y = -INFINITY;
    }
}

// -------------------------------------------------------------- pieces, tiles

// The rows of a unit and the blobs that they see. Tiles are taken from both ends in turn, so that
// neighbouring pieces of a prompt see equally much.
struct Tile {
    int32_t row0, rows;      // of the request's KV head
    int32_t x_lo, x_hi;      // positions of the first and the last
    Span span;
};

template <int RU>
__device__ __forceinline__ Tile tile_of(const AttnArgs &p, const Unit &u)
{
    Tile t;
    t.row0 = RU * (u.rt & 1 ? u.tiles - 1 - (u.rt >> 1) : u.rt >> 1);
    t.rows = min(RU, u.q.rows - t.row0);
    t.x_lo = u.q.x0 + t.row0 / p.ratio;
    t.x_hi = u.q.x0 + (t.row0 + t.rows - 1) / p.ratio;
    const int32_t end = t.x_hi < 0 ? 0 : t.x_hi / 16 + 1;
    t.span = {end, 0, 0, end};
    const int64_t low = (int64_t)t.x_lo + 1 - p.a.window;
    if (p.a.window > 0 && low > 0) {
        const int32_t first = (int32_t)(low / 16);
        const int64_t sb = ((int64_t)p.a.sinks + 15) / 16;
        t.span.sink = sb < first ? (int32_t)sb : first;
        t.span.skip = first - t.span.sink;
        t.span.nb = end - t.span.skip;
    }
    return t;
}

// The warp's stretch of the tile's blobs: the unit's piece is [b0, b1) of span.nb blobs of the
// request, and takes as large a part of the tile's.
__device__ __forceinline__ void tile_range(const Unit &u, const Tile &t, int warp, int *b, int *e)
{
    const int b0 = (int)((int64_t)u.b0 * t.span.nb / u.span.nb), b1 = (int)((int64_t)u.b1 * t.span.nb / u.span.nb);
    *b = b0 + (int)((int64_t)(b1 - b0) * warp / kWarps);
    *e = b0 + (int)((int64_t)(b1 - b0) * (warp + 1) / kWarps);
}

// ------------------------------------------------------------------- copies

// Where a warp stands in its block's piece: in shared memory, since it is looked at seldom and would
// take a third of the registers.
struct Stand {
    Unit u;
    Tile t;
    int64_t pos;     // blobs of the piece up to the end of the unit
    int32_t b, e;    // blobs of the tile that are left of the warp's stretch
};

// The warp's copies, HB blobs at a time and kStages of those ahead of it: 32 blobs are looked up at once,
// one by each lane, which then issues its own blob's copy.
template <typename B, int RU, int HB, int kStages>
struct Feeder {
    uint8_t (*ring)[HB][B::kVCodes];
    uint64_t *full;                // barriers, HB arrivals each
    Stand *at;
    int32_t i, n;                  // blobs issued and looked up of the current 32
    uint32_t off, ok;              // the lane's blob (in 128-byte units of the layer); valid lanes
    uint32_t issued, ahead;        // steps issued; which blobs of the steps in flight are there

    __device__ __forceinline__ void start(const AttnArgs &p, int64_t count, const Unit &u, int warp, int lane)
    {
        const Tile t = tile_of<RU>(p, u);
        int b, e;
        tile_range(u, t, warp, &b, &e);
        if (lane == 0)
            *at = {u, t, u.b1 - u.b0, b, e};
        i = n = 0;
        off = ok = issued = ahead = 0;
        __syncwarp();
        for (int k = 0; k < kStages; ++k)
            feed(p, count, warp, lane);
    }

    __device__ __forceinline__ bool look(const AttnArgs &p, int64_t count, int warp, int lane)
    {
        int b = at->b, e = at->e;
        if (b >= e) {
            Unit u = at->u;
            Tile t;
            int64_t pos = at->pos;
            do {
                if (pos >= count)
                    return false;
                unit_next<RU, WeighBatch>(p, count - pos, &u);
                t = tile_of<RU>(p, u);
                pos += u.b1 - u.b0;
                tile_range(u, t, warp, &b, &e);
            } while (b >= e);
            __syncwarp();
            if (lane == 0)
                *at = {u, t, pos, b, e};
            __syncwarp();
        }
        i = 0;
        n = e - b < 32 ? e - b : 32;
        int id = -1;
        if (lane < n) {
            const int bpp = p.page_tokens / 16, vb = b + lane, ab = vb < at->t.span.sink ? vb : vb + at->t.span.skip;
            const int page = ab / bpp;
            id = p.a.block_table[at->u.r * p.a.table_stride + page];
            if ((unsigned)id >= (unsigned)p.num_pages)
                int4_set_status(p.status, CG_ERR_CORRUPT);
            off = (((uint32_t)id * p.heads + at->u.h) * bpp + (ab - page * bpp)) * (B::kBytes / 128);
        }
        ok = __ballot_sync(0xFFFFFFFFu, (unsigned)id < (unsigned)p.num_pages);
        if (lane == 0)
            at->b = b + n;
        __syncwarp();
        return true;
    }

    __device__ __forceinline__ void feed(const AttnArgs &p, int64_t count, int warp, int lane)
    {
        ahead >>= HB;
        if (i >= n && !look(p, count, warp, lane))
            return;
        const int st = issued % kStages;
        if ((unsigned)(lane - i) < (unsigned)HB) {
            if (ok >> lane & 1) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                bar_expect(&full[st], B::kVCodes);
                bulk_copy(ring[st][lane - i], p.layer + (uint64_t)off * 128, B::kVCodes, &full[st]);
            } else {
                bar_arrive(&full[st]);
            }
        }
        ahead |= (ok >> i & ((1u << HB) - 1)) << (HB * (kStages - 1));
        i += HB;
        ++issued;
    }
};

// -------------------------------------------------------- maximum and sum

template <typename B, int NT>
struct StatShared {
    uint8_t ring[kWarps][kRing][1][B::kVCodes];   // the K half of blobs
    uint4 qf[NT][B::kWords][32];                  // the rows' second factors, as the lanes have them
    float2 factors[NT][B::kGroups + 1][4];        // rho, sq
    float m[kWarps][8 * NT], l[kWarps][8 * NT];
    uint64_t full[kWarps][kRing];
    Stand feed[kWarps], now[kWarps];
};

// A row's maximum set by its first score or raised by a later one, `top` above it: by how much. *limit
// stays below every score while a row that is there waits for its first.
__device__ __forceinline__ float raise(float top, bool no_row, float *m, float *l, float *limit)
{
    const bool none = *l == 0.0f;
    const float up = none ? (top > kNone ? top : 0.0f) : fmaxf(top, 0.0f);
    *m += up;
    *l = none ? 0.0f : *l * exp2_fast(-up);
    if (none && !(top > kNone) && !no_row)
        *limit = kNone;
    return up;
}

// Blocks on an SM.
constexpr int kStatBlocks = 3;

// For 8 NT rows of a (request, KV head) at a time. 12 rows of 32768 tokens, 8 KV heads: 31 us with all that
// follows, 32 rows 41, 64 rows 63. What bounds it is instructions: a blob's keys are made once (4 a pair of codes) and
// meet NT tiles of 8 rows, each of whose scores takes an exponential and a store.
//
// kStored: scores are left for the sums, else the queries.
template <typename B, int NT, bool kStored>
__global__ void __launch_bounds__(kThreads, kStatBlocks) k_weigh_stats(AttnArgs p, WeighArgs a)
{
    using S = StatShared<B, NT>;
    constexpr int NW = B::kWords, NG = B::kGroups, RU = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);
    const int lane = lane_once(), warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;

    grid_next();
    if (a.taken != nullptr && blockIdx.x == 0 && threadIdx.x < 2)
        a.taken[threadIdx.x] = 0;
    if (lane == 0)
        for (int i = 0; i < kRing; ++i)
            bar_init(&sm.full[warp][i], 1);
    bar_init_fence();
    int64_t total, chunk;
    const Place at = schedule<RU, WeighBatch>(p, gridDim.x, blockIdx.x, 0, blockIdx.x == 0, &total, &chunk);
    const int64_t begin = blockIdx.x * chunk;
    if (begin >= total)
        return;
    const int64_t count = (begin + chunk < total ? begin + chunk : total) - begin;
    Unit first;
    unit_at<RU, WeighBatch>(p, at, count, &first);
    Feeder<B, RU, 1, kRing> feeder;
    feeder.ring = sm.ring[warp];
    feeder.full = sm.full[warp];
    feeder.at = &sm.feed[warp];
    feeder.start(p, count, first, warp, lane);
    Stand &now = sm.now[warp];
    if (lane == 0)
        now = {first, tile_of<RU>(p, first), 0, 0, 0};
    __syncwarp();

    const int window = p.a.window > 0 ? p.a.window : INT32_MAX;
    bool alive = true;               // no wait has run out
    uint32_t used = 0;
    for (;;) {
        const Unit u = now.u;
        const Tile tile = now.t;
        const int slot = first_slot(p, u.r, u.q.row0) + tile.row0 / 8;
        // a warp to a tile of 8 rows; the unit's first piece leaves them for the sums
        if (warp < NT) {
            Queries<B> q;
            load_rows<B>(p, u.q, u.h, tile.row0 + 8 * warp, &q);
            const int64_t at_slot = (int64_t)u.h * a.slots + slot + warp;
            uint4 *to = a.queries + at_slot * NW * 32 + lane;
            float2 *f = reinterpret_cast<float2 *>(a.factors + at_slot * (NG + 1) * 8) + t;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                sm.qf[warp][w][lane] = make_uint4(q.qf[w][0], q.qf[w][1], q.qf[w][2], q.qf[w][3]);
                if (!kStored && u.b0 == 0 && 8 * warp < tile.rows)
                    to[32 * w] = sm.qf[warp][w][lane];
            }
            if (g == 0) {
#pragma unroll
                for (int i = 0; i <= NG; ++i) {
                    sm.factors[warp][i][t] = i ? q.sq[i ? i - 1 : 0] : q.rho;
                    if (!kStored && u.b0 == 0 && 8 * warp < tile.rows)
                        f[4 * i] = sm.factors[warp][i][t];
                }
            }
        }
        __syncthreads();
        int x[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int in = 8 * nt + 2 * t + j;
                x[nt][j] = in < tile.rows ? u.q.x0 + (tile.row0 + in) / p.ratio : -1;
            }
        // Each lane keeps a maximum (0 before the first score) and a sum of its own, over tokens g and g + 8
        // of the blobs. The maximum is set by a row's first score, and raised only when a score exceeds it by
        // 2^8: `limit` is below every score while a row of the lane waits for its first.
        float2 m[NT], l[NT];
        float limit = kNone;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            m[nt] = l[nt] = make_float2(0.0f, 0.0f);
        int b, e;
        tile_range(u, tile, warp, &b, &e);
        for (; b < e; ++b) {
            const int st = used % kRing;
            if (alive) {
                const bool give_up = kTestTimeout && used == 1;
                if (give_up || !__all_sync(0xFFFFFFFFu, bar_wait(&sm.full[warp][st], (used / kRing) & 1))) {
                    alive = false;   // `used` stays: the first blob not waited for
                    int4_set_status(p.status, CG_ERR_TIMEOUT);
                } else {
                    ++used;
                }
            }
            if (alive && (feeder.ahead & 1)) {
                Keys<B> k;
                load_keys<B>(sm.ring[warp][st][0], lane, &k);
                const int tok = 16 * (b < tile.span.sink ? b : b + tile.span.skip);
                const bool whole = tok + 15 <= tile.x_lo && (tile.x_hi - tok < window || tok + 15 < p.a.sinks);
                // rows that are not there have q = 0: what they get is dropped at the end
                float2 z[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    Queries<B> q;
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const uint4 v = sm.qf[nt][w][lane];
                        q.qf[w][0] = v.x, q.qf[w][1] = v.y, q.qf[w][2] = v.z, q.qf[w][3] = v.w;
                    }
                    q.rho = sm.factors[nt][0][t];
#pragma unroll
                    for (int i = 0; i < NG; ++i)
                        q.sq[i] = sm.factors[nt][i + 1][t];
                    scores_of<B>(k, q, m[nt], z[nt]);
                }
                if (!whole)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        hide(p, tok, g, x[nt], window, z[nt]);
                if (kStored) {
                    float *to = a.scores + (((int64_t)u.r * p.heads + u.h) * a.rows + tile.row0 + 2 * t) * a.tokens + tok + g;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int row = 8 * nt + 2 * t;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if (row < tile.rows)
                                to[(int64_t)(8 * nt) * a.tokens + 8 * j] = z[nt][j].x + m[nt].x;
                            if (row + 1 < tile.rows)
                                to[(int64_t)(8 * nt + 1) * a.tokens + 8 * j] = z[nt][j].y + m[nt].y;
                        }
                    }
                }
                float top = -INFINITY;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    top = fmaxf(fmaxf(top, z[nt][0].x), z[nt][0].y);
                    top = fmaxf(fmaxf(top, z[nt][1].x), z[nt][1].y);
                }
                if (top > limit) {
                    limit = 8.0f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float up_x = raise(fmaxf(z[nt][0].x, z[nt][1].x), x[nt][0] < 0, &m[nt].x, &l[nt].x, &limit);
                        const float up_y = raise(fmaxf(z[nt][0].y, z[nt][1].y), x[nt][1] < 0, &m[nt].y, &l[nt].y, &limit);
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            z[nt][j] = make_float2(z[nt][j].x - up_x, z[nt][j].y - up_y);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    l[nt].x += exp2_fast(z[nt][0].x) + exp2_fast(z[nt][1].x);
                    l[nt].y += exp2_fast(z[nt][0].y) + exp2_fast(z[nt][1].y);
                }
            }
            if (kStored && alive && !(feeder.ahead & 1)) {   // a page that is not there
                const int tok = 16 * (b < tile.span.sink ? b : b + tile.span.skip);
                float *to = a.scores + (((int64_t)u.r * p.heads + u.h) * a.rows + tile.row0) * a.tokens + tok;
                for (int i = lane; i < 16 * tile.rows; i += 32)
                    to[(int64_t)(i / 16) * a.tokens + i % 16] = -INFINITY;
            }
            __syncwarp();   // every lane has read the place
            if (alive)
                feeder.feed(p, count, warp, lane);
        }
        // ---- joined over the lanes of a row, the warps, and with other pieces in a second kernel
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float lj = j ? l[nt].y : l[nt].x, mj = lj == 0.0f ? kNone : j ? m[nt].y : m[nt].x;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    const float om = __shfl_xor_sync(0xFFFFFFFFu, mj, d);
                    const float ol = __shfl_xor_sync(0xFFFFFFFFu, lj, d), mx = fmaxf(mj, om);
                    lj = lj * exp2_fast(mj - mx) + ol * exp2_fast(om - mx);
                    mj = mx;
                }
                if (g == 0) {
                    sm.m[warp][8 * nt + 2 * t + j] = mj;
                    sm.l[warp][8 * nt + 2 * t + j] = lj;
                }
            }
        __syncthreads();
        Unit end = now.u;
        const bool from_before = end.b0 > 0, goes_on = end.b1 < end.span.nb;
        if (threadIdx.x < RU) {
            const int row = threadIdx.x, rows = now.t.rows;
            float mx = kNone, ls = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                mx = fmaxf(mx, sm.m[w][row]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                ls += sm.l[w][row] * exp2_fast(sm.m[w][row] - mx);
            if (row >= rows)
                ls = 0.0f;
            if (from_before || goes_on)
                a.parts[((int64_t)blockIdx.x * 2 + (from_before ? 0 : 1)) * RU + row] = make_float2(mx, ls);
            else if (row < (rows + 7) / 8 * 8)
                a.stats[((int64_t)end.h * a.slots + first_slot(p, end.r, end.q.row0) + now.t.row0 / 8) * 8 + row] =
                    row_stats_of(mx, ls);
        }
        const int64_t pos = now.pos + end.b1 - end.b0;
        __syncthreads();
        if (pos >= count)
            break;
        unit_next<RU, WeighBatch>(p, count - pos, &end);
        if (lane == 0)
            now = {end, tile_of<RU>(p, end), pos, 0, 0};
        __syncwarp();
    }
    // a wait that ran out: the copies still in flight must land before the block's memory goes
    if (!alive)
        for (; used < feeder.issued; ++used)
            bar_wait(&sm.full[warp][used % kRing], (used / kRing) & 1);
}

// ---- up to 8 rows: scores are stored

// Half the words' instructions: a code enters as a bf16 whose bits are the code's, n 2^-133 or, for the
// upper codes, n 2^-129 (against 1/16 of the query), and 8 times the sum of the queries comes off where the
// products of a group are summed: its accumulator begins with that.
template <typename B, int P>
struct FewQueries {
    uint32_t qf[P][B::kWords][4];
    float2 off[B::kGroups];          // -8 sum q of a group, as the products count them
    float2 rho, sq[B::kGroups];
};

// P = 2: columns 4 .. 7 of the instruction have the rows 0 .. 3 again. A blob's products with the rows in
// columns 0 .. 3 and the next one's with those in 4 .. 7 go to one accumulator, and all that follows is
// done for both at once.
template <typename B, int P>
__device__ __forceinline__ void load_few(const AttnArgs &p, const AttnRequest &rq, int h, FewQueries<B, P> *to)
{
    constexpr int NW = B::kWords, NG = B::kGroups, WPG = NW / NG;
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3, row = P == 2 ? g & 3 : g;
    const bool there = row < rq.rows;
    const int qt = there ? row / p.ratio : 0, qh = h * p.ratio + (there ? row - qt * p.ratio : 0);
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.a.q) +
                             (int64_t)(rq.row0 + qt) * p.a.q_token_stride + qh * p.a.q_head_stride;
    uint4 v[NW];
    uint32_t top = 0;        // largest |q| of the row (as bf16 bits, in both halves)
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        v[w] = there ? *reinterpret_cast<const uint4 *>(q + 32 * w + 8 * t) : make_uint4(0, 0, 0, 0);
        top = __vmaxu2(__vmaxu2(top, v[w].x & 0x7FFF7FFFu), v[w].y & 0x7FFF7FFFu);
        top = __vmaxu2(__vmaxu2(top, v[w].z & 0x7FFF7FFFu), v[w].w & 0x7FFF7FFFu);
    }
    top = max(top & 0xFFFFu, top >> 16);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    // exact: |q| 2^fe stays below 2^127; small rows (and 0) take the largest factor
    const int fe = min(126 - ((int)(top >> 7) - 127), 127);
    const float up = pow2(fe), up16 = pow2(fe - 4);
    // scale2 2^(133 - fe) in two steps, both upwards: the power alone may pass 2^127, and what
    // lies between passes fp32's range only where the result does
    const float back = p.scale2 * pow2((133 - fe) >> 1) * pow2((134 - fe) >> 1);
    const float o0 = pow2((fe - 130) >> 1), o1 = -pow2((fe - 129) >> 1);
    to->rho = make_float2(__shfl_sync(0xFFFFFFFFu, back, 8 * t), __shfl_sync(0xFFFFFFFFu, back, 8 * t + 4));
    float sum[NG] = {};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const uint4 c = v[w];
        // channels i and i + 4 side by side, as the codes of a word come
        const uint32_t f[4] = {pack_bf16(par_s(c.x) * up, par_s(c.z) * up), pack_bf16(par_lo(c.x) * up16, par_lo(c.z) * up16),
                               pack_bf16(par_s(c.y) * up, par_s(c.w) * up), pack_bf16(par_lo(c.y) * up16, par_lo(c.w) * up16)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            to->qf[0][w][i] = P == 2 && g >= 4 ? 0 : f[i];
            if (P == 2)
                to->qf[P - 1][w][i] = g >= 4 ? f[i] : 0;
        }
        sum[w / WPG] += ((par_s(c.x) + par_s(c.z)) + (par_lo(c.x) + par_lo(c.z))) +
                        ((par_s(c.y) + par_s(c.w)) + (par_lo(c.y) + par_lo(c.w)));
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 2);
        const float off = sum[i] * o0 * o1, mine = p.scale2 * sum[i];
        to->off[i] = make_float2(__shfl_sync(0xFFFFFFFFu, off, 8 * t), __shfl_sync(0xFFFFFFFFu, off, 8 * t + 4));
        to->sq[i] = make_float2(__shfl_sync(0xFFFFFFFFu, mine, 8 * t), __shfl_sync(0xFFFFFFFFu, mine, 8 * t + 4));
    }
}

// z[j]: token g + 8 j with rows 2t and 2t + 1 (of their blob). `par`: the lane's blob, for its parameters.
template <typename B, int P>
__device__ __forceinline__ void few_scores(const uint8_t *(&blob)[P], const uint8_t *par, const FewQueries<B, P> &q,
                                           int lane, float2 (&z)[2])
{
    constexpr int D = B::kD, NW = B::kWords, NG = B::kGroups, WPG = NW / NG;
    const int g = lane >> 2, t = lane & 3;
    uint32_t k[P][2][NW];
#pragma unroll
    for (int b = 0; b < P; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            load_words(k[b][j], blob[b] + B::kKCodes + (g + 8 * j) * (D / 2) + t * (D / 8));
    uint32_t pw[2][NG];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        load_words(pw[j], par + B::kKParams + (g + 8 * j) * 4 * NG);
    float2 y[2];
#pragma unroll
    for (int gi = 0; gi < NG; ++gi) {
        float x[4] = {q.off[gi].x, q.off[gi].y, q.off[gi].x, q.off[gi].y};
#pragma unroll
        for (int b = 0; b < P; ++b)
#pragma unroll
            for (int w = gi * WPG; w < (gi + 1) * WPG; ++w)
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const uint32_t a[4] = {codes_of(k[b][0][w], i), codes_of(k[b][1][w], i),
                                           codes_of(k[b][0][w], i + 1), codes_of(k[b][1][w], i + 1)};
                    mma(x, a, q.qf[b][w][i], q.qf[b][w][i + 1], x);
                }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float s = par_s(pw[j][gi]), mid = fmaf(8.0f, s, par_lo(pw[j][gi]));
            const float2 s2 = make_float2(s, s), mid2 = make_float2(mid, mid), x2 = make_float2(x[2 * j], x[2 * j + 1]);
            y[j] = gi ? fma2(s2, x2, y[j]) : mul2(s2, x2);
            z[j] = gi ? fma2(mid2, q.sq[gi], z[j]) : mul2(mid2, q.sq[0]);
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
        z[j] = fma2(y[j], q.rho, z[j]);
}

constexpr int kFewBlocks = 3;    // on an SM

// A warp takes two accumulators' blobs in one step, two P: their chains mix, and what a step costs
// besides (waits, copies, the look at the maximum) is halved.
template <typename B, int P>
struct FewShared {
    static constexpr int HB = 2 * P, kSteps = P == 2 ? 3 : 4;
    uint8_t ring[kWarps][kSteps][HB][B::kVCodes];
    float m[kWarps][8], l[kWarps][8];
    uint64_t full[kWarps][kSteps];
    Stand feed[kWarps], now[kWarps];
};

template <typename B, int P>
__global__ void __launch_bounds__(kThreads, kFewBlocks) k_weigh_few(AttnArgs p, WeighArgs a)
{
    using S = FewShared<B, P>;
    constexpr int HB = S::HB, kSteps = S::kSteps;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);
    const int lane = lane_once(), warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;

    grid_next();
    if (lane == 0)
        for (int i = 0; i < kSteps; ++i)
            bar_init(&sm.full[warp][i], HB);
    bar_init_fence();
    int64_t total, chunk;
    const Place at = schedule<8, WeighBatch>(p, gridDim.x, blockIdx.x, 0, blockIdx.x == 0, &total, &chunk);
    const int64_t begin = blockIdx.x * chunk;
    if (begin >= total)
        return;
    const int64_t count = (begin + chunk < total ? begin + chunk : total) - begin;
    Unit first;
    unit_at<8, WeighBatch>(p, at, count, &first);
    Feeder<B, 8, HB, kSteps> feeder;
    feeder.ring = sm.ring[warp];
    feeder.full = sm.full[warp];
    feeder.at = &sm.feed[warp];
    feeder.start(p, count, first, warp, lane);
    Stand &now = sm.now[warp];
    if (lane == 0)
        now = {first, tile_of<8>(p, first), 0, 0, 0};
    __syncwarp();

    const int window = p.a.window > 0 ? p.a.window : INT32_MAX;
    const int side = P == 2 ? t >> 1 : 0;            // which blob of a pair the lane's columns are of
    const int row = P == 2 ? 2 * (t & 1) : 2 * t;    // the first of the lane's two rows
    bool alive = true;               // no wait has run out
    uint32_t used = 0;
    for (;;) {
        const Unit u = now.u;
        const Tile tile = now.t;
        FewQueries<B, P> q;
        load_few<B, P>(p, u.q, u.h, &q);
        const int x[2] = {row < tile.rows ? u.q.x0 + row / p.ratio : -1, row + 1 < tile.rows ? u.q.x0 + (row + 1) / p.ratio : -1};
        const bool has[2] = {row < tile.rows, row + 1 < tile.rows};
        float *to0 = a.scores + (((int64_t)u.r * p.heads + u.h) * a.rows + row) * a.tokens + g;
        float *to1 = to0 + a.tokens;
        float2 m = make_float2(kNone, kNone), l = make_float2(0.0f, 0.0f);
        int b, e;
        tile_range(u, tile, warp, &b, &e);
        for (; b < e; b += HB) {
            const int st = used % kSteps;
            if (alive) {
                const bool give_up = kTestTimeout && used == 1;
                if (give_up || !__all_sync(0xFFFFFFFFu, bar_wait(&sm.full[warp][st], (used / kSteps) & 1))) {
                    alive = false;   // `used` stays: the first step not waited for
                    int4_set_status(p.status, CG_ERR_TIMEOUT);
                } else {
                    ++used;
                }
            }
            if (alive) {
                auto token = [&](int vb) { return 16 * (vb < tile.span.sink ? vb : vb + tile.span.skip); };
                const uint8_t(&ring)[HB][B::kVCodes] = sm.ring[warp][st];
                float2 z[2][2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint8_t *blobs[P];
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        blobs[i] = ring[P * k + i];
                    few_scores<B, P>(blobs, ring[P * k + side], q, lane, z[k]);
                }
                // every row sees all of the step's tokens: from the first to the last, or to the last of the sinks
                const int t0 = token(b), t1 = token(b + HB - 1) + 15;
                const bool whole = t1 <= tile.x_lo && (tile.x_hi - t0 < window || t1 < p.a.sinks);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int vb = b + P * k + side, tok = token(vb);
                    if (!whole)
                        hide(p, tok, g, x, window, z[k]);
                    if (!(feeder.ahead >> (P * k + side) & 1))
                        z[k][0] = z[k][1] = make_float2(-INFINITY, -INFINITY);
                    if (vb < e && has[0]) {
                        to0[tok] = z[k][0].x;
                        to0[tok + 8] = z[k][1].x;
                    }
                    if (vb < e && has[1]) {
                        to1[tok] = z[k][0].y;
                        to1[tok + 8] = z[k][1].y;
                    }
                }
                // the maximum is raised only when a score exceeds it by 2^8
                const float top0 = fmaxf(fmaxf(z[0][0].x, z[0][1].x), fmaxf(z[1][0].x, z[1][1].x));
                const float top1 = fmaxf(fmaxf(z[0][0].y, z[0][1].y), fmaxf(z[1][0].y, z[1][1].y));
                if (fmaxf(top0 - m.x, top1 - m.y) > 8.0f) {
                    const float m0 = fmaxf(m.x, top0), m1 = fmaxf(m.y, top1);
                    l.x *= exp2_fast(m.x - m0);
                    l.y *= exp2_fast(m.y - m1);
                    m = make_float2(m0, m1);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    l.x += exp2_fast(z[k][0].x - m.x) + exp2_fast(z[k][1].x - m.x);
                    l.y += exp2_fast(z[k][0].y - m.y) + exp2_fast(z[k][1].y - m.y);
                }
            }
            __syncwarp();   // every lane has read the place
            if (alive)
                feeder.feed(p, count, warp, lane);
        }
        // ---- joined over the lanes of a row, the warps, and with other pieces in a second kernel
#pragma unroll
        for (int d = P == 2 ? 2 : 4; d < 32; d <<= 1) {
            const float2 om = make_float2(__shfl_xor_sync(0xFFFFFFFFu, m.x, d), __shfl_xor_sync(0xFFFFFFFFu, m.y, d));
            const float2 ol = make_float2(__shfl_xor_sync(0xFFFFFFFFu, l.x, d), __shfl_xor_sync(0xFFFFFFFFu, l.y, d));
            const float2 mx = make_float2(fmaxf(m.x, om.x), fmaxf(m.y, om.y));
            l.x = l.x * exp2_fast(m.x - mx.x) + ol.x * exp2_fast(om.x - mx.x);
            l.y = l.y * exp2_fast(m.y - mx.y) + ol.y * exp2_fast(om.y - mx.y);
            m = mx;
        }
        if (g == 0 && side == 0) {
            sm.m[warp][row] = m.x;
            sm.m[warp][row + 1] = m.y;
            sm.l[warp][row] = l.x;
            sm.l[warp][row + 1] = l.y;
        }
        __syncthreads();
        Unit end = now.u;
        const bool from_before = end.b0 > 0, goes_on = end.b1 < end.span.nb;
        if (threadIdx.x < 8) {
            const int i = threadIdx.x;
            float mx = kNone, ls = 0.0f;
            if (i < now.t.rows) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    mx = fmaxf(mx, sm.m[w][i]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    ls += sm.l[w][i] * exp2_fast(sm.m[w][i] - mx);
            }
            if (from_before || goes_on)
                a.parts[((int64_t)blockIdx.x * 2 + (from_before ? 0 : 1)) * 8 + i] = make_float2(mx, ls);
            else
                a.stats[((int64_t)end.h * a.slots + first_slot(p, end.r, end.q.row0)) * 8 + i] = row_stats_of(mx, ls);
        }
        const int64_t pos = now.pos + end.b1 - end.b0;
        __syncthreads();
        if (pos >= count)
            break;
        unit_next<8, WeighBatch>(p, count - pos, &end);
        if (lane == 0)
            now = {end, tile_of<8>(p, end), pos, 0, 0};
        __syncwarp();
    }
    // a wait that ran out: the copies still in flight must land before the block's memory goes
    if (!alive)
        for (; used < feeder.issued; ++used)
            bar_wait(&sm.full[warp][used % kSteps], (used / kSteps) & 1);
}

// Block c joins the unit that begins in block c of the first kernel and goes on behind it.
template <int RU>
__global__ void __launch_bounds__(kThreads) k_weigh_join(AttnArgs p, int pieces, WeighArgs a)
{
    grid_next();
    int64_t total, chunk;
    const int c = blockIdx.x;
    const Place at = schedule<RU, WeighBatch>(p, pieces, c + 1, 0, false, &total, &chunk);
    const int64_t border = (c + 1) * chunk;
    Unit u;
    if (border < total)
        unit_at<RU, WeighBatch>(p, at, 1, &u);
    grid_wait();
    if (border >= total || u.b0 == 0 || u.b0 > chunk)
        return;   // nothing there, or begins at the border, or before block c
    const int64_t end = border - u.b0 + u.span.nb;
    const int n = (int)((end + chunk - 1) / chunk) - c;
    const Tile tile = tile_of<RU>(p, u);
    const int slot = first_slot(p, u.r, u.q.row0) + tile.row0 / 8;
    // rows side by side, the parts shared by slices of the block
    constexpr int kSlices = kThreads / RU;
    __shared__ float2 slices[kSlices][RU];
    const int row = threadIdx.x % RU, slice = threadIdx.x / RU;
    float mx = kNone, l = 0.0f;
#pragma unroll 4
    for (int k = slice; k < n; k += kSlices) {
        const float2 part = a.parts[((int64_t)(c + k) * 2 + (k == 0)) * RU + row];
        const float up = fmaxf(mx, part.x);
        l = l * exp2_fast(mx - up) + part.y * exp2_fast(part.x - up);
        mx = up;
    }
    slices[slice][row] = make_float2(mx, l);
    __syncthreads();
    if (threadIdx.x < (tile.rows + 7) / 8 * 8) {
        for (int k = 0; k < kSlices; ++k)
            mx = fmaxf(mx, slices[k][row].x);
        l = 0.0f;
        for (int k = 0; k < kSlices; ++k)
            l = fmaf(slices[k][row].y, exp2_fast(slices[k][row].x - mx), l);
        a.stats[((int64_t)u.h * a.slots + slot) * 8 + row] = row_stats_of(mx, l);
    }
}

// -------------------------------------------------------------- sums of tokens

// A warp takes a blob of a (request, KV head), whose keys stay in its registers, over the rows that see any
// of its tokens: all of those, or where there are many a quarter, every fourth tile of 8.
template <typename B>
__global__ void __launch_bounds__(kThreads, 3) k_weigh_sums(AttnArgs p, WeighArgs a)
{
    constexpr int NW = B::kWords, NG = B::kGroups;
    __shared__ float parts[kWarps][16];
    const int lane = lane_once(), warp = threadIdx.x >> 5, t = lane & 3;
    const int window = p.a.window > 0 ? p.a.window : INT32_MAX;
    const int bpp = p.page_tokens / 16;
    grid_next();   // the kernels for many rows may come up: they work on other rows
    grid_wait();
    Items items = {0, 0};
    for (int64_t item = blockIdx.x;; item += gridDim.x) {
        AttnRequest q;
        int r, h, t0;
        if (!find_item(p, item, [&](const AttnRequest &x) { return x.rows > p.few_rows ? 0 : x.rows >= kManyRows ? 16 : kItemTokens; }, &items, &q,
                       &r, &h, &t0))
            return;
        const bool shared = q.rows >= kManyRows;   // the block's warps have the same tokens
        if (!shared) {
            t0 += 16 * warp;
            if (t0 >= q.kv)
                continue;
        }
        const int page = t0 / p.page_tokens, id = p.a.block_table[r * p.a.table_stride + page];
        const bool there = (unsigned)id < (unsigned)p.num_pages;
        if (!there)
            int4_set_status(p.status, CG_ERR_CORRUPT);
        const uint64_t blob = there ? ((uint64_t)id * p.heads + h) * bpp + (t0 - page * p.page_tokens) / 16 : 0;
        Keys<B> keys;
        load_keys<B>(p.layer + blob * B::kBytes, lane, &keys);
        // ---- rows that see any of the tokens
        const int64_t lo = min((int64_t)max(0, t0 - q.x0) * p.ratio, (int64_t)q.rows);
        int64_t hi = q.rows;
        if (p.a.window > 0 && t0 >= p.a.sinks)
            hi = min(hi, ((int64_t)t0 + 15 + window - q.x0) * p.ratio);
        const int step = shared ? kWarps : 1, i0 = (int)(lo / 8) + (shared ? warp : 0);
        const int i1 = hi < 0 ? 0 : (int)((hi + 7) / 8);
        const int64_t slot = (int64_t)h * a.slots + first_slot(p, r, q.row0);
        const uint4 *from = a.queries + slot * NW * 32 + lane;
        const float2 *factors = reinterpret_cast<const float2 *>(a.factors + slot * (NG + 1) * 8) + t;
        const float4 *stats = reinterpret_cast<const float4 *>(a.stats + slot * 8 + 2 * t);
        // Whether a row sees a token goes by rows: position x0 + row / ratio is at least x from row
        // (x - x0) ratio on. All 8 rows of a tile see the whole blob from row `from_row` on, up to `to_row`.
        auto row_of = [&](int64_t x) {   // (a tile's rows end at 2^31 - 8 at most)
            return (int)max(min((x - q.x0) * p.ratio, (int64_t)INT32_MAX), (int64_t)-1);
        };
        const int from_row = row_of((int64_t)t0 + 15);
        const int to_row = p.a.window == 0 || t0 + 15 < p.a.sinks ? INT32_MAX : row_of((int64_t)t0 + window);
        float total[2] = {}, sum[2] = {};
        int count = 0;
        auto scores = [&](int i, float4 *st, float2 (&z)[2]) {   // of row tile i
            Queries<B> rows;
            const uint4 *qi = from + (int64_t)i * (NW * 32);
            const float2 *fi = factors + (int64_t)i * ((NG + 1) * 4);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const uint4 v = qi[32 * w];
                rows.qf[w][0] = v.x, rows.qf[w][1] = v.y, rows.qf[w][2] = v.z, rows.qf[w][3] = v.w;
            }
            rows.rho = fi[0];
#pragma unroll
            for (int k = 0; k < NG; ++k)
                rows.sq[k] = fi[4 * (k + 1)];
            *st = stats[4 * (int64_t)i];
            scores_of<B>(keys, rows, make_float2(st->x, st->z), z);
        };
        auto add = [&](const float4 &st, const float2 (&z)[2]) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                sum[j] = fmaf(exp2_fast(z[j].y), st.w, fmaf(exp2_fast(z[j].x), st.y, sum[j]));
        };
        auto carry = [&]() {   // sums of sums: their roundings grow with the root of either's length
            if ((++count & 31) == 0)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    total[j] += sum[j];
                    sum[j] = 0.0f;
                }
        };
        // tiles [f0, f1) see the whole blob: two at a time, whose instructions mix
        const int f0 = from_row < 0 ? i0 : from_row > 8 * (int64_t)i1 ? i1 : max(i0, (from_row + 7) / 8);
        const int f1 = min(i1, to_row < 0 ? 0 : to_row / 8);
        for (int i = i0; i < i1; i += step) {
            if (i >= f0 && i + step < f1) {
                float4 st[2];
                float2 z[2][2];
                scores(i, &st[0], z[0]);
                scores(i + step, &st[1], z[1]);
                add(st[0], z[0]);
                add(st[1], z[1]);
                carry();
                i += step;
                continue;
            }
            float4 st;
            float2 z[2];
            scores(i, &st, z);
            if (i < f0 || i >= f1) {
                const int row = 8 * i + 2 * t;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t tok = t0 + 8 * j + (lane >> 2);
                    const int first = row_of(tok), end = p.a.window == 0 || tok < p.a.sinks ? INT32_MAX : row_of(tok + window);
                    if (row < first || row >= end)
                        z[j].x = -INFINITY;
                    if (row + 1 < first || row + 1 >= end)
                        z[j].y = -INFINITY;
                }
            }
            add(st, z);
            carry();
        }
        float mine = 0.0f;   // of token t0 + lane
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float s = total[j] + sum[j];
            s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
            s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
            s = __shfl_sync(0xFFFFFFFFu, s, 4 * (lane & 7));
            if (lane >> 3 == j)
                mine = there ? s : 0.0f;
        }
        if (shared) {
            if (lane < 16)
                parts[warp][lane] = mine;
            __syncthreads();
            if (lane < 16)
                mine = (parts[0][lane] + parts[1][lane]) + (parts[2][lane] + parts[3][lane]);
            __syncthreads();
        }
        const int tok = t0 + lane;
        if ((!shared || warp == 0) && lane < 16 && tok < q.kv) {
            const float had = a.w.in == nullptr ? 0.0f : a.w.in[r * a.w.in_request_stride + h * a.w.in_head_stride + tok];
            a.w.out[r * a.w.out_request_stride + h * a.w.out_head_stride + tok] = had + mine;
        }
    }
}

// The same from stored scores, kEach tokens to a thread, kRows rows at a time: as many loads in flight as a
// thread has registers for, whether a request has few rows and many tokens or the other way round.
template <int kEach, int kRows>
__global__ void __launch_bounds__(kThreads) k_weigh_apply(AttnArgs p, WeighArgs a)
{
    constexpr int kTokens = kEach * kThreads;
    grid_next();   // as there
    grid_wait();
    Items items = {0, 0};
    for (int64_t item = blockIdx.x;; item += gridDim.x) {
        AttnRequest q;
        int r, h, t0;
        if (!find_item(p, item, [&](const AttnRequest &x) { return x.rows > p.few_rows ? 0 : kTokens; }, &items, &q, &r, &h, &t0))
            return;
        t0 += threadIdx.x;
        const float *in = a.w.in == nullptr ? nullptr : a.w.in + r * a.w.in_request_stride + h * a.w.in_head_stride;
        float *out = a.w.out + r * a.w.out_request_stride + h * a.w.out_head_stride;
        const float *scores = a.scores + ((int64_t)r * p.heads + h) * a.rows * a.tokens + t0;
        const float4 *stats = reinterpret_cast<const float4 *>(a.stats + ((int64_t)h * a.slots + first_slot(p, r, q.row0)) * 8);
        // A blob has scores for the rows of a tile (of 8, 16 or 32, where the first pass has several) that
        // sees it, whose own rows may see less of it.
        const int64_t sinks = ((int64_t)p.a.sinks + 15) / 16 * 16;
        float had[kEach], sum[kEach], total[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int tok = t0 + k * kThreads;
            had[k] = in != nullptr && tok < q.kv ? in[tok] : 0.0f;
            sum[k] = total[k] = 0.0f;
        }
        for (int row = 0; row < q.rows; row += kRows) {
            // the tokens from `low` on (or below sinks) up to x_last: those of these rows
            const int x_first = q.x0 + row / p.ratio, x_last = q.x0 + min(row + kRows - 1, q.rows - 1) / p.ratio;
            const int64_t low = p.a.window > 0 ? (int64_t)x_first + 1 - p.a.window : 0;
            float z[kRows][kEach];
#pragma unroll
            for (int j = 0; j < kRows; ++j)
#pragma unroll
                for (int k = 0; k < kEach; ++k) {
                    const int tok = t0 + k * kThreads;
                    const bool seen = tok <= x_last && (tok >= low || tok < sinks) && row + j < q.rows;
                    z[j][k] = seen ? scores[(int64_t)(row + j) * a.tokens + k * kThreads] : -INFINITY;
                }
#pragma unroll
            for (int j = 0; j < kRows; j += 2) {
                // of two rows (0, 0 where only the second is not there)
                const float4 st = row + j < q.rows ? stats[(row + j) / 2] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < kEach; ++k)
                    sum[k] = fmaf(exp2_fast(z[j + 1][k] - st.z), st.w, fmaf(exp2_fast(z[j][k] - st.x), st.y, sum[k]));
            }
            if (row % 256 == 256 - kRows)   // sums of sums: their roundings grow with the root of either's length
#pragma unroll
                for (int k = 0; k < kEach; ++k) {
                    total[k] += sum[k];
                    sum[k] = 0.0f;
                }
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if (t0 + k * kThreads < q.kv)
                out[t0 + k * kThreads] = had[k] + (total[k] + sum[k]);
    }
}

template <int RU, typename Sh, typename B>
cudaError_t launch(void (*kernel)(AttnArgs, WeighArgs), int per_sm, const AttnArgs &p, const WeighArgs &a, bool stored,
                   cudaStream_t s)
{
    int sms = 0;
    cudaError_t err = attn_sm_count(&sms);
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Sh));
    if (err != cudaSuccess)
        return err;
    const int blocks = per_sm * sms < kMaxBlocks ? per_sm * sms : kMaxBlocks;
    kernel<<<blocks, kThreads, sizeof(Sh), s>>>(p, a);
    err = cudaGetLastError();
    if (err == cudaSuccess)
        err = launch_under(k_weigh_join<RU>, dim3(blocks), kThreads, 0, s, p, blocks, a);
    if (err != cudaSuccess)
        return err;
    if (stored && RU == 8)
        return launch_under(k_weigh_apply<4, 4>, dim3(8 * sms), kThreads, 0, s, p, a);
    if (stored)
        return launch_under(k_weigh_apply<1, 16>, dim3(16 * sms), kThreads, 0, s, p, a);
    return launch_under(k_weigh_sums<B>, dim3(3 * sms), kThreads, 0, s, p, a);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// How a call goes, and the parts of its workspace.
struct WeighSizes {
    int32_t slots, rows, tokens;   // rows of a request's KV head, and tokens, at most
    bool stored, tiles;            // scores are stored; requests with many rows go by tiles
    size_t parts, stats, queries, factors, scores, many;
    size_t bytes() const { return parts + stats + queries + factors + scores + many; }
};

// Requests with more rows than this go to the kernels for many (cachegen_weigh_many.cu), where there is room
// for their sums by row tiles. Here and there, 8 KV heads of 128: one request of 32768 tokens with 32 rows 41 us and
// 75, 48 rows 58 and 75, 64 rows 63 and 76; eight of 16384 with 64 rows 199 and 231, 64 of 1024 with 64 rows 118
// and 138. More rows here would read K again for each 32.
// Their seven launches take 31 us where there is little to do, so small batches stay here up to twice the rows: of 80
// rows, one head of 1024 tokens 25 and 31, eight of 4096 29 and 39, of 16384 55 and 53; of 128 rows, eight heads of
// 1024 tokens 31 and 35, of 4096 41 and 39.
constexpr int kTileRows = 64;
constexpr int64_t kFewPairs = 3 << 20;   // of a row and a token
// Bytes. Both bound the workspace and cost time: they go by what the table may hold (lengths are known to the GPU
// alone), and what passes them is read and computed again instead. Here and with room for
// them, 32 query and 8 KV heads of 128: a prompt of 32768 tokens (1.02 GB of sums) 49 ms and 18.7, one of 16384 has
// the room and takes 4.8; a chunk of 8192 of 16384 tokens under a table for 131072 9.1 ms and 3.7. 64 requests of
// 4096 to 8192 tokens, a query each, under a table for 65536 (537 MB of scores) 462 us and 88.
constexpr size_t kMostSums = (size_t)1 << 30;

constexpr size_t kMostScores = (size_t)256 << 20;
constexpr int32_t kMostTokens = INT32_MAX - 65535;

WeighSizes sizes_of(const cg_int4_cache *c, const cg_attention *a, const cg_token_weights *w)
{
    WeighSizes z = {};
    const int ratio = a->q_heads / c->num_heads;
    const int n = a->max_q_len > 0 && a->max_q_len < a->tokens ? a->max_q_len : a->tokens;
    const int64_t rows = (int64_t)n * ratio, limit = (int64_t)a->table_width * c->page_tokens;
    z.slots = (int32_t)((int64_t)a->tokens * ratio / 8 + a->requests + 1);
    z.tokens = (int32_t)(((limit < w->width ? limit : w->width) + 15) / 16 * 16);
    const size_t lists = (size_t)a->requests * c->num_heads;
    if (rows > kTileRows && (rows > 2 * kTileRows || (double)lists * rows * z.tokens > kFewPairs)) {
        z.many = weigh_many_workspace(c, a, z.tokens);
        z.tiles = z.many <= kMostSums;
        z.many = z.tiles ? align256(z.many) : 0;
    }
    z.rows = (int32_t)(z.tiles ? kTileRows : rows);
    // Scores are stored, and not computed again, where there is room for those that the batch can have: one
    // request of 32768 tokens, 128 rows and 8 heads (134 MB) took 115 us so and 123 computed again; with two of
    // 2048 tokens and 8192 rows each (1 GB), which the L2 does not hold, either took as long.
    z.stored = lists == 0 || (size_t)z.rows * z.tokens <= kMostScores / sizeof(float) / lists;
    z.parts = align256((size_t)kMaxBlocks * 2 * 32 * sizeof(float2));
    z.stats = align256((size_t)c->num_heads * z.slots * 8 * sizeof(float2));
    if (z.stored) {
        z.scores = align256(lists * z.rows * z.tokens * sizeof(float));
    } else {
        z.queries = align256((size_t)c->num_heads * z.slots * (c->head_size / 32) * 512);
        z.factors = align256((size_t)c->num_heads * z.slots * (c->head_size / c->group + 1) * 32);
    }
    return z;
}

cg_status check_weights(const cg_token_weights *w)
{
    if (w->width < 0 || w->out_request_stride < 0 || w->out_head_stride < 0 ||
        (w->in != nullptr && (w->in_request_stride < 0 || w->in_head_stride < 0)))
        return CG_ERR_INVALID_ARG;
    return CG_OK;
}

}  // namespace

extern "C" cg_status cg_int4_weigh_workspace(const cg_int4_cache *c, const cg_attention *a,
                                             const cg_token_weights *w, size_t *bytes)
{
    if (c == nullptr || a == nullptr || w == nullptr || bytes == nullptr)
        return CG_ERR_INVALID_ARG;
    cg_status st = attn_check_sizes(c, a);
    if (st == CG_OK)
        st = check_weights(w);
    // (a block's last tokens count past a request's)
    if (st == CG_OK && (int64_t)a->table_width * c->page_tokens > kMostTokens && w->width > kMostTokens)
        st = CG_ERR_UNSUPPORTED;
    if (st == CG_OK)
        *bytes = sizes_of(c, a, w).bytes();
    return st;
}

extern "C" cg_status cg_int4_weigh(const cg_int4_cache *c, int32_t layer, const cg_attention *a,
                                   const cg_token_weights *w, void *workspace, size_t workspace_bytes,
                                   cg_stream_t stream)
{
    cg_status st = int4_check(c);
    if (st != CG_OK)
        return st;
    size_t need = 0;
    st = cg_int4_weigh_workspace(c, a, w, &need);
    if (st != CG_OK)
        return st;
    if (layer < 0 || layer >= c->num_layers)
        return CG_ERR_INVALID_ARG;
    if (a->requests == 0)
        return CG_OK;
    st = attn_check_arrays(a, false);
    if (st != CG_OK || (w->out == nullptr && w->width > 0) || !int4_aligned(w->in, 4) || !int4_aligned(w->out, 4) ||
        !int4_aligned(workspace, 256))
        return CG_ERR_INVALID_ARG;
    if (w->in != nullptr && w->in == w->out &&
        (w->in_request_stride != w->out_request_stride || w->in_head_stride != w->out_head_stride))
        return CG_ERR_INVALID_ARG;
    if (workspace_bytes < need || workspace == nullptr)
        return CG_ERR_CAPACITY;
    AttnArgs p = attn_args(c, layer, a);
    const WeighSizes z = sizes_of(c, a, w);
    p.few_rows = z.tiles ? kTileRows : INT32_MAX;
    // short units are not strung together, as behind shared tokens (3 requests of 11 queries and 12 tokens, 8
    // heads: 103 us with, 17 without)
    p.least_unit = 16;
    if (p.kv_limit > w->width)
        p.kv_limit = w->width;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    auto take = [&](size_t n) {
        uint8_t *at = ws;
        ws += n;
        return at;
    };
    WeighArgs args;
    args.w = *w;
    args.slots = z.slots;
    args.rows = z.rows;
    args.tokens = z.tokens;
    args.parts = reinterpret_cast<float2 *>(take(z.parts));
    args.stats = reinterpret_cast<float2 *>(take(z.stats));
    args.queries = reinterpret_cast<uint4 *>(take(z.queries));
    args.factors = reinterpret_cast<float *>(take(z.factors));
    args.scores = reinterpret_cast<float *>(take(z.scores));
    args.sums = nullptr;
    args.tiles = 0;
    args.taken = z.tiles ? weigh_many_taken(ws) : nullptr;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err = int4_dispatch(c->head_size, c->group, [&](auto blob) {
        using B = decltype(blob);
        if (z.stored && z.rows <= 8)
            return z.rows <= 4 ? launch<8, FewShared<B, 2>, B>(k_weigh_few<B, 2>, kFewBlocks, p, args, true, s)
                               : launch<8, FewShared<B, 1>, B>(k_weigh_few<B, 1>, kFewBlocks, p, args, true, s);
        if (z.stored && z.rows <= 16)
            return launch<16, StatShared<B, 2>, B>(k_weigh_stats<B, 2, true>, kStatBlocks, p, args, true, s);
        return launch<32, StatShared<B, 4>, B>(z.stored ? k_weigh_stats<B, 4, true> : k_weigh_stats<B, 4, false>,
                                               kStatBlocks, p, args, z.stored, s);
    });
    if (err == cudaSuccess && z.tiles)
        err = weigh_many_launch(p, args, c, ws, s);
    return err == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

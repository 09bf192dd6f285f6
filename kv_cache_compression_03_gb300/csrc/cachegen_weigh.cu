// cg_int4_weigh: the attention weight that every token of the 4-bit cache gets, sum over a
// request's new tokens i and the query heads g of a KV head of p_igj = 2^(z_igj - m_ig) / l_ig,
// z the scores in powers of two.
//
// The maximum m and the sum l of a row are over all of its tokens, so K is met twice: once for
// m and l of every row, once for the sums over the rows of every token.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cg_few.h"

namespace {

constexpr int kRing = 8;           // blobs in a warp's ring
constexpr int kItemTokens = 128;   // of a block in the second pass, 32 to a warp
constexpr int kApplyTokens = 512;  // of a block in the second pass over stored scores
constexpr int kMaxBlocks = 960;    // of the first pass

struct WeighArgs {
    cg_token_weights w;
    float2 *parts;       // [block][2][rows of a tile]: m, l of pieces; slot 0 began in an earlier block
    float2 *stats;       // [heads][slots][8]: m, 1 / l (0, 0: no such row, or it sees nothing)
    int32_t slots;       // row tiles of 8 of all requests
    // what the second pass works from, either
    uint4 *queries;      // [heads][slots][words][32]: the second factor, as a lane of the warp has it
    float *factors;      // [heads][slots][groups + 1][8]: rho, sq
    // or
    float *scores;       // [requests][heads][rows][tokens]
    int32_t rows, tokens;
};

// Row tiles of 8 of request r lie from here on. (Of a rows before it and b of its own, ceil(b / 8)
// is at most floor((a + b) / 8) - floor(a / 8) + 1.)
__device__ __forceinline__ int32_t first_slot(const AttnArgs &p, int r, int32_t row0)
{
    return (int32_t)((int64_t)row0 * p.ratio / 8) + r;
}

// ------------------------------------------------------------------- scores

// With mid = lo + 8 s and m = n - 8 in [-8, 7], q.k^ = sum_g s_g (q.m)_g + mid_g (sum q)_g. Where a
// few channels of a group are large, s and lo follow those and the others' codes lie near 8:
// q.n and lo (sum q) would be large and cancel (an error of 1.3e-5 in the weights, of 2e-7 so). The
// products of bf16 pairs are exact, everything else is fp32.

// Codes i and i + 4 of a word, less 8, as a bf16 pair: exact out of the mantissa of 128 + n.
__device__ __forceinline__ uint32_t centred(uint32_t w, int i)
{
    const uint32_t x = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    uint32_t y;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x43084308u));
    return y;
}

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
__device__ __forceinline__ void load_keys(const uint8_t *blob, Keys<B> *to)
{
    constexpr int D = B::kD, NW = B::kWords, NG = B::kGroups;
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
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

// Scores in powers of two: z[j] are token g + 8 j's with rows 2t and 2t + 1.
template <typename B>
__device__ __forceinline__ void scores_of(const Keys<B> &k, const Queries<B> &q, float2 (&z)[2])
{
    constexpr int NW = B::kWords, NG = B::kGroups, WPG = NW / NG;
    float2 y[2];
#pragma unroll
    for (int gi = 0; gi < NG; ++gi) {
        float acc[4];
#pragma unroll
        for (int w = gi * WPG; w < (gi + 1) * WPG; ++w)
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                if (w == gi * WPG && i == 0)
                    mma16816_first(acc, k.a[w][0], k.a[w][1], k.a[w][2], k.a[w][3], q.qf[w][0], q.qf[w][1]);
                else
                    mma16816(acc, k.a[w][2 * i], k.a[w][2 * i + 1], k.a[w][2 * i + 2], k.a[w][2 * i + 3], q.qf[w][i],
                             q.qf[w][i + 1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 s = make_float2(k.s[j][gi], k.s[j][gi]), mid = make_float2(k.mid[j][gi], k.mid[j][gi]);
            const float2 x = make_float2(acc[2 * j], acc[2 * j + 1]);
            y[j] = gi ? fma2(s, x, y[j]) : make_float2(s.x * x.x, s.y * x.y);
            z[j] = gi ? fma2(mid, q.sq[gi], z[j]) : make_float2(mid.x * q.sq[0].x, mid.y * q.sq[0].y);
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
        z[j] = fma2(y[j], q.rho, z[j]);
}

// Where not every token is seen by every row: -inf for those that are not. x: positions of the rows.
__device__ __forceinline__ void hide(const AttnArgs &p, int tok, const int (&x)[2], int window, float2 (&z)[2])
{
    const int g = (threadIdx.x & 31) >> 2;
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

// -------------------------------------------------------- maximum and sum

template <typename B, int NT>
struct StatShared {
    uint8_t ring[kWarps][kRing][B::kVCodes];   // the K half of blobs
    float m[kWarps][8 * NT], l[kWarps][8 * NT];
    uint64_t full[kWarps][kRing];
};

__device__ __forceinline__ float2 row_stats_of(float m, float l)
{
    return l == 0.0f ? make_float2(0.0f, 0.0f) : make_float2(m, 1.0f / l);
}

// Blocks of the first pass on an SM.
constexpr int stat_blocks(int NT) { return NT == 1 ? 4 : NT == 2 ? 3 : 2; }

// kStored: scores are left for the second pass, else the queries.
template <typename B, int NT, bool kStored>
__global__ void __launch_bounds__(kThreads, stat_blocks(NT)) k_weigh_stats(AttnArgs p, WeighArgs a)
{
    using S = StatShared<B, NT>;
    constexpr int NW = B::kWords, NG = B::kGroups, RU = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;

    grid_next();
    if (lane == 0)
        for (int i = 0; i < kRing; ++i)
            bar_init(&sm.full[warp][i], 1);
    bar_init_fence();
    int64_t total, chunk;
    const Place at = schedule<RU>(p, gridDim.x, blockIdx.x, 0, blockIdx.x == 0, &total, &chunk);
    const int64_t begin = blockIdx.x * chunk;
    if (begin >= total)
        return;
    const int64_t count = (begin + chunk < total ? begin + chunk : total) - begin;
    const int bpp = p.page_tokens / 16;
    // ---- the warp's copies, some blobs ahead of it: 32 are looked up at once, one by each lane,
    // which then issues its own blob's copy
    Unit first;
    unit_at<RU>(p, at, count, &first);
    Unit fu = first;
    Tile ft = tile_of<RU>(p, fu);
    int64_t f_pos = fu.b1 - fu.b0;
    int f_b, f_e, f_i = 0, f_n = 0;
    tile_range(fu, ft, warp, &f_b, &f_e);
    uint32_t f_off = 0, f_ok = 0, issued = 0, ahead = 0;
    auto feed = [&]() {
        ahead >>= 1;
        if (f_i >= f_n) {
            while (f_b >= f_e) {
                if (f_pos >= count)
                    return;
                unit_next<RU>(p, count - f_pos, &fu);
                ft = tile_of<RU>(p, fu);
                f_pos += fu.b1 - fu.b0;
                tile_range(fu, ft, warp, &f_b, &f_e);
            }
            f_i = 0;
            f_n = f_e - f_b < 32 ? f_e - f_b : 32;
            int id = -1;
            if (lane < f_n) {
                const int vb = f_b + lane, ab = vb < ft.span.sink ? vb : vb + ft.span.skip;
                const int page = ab / bpp;
                id = p.a.block_table[fu.r * p.a.table_stride + page];
                if ((unsigned)id >= (unsigned)p.num_pages)
                    int4_set_status(p.status, CG_ERR_CORRUPT);
                f_off = (((uint32_t)id * p.heads + fu.h) * bpp + (ab - page * bpp)) * (B::kBytes / 128);
            }
            f_ok = __ballot_sync(0xFFFFFFFFu, (unsigned)id < (unsigned)p.num_pages);
            f_b += f_n;
        }
        const int st = issued % kRing;
        if (lane == f_i) {
            uint64_t *bar = &sm.full[warp][st];
            if (f_ok >> lane & 1) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                bar_expect(bar, B::kVCodes);
                bulk_copy(sm.ring[warp][st], p.layer + (uint64_t)f_off * 128, B::kVCodes, bar);
            } else {
                bar_arrive(bar);
            }
        }
        ahead |= (f_ok >> f_i & 1) << (kRing - 1);
        ++f_i;
        ++issued;
    };
    __syncwarp();
    for (int i = 0; i < kRing; ++i)
        feed();

    const int window = p.a.window > 0 ? p.a.window : INT32_MAX;
    bool alive = true;               // no wait has run out
    uint32_t used = 0;
    Unit u = first;
    int64_t pos = 0;
    for (;;) {
        const Tile tile = tile_of<RU>(p, u);
        const int slot = first_slot(p, u.r, u.q.row0) + tile.row0 / 8;
        Queries<B> q[NT];
        int x[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            load_rows<B>(p, u.q, u.h, tile.row0 + 8 * nt, &q[nt]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int in = 8 * nt + 2 * t + j;
                x[nt][j] = in < tile.rows ? u.q.x0 + (tile.row0 + in) / p.ratio : -1;
            }
            if (!kStored && u.b0 == 0 && warp == 0 && 8 * nt < tile.rows) {   // by the unit's first piece
                const int64_t at_slot = (int64_t)u.h * a.slots + slot + nt;
                uint4 *to = a.queries + at_slot * NW * 32 + lane;
#pragma unroll
                for (int w = 0; w < NW; ++w)
                    to[32 * w] = make_uint4(q[nt].qf[w][0], q[nt].qf[w][1], q[nt].qf[w][2], q[nt].qf[w][3]);
                if (g == 0) {
                    float2 *f = reinterpret_cast<float2 *>(a.factors + at_slot * (NG + 1) * 8) + t;
                    f[0] = q[nt].rho;
#pragma unroll
                    for (int i = 0; i < NG; ++i)
                        f[4 * (i + 1)] = q[nt].sq[i];
                }
            }
        }
        // each lane keeps a maximum and a sum of its own, over tokens g and g + 8 of the blobs
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[nt][j] = kNone;
                l[nt][j] = 0.0f;
            }
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
            if (alive && (ahead & 1)) {
                Keys<B> k;
                load_keys<B>(sm.ring[warp][st], &k);
                const int tok = 16 * (b < tile.span.sink ? b : b + tile.span.skip);
                const bool whole = tok + 15 <= tile.x_lo && (tile.x_hi - tok < window || tok + 15 < p.a.sinks);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float2 z[2];
                    scores_of<B>(k, q[nt], z);
                    if (!whole)
                        hide(p, tok, x[nt], window, z);
                    if (kStored) {
                        float *to = a.scores + ((int64_t)u.r * p.heads + u.h) * a.rows * a.tokens + tok + g;
                        const int row = 2 * t;
                        if (row < tile.rows) {
                            to[(int64_t)row * a.tokens] = z[0].x;
                            to[(int64_t)row * a.tokens + 8] = z[1].x;
                        }
                        if (row + 1 < tile.rows) {
                            to[(int64_t)(row + 1) * a.tokens] = z[0].y;
                            to[(int64_t)(row + 1) * a.tokens + 8] = z[1].y;
                        }
                    }
                    // raised only when a score exceeds it by 2^8
                    const float2 top = make_float2(fmaxf(z[0].x, z[1].x), fmaxf(z[0].y, z[1].y));
                    if (top.x > m[nt][0] + 8.0f) {
                        l[nt][0] *= exp2_fast(m[nt][0] - top.x);
                        m[nt][0] = top.x;
                    }
                    if (top.y > m[nt][1] + 8.0f) {
                        l[nt][1] *= exp2_fast(m[nt][1] - top.y);
                        m[nt][1] = top.y;
                    }
                    l[nt][0] += exp2_fast(z[0].x - m[nt][0]) + exp2_fast(z[1].x - m[nt][0]);
                    l[nt][1] += exp2_fast(z[0].y - m[nt][1]) + exp2_fast(z[1].y - m[nt][1]);
                }
            } else if (kStored && alive) {   // a page that is not there
                const int tok = 16 * (b < tile.span.sink ? b : b + tile.span.skip);
                float *to = a.scores + ((int64_t)u.r * p.heads + u.h) * a.rows * a.tokens + tok;
                for (int i = lane; i < 16 * tile.rows; i += 32)
                    to[(int64_t)(i / 16) * a.tokens + i % 16] = -INFINITY;
            }
            __syncwarp();   // every lane has read the place
            if (alive)
                feed();
        }
        // ---- joined over the lanes of a row, the warps, and with other pieces in a second kernel
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    const float om = __shfl_xor_sync(0xFFFFFFFFu, m[nt][j], d);
                    const float ol = __shfl_xor_sync(0xFFFFFFFFu, l[nt][j], d), mx = fmaxf(m[nt][j], om);
                    l[nt][j] = l[nt][j] * exp2_fast(m[nt][j] - mx) + ol * exp2_fast(om - mx);
                    m[nt][j] = mx;
                }
                if (g == 0) {
                    sm.m[warp][8 * nt + 2 * t + j] = m[nt][j];
                    sm.l[warp][8 * nt + 2 * t + j] = l[nt][j];
                }
            }
        __syncthreads();
        const bool from_before = u.b0 > 0, goes_on = u.b1 < u.span.nb;
        if (tid < RU) {
            float mx = kNone, ls = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                mx = fmaxf(mx, sm.m[w][tid]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                ls += sm.l[w][tid] * exp2_fast(sm.m[w][tid] - mx);
            if (tid >= tile.rows)
                ls = 0.0f;
            if (from_before || goes_on)
                a.parts[((int64_t)blockIdx.x * 2 + (from_before ? 0 : 1)) * RU + tid] = make_float2(mx, ls);
            else if (tid < (tile.rows + 7) / 8 * 8)
                a.stats[((int64_t)u.h * a.slots + slot) * 8 + tid] = row_stats_of(mx, ls);
        }
        __syncthreads();
        pos += u.b1 - u.b0;
        if (pos >= count)
            break;
        unit_next<RU>(p, count - pos, &u);
    }
    // a wait that ran out: the copies still in flight must land before the block's memory goes
    if (!alive)
        for (; used < issued; ++used)
            bar_wait(&sm.full[warp][used % kRing], (used / kRing) & 1);
}

// Block c joins the unit that begins in block c of the first kernel and goes on behind it.
template <int RU>
__global__ void __launch_bounds__(kThreads) k_weigh_join(AttnArgs p, int pieces, WeighArgs a)
{
    grid_next();
    int64_t total, chunk;
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Place at = schedule<RU>(p, pieces, c + 1, 0, false, &total, &chunk);
    const int64_t border = (c + 1) * chunk;
    Unit u;
    if (border < total)
        unit_at<RU>(p, at, 1, &u);
    grid_wait();
    if (border >= total || u.b0 == 0 || u.b0 > chunk)
        return;   // nothing there, or begins at the border, or before block c
    const int64_t end = border - u.b0 + u.span.nb;
    const int n = (int)((end + chunk - 1) / chunk) - c;
    const Tile tile = tile_of<RU>(p, u);
    const int slot = first_slot(p, u.r, u.q.row0) + tile.row0 / 8;
    for (int row = warp; row < (tile.rows + 7) / 8 * 8; row += kWarps) {
        float mx = kNone, l = 0.0f;
        for (int k = lane; k < n; k += 32)
            mx = fmaxf(mx, a.parts[((int64_t)(c + k) * 2 + (k == 0)) * RU + row].x);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
        for (int k = lane; k < n; k += 32) {
            const float2 part = a.parts[((int64_t)(c + k) * 2 + (k == 0)) * RU + row];
            l = fmaf(part.y, exp2_fast(part.x - mx), l);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
            l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        if (lane == 0)
            a.stats[((int64_t)u.h * a.slots + slot) * 8 + row] = row_stats_of(mx, l);
    }
}

// -------------------------------------------------------------- sums of tokens

// Items of `each` tokens of a (request, KV head), those of all heads of the first tokens first. One
// warp finds its item, going on from where the last call stood (32 requests from r0 on, `before`
// items ahead of them): false when there are no more. Requests without rows have items too.
struct Items {
    int r0;
    int64_t before;
};

__device__ __forceinline__ bool find_item(const AttnArgs &p, int64_t item, int each, Items *at, AttnRequest *q, int *r,
                                          int *h, int *tok)
{
    const int lane = threadIdx.x & 31;
    for (;; at->r0 += 32) {
        if (at->r0 >= p.a.requests)
            return false;
        uint32_t error;
        int64_t w = 0;
        if (at->r0 + lane < p.a.requests) {
            attn_request(p, at->r0 + lane, q, &error);
            if (error == CG_OK)
                w = (int64_t)((q->kv + each - 1) / each) * p.heads;
        }
        int64_t inc = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
            if (lane >= d)
                inc += o;
        }
        const int64_t start = at->before + inc - w;
        const uint32_t mine = __ballot_sync(0xFFFFFFFFu, item >= start && item < start + w);
        if (mine == 0) {
            at->before += __shfl_sync(0xFFFFFFFFu, inc, 31);
            continue;
        }
        const int src = __ffs(mine) - 1;
        const int64_t off = __shfl_sync(0xFFFFFFFFu, item - start, src);
        *r = at->r0 + src;
        attn_request(p, *r, q, &error);
        *h = (int)(off % p.heads);
        *tok = (int)(off / p.heads) * each;
        return true;
    }
}

// A block to 128 tokens of a (request, KV head), two blobs to a warp, over all rows that see any
// of them.
template <typename B>
__global__ void __launch_bounds__(kThreads, 3) k_weigh_sums(AttnArgs p, WeighArgs a)
{
    constexpr int NW = B::kWords, NG = B::kGroups;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int window = p.a.window > 0 ? p.a.window : INT32_MAX;
    const int bpp = p.page_tokens / 16;
    grid_wait();
    Items items = {0, 0};
    for (int64_t item = blockIdx.x;; item += gridDim.x) {
        AttnRequest q;
        int r, h, t0;
        if (!find_item(p, item, kItemTokens, &items, &q, &r, &h, &t0))
            return;
        t0 += 32 * warp;
        if (t0 >= q.kv)
            continue;
        Keys<B> keys[2];
        bool there[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int tok = min(t0 + 16 * b, q.kv - 1) & ~15, page = tok / p.page_tokens;
            const int id = p.a.block_table[r * p.a.table_stride + page];
            there[b] = (unsigned)id < (unsigned)p.num_pages;
            if (!there[b])
                int4_set_status(p.status, CG_ERR_CORRUPT);
            // (a blob behind the last token is the one before it again: its sums are not written)
            const uint64_t blob = there[b] ? ((uint64_t)id * p.heads + h) * bpp + (tok - page * p.page_tokens) / 16 : 0;
            load_keys<B>(p.layer + blob * B::kBytes, &keys[b]);
        }
        // ---- rows that see any of the warp's tokens
        const int64_t lo = min((int64_t)max(0, t0 - q.x0) * p.ratio, (int64_t)q.rows);
        int64_t hi = q.rows;
        if (p.a.window > 0 && t0 >= p.a.sinks)
            hi = min(hi, ((int64_t)t0 + 31 + window - q.x0) * p.ratio);
        const int i0 = (int)(lo / 8), i1 = hi < 0 ? 0 : (int)((hi + 7) / 8);
        const int64_t slot = (int64_t)h * a.slots + first_slot(p, r, q.row0);
        float total[2][2] = {}, sum[2][2] = {};
        for (int i = i0; i < i1; ++i) {
            Queries<B> rows;
            const uint4 *from = a.queries + (slot + i) * NW * 32 + lane;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const uint4 v = from[32 * w];
                rows.qf[w][0] = v.x, rows.qf[w][1] = v.y, rows.qf[w][2] = v.z, rows.qf[w][3] = v.w;
            }
            const float2 *f = reinterpret_cast<const float2 *>(a.factors + (slot + i) * (NG + 1) * 8) + t;
            rows.rho = f[0];
#pragma unroll
            for (int k = 0; k < NG; ++k)
                rows.sq[k] = f[4 * (k + 1)];
            const float4 st = *reinterpret_cast<const float4 *>(a.stats + (slot + i) * 8 + 2 * t);
            const int x_lo = q.x0 + 8 * i / p.ratio, x_hi = q.x0 + min(8 * i + 7, q.rows - 1) / p.ratio;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int tok = t0 + 16 * b;
                float2 z[2];
                scores_of<B>(keys[b], rows, z);
                if (!(tok + 15 <= x_lo && (x_hi - tok < window || tok + 15 < p.a.sinks))) {
                    const int row = 8 * i + 2 * t;
                    const int x[2] = {row < q.rows ? q.x0 + row / p.ratio : -1,
                                      row + 1 < q.rows ? q.x0 + (row + 1) / p.ratio : -1};
                    hide(p, tok, x, window, z);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    sum[b][j] = fmaf(exp2_fast(z[j].y - st.z), st.w, fmaf(exp2_fast(z[j].x - st.x), st.y, sum[b][j]));
            }
            if ((i & 31) == 31)   // sums of sums: their roundings grow with the root of either's length
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        total[b][j] += sum[b][j];
                        sum[b][j] = 0.0f;
                    }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float s = total[b][j] + sum[b][j];
                s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
                s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
                const int tok = t0 + 16 * b + 8 * j + g;
                if (t == 0 && tok < q.kv) {
                    const float had = a.w.in == nullptr ? 0.0f
                                                        : a.w.in[r * a.w.in_request_stride + h * a.w.in_head_stride + tok];
                    a.w.out[r * a.w.out_request_stride + h * a.w.out_head_stride + tok] = there[b] ? had + s : had;
                }
            }
    }
}

// The same from stored scores, a thread to a token.
__global__ void __launch_bounds__(kThreads) k_weigh_apply(AttnArgs p, WeighArgs a)
{
    constexpr int kEach = kApplyTokens / kThreads;
    grid_wait();
    Items items = {0, 0};
    for (int64_t item = blockIdx.x;; item += gridDim.x) {
        AttnRequest q;
        int r, h, t0;
        if (!find_item(p, item, kApplyTokens, &items, &q, &r, &h, &t0))
            return;
        const float *in = a.w.in == nullptr ? nullptr : a.w.in + r * a.w.in_request_stride + h * a.w.in_head_stride;
        float *out = a.w.out + r * a.w.out_request_stride + h * a.w.out_head_stride;
        const float *scores = a.scores + ((int64_t)r * p.heads + h) * a.rows * a.tokens;
        const float2 *stats = a.stats + ((int64_t)h * a.slots + first_slot(p, r, q.row0)) * 8;
        // blobs that no row sees have no scores
        const int x_last = q.x0 + (q.rows > 0 ? (q.rows - 1) / p.ratio : 0);
        const int64_t low = p.a.window > 0 ? ((int64_t)q.x0 + 1 - p.a.window) / 16 * 16 : 0;
        const int64_t sinks = ((int64_t)p.a.sinks + 15) / 16 * 16;
        float sum[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            sum[k] = 0.0f;
        for (int row = 0; row < q.rows; ++row) {
            const float2 st = stats[row];
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int tok = t0 + k * kThreads + threadIdx.x;
                if (tok <= x_last && (tok >= low || tok < sinks))
                    sum[k] = fmaf(exp2_fast(scores[(int64_t)row * a.tokens + tok] - st.x), st.y, sum[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int tok = t0 + k * kThreads + threadIdx.x;
            if (tok < q.kv)
                out[tok] = (in == nullptr ? 0.0f : in[tok]) + sum[k];
        }
    }
}

template <typename B, int NT, bool kStored>
cudaError_t launch(const AttnArgs &p, const WeighArgs &a, cudaStream_t s)
{
    using Sh = StatShared<B, NT>;
    int sms = 0;
    cudaError_t err = attn_sm_count(&sms);
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(k_weigh_stats<B, NT, kStored>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)sizeof(Sh));
    if (err != cudaSuccess)
        return err;
    const int blocks = stat_blocks(NT) * sms < kMaxBlocks ? stat_blocks(NT) * sms : kMaxBlocks;
    k_weigh_stats<B, NT, kStored><<<blocks, kThreads, sizeof(Sh), s>>>(p, a);
    err = cudaGetLastError();
    if (err == cudaSuccess)
        err = launch_under(k_weigh_join<8 * NT>, dim3(blocks), kThreads, 0, s, p, blocks, a);
    if (err != cudaSuccess)
        return err;
    if (kStored)
        return launch_under(k_weigh_apply, dim3(8 * sms), kThreads, 0, s, p, a);
    return launch_under(k_weigh_sums<B>, dim3(3 * sms), kThreads, 0, s, p, a);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// How a call goes, and the parts of its workspace.
struct WeighSizes {
    int32_t slots, rows, tokens;   // rows of a request's KV head, and tokens, at most
    bool stored;
    size_t parts, stats, queries, factors, scores;
    size_t bytes() const { return parts + stats + queries + factors + scores; }
};

constexpr size_t kMostScores = (size_t)256 << 20;   // bytes

WeighSizes sizes_of(const cg_int4_cache *c, const cg_attention *a, const cg_token_weights *w)
{
    WeighSizes z = {};
    const int ratio = a->q_heads / c->num_heads;
    const int n = a->max_q_len > 0 && a->max_q_len < a->tokens ? a->max_q_len : a->tokens;
    const int64_t rows = (int64_t)n * ratio, limit = (int64_t)a->table_width * c->page_tokens;
    z.slots = (int32_t)((int64_t)a->tokens * ratio / 8 + a->requests + 1);
    z.rows = (int32_t)(rows < INT32_MAX ? rows : INT32_MAX);
    z.tokens = (int32_t)(((limit < w->width ? limit : w->width) + 15) / 16 * 16);
    // of up to 8 rows a token's scores are fewer bytes than its keys and are not computed again; a batch
    // with more room in its tables than this goes without
    const size_t lists = (size_t)a->requests * c->num_heads;
    z.stored = z.rows <= 8 && (lists == 0 || (size_t)z.rows * z.tokens <= kMostScores / sizeof(float) / lists);
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
    if (a->requests == 0 || w->width == 0)
        return CG_OK;
    st = attn_check_arrays(a, false);
    if (st != CG_OK || w->out == nullptr || !int4_aligned(w->in, 4) || !int4_aligned(w->out, 4) ||
        !int4_aligned(workspace, 256))
        return CG_ERR_INVALID_ARG;
    if (w->in == w->out &&
        (w->in_request_stride != w->out_request_stride || w->in_head_stride != w->out_head_stride))
        return CG_ERR_INVALID_ARG;
    if (workspace_bytes < need || workspace == nullptr)
        return CG_ERR_CAPACITY;
    AttnArgs p = attn_args(c, layer, a);
    p.few_rows = INT32_MAX;
    if (p.kv_limit > w->width)
        p.kv_limit = w->width;
    const WeighSizes z = sizes_of(c, a, w);
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
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = int4_dispatch(c->head_size, c->group, [&](auto blob) {
        using B = decltype(blob);
        if (z.rows <= 8)
            return z.stored ? launch<B, 1, true>(p, args, s) : launch<B, 1, false>(p, args, s);
        return z.rows <= 16 ? launch<B, 2, false>(p, args, s) : launch<B, 4, false>(p, args, s);
    });
    return err == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

// Attention over the 4-bit cache for many query rows (prompts, chunks of
// them, more than a few drafted tokens): 4 D flops per query head and visible
// pair, bound by the tensor cores in the limit.
//
// One block per 256 rows of a (request, KV head), rows being the head's query
// heads of one token after another: the group shares its K and V, and codes are
// expanded once for 256 rows, beside 2 x 2 products of 128 x 128 x 128. Per tile of
// 128 tokens, S = Q K^T and O += P V by tcgen05.mma (128 x 128 x 16, bf16 in, fp32
// accumulators in tensor memory), two row tiles of 128 in turn, so that the
// softmax of one runs under the products of the other:
//   warps 0-3, 4-7   softmax of row tile 0, 1: a thread owns a row. It reads S
//                    from tensor memory, keeps the running maximum and sum
//                    and writes P as bf16 over S, where the next product reads
//                    it, half a tile at a time. O is rescaled in place, only when
//                    a maximum rises by more than 2^8.
//   warps 8-15       4-bit codes to bf16 tiles in shared memory, a blob of 16 tokens
//                    at a time: K as rows of tokens, V transposed (rows of channels)
//   warp 16          finds the units and copies their blobs into a ring, four lanes at once
//   warp 17          one thread issues all products
// K rows keep the channel order in which a word's codes come apart (0 4 1 5 2 6
// 3 7 of each eight); Q is laid out alike. V's words hold a pair of tokens each, as
// the transposed rows need them. Tensor memory is full: two S, two O, 128 columns each.
//
// At most half as many units as blocks: each is cut along its tokens, and a second kernel
// joins the pieces in their order; with one row tile the softmax groups take turns at the
// tiles of tokens. More units are dealt to the blocks in turns, the longest first.
//
// Roundings: k^ and v^ = lo + s n to bf16 (one rounding, 2^-8 relative at most), p to
// bf16: the products need 16-bit operands, and bf16 keeps the range of s and lo. Against
// 64 bits the error is 0.0026 to 0.0039 of the result (prompt 0.0034, drafts 0.0038; the largest
// part is k^'s, which moves scores), where rounding the result alone gives 0.0017. Scores,
// sums and O stay in fp32.
//
// Measured (8 KV heads of 128, 32 query heads, groups of 32): a prompt of 8192 tokens 547 us,
// 1005 TFLOP/s, the tensor pipe active for 48 % of the time (its floor at 1909 TFLOP/s is
// 288 us); four drafted tokens of each of four requests at 128K tokens (2 KV heads, 32 query
// heads, groups of 64) 116 us, 1.25 TB/s. A tile of 128 tokens takes 4300 cycles: a softmax of 2700 (two reads of S, 1000 for the
// maximum and 1500 for the exponentials) and the products of both row tiles, 4 x 512, which
// the chain S -> P -> O -> next S of each row tile overlaps only in part. The kernel's time is
// that of its longest block: 250 tiles of the 8192-token prompt where the mean is 219, 66
// where it is 56 of a 2048-token chunk under a window of 4096 tokens. What was tried
// against that and is slower: tiles of 64 tokens with the next S ready beforehand (650 us),
// one pass over S that raises the maximum as it goes (594), 64 columns at a time (625: spills),
// V kept in registers until the next K is written (583). Six expanding warps: 601 us; one blob
// copied at a time: 624; products issued under a lane test instead of elect.sync: 150 cycles
// each instead of 64.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cg_tiles.h"

namespace {

constexpr int kSoftWarps = 8, kExpandWarps = 8;
constexpr int kWarps = kSoftWarps + kExpandWarps + 2;
constexpr int kThreads = 32 * kWarps;
constexpr int kRing = 12;   // blobs copied ahead
constexpr int kIssue = 4;        // of those, copied at once
constexpr int kRows = 256;       // of a block
constexpr int kTile = 128;       // tokens
constexpr int kBlobs = kTile / 16;
// every expanding warp has a blob of every tile, so that it waits for each use of a barrier
static_assert(kExpandWarps <= kBlobs);
constexpr float kNone = -3.0e38f;

// The scale (in powers of two) as a factor of Q and one of the scores. Q takes its sign, so
// that the largest score is the largest product, and a scale of 0 (masked products are -inf;
// what is not finite times 0 stays so), and the power of two of one below 2^-24, so that no
// q.k overflows whose score is below 2^100. Exact, unless q 2^e is below bf16's normal range.
constexpr float kSmallScale = 0x1p-24f;

__device__ __forceinline__ uint32_t q_factor(float scale2)   // a bf16, twice
{
    const uint32_t bits = __float_as_uint(scale2), sign = bits >> 16 & 0x8000u;
    const uint32_t e = max(bits >> 23 & 0xFF, 1u);           // (subnormal ones go by 2^-126)
    const uint32_t f = scale2 == 0.0f ? 0u : sign | (fabsf(scale2) < kSmallScale ? e << 7 : 0x3F80u);
    return f | f << 16;
}

__device__ __forceinline__ float soft_scale(float scale2)
{
    const float a = fabsf(scale2);
    if (a >= kSmallScale)
        return a;
    const uint32_t e = max(__float_as_uint(a) >> 23, 1u);
    return a == 0.0f ? 1.0f : a * __uint_as_float((254u - e) << 23);
}

// ------------------------------------------------------------------ schedule

constexpr int kUnits = 4;       // units known at a time
constexpr int kBadTiles = 16;   // more than the copies can be ahead of the softmax

// 256 rows of a (request, KV head), and of the blobs that they see ([0, sink) and
// [sink + skip, ..), nb of them) those of one piece, from v0 on in n tiles of 8.
// Where there are fewer units than blocks, each is cut into pieces along its
// tokens, an item to a block, whose results a second kernel joins.
struct Unit {
    int32_t there;        // 0: no more items
    int32_t item, parts;  // the item's number; how many the unit is cut into
    int32_t r, h, q_row0; // request, KV head, the request's first query row
    int32_t rows, row0;   // rows of the request's KV head, first row of the unit
    int32_t tiles_q;      // row tiles of 128: 1 or 2
    int32_t x0, kv;       // position of the request's first query row; its tokens
    int32_t n, nb, sink, skip;
    int32_t v0;           // the piece's first visible blob
    // With one row tile in a cut unit the two softmax groups take turns at the tiles of tokens,
    // each with a maximum, a sum and an accumulator of its own.
    __device__ __forceinline__ bool turns() const { return tiles_q == 1 && parts > 1; }
    __device__ __forceinline__ int32_t blob(int32_t vb) const { return vb < sink ? vb : vb + skip; }
};

template <typename B>
struct ManyShared {
    uint8_t q[2][kTile * B::kD * 2];
    uint8_t k[2][kTile * B::kD * 2];
    uint8_t v[2][kTile * B::kD * 2];
    uint8_t ring[kRing][B::kBytes];
    uint64_t q_full, q_empty, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_half[2], p_full[2],
        o_full[2], last;
    uint64_t u_full[kUnits], u_empty[kUnits], raw_full[kRing], raw_empty[kRing];
    Unit unit[kUnits];
    uint32_t raw_blob[kRing];    // which of the block's blobs is in a place (times 2), and whether it was copied (1)
    uint32_t bad[kBadTiles];     // of the last tiles: blobs whose page id is outside the cache
    uint32_t tmem;
    int32_t units;       // of the whole batch
    uint32_t gave_up;    // a wait ran out: everyone leaves
};

// Most blocks, hence most items of a batch that is cut; and most items of shared tokens, whose units
// are cut in more pieces than blocks.
constexpr int kMaxBlocks = 160, kMaxItems = 640, kMaxSplit = 31;

// Workspace: how the batch was cut, the units, and of each item 256 rows of
// { float o[D] }, then { float m }, { float l }. Where the softmax groups take
// turns, rows 128 .. 255 are the second group's results for rows 0 .. 127.
struct ManyWork {
    int32_t items;       // that there is room for
    int32_t *cut;        // units, pieces of each
    Unit *heads;
    float *parts;
};

template <int D>
constexpr size_t kPartFloats = (size_t)kRows * (D + 2);

// (kShared as attn_request has it)
template <bool kShared>
__device__ __forceinline__ int32_t units_of(const AttnArgs &p, int r, AttnRequest *q)
{
    uint32_t error;
    if (r >= p.a.requests || !attn_request<kShared>(p, r, q, &error) || q->rows <= p.few_rows)
        return 0;
    return (q->rows + kRows - 1) / kRows * p.heads;   // at most tokens * q_heads
}

// One warp: unit `want` of the batch into *u. It goes on from where the last
// call stood (32 requests from *r0 on, `*before` units ahead of them).
template <bool kShared>
__device__ __forceinline__ void find_unit(const AttnArgs &p, int64_t item, int split, int *r0, int64_t *before,
                                          Unit *u, Unit *heads)
{
    const int lane = threadIdx.x & 31;
    const int64_t want = item / split;
    const int piece = (int)(item - want * split);
    for (;; *r0 += 32) {
        if (*r0 >= p.a.requests) {
            if (lane == 0)
                u->there = 0;
            __syncwarp();
            return;
        }
        AttnRequest q;
        const int w = units_of<kShared>(p, *r0 + lane, &q);
        int64_t inc = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
            if (lane >= d)
                inc += o;
        }
        const int64_t start = *before + inc - w;
        const uint32_t mine = __ballot_sync(0xFFFFFFFFu, want >= start && want < start + w);
        if (mine == 0) {
            *before += __shfl_sync(0xFFFFFFFFu, inc, 31);
            continue;
        }
        const int src = __ffs(mine) - 1;
        const int off = __shfl_sync(0xFFFFFFFFu, (int)(want - start), src);
        const int r = *r0 + src;
        units_of<kShared>(p, r, &q);
        // the last rows, which see most, first
        const int tile = (q.rows + kRows - 1) / kRows - 1 - off / p.heads;
        const int row0 = tile * kRows, rows = min(kRows, q.rows - row0), x0 = q.x0;
        const int pos_ratio = kShared ? p.pos_ratio : p.ratio;
        const int x_first = x0 + row0 / pos_ratio, x_last = x0 + (row0 + rows - 1) / pos_ratio;
        const int end = x_last < 0 ? 0 : x_last / 16 + 1;
        int sink = 0, skip = 0;
        const int64_t low = (int64_t)x_first + 1 - p.a.window;
        if (p.a.window > 0 && low > 0) {
            const int first = (int)(low / 16);
            const int64_t sb = ((int64_t)p.a.sinks + 15) / 16;
            sink = sb < first ? (int)sb : first;
            skip = first - sink;
        }
        const int nb = end - skip, n = (nb + kBlobs - 1) / kBlobs;
        // at least two tiles to a piece; the pieces behind the last are empty
        const int parts = min(split, max(n / 2, 1));
        const int t0 = piece < parts ? (int)((int64_t)n * piece / parts) : 0;
        const int t1 = piece < parts ? (int)((int64_t)n * (piece + 1) / parts) : 0;
        if (lane == 0) {
            const Unit found = {piece < parts ? 1 : 2, (int)item, parts, r, off % p.heads, q.row0, q.rows, row0,
                                rows > 128 ? 2 : 1, x0, q.kv, t1 - t0, nb, sink, skip, t0 * kBlobs};
            *u = found;
            if (split > 1 && piece == 0)
                heads[want] = found;
        }
        __syncwarp();
        return;
    }
}

// Units of shared tokens have n tiles each: as many pieces of each as make the longest block shortest,
// a piece counting its tiles and what it costs to begin and end it (some 3 of them: 197 units of 256
// tiles on 152 SMs take two turns whole, and 4/3 in three pieces). Every piece has two tiles at least,
// so none is empty.
__device__ __forceinline__ int split_of_equals(int units, int n, int items)
{
    const int lane = threadIdx.x & 31, whole = units > 0 ? (int)gridDim.x / units : 0;
    const int s = lane < kMaxSplit ? lane + 1 : max(whole, 1);
    const int64_t turns = ((int64_t)units * s + gridDim.x - 1) / gridDim.x;
    const int64_t cost = turns * ((n + s - 1) / s + 3);
    const bool can = s == 1 || (s <= n / 2 && (int64_t)units * s <= items);
    // the least cost, and of equal ones the least s
    const uint32_t least = __reduce_min_sync(0xFFFFFFFFu, can ? (uint32_t)min(cost, (int64_t)0x7FFFFFFF) : 0xFFFFFFFFu);
    const bool mine = can && (uint32_t)min(cost, (int64_t)0x7FFFFFFF) == least;
    return (int)__reduce_min_sync(0xFFFFFFFFu, mine ? (uint32_t)s : 0xFFFFFFFFu);
}

// -------------------------------------------------------------------- kernel

// kShared: there are shared tokens, and where they have a pass of their own (p.rows), this is one of the two.
template <typename B, bool kShared>
__global__ void __launch_bounds__(kThreads, 1) k_attention_many(AttnArgs p, ManyWork work)
{
    constexpr int D = B::kD, NW = B::kWords, NG = B::kGroups, WPG = NW / NG;
    constexpr int kQSub = kTile * 128;           // bytes of a 64-channel part of a Q or K tile
    constexpr int kVSub = D * 128;               // bytes of a 64-token part of a V tile
    // all 512 columns of tensor memory, so they start at 0: S0, S1, O0, O1
    constexpr uint32_t kS = 0, kO = 256;
    using S = ManyShared<B>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    grid_next();
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            bar_init(&sm.k_full[i], kBlobs);
            bar_init(&sm.v_full[i], kBlobs);
            bar_init(&sm.p_half[i], 128);
            bar_init(&sm.p_full[i], 128);
            bar_init(&sm.k_empty[i], 1);
            bar_init(&sm.v_empty[i], 1);
            bar_init(&sm.s_full[i], 1);
            bar_init(&sm.o_full[i], 1);
        }
        bar_init(&sm.last, 1);
        for (int i = 0; i < kUnits; ++i) {
            bar_init(&sm.u_full[i], 1);
            bar_init(&sm.u_empty[i], kWarps);
        }
        for (int i = 0; i < kRing; ++i) {
            bar_init(&sm.raw_full[i], 1);
            bar_init(&sm.raw_empty[i], 1);
            sm.raw_blob[i] = 0xFFFFFFFFu;   // none: a block has fewer
        }
        bar_init(&sm.q_full, kExpandWarps);
        bar_init(&sm.q_empty, 1);
        bar_init_fence();
        sm.gave_up = 0;
        sm.units = 0;
    }
    __syncthreads();
    {
        int64_t mine = 0;
        for (int r = tid; r < p.a.requests; r += kThreads) {
            AttnRequest q;
            mine += units_of<kShared>(p, r, &q);
        }
        // only whether there are fewer than blocks matters
        const int few = __reduce_add_sync(0xFFFFFFFFu, (int)min(mine, (int64_t)(1 << 20)));
        if (lane == 0)
            atomicAdd(&sm.units, few);
    }
    if (warp == kWarps - 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_addr(&sm.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tmem_fence_before();
    }
    __syncthreads();
    tmem_fence_after();
    if (sm.tmem != 0 && tid == 0)   // never: the block took all of it
        int4_set_status(p.status, CG_ERR_CUDA);
    const int split = kShared && p.first ? split_of_equals(sm.units, ((p.shared + 15) / 16 + kBlobs - 1) / kBlobs, work.items)
                      : sm.units > 0 && sm.units < gridDim.x ? gridDim.x / sm.units : 1;
    if (blockIdx.x == 0 && tid == 0) {
        work.cut[0] = sm.units;
        work.cut[1] = split;
    }
    const int bpp = p.page_tokens / 16;
    const int pos_ratio = kShared ? p.pos_ratio : p.ratio;
    const bool passes = kShared && p.rows != nullptr;
    // Every role walks the block's units on its own and meets the others at the barriers only,
    // so that the next unit's queries, keys and values come in under the last one's products.
    uint32_t un = 0;             // units begun
    uint32_t tiles_done = 0;     // K and V tiles of earlier units
    auto wait = [&](uint64_t *bar, uint32_t parity, bool at_once = false) {   // one thread's view
        return wait_or_leave(bar, parity, &sm.gave_up, p.status, at_once);
    };
    auto wait_all = [&](uint64_t *bar, uint32_t parity, bool at_once = false) {   // the warp's
        return __all_sync(0xFFFFFFFFu, wait_or_leave(bar, parity, &sm.gave_up, p.status, at_once));
    };
    // test builds: which role of this block gives up
    auto gives_up = [&](uint32_t role) { return kTestTimeout && blockIdx.x % 4 == role; };
    uint32_t issued = 0;         // blobs whose copies the copying warp has issued
    auto next_unit = [&]() -> const Unit * {   // the warp's next unit, or none
        if (!wait_all(&sm.u_full[un % kUnits], un / kUnits & 1))
            return nullptr;
        const Unit *u = &sm.unit[un % kUnits];
        return u->there == 1 ? u : nullptr;   // (a piece that is empty is a block's only item)
    };
    auto unit_over = [&](int n) {
        tiles_done += n;
        __syncwarp();
        if (lane == 0)
            bar_arrive(&sm.u_empty[un % kUnits]);
        ++un;
    };

    if (warp < kSoftWarps) {
        // ===================================================== softmax of a row
        // exponents in powers of two; what q_factor puts into Q does not come here
        const float sc = soft_scale(p.scale2);
        const int window = p.a.window > 0 ? p.a.window : INT32_MAX;
        const int i = warp >> 2;
        const uint32_t lane_at = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t s_at = lane_at + kS + 128 * i, o_at = lane_at + kO + 128 * i;
        uint32_t s_done = 0, o_done = 0;
        while (const Unit *up = next_unit()) {
            const Unit &u = *up;
            const int n = u.n;
            const bool turns = u.turns();
            const int tile = turns ? 0 : i, first = turns ? i : 0, step = turns ? 2 : 1;
            if (tile < u.tiles_q) {
                const int rr = u.row0 + 128 * tile + 32 * (warp & 3) + lane;
                const int x = rr < u.rows ? u.x0 + rr / pos_ratio : -1;
                const int last_row = min(u.row0 + 128 * tile + 128, u.rows) - 1;
                const int x_lo = u.x0 + (u.row0 + 128 * tile) / pos_ratio;
                const int x_hi = u.x0 + last_row / pos_ratio;
                float m = kNone, l = 0.0f;
                bool alive = true;
                for (int j = first; j < n; j += step) {
                    alive = wait_all(&sm.s_full[i], s_done & 1, gives_up(0) && s_done == 1);
                    ++s_done;
                    if (!alive)
                        break;
                    tmem_fence_after();
                    const int vb0 = u.v0 + j * kBlobs;
                    const int t0 = 16 * u.blob(vb0), t1 = 16 * u.blob(vb0 + kBlobs - 1) + 15;
                    const uint32_t bad = *reinterpret_cast<volatile uint32_t *>(&sm.bad[(tiles_done + j) % kBadTiles]);
                    const bool whole = bad == 0 && vb0 + kBlobs <= u.nb && t1 <= x_lo &&
                                       (x_hi - t0 < window || t1 < p.a.sinks);
                    // S is read twice, 32 columns at a time: rolled loops, because the roles of the
                    // block run side by side and have to share the instruction caches
                    constexpr int C = 32;
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < kTile / C; ++c) {
                        float s[C];
#pragma unroll
                        for (int k = 0; k < C / 32; ++k)
                            tmem_ld32(s + 32 * k, s_at + C * c + 32 * k);
                        tmem_wait_ld();
                        if (!whole) {
#pragma unroll
                            for (int b = 0; b < C / 16; ++b) {
                                const int in = C / 16 * c + b, vb = vb0 + in, tok = 16 * u.blob(vb);
                                // of the blob's 16 tokens the row sees those below `end`, from `low` on or below `sink`
                                const int end = vb < u.nb && !(bad >> in & 1) ? x + 1 - tok : 0;
                                const int64_t low64 = (int64_t)x + 1 - window - tok;
                                const int low = low64 < 0 ? 0 : (int)min(low64, (int64_t)16);
                                const int sink = p.a.sinks - tok;
                                uint32_t back[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    s[16 * b + e] = e < end && (e >= low || e < sink) ? s[16 * b + e] : -INFINITY;
                                    back[e] = __float_as_uint(s[16 * b + e]);
                                }
                                tmem_st16(s_at + C * c + 16 * b, back);
                            }
                        }
                        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                        for (int e = 4; e + 8 <= C; e += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                top[k] = fmaxf(fmaxf(top[k], s[e + 2 * k]), s[e + 2 * k + 1]);
#pragma unroll
                        for (int e = C - 4; e < C; ++e)
                            top[e & 3] = fmaxf(top[e & 3], s[e]);
                        mx = fmaxf(fmaxf(mx, fmaxf(top[0], top[1])), fmaxf(top[2], top[3]));
                    }
                    if (!whole)
                        tmem_wait_st();
                    mx *= sc;
                    if (__any_sync(0xFFFFFFFFu, mx > m + 8.0f)) {
                        const float mn = fmaxf(mx, m), f = exp2_fast(m - mn);
                        m = mn;
                        l *= f;
                        if (j > first) {
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t o[16];
                                tmem_ld16(o, o_at + 16 * c);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st16(o_at + 16 * c, o);
                            }
                        }
                    }
                    float2 sum = make_float2(0.0f, 0.0f), sum_b = sum;
                    const float2 sc2 = make_float2(sc, sc), m2 = make_float2(-m, -m);
#pragma unroll 1
                    for (int c = 0; c < kTile / C; ++c) {
                        float s[C];
#pragma unroll
                        for (int k = 0; k < C / 32; ++k)
                            tmem_ld32(s + 32 * k, s_at + C * c + 32 * k);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < C / 32; ++k) {
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float2 z = fma2(make_float2(s[32 * k + 2 * e], s[32 * k + 2 * e + 1]), sc2, m2);
                                z.x = exp2_fast(z.x);
                                z.y = exp2_fast(z.y);
                                if (e & 1)
                                    sum_b = add2(sum_b, z);
                                else
                                    sum = add2(sum, z);
                                pk[e] = pack_bf16(z.x, z.y);
                            }
                            tmem_st16(s_at + C / 2 * c + 16 * k, pk);   // over columns already read
                        }
                        if (c == kTile / C / 2 - 1) {   // the products of half the tile may begin
                            tmem_wait_st();
                            tmem_fence_before();
                            bar_arrive(&sm.p_half[i]);
                        }
                    }
                    sum = add2(sum, sum_b);
                    l += sum.x + sum.y;
                    tmem_wait_st();
                    tmem_fence_before();
                    bar_arrive(&sm.p_full[i]);
                }
                const bool any = n > first;
                if (alive && any) {
                    alive = wait_all(&sm.o_full[i], o_done & 1);
                    ++o_done;
                    tmem_fence_after();
                }
                if (!alive)
                    break;
                float inv = l == 0.0f ? 0.0f : 1.0f / l;
                if (passes && !p.first)   // for the rows of the shared tokens
                    grid_wait();
                const int qt = rr / p.ratio, qh = u.h * p.ratio + rr - qt * p.ratio;
                float *shared_row = nullptr, shared_f = 0.0f;
                if (passes && u.parts == 1 && rr < u.rows) {
                    const int64_t row = (int64_t)(u.q_row0 + qt) * p.a.q_heads + qh;
                    shared_row = p.rows + row * D;
                    if (p.first) {
                        p.row_stats[row] = make_float2(m, l);
                    } else {
                        const float2 f = join_factors(p, row, m, l);
                        inv *= f.x;
                        shared_f = f.y;
                    }
                }
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) +
                                     (int64_t)(u.q_row0 + qt) * p.a.out_token_stride + qh * p.a.out_head_stride;
                float *part = work.parts + u.item * kPartFloats<D>;
                const int part_row = 128 * i + 32 * (warp & 3) + lane;
                if (u.parts > 1) {
                    part[(size_t)kRows * D + part_row] = m;
                    part[(size_t)kRows * (D + 1) + part_row] = l;
                }
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    if (any) {
                        tmem_ld32(o, o_at + 32 * c);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = 0.0f;
                    }
                    if (rr >= u.rows)
                        continue;
                    // column 8 i + g is channel 4 g + i, as V's rows are
                    if (u.parts > 1) {
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            *reinterpret_cast<float4 *>(part + (size_t)part_row * D + 32 * c + 4 * g) =
                                make_float4(o[g], o[8 + g], o[16 + g], o[24 + g]);
                    } else if (passes && shared_row != nullptr) {
#pragma unroll
                        for (int g = 0; g < 8; ++g) {
                            float4 *there = reinterpret_cast<float4 *>(shared_row + 32 * c + 4 * g);
                            float4 v = make_float4(o[g] * inv, o[8 + g] * inv, o[16 + g] * inv, o[24 + g] * inv);
                            if (p.first) {
                                *there = v;
                            } else {
                                const float4 b = *there;
                                v = make_float4(fmaf(b.x, shared_f, v.x), fmaf(b.y, shared_f, v.y),
                                                fmaf(b.z, shared_f, v.z), fmaf(b.w, shared_f, v.w));
                                *reinterpret_cast<uint2 *>(out + 32 * c + 4 * g) =
                                    make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
                            }
                        }
                    } else {
#pragma unroll
                        for (int g = 0; g < 8; g += 2)
                            *reinterpret_cast<uint4 *>(out + 32 * c + 4 * g) = make_uint4(
                                pack_bf16(o[g] * inv, o[8 + g] * inv), pack_bf16(o[16 + g] * inv, o[24 + g] * inv),
                                pack_bf16(o[g + 1] * inv, o[9 + g] * inv), pack_bf16(o[17 + g] * inv, o[25 + g] * inv));
                    }
                }
                tmem_fence_before();   // the next unit's first p_half orders these reads before its O
            }
            unit_over(n);
        }
    } else {
        if (warp < kSoftWarps + kExpandWarps) {
            // ======================================================= queries, K and V tiles
            // Blobs go round the warps. K: 8 tokens at a time, lane t + 4 k has words t of token
            // (k & 1) * 4 + (k >> 1). V: 4 pairs of tokens at a time, lane g + 8 w has the words
            // (g, w), channels 32 w + 4 g + i, which become rows 32 w + 8 i + g. Either way eight
            // lanes' 16-byte stores meet all banks.
            const int wi = warp - kSoftWarps, t = lane & 3, k8 = lane >> 2;
            const int half_tok = (k8 & 1) * 4 + (k8 >> 1);
            const int g = lane & 7, vw = (lane >> 3) % NW, v_half = NW == 2 ? lane >> 4 : 0;
            const uint32_t factor = q_factor(p.scale2);
            auto blob_issued = [&](uint32_t slot, uint32_t at) {   // false: a wait ran out
                const volatile uint32_t *blob = &sm.raw_blob[slot];
                uint64_t start = 0;
                for (uint32_t i = 0; (*blob ^ 2 * at) >> 1; ++i) {
                    if ((i & 63) != 63)
                        continue;
                    if (*reinterpret_cast<volatile uint32_t *>(&sm.gave_up))
                        return false;
                    const uint64_t now = now_ns();
                    if (start == 0) {
                        start = now;
                    } else if (now - start > kBarWaitNs) {
                        *reinterpret_cast<volatile uint32_t *>(&sm.gave_up) = 1;
                        int4_set_status(p.status, CG_ERR_TIMEOUT);
                        return false;
                    }
                }
                return true;
            };
            uint32_t seq = 0;            // blobs of earlier units
            while (const Unit *up = next_unit()) {
                const Unit &u = *up;
                const int n = u.n;
                auto queries = [&]() {   // false: a wait ran out
                    if (!wait_all(&sm.q_empty, (un & 1) ^ 1))   // the last unit's scores are done
                        return false;
                    constexpr int kC = D / 8, kStep = 32 * kExpandWarps / kC;   // rows apart
                    const int vt = 32 * wi + lane, c = vt % kC;
                    int in = vt / kC;
                    int qt = (u.row0 + in) / p.ratio, qr = (u.row0 + in) - qt * p.ratio;
                    const int step_t = kStep / p.ratio, step_r = kStep - step_t * p.ratio;
                    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.a.q) +
                                             (int64_t)u.q_row0 * p.a.q_token_stride +
                                             (int64_t)u.h * p.ratio * p.a.q_head_stride + 8 * c;
                    const int end = 128 * u.tiles_q, rows = u.rows - u.row0;
#pragma unroll 1
                    while (in < end) {
                        uint4 v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v[e] = in + e * kStep < rows
                                       ? *reinterpret_cast<const uint4 *>(q + qt * p.a.q_token_stride +
                                                                          qr * p.a.q_head_stride)
                                       : make_uint4(0, 0, 0, 0);
                            qt += step_t;
                            qr += step_r;
                            if (qr >= p.ratio) {
                                qr -= p.ratio;
                                ++qt;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e, in += kStep)
                            if (in < end)
                                *reinterpret_cast<uint4 *>(sm.q[in >> 7] + (c >> 3) * kQSub + (in & 127) * 128 +
                                                           (((c & 7) ^ (in & 7)) << 4)) =
                                    make_uint4(mul_bf16x2(__byte_perm(v[e].x, v[e].z, 0x5410), factor),
                                               mul_bf16x2(__byte_perm(v[e].x, v[e].z, 0x7632), factor),
                                               mul_bf16x2(__byte_perm(v[e].y, v[e].w, 0x5410), factor),
                                               mul_bf16x2(__byte_perm(v[e].y, v[e].w, 0x7632), factor));
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(&sm.q_full);
                    return true;
                };
                bool have_q = false, alive = true;
                int b = (int)((wi + kExpandWarps - seq % kExpandWarps) % kExpandWarps);
                for (; b < n * kBlobs && alive; b += kExpandWarps) {
                    if (!have_q && b >= kBlobs) {   // after the first tile, which can be begun without
                        have_q = true;
                        if (!(alive = queries()))
                            break;
                    }
                    const uint32_t use = tiles_done + (uint32_t)b / kBlobs, sl = use & 1, at = seq + b;
                    const uint32_t slot = at % kRing;
                    const int in_tile = b % kBlobs;
                    // The place's blob before this one is another warp's and may still be on its way, where
                    // the barrier's parity would say the same as when this one is there: so first, that
                    // this one was issued, which it is only into a place that was read.
                    alive = __all_sync(0xFFFFFFFFu, blob_issued(slot, at)) &&
                            wait_all(&sm.raw_full[slot], at / kRing & 1, gives_up(1) && at == 5) &&
                            wait_all(&sm.k_empty[sl], (use >> 1 & 1) ^ 1);
                    if (!alive)
                        break;
                    const uint8_t *blob = sm.ring[slot];
                    const bool there = sm.raw_blob[slot] & 1;
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        const int tok = 8 * a + half_tok, row = 16 * in_tile + tok;
                        uint32_t code[NW], par[NG];
                        load_words(code, blob + B::kKCodes + tok * (D / 2) + t * (D / 8));
                        load_words(par, blob + B::kKParams + tok * 4 * NG);
#pragma unroll
                        for (int w = 0; w < NW; ++w) {
                            const uint32_t q = there ? par[w / WPG] : 0;   // (0 + 0 n)
                            const uint32_t s2 = __byte_perm(q, q, 0x1010), lo2 = __byte_perm(q, q, 0x3232);
                            const uint4 o = make_uint4(expand(code[w], 0, s2, lo2), expand(code[w], 1, s2, lo2),
                                                 expand(code[w], 2, s2, lo2), expand(code[w], 3, s2, lo2));
                            const int c = 4 * w + t;
                            *reinterpret_cast<uint4 *>(sm.k[sl] + (c >> 3) * kQSub + row * 128 +
                                                       (((c & 7) ^ (row & 7)) << 4)) = o;
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(&sm.k_full[sl]);
                    alive = wait_all(&sm.v_empty[sl], (use >> 1 & 1) ^ 1);
                    if (!alive)
                        break;
                    // tokens that are not there get 0, whatever the cache holds in their place
                    const int left = there ? u.kv - 16 * u.blob(u.v0 + b) : 0;
#pragma unroll
                    for (int a = 0; a < (NW == 2 ? 1 : 2); ++a) {
                        const int hf = NW == 2 ? v_half : a, chunk = 2 * in_tile + hf;
                        uint32_t code[4], s2[4], lo2[4];
                        const uint32_t *par = reinterpret_cast<const uint32_t *>(blob + B::kVParams) + 8 * hf * NG +
                                              vw / WPG;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            code[e] = *reinterpret_cast<const uint32_t *>(blob + B::kVCodes + (4 * hf + e) * D +
                                                                          g * (D / 8) + 4 * vw);
                            const int tok = 8 * hf + 2 * e;
                            const uint32_t p0 = tok < left ? par[2 * e * NG] : 0;
                            const uint32_t p1 = tok + 1 < left ? par[(2 * e + 1) * NG] : 0;
                            s2[e] = __byte_perm(p0, p1, 0x5410);
                            lo2[e] = __byte_perm(p0, p1, 0x7632);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = 32 * vw + 8 * i + g;
                            *reinterpret_cast<uint4 *>(sm.v[sl] + (chunk >> 3) * kVSub + row * 128 +
                                                       (((chunk & 7) ^ (row & 7)) << 4)) =
                                make_uint4(expand(code[0], i, s2[0], lo2[0]), expand(code[1], i, s2[1], lo2[1]),
                                           expand(code[2], i, s2[2], lo2[2]), expand(code[3], i, s2[3], lo2[3]));
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        bar_arrive(&sm.v_full[sl]);
                        bar_arrive(&sm.raw_empty[slot]);
                    }
                }
                if (alive && !have_q)
                    alive = queries();
                if (!alive)
                    break;
                seq += n * kBlobs;
                unit_over(n);
            }
        } else if (warp == kSoftWarps + kExpandWarps) {
            // ======================================================= units, copies
            int u_r0 = 0;
            int64_t u_before = 0;
            auto find = [&](uint32_t which) {   // false: a wait ran out
                const uint32_t slot = which % kUnits;
                if (!wait_all(&sm.u_empty[slot], (which / kUnits & 1) ^ 1))
                    return false;
                find_unit<kShared>(p, blockIdx.x + (int64_t)which * gridDim.x, split, &u_r0, &u_before, &sm.unit[slot],
                          work.heads);
                if (lane == 0)
                    bar_arrive(&sm.u_full[slot]);
                __syncwarp();
                return true;
            };
            find(0);   // a place that was never used: no wait
            while (const Unit *up = next_unit()) {
                const Unit &u = *up;
                const int32_t *table = p.a.block_table + u.r * p.a.table_stride;
                const int n = u.n;
                bool alive = true;
                for (int b0 = 0; b0 < n * kBlobs && alive; b0 += 32) {
                    // 32 blobs (four tiles) are looked up at once, one by each lane
                    const int vb = u.v0 + b0 + lane;
                    const bool wanted = b0 + lane < n * kBlobs && vb < u.nb;
                    const int blob = wanted ? u.blob(vb) : 0, page = blob / bpp;
                    const int id = wanted ? (kShared && 16 * blob < p.front ? p.a.block_table : table)[page] : -1;
                    const bool there = (unsigned)id < (unsigned)p.num_pages;
                    const uint32_t bad = __ballot_sync(0xFFFFFFFFu, wanted && !there);
                    if (bad && lane == 0)
                        int4_set_status(p.status, CG_ERR_CORRUPT);
                    // in 128-byte units of the layer (it fits, cg_int4.h)
                    const uint32_t place = there ? (((uint32_t)id * p.heads + u.h) * bpp + (blob - page * bpp)) *
                                                       (B::kBytes / 128)
                                                 : 0;
                    const int count = min(32, n * kBlobs - b0);
                    // kIssue at a time: as many lanes wait for a place in the ring each, and copy
                    for (int k = 0; k < count; k += kIssue) {
                        const uint32_t at = issued + lane % kIssue, slot = at % kRing;
                        alive = wait_all(&sm.raw_empty[slot], (at / kRing & 1) ^ 1, gives_up(2) && issued == kRing);
                        if (!alive)
                            break;
                        issued += kIssue;
                        if ((unsigned)(lane - k) < kIssue) {
                            if (lane % kBlobs == 0)
                                *reinterpret_cast<volatile uint32_t *>(
                                    &sm.bad[(tiles_done + (b0 + lane) / kBlobs) % kBadTiles]) = bad >> lane & 0xFFu;
                            *reinterpret_cast<volatile uint32_t *>(&sm.raw_blob[slot]) = 2 * at + there;
                            if (there) {
                                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                                bar_expect(&sm.raw_full[slot], B::kBytes);
                                bulk_copy(sm.ring[slot], p.layer + (uint64_t)place * 128, B::kBytes,
                                          &sm.raw_full[slot]);
                            } else {
                                bar_arrive(&sm.raw_full[slot]);
                            }
                        }
                        __syncwarp();
                    }
                    if (b0 == 0 && alive)
                        alive = find(un + 1);
                }
                if (n == 0)
                    alive = find(un + 1);
                if (!alive)
                    break;
                unit_over(n);
            }
        } else {
            // ========================================================== products
            const uint32_t q_at = smem_addr(sm.q[0]), k_at = smem_addr(sm.k[0]), v_at = smem_addr(sm.v[0]);
            // S of accumulator i: row tile `rows` with the K tile in place sl
            auto scores = [&](int i, int rows, uint32_t sl) {
                const uint32_t a = smem_desc(q_at + rows * (kTile * D * 2)), b = smem_desc(k_at + sl * (kTile * D * 2));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * kQSub + (kk & 3) * 32) >> 4;
                    mma_ss(kS + 128 * i, a + off, b + off, mma_desc(kTile), kk > 0);
                }
                mma_commit(&sm.s_full[i]);
            };
            uint32_t p_done = 0;     // parity of each row tile's p_full
            while (const Unit *up = next_unit()) {
                const int n = up->n, tiles_q = up->tiles_q;
                const bool turns = up->turns();
                bool left = false;       // a wait ran out
                if (elect_one()) {
                    // O of accumulator i, with the V tile of the t-th tile of all
                    auto values = [&](int i, int half, uint32_t t, bool add) {
                        const uint32_t b = smem_desc(v_at + (t & 1) * (kTile * D * 2) + half * kVSub);
#pragma unroll
                        for (int kk = 0; kk < kTile / 32; ++kk)
                            mma_ts(kO + 128 * i, kS + 128 * i + 32 * half + 8 * kk, b + (kk * 32 >> 4), mma_desc(D),
                                   add || kk > 0);
                    };
                    auto k_there = [&](uint32_t t) { return wait(&sm.k_full[t & 1], t >> 1 & 1); };
                    auto v_there = [&](uint32_t t) { return wait(&sm.v_full[t & 1], t >> 1 & 1); };
                    auto p_there = [&](int i) {
                        const bool ok = wait(&sm.p_full[i], p_done >> i & 1);
                        p_done ^= 1u << i;
                        return ok;
                    };
                    auto half_there = [&](int i, bool at_once) {
                        return wait(&sm.p_half[i], p_done >> i & 1, at_once);
                    };
                    bool alive = wait(&sm.q_full, un & 1);
                    const uint32_t t0 = tiles_done;
                    // the first scores of both accumulators
                    const int head = turns ? min(n, 2) : min(n, 1);
                    for (int j = 0; j < head && alive; ++j) {
                        alive = k_there(t0 + j);
                        if (!alive)
                            break;
                        tmem_fence_after();
                        scores(turns ? j : 0, 0, (t0 + j) & 1);
                        if (!turns && tiles_q > 1)
                            scores(1, 1, (t0 + j) & 1);
                        mma_commit(&sm.k_empty[(t0 + j) & 1]);
                    }
                    if (n <= head) {   // no more scores
                        if (n == 0)
                            bar_arrive(&sm.q_empty);
                        else if (alive)
                            mma_commit(&sm.q_empty);
                    }
                    for (int j = 0; j < n && alive; ++j) {
                        const uint32_t t = t0 + j, nx = t + head;   // nx: the next tile of this accumulator
                        const bool more = j + head < n;
                        for (int k = 0; k < (turns ? 1 : tiles_q); ++k) {
                            const int i = turns ? j & 1 : k;
                            alive = half_there(i, gives_up(3) && t == 1);
                            if (alive && k == 0)
                                alive = v_there(t);
                            if (!alive)
                                break;
                            tmem_fence_after();
                            values(i, 0, t, j >= head);
                            if (!(alive = p_there(i)))
                                break;
                            tmem_fence_after();
                            values(i, 1, t, true);
                            if (turns || k + 1 == tiles_q)
                                mma_commit(&sm.v_empty[t & 1]);
                            // only now: a warp that expands tile nx may have to write V where tile t lies
                            // before it comes to the last of nx's K
                            if (more && k == 0 && !(alive = k_there(nx)))
                                break;
                            if (more)
                                scores(i, turns ? 0 : i, nx & 1);
                            else
                                mma_commit(&sm.o_full[i]);
                        }
                        if (alive && more)
                            mma_commit(&sm.k_empty[nx & 1]);
                        if (alive && j + head + 1 == n)
                            mma_commit(&sm.q_empty);
                    }
                    left = !alive;
                }
                if (__any_sync(0xFFFFFFFFu, left))
                    break;
                unit_over(n);
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    // Every role has left, so nothing is issued any more. After a wait that ran out, whichever
    // role it was, what is in flight ends before shared and tensor memory go.
    if (sm.gave_up) {
        if (warp == kSoftWarps + kExpandWarps) {
            for (uint32_t at = issued < kRing ? 0 : issued - kRing; at < issued; ++at)
                bar_wait(&sm.raw_full[at % kRing], at / kRing & 1);
        } else if (warp == kWarps - 1) {
            if (elect_one()) {   // the thread that issued the products
                mma_commit(&sm.last);
                bar_wait(&sm.last, 0);
            }
            __syncwarp();
        }
        __syncthreads();
    }
    if (warp == kWarps - 1) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sm.tmem) : "memory");
    }
    grid_wait();
}

// ------------------------------------------------------------------- joining

// Rows of units that were cut, a warp to a row: the parts' accumulators, weighted by
// 2^(m - max m), in the order of the parts.
constexpr int kJoinThreads = 128;

// Blocks: four on each of 152 SMs, and ten for shared tokens, where there may be 50000 rows and what counts is
// how many loads are under way (25200 rows in three parts: 30 us with ten, 64 with four).
constexpr int join_blocks(bool first) { return first ? 1520 : 608; }

template <int D, bool kShared>
__global__ void __launch_bounds__(kJoinThreads) k_attention_many_join(AttnArgs p, ManyWork work)
{
    constexpr int kC = D / 32;   // channels of a lane
    if (kShared)
        grid_next();   // the pass behind the shared tokens may come up
    grid_wait();
    if (work.cut[1] == 1)
        return;
    const int lane = threadIdx.x & 31, rows = work.cut[0] * kRows;   // (units that are cut are no more than items)
    for (int at = (blockIdx.x * kJoinThreads + threadIdx.x) >> 5; at < rows; at += gridDim.x * kJoinThreads / 32) {
        const Unit &u = work.heads[at / kRows];
        const int row = at % kRows, rr = u.row0 + row;
        if (u.parts == 1 || rr >= u.rows)
            continue;
        const int each = u.turns() ? 2 : 1, n = u.parts * each;
        // part k: its item, and its row there
        const float *first = work.parts + u.item * kPartFloats<D>;
        auto part_of = [&](int k) { return first + (k / each) * kPartFloats<D>; };
        auto row_of = [&](int k) { return row + 128 * (k % each); };
        float mx = kNone;
        for (int k = lane; k < n; k += 32)
            mx = fmaxf(mx, part_of(k)[(size_t)kRows * D + row_of(k)]);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
        float l = 0.0f, sum[kC] = {};
        for (int k0 = 0; k0 < n; k0 += 32) {
            float f = 0.0f;
            if (k0 + lane < n) {
                const float *stats = part_of(k0 + lane) + (size_t)kRows * D + row_of(k0 + lane);
                f = exp2_fast(stats[0] - mx);
                l = fmaf(stats[kRows], f, l);
            }
            const int here = min(32, n - k0);
#pragma unroll 8
            for (int k = 0; k < here; ++k) {
                const float *o = part_of(k0 + k) + (size_t)row_of(k0 + k) * D + kC * lane;
                const float w = __shfl_sync(0xFFFFFFFFu, f, k);
                float v[kC];
                if constexpr (kC == 4)
                    *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(o);
                else
                    *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(o);
#pragma unroll
                for (int c = 0; c < kC; ++c)
                    sum[c] = fmaf(v[c], w, sum[c]);
            }
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
            l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int qt = rr / p.ratio, qh = u.h * p.ratio + rr - qt * p.ratio;
#pragma unroll
        for (int c = 0; c < kC; ++c)
            sum[c] *= inv;
        if (kShared && p.rows != nullptr) {
            const int64_t at_row = (int64_t)(u.q_row0 + qt) * p.a.q_heads + qh;
            float *there = p.rows + at_row * D + kC * lane;
            if (p.first) {
#pragma unroll
                for (int c = 0; c < kC; ++c)
                    there[c] = sum[c];
                if (lane == 0)
                    p.row_stats[at_row] = make_float2(mx, l);
                continue;
            }
            const float2 f = join_factors(p, at_row, mx, l);
#pragma unroll
            for (int c = 0; c < kC; ++c)
                sum[c] = fmaf(there[c], f.y, sum[c] * f.x);
        }
        uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.a.out) +
                                                     (int64_t)(u.q_row0 + qt) * p.a.out_token_stride +
                                                     qh * p.a.out_head_stride + kC * lane);
        if constexpr (kC == 4)
            *reinterpret_cast<uint2 *>(out) =
                make_uint2(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]));
        else
            *out = pack_bf16(sum[0], sum[1]);
    }
}

constexpr size_t head_bytes(int items) { return 256 + (sizeof(Unit) * items + 255) / 256 * 256; }

template <typename B, bool kShared>
cudaError_t launch(const AttnArgs &p, uint8_t *ws, cudaStream_t s)
{
    int sms = 0;
    cudaError_t err = attn_sm_count(&sms);
    const int smem = (int)sizeof(ManyShared<B>);
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(k_attention_many<B, kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess)
        return err;
    const int items = p.first ? p.items : kMaxBlocks, blocks = sms < kMaxBlocks ? sms : kMaxBlocks;
    const ManyWork work = {items, reinterpret_cast<int32_t *>(ws), reinterpret_cast<Unit *>(ws + 256),
                           reinterpret_cast<float *>(ws + head_bytes(items))};
    if (p.first) {   // the call's first kernel: it follows what is in the stream
        k_attention_many<B, kShared><<<blocks, kThreads, smem, s>>>(p, work);
        err = cudaGetLastError();
    } else {   // under the kernels for few rows: it works on other rows, with a workspace of its own
        err = launch_under(k_attention_many<B, kShared>, dim3(blocks), kThreads, smem, s, p, work);
    }
    if (err == cudaSuccess)
        err = launch_under(k_attention_many_join<B::kD, kShared>, dim3(join_blocks(p.first)), kJoinThreads, 0, s, p, work);
    return err;
}

}  // namespace

int attn_many_items(int64_t rows, int heads)
{
    const int64_t most = (rows + kRows - 1) / kRows * heads * kMaxSplit;
    return most < kMaxBlocks ? kMaxBlocks : most < kMaxItems ? (int)most : kMaxItems;
}

size_t attn_many_workspace(int head_size, int items)
{
    items = items > 0 ? items : kMaxBlocks;
    return head_bytes(items) + items * (size_t)kRows * (head_size + 2) * sizeof(float);
}

cudaError_t attn_many_launch(const AttnArgs &p, int head_size, int group, void *ws, cudaStream_t s)
{
    return int4_dispatch(head_size, group, [&](auto blob) {
        using B = decltype(blob);
        uint8_t *at = static_cast<uint8_t *>(ws);
        return p.shared + p.front > 0 ? launch<B, true>(p, at, s) : launch<B, false>(p, at, s);
    });
}

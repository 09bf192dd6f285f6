// cg_int4_weigh for requests with many query rows: their scores by tcgen05, twice, once for the maximum
// and sum of every row and once for the sums of every token over the rows.
//
// Exact products of 16-bit operands. With c the code whose value is nearest to 0, m = n - c and mid = lo + c s,
// q.k^ = sum q (s m) + sum mid (sum q), over channels and over groups. (Where a few channels of a group are
// large, s follows them and the others' codes lie at c: so their terms are small and none cancel. With 8
// for c the error was 3e-7 to 1e-6 of the prompts' weights, so 1.5e-7, for 4 % of the time.) s m has 13
// bits: two bf16 values hold it. mid and sum q are fp32, three bf16 values each, of whose nine products
// the six largest count (the others are below 2^-24). So a tile of scores is 2 D / 16 instructions for the
// codes and one or two for the groups, all into one accumulator, and differs from the sums in 64 bits by
// fp32 roundings alone.
//
// One block per 128 rows of a (request, KV head), which stay in shared memory, and tiles of 128 tokens, whose
// keys eight warps expand, 16 tokens each. Either pass is 128 x 128 x (2 D + 16 or 32):
//   warps 0-3, 4-7   take the scores of every other tile out of tensor memory. First pass: S = Q K^T, a
//                    thread has a row and keeps its maximum and sum. Second: S = K Q^T, a thread has a token
//                    and sums over the 128 rows; sums of several row tiles are added, in order, by a third
//                    kernel.
//   warps 8-15       queries of a unit; keys of a blob at a time
//   warp 16          finds the units and copies the K half of their blobs into a ring
//   warp 17          one thread issues all products
// With fewer units than blocks each is cut along its tokens; of more, whichever block is free takes the next, the
// longest of a request first (two prompts of 2048: 195 us so, 210 dealt in turns).
//
// What bounds it: a tile takes some 2300 cycles in the first pass and 3000 in the second. Its products are 1280,
// which the shared memory's rate sets (two operands of 4 KB in 64 cycles), the expansion of its keys and its
// exponentials about as much each; they overlap, but hand the two buffers of keys and scores on by barriers.
// One request of 32768 tokens, 128 rows, 32 query and 8 KV heads: 29 + 32 us, with all else 76; two prompts of
// 2048 at 4 rows to a token: 190. Products alone would be 9 of the 29. (Built, and not better, when those two took
// 76 and 188: 256 rows to a block, whose low parts had one buffer, 88 and 183; 16 expanding warps of half a blob, 84 and
// 224; two accumulators for a tile of scores, 81 and 208, for a fifth less of error.)

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cg_tiles.h"
#include "cg_weigh.h"

namespace {

constexpr int kSoftWarps = 8, kExpandWarps = 8;
constexpr int kAllWarps = kSoftWarps + kExpandWarps + 2, kAllThreads = 32 * kAllWarps;
constexpr int kPlaces = 24;      // blobs copied ahead
constexpr int kIssue = 8;        // of those, copied at once
constexpr int kTile = 128;       // rows, and tokens
constexpr int kBlobs = kTile / 16;
constexpr int kKnown = 4;        // units known at a time, and their rows' factors kept
constexpr int kBadTiles = 16;    // more than the copies can be ahead of the scores
constexpr int kMaxBlocks = 160;

// 128 rows of a (request, KV head), and of the blobs that they see ([0, sink) and [sink + skip, ..), nb of
// them) those of one piece, from v0 on in n tiles of 8.
struct Piece {
    int32_t there;          // 0: no more; 2: an empty piece, its block's only one
    int32_t item, parts;    // the item's number; how many the unit is cut into
    int32_t r, h, q_row0;   // request, KV head, the request's first query row
    int32_t rows, row0;     // rows of the request's KV head, first row of the unit
    int32_t x0, kv;         // position of the request's first query row; its tokens
    int32_t n, nb, sink, skip;
    int32_t v0;             // the piece's first visible blob
    __device__ __forceinline__ int32_t blob(int32_t vb) const { return vb < sink ? vb : vb + skip; }
};

// The groups' columns: 8 of a 16-byte chunk for each group (six count), whole instructions of 16.
template <typename B>
constexpr int kGroupSteps = B::kGroups == 4 ? 2 : 1;

template <typename B>
struct TileShared {
    uint8_t q[kTile * B::kD * 2];
    uint8_t qx[kTile * 64];
    uint8_t k[2][2][kTile * B::kD * 2];     // high and low parts
    uint8_t kx[2][kTile * 64];
    uint8_t ring[kPlaces][B::kVCodes];
    float4 row[kKnown][kTile / 2];          // of two rows: rho, rho, -m, -m
    float2 inv[kKnown][kTile / 2];          // and 1 / l
    uint64_t q_full, q_empty, k_full[2], k_empty[2], s_full[2], s_empty[2], last;
    uint64_t u_full[kKnown], u_empty[kKnown], row_full[kKnown], raw_full[kPlaces], raw_empty[kPlaces];
    Piece piece[kKnown];
    uint32_t raw_blob[kPlaces];  // which of the block's blobs is in a place (times 2), and whether it was copied (1)
    uint32_t bad[kBadTiles];     // of the last tiles: blobs whose page id is outside the cache
    uint32_t tmem;
    int32_t units;
    uint32_t gave_up;            // a wait ran out: everyone leaves
};

struct TileWork {
    int32_t most;        // units that there is room for
    int32_t *cut;        // units; then, of either pass, items taken behind the blocks' first
    Piece *heads;        // [units]: their first pieces
    float2 *parts;       // [items][2][128]: m, l of an item's even tiles and of its odd ones
};

__device__ __forceinline__ int32_t units_of(const AttnArgs &p, int r, AttnRequest *q)
{
    uint32_t error;
    if (r >= p.a.requests || !attn_request<WeighBatch::kShared>(p, r, q, &error) || q->rows <= p.few_rows)
        return 0;
    return (q->rows + kTile - 1) / kTile * p.heads;
}

// Tiles of 128 rows of request r lie from here on (as first_slot has those of 8).
__device__ __forceinline__ int32_t first_tile(const AttnArgs &p, int r, int32_t row0)
{
    return (int32_t)((int64_t)row0 * p.ratio / kTile) + r;
}

// The blobs that rows row0 .. row0 + rows - 1 see.
__device__ __forceinline__ void blobs_of(const AttnArgs &p, int32_t x0, int32_t row0, int32_t rows, int *nb, int *sink, int *skip)
{
    const int x_first = x0 + row0 / p.ratio, x_last = x0 + (row0 + rows - 1) / p.ratio;
    const int end = x_last < 0 ? 0 : x_last / 16 + 1;
    *sink = *skip = 0;
    const int64_t low = (int64_t)x_first + 1 - p.a.window;
    if (p.a.window > 0 && low > 0) {
        const int first = (int)(low / 16);
        const int64_t sb = ((int64_t)p.a.sinks + 15) / 16;
        *sink = sb < first ? (int)sb : first;
        *skip = first - *sink;
    }
    *nb = end - *skip;
}

// One warp: piece `item` of the batch into *u. It goes on from where the last call stood.
__device__ __forceinline__ void find_piece(const AttnArgs &p, int64_t item, int split, int *r0, int64_t *before, Piece *u,
                                           const TileWork &work, Piece *heads)
{
    const int lane = threadIdx.x & 31;
    const int64_t want = item / split;
    const int piece = (int)(item - want * split);
    for (;; *r0 += 32) {
        if (*r0 >= p.a.requests || want >= work.most) {
            if (lane == 0)
                u->there = 0;
            __syncwarp();
            return;
        }
        AttnRequest q;
        const int w = units_of(p, *r0 + lane, &q);
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
        units_of(p, r, &q);
        // the last rows, which see most, first
        const int tile = (q.rows + kTile - 1) / kTile - 1 - off / p.heads;
        const int row0 = tile * kTile, rows = min(kTile, q.rows - row0);
        int nb, sink, skip;
        blobs_of(p, q.x0, row0, rows, &nb, &sink, &skip);
        const int n = (nb + kBlobs - 1) / kBlobs;
        // at least two tiles to a piece; the pieces behind the last are empty
        const int parts = min(split, max(n / 2, 1));
        const int t0 = piece < parts ? (int)((int64_t)n * piece / parts) : 0;
        const int t1 = piece < parts ? (int)((int64_t)n * (piece + 1) / parts) : 0;
        if (lane == 0) {
            const Piece found = {piece < parts ? 1 : 2, (int)item, parts, r, off % p.heads, q.row0, q.rows, row0,
                                 q.x0, q.kv, t1 - t0, nb, sink, skip, t0 * kBlobs};
            *u = found;
            if (piece == 0 && heads != nullptr)
                heads[want] = found;
        }
        __syncwarp();
        return;
    }
}

// c s - hi of bf16 pairs, exact where hi is the product rounded.
__device__ __forceinline__ uint32_t rest_of(uint32_t c, uint32_t s, uint32_t hi)
{
    const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&c),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&s),
                                     __hneg2(*reinterpret_cast<const __nv_bfloat162 *>(&hi)));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// The code whose value is nearest to 0 (0 where s is; any code gives the same score but for roundings).
__device__ __forceinline__ float code_of_zero(uint32_t par)
{
    return fminf(fmaxf(rintf(__fdividef(-par_lo(par), par_s(par))), 0.0f), 15.0f);
}

// x in three bf16 values (the high halves): 24 bits.
__device__ __forceinline__ void three_parts(float x, uint32_t (&part)[3])
{
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        part[i] = pack_bf16(0.0f, x) & 0xFFFF0000u;
        x -= __uint_as_float(part[i]);
    }
}

template <typename B, bool kSums>
__global__ void __launch_bounds__(kAllThreads, 1) k_weigh_tiles(AttnArgs p, WeighArgs a, TileWork work)
{
    constexpr int D = B::kD, NW = B::kWords, NG = B::kGroups, WPG = NW / NG;
    constexpr int kSub = kTile * 128;            // bytes of a 64-channel part of a tile
    constexpr int kGroupChunks = 2 * kGroupSteps<B>;
    using S = TileShared<B>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    grid_next();
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            bar_init(&sm.k_full[i], kExpandWarps);
            bar_init(&sm.k_empty[i], 1);
            bar_init(&sm.s_full[i], 1);
            bar_init(&sm.s_empty[i], 128);
        }
        bar_init(&sm.last, 1);
        for (int i = 0; i < kKnown; ++i) {
            bar_init(&sm.u_full[i], 1);
            bar_init(&sm.u_empty[i], kAllWarps);
            bar_init(&sm.row_full[i], kExpandWarps);
        }
        for (int i = 0; i < kPlaces; ++i) {
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
        for (int r = tid; r < p.a.requests; r += kAllThreads) {
            AttnRequest q;
            mine += units_of(p, r, &q);
        }
        // exact where the batch is right: parts of 2 KB a unit are within the bound on the workspace, so units are
        // fewer than 2^20; of more, only that they are too many matters
        const int few = __reduce_add_sync(0xFFFFFFFFu, (int)min(mine, (int64_t)(1 << 20)));
        if (lane == 0)
            atomicAdd(&sm.units, few);
    }
    if (warp == kAllWarps - 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_addr(&sm.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tmem_fence_before();
    }
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = sm.tmem;
    const int split = sm.units > 0 && sm.units < gridDim.x ? gridDim.x / sm.units : 1;
    if (!kSums && blockIdx.x == 0 && tid == 0) {
        work.cut[0] = min(sm.units, work.most);
        if (sm.units > work.most)   // more than a batch of so many tokens has: requests that share rows of q
            int4_set_status(p.status, CG_ERR_CORRUPT);
    }
    const int bpp = p.page_tokens / 16;
    // Every role walks the block's pieces on its own and meets the others at the barriers only.
    uint32_t un = 0;             // pieces begun
    uint32_t qn = 0;             // those with tiles
    uint32_t tiles_done = 0;     // tiles of earlier pieces
    auto wait = [&](uint64_t *bar, uint32_t parity, bool at_once = false) {   // one thread's view
        return wait_or_leave(bar, parity, &sm.gave_up, p.status, at_once);
    };
    auto wait_all = [&](uint64_t *bar, uint32_t parity, bool at_once = false) {   // the warp's
        return __all_sync(0xFFFFFFFFu, wait_or_leave(bar, parity, &sm.gave_up, p.status, at_once));
    };
    // test builds: which role of this block gives up
    auto gives_up = [&](uint32_t role) { return kTestTimeout && blockIdx.x % 4 == role; };
    uint32_t issued = 0;         // blobs whose copies the copying warp has issued
    auto next_piece = [&]() -> const Piece * {   // the warp's next one, or none
        if (!wait_all(&sm.u_full[un % kKnown], un / kKnown & 1))
            return nullptr;
        const Piece *u = &sm.piece[un % kKnown];
        return u->there == 1 ? u : nullptr;
    };
    auto piece_over = [&](int n) {
        tiles_done += n;
        qn += n > 0;
        __syncwarp();
        if (lane == 0)
            bar_arrive(&sm.u_empty[un % kKnown]);
        ++un;
    };

    if (warp < kSoftWarps) {
        // ============================================================ scores
        const int i = warp >> 2, my = 32 * (warp & 3) + lane;   // accumulator; row or token of the tile
        const uint32_t s_at = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128 * i;
        const int window = p.a.window > 0 ? p.a.window : INT32_MAX;
        while (const Piece *up = next_piece()) {
            const Piece &u = *up;
            const int n = u.n, rows = min(kTile, u.rows - u.row0);
            const int x_lo = u.x0 + u.row0 / p.ratio, x_hi = u.x0 + (u.row0 + rows - 1) / p.ratio;
            const int rr = u.row0 + my;
            const int x = rr < u.rows ? u.x0 + rr / p.ratio : -1;       // (first pass)
            const float4 *row_f = sm.row[qn % kKnown];
            const float2 *inv_f = sm.inv[qn % kKnown];
            float m = kNone, l = 0.0f;
            float *out = a.sums + ((int64_t)u.h * a.tiles + first_tile(p, u.r, u.q_row0) + u.row0 / kTile) * a.tokens;
            // (not q_full, which may have gone on: a short piece's products do not wait for these warps)
            bool alive = n == 0 || wait_all(&sm.row_full[qn % kKnown], qn / kKnown & 1);
            float rho = 0.0f;
            if (!kSums && n > 0 && alive)
                rho = my & 1 ? row_f[my >> 1].y : row_f[my >> 1].x;
            // which of the piece's tiles are in the accumulator goes by how many the block has had, hence by timing;
            // the parts go by the tiles, so that the join adds in the same order whatever block had the piece
            const int half = (int)((i - tiles_done) & 1u);
            for (int j = half; j < n && alive; j += 2) {
                const uint32_t use = tiles_done + j;
                alive = wait_all(&sm.s_full[i], use >> 1 & 1, gives_up(0) && use == 2);
                if (!alive)
                    break;
                tmem_fence_after();
                const int vb0 = u.v0 + j * kBlobs;
                const int t0 = 16 * u.blob(vb0), t1 = 16 * u.blob(vb0 + kBlobs - 1) + 15;
                const uint32_t bad = *reinterpret_cast<volatile uint32_t *>(&sm.bad[use % kBadTiles]);
                const bool whole = bad == 0 && vb0 + kBlobs <= u.nb && t1 <= x_lo && (x_hi - t0 < window || t1 < p.a.sinks);
                if (!kSums) {
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float s[32];
                        tmem_ld32(s, s_at + 32 * c);
                        tmem_wait_ld();
                        float2 *z = reinterpret_cast<float2 *>(s);
                        const float2 rho2 = make_float2(rho, rho);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            z[e] = mul2(z[e], rho2);
                        if (!whole) {
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                const int in = 2 * c + b, vb = vb0 + in, tok = 16 * u.blob(vb);
                                // of the blob's 16 tokens the row sees those below `end`, from `low` on or below `sink`
                                const int end = vb < u.nb && !(bad >> in & 1) ? x + 1 - tok : 0;
                                const int64_t low64 = (int64_t)x + 1 - window - tok;
                                const int low = low64 < 0 ? 0 : (int)min(low64, (int64_t)16);
                                const int sink = p.a.sinks - tok;
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    s[16 * b + e] = e < end && (e >= low || e < sink) ? s[16 * b + e] : -INFINITY;
                            }
                        }
                        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                        for (int e = 4; e + 8 <= 32; e += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                top[k] = fmaxf(fmaxf(top[k], s[e + 2 * k]), s[e + 2 * k + 1]);
#pragma unroll
                        for (int e = 28; e < 32; ++e)
                            top[e & 3] = fmaxf(top[e & 3], s[e]);
                        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                        if (mx > m + 8.0f) {   // raised only when a score exceeds it by 2^8
                            l *= exp2_fast(m - mx);
                            m = mx;
                        }
                        const float2 m2 = make_float2(-m, -m);
                        float2 sum = make_float2(0.0f, 0.0f), sum_b = sum;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float2 y = add2(z[e], m2);
                            y.x = exp2_fast(y.x);
                            y.y = exp2_fast(y.y);
                            if (e & 1)
                                sum_b = add2(sum_b, y);
                            else
                                sum = add2(sum, y);
                        }
                        sum = add2(sum, sum_b);
                        l += sum.x + sum.y;
                    }
                    tmem_fence_before();
                    bar_arrive(&sm.s_empty[i]);
                } else {
                    // of the tile's rows the token is seen by those from c_lo on, below c_hi
                    const int vb = vb0 + (my >> 4), tok = 16 * u.blob(vb) + (my & 15);
                    const bool there = vb < u.nb && tok < u.kv && !(bad >> (my >> 4) & 1);
                    auto column = [&](int64_t x1) {
                        return (int)max(min((x1 - u.x0) * p.ratio - u.row0, (int64_t)kTile), (int64_t)0);
                    };
                    int c_lo = 0, c_hi = kTile;
                    if (!whole) {
                        c_lo = column(tok);
                        if (p.a.window > 0 && tok >= p.a.sinks)
                            c_hi = column((int64_t)tok + window);
                    }
                    float2 total = make_float2(0.0f, 0.0f);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float s[32];
                        tmem_ld32(s, s_at + 32 * c);
                        tmem_wait_ld();
                        float2 *z = reinterpret_cast<float2 *>(s);
                        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float4 f = row_f[16 * c + e];
                            z[e] = fma2(z[e], make_float2(f.x, f.y), make_float2(f.z, f.w));
                        }
                        if (!whole)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                s[e] = 32 * c + e >= c_lo && 32 * c + e < c_hi ? s[e] : -INFINITY;
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            sum = fma2(make_float2(exp2_fast(z[e].x), exp2_fast(z[e].y)), inv_f[16 * c + e], sum);
                        total = add2(total, sum);
                    }
                    tmem_fence_before();
                    bar_arrive(&sm.s_empty[i]);
                    if (vb < u.nb && tok < u.kv)
                        out[tok] = there ? total.x + total.y : 0.0f;
                }
            }
            if (!alive)
                break;
            if (!kSums)
                work.parts[((int64_t)u.item * 2 + half) * kTile + my] = make_float2(m, l);
            piece_over(n);
        }
    } else if (warp < kSoftWarps + kExpandWarps) {
        // ==================================================== queries, keys
        const int wi = warp - kSoftWarps, t = lane & 3, k8 = lane >> 2;
        const int half_tok = (k8 & 1) * 4 + (k8 >> 1);   // eight lanes' 16-byte stores meet all banks
        auto blob_issued = [&](uint32_t slot, uint32_t at) {   // false: a wait ran out
            const volatile uint32_t *blob = &sm.raw_blob[slot];
            uint64_t start = 0;
            for (uint32_t k = 0; (*blob ^ 2 * at) >> 1; ++k) {
                if ((k & 63) != 63)
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
        // chunk c of 8 columns of a row, in a tile of 64-column parts
        auto put = [&](uint8_t *tile, int row, int c, uint4 v) {
            *reinterpret_cast<uint4 *>(tile + (c >> 3) * kSub + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v;
        };
        // and of a row of 64 bytes
        auto put_group = [&](uint8_t *tile, int row, int c, uint4 v) {
            *reinterpret_cast<uint4 *>(tile + row * 64 + ((c ^ (row >> 1 & 3)) << 4)) = v;
        };
        uint32_t seq = 0;            // blobs of earlier pieces
        while (const Piece *up = next_piece()) {
            const Piece &u = *up;
            const int n = u.n;
            auto queries = [&]() {   // false: a wait ran out
                const int64_t slot = (int64_t)u.h * a.slots + first_slot(p, u.r, u.q_row0) + u.row0 / 8;
                constexpr int kRounds = kTile / 8 / kExpandWarps;
                uint4 v[kRounds][NW];      // on their way while the last piece's products end
#pragma unroll
                for (int i = 0; i < kRounds; ++i) {
                    const int row = u.row0 + 8 * (wi + kExpandWarps * i) + k8;
                    const bool there = row < u.rows;
                    const int qt = there ? row / p.ratio : 0, qh = u.h * p.ratio + (there ? row - qt * p.ratio : 0);
                    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.a.q) +
                                             (int64_t)(u.q_row0 + qt) * p.a.q_token_stride + qh * p.a.q_head_stride;
#pragma unroll
                    for (int w = 0; w < NW; ++w)
                        v[i][w] = there ? *reinterpret_cast<const uint4 *>(q + 32 * w + 8 * t) : make_uint4(0, 0, 0, 0);
                }
                if (!wait_all(&sm.q_empty, (qn & 1) ^ 1))   // the last piece's scores are done
                    return false;
                if (kSums)
                    grid_wait();   // for the rows' maxima and sums
#pragma unroll
                for (int i = 0; i < kRounds; ++i) {
                    const int in = 8 * (wi + kExpandWarps * i) + k8;
                    const bool there = u.row0 + in < u.rows;
                    uint32_t top = 0;        // largest |q| of the row (as bf16 bits, in both halves)
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        top = __vmaxu2(__vmaxu2(top, v[i][w].x & 0x7FFF7FFFu), v[i][w].y & 0x7FFF7FFFu);
                        top = __vmaxu2(__vmaxu2(top, v[i][w].z & 0x7FFF7FFFu), v[i][w].w & 0x7FFF7FFFu);
                    }
                    top = max(top & 0xFFFFu, top >> 16);
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    // the row times a power of two that brings it below 2^-7, and the sign of the scale
                    const int e = max((int)(top >> 7) - 127, -118);
                    const float up = pow2((-8 - e) >> 1), up2 = copysignf(pow2((-7 - e) >> 1), p.scale2);
                    const float rho = fabsf(p.scale2) * pow2((8 + e) >> 1) * pow2((9 + e) >> 1);
                    float sum[NG] = {};
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const uint4 c = v[i][w];
                        // channels i and i + 4 side by side, as the codes of a word come
                        const float f[8] = {par_s(c.x), par_s(c.z), par_lo(c.x), par_lo(c.z),
                                            par_s(c.y), par_s(c.w), par_lo(c.y), par_lo(c.w)};
                        put(sm.q, in, 4 * w + t, make_uint4(pack_bf16(f[0] * up * up2, f[1] * up * up2),
                                                            pack_bf16(f[2] * up * up2, f[3] * up * up2),
                                                            pack_bf16(f[4] * up * up2, f[5] * up * up2),
                                                            pack_bf16(f[6] * up * up2, f[7] * up * up2)));
                        sum[w / WPG] += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
                    }
                    float mine = 0.0f;       // of group t
#pragma unroll
                    for (int k = 0; k < NG; ++k) {
                        sum[k] += __shfl_xor_sync(0xFFFFFFFFu, sum[k], 1);
                        sum[k] += __shfl_xor_sync(0xFFFFFFFFu, sum[k], 2);
                        if (t == k)
                            mine = sum[k] * up * up2;
                    }
                    uint32_t part[3];
                    three_parts(mine, part);
                    if (t < kGroupChunks)   // 0 1 2 0 1 0 beside 0 0 0 1 1 2 of the keys
                        put_group(sm.qx, in, t, make_uint4(part[0] >> 16 | part[1], part[2] >> 16 | part[0], part[1] >> 16 | part[0], 0));
                    if (t == 0) {
                        float *f = reinterpret_cast<float *>(&sm.row[qn % kKnown][in >> 1]) + (in & 1);
                        f[0] = rho;
                        if (kSums) {
                            const float2 st = there ? a.stats[slot * 8 + in] : make_float2(0.0f, 0.0f);
                            f[2] = -st.x;
                            reinterpret_cast<float *>(&sm.inv[qn % kKnown][in >> 1])[in & 1] = st.y;
                        }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(&sm.row_full[qn % kKnown]);
                    bar_arrive(&sm.q_full);
                }
                return true;
            };
            bool alive = n == 0 || queries();
            static_assert(kExpandWarps == kBlobs);
            for (int b = wi; b < n * kBlobs && alive; b += kBlobs) {   // a blob of each tile
                const uint32_t use = tiles_done + (uint32_t)b / kBlobs, sl = use & 1, at = seq + b;
                const uint32_t slot = at % kPlaces;
                const int in_tile = b % kBlobs;
                // first that this blob was issued, which it is only into a place that was read: the barrier's
                // parity alone would say the same while the blob before it is on its way
                alive = __all_sync(0xFFFFFFFFu, blob_issued(slot, at)) &&
                        wait_all(&sm.raw_full[slot], at / kPlaces & 1, gives_up(1) && at == 5) &&
                        wait_all(&sm.k_empty[sl], (use >> 1 & 1) ^ 1);
                if (!alive)
                    break;
                const uint8_t *blob = sm.ring[slot];
                const bool there = sm.raw_blob[slot] & 1;
#pragma unroll
                for (int c8 = 0; c8 < 2; ++c8) {
                    const int tok = 8 * c8 + half_tok, row = 16 * in_tile + tok;
                    uint32_t code[NW], par[NG];
                    load_words(code, blob + B::kKCodes + tok * (D / 2) + t * (D / 8));
                    load_words(par, blob + B::kKParams + tok * 4 * NG);
                    // a lane of the token's four finds c of group t % NG; 128 + c, twice, for all
                    const uint32_t own = *reinterpret_cast<const uint32_t *>(blob + B::kKParams + (tok * NG + t % NG) * 4);
                    const float c_own = code_of_zero(own);
                    const uint32_t own_from = (0x4300u + (uint32_t)c_own) * 0x10001u;
                    uint32_t from[NG];
#pragma unroll
                    for (int k = 0; k < NG; ++k)
                        from[k] = NG == 1 ? own_from : __shfl_sync(0xFFFFFFFFu, own_from, (lane & ~3) | k);
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const uint32_t q = there ? par[w / WPG] : 0;
                        const uint32_t s2 = __byte_perm(q, q, 0x1010);
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t c = centred(code[w], k, from[w / WPG]);
                            hi[k] = mul_bf16x2(c, s2);
                            lo[k] = rest_of(c, s2, hi[k]);
                        }
                        put(sm.k[sl][0], row, 4 * w + t, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                        put(sm.k[sl][1], row, 4 * w + t, make_uint4(lo[0], lo[1], lo[2], lo[3]));
                    }
                    if (t < kGroupChunks) {
                        uint32_t part[3];
                        three_parts(t < NG && there ? fmaf(c_own, par_s(own), par_lo(own)) : 0.0f, part);
                        put_group(sm.kx[sl], row, t, make_uint4(part[0] >> 16 | part[0], part[0] >> 16 | part[1],
                                                          part[1] >> 16 | part[2], 0));
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(&sm.k_full[sl]);
                    bar_arrive(&sm.raw_empty[slot]);
                }
            }
            if (!alive)
                break;
            seq += n * kBlobs;
            piece_over(n);
        }
    } else if (warp == kSoftWarps + kExpandWarps) {
        // ==================================================== pieces, copies
        int u_r0 = 0;
        int64_t u_before = 0;
        auto find = [&](uint32_t which) {   // false: a wait ran out
            const uint32_t slot = which % kKnown;
            if (!wait_all(&sm.u_empty[slot], (which / kKnown & 1) ^ 1))
                return false;
            int64_t item = blockIdx.x;
            if (which > 0) {   // the next one that no block has
                grid_wait();   // for the counter's 0
                int32_t taken = 0;
                if (lane == 0)
                    taken = atomicAdd(a.taken + kSums, 1);
                item = gridDim.x + (int64_t)__shfl_sync(0xFFFFFFFFu, taken, 0);
            }
            find_piece(p, item, split, &u_r0, &u_before, &sm.piece[slot],
                       work, kSums ? nullptr : work.heads);
            if (lane == 0)
                bar_arrive(&sm.u_full[slot]);
            __syncwarp();
            return true;
        };
        find(0);   // a place that was never used: no wait
        while (const Piece *up = next_piece()) {
            const Piece &u = *up;
            const int32_t *table = p.a.block_table + u.r * p.a.table_stride;
            const int n = u.n;
            bool alive = true;
            for (int b0 = 0; b0 < n * kBlobs && alive; b0 += 32) {
                // 32 blobs (four tiles) are looked up at once, one by each lane
                const int vb = u.v0 + b0 + lane;
                const bool wanted = b0 + lane < n * kBlobs && vb < u.nb;
                const int blob = wanted ? u.blob(vb) : 0, page = blob / bpp;
                const int id = wanted ? table[page] : -1;
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
                    const uint32_t at = issued + lane % kIssue, slot = at % kPlaces;
                    alive = wait_all(&sm.raw_empty[slot], (at / kPlaces & 1) ^ 1, gives_up(2) && issued == kPlaces);
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
                            bar_expect(&sm.raw_full[slot], B::kVCodes);
                            bulk_copy(sm.ring[slot], p.layer + (uint64_t)place * 128, B::kVCodes, &sm.raw_full[slot]);
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
            piece_over(n);
        }
    } else {
        // ============================================================ products
        const uint32_t q_at = smem_addr(sm.q), qx_at = smem_addr(sm.qx), k_at = smem_addr(sm.k[0][0]), kx_at = smem_addr(sm.kx[0]);
        constexpr uint32_t kHalf = kTile * D * 2;   // bytes of the high or low parts of a tile
        while (const Piece *up = next_piece()) {
            const int n = up->n;
            bool left = false;       // a wait ran out
            if (elect_one()) {
                bool alive = n == 0 || wait(&sm.q_full, qn & 1);
                for (int j = 0; j < n && alive; ++j) {
                    const uint32_t use = tiles_done + j, sl = use & 1;
                    alive = wait(&sm.k_full[sl], use >> 1 & 1, gives_up(3) && use == 1) &&
                            wait(&sm.s_empty[sl], (use >> 1 & 1) ^ 1);
                    if (!alive)
                        break;
                    tmem_fence_after();
                    auto product = [&](uint32_t q, uint32_t k, uint32_t off, bool add) {
                        const uint32_t dq = smem_desc(q) + off, dk = smem_desc(k) + off;
                        mma_ss(tmem + 128 * sl, kSums ? dk : dq, kSums ? dq : dk, mma_desc(kTile), add);
                    };
                    const uint32_t dqx = smem_desc(qx_at), dkx = smem_desc(kx_at + sl * (kTile * 64));
                    // the small parts first: an accumulator loses most where it is large
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        product(q_at, k_at + (2 * sl + 1) * kHalf, ((kk >> 2) * kSub + (kk & 3) * 32) >> 4, kk > 0);
#pragma unroll
                    for (int kk = 0; kk < kGroupSteps<B>; ++kk)
                        mma_ss<kDescHigh64>(tmem + 128 * sl, (kSums ? dkx : dqx) + 2 * kk, (kSums ? dqx : dkx) + 2 * kk,
                                            mma_desc(kTile), true);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        product(q_at, k_at + 2 * sl * kHalf, ((kk >> 2) * kSub + (kk & 3) * 32) >> 4, true);
                    mma_commit(&sm.s_full[sl]);
                    mma_commit(&sm.k_empty[sl]);
                    if (j + 1 == n)
                        mma_commit(&sm.q_empty);
                }
                left = !alive;
            }
            if (__any_sync(0xFFFFFFFFu, left))
                break;
            piece_over(n);
        }
    }
    tmem_fence_before();
    __syncthreads();
    // Every role has left, so nothing is issued any more. After a wait that ran out, whichever
    // role it was, what is in flight ends before shared and tensor memory go.
    if (sm.gave_up) {
        if (warp == kSoftWarps + kExpandWarps) {
            for (uint32_t at = issued < kPlaces ? 0 : issued - kPlaces; at < issued; ++at)
                bar_wait(&sm.raw_full[at % kPlaces], at / kPlaces & 1);
        } else if (warp == kAllWarps - 1) {
            if (elect_one()) {   // the thread that issued the products
                mma_commit(&sm.last);
                bar_wait(&sm.last, 0);
            }
            __syncwarp();
        }
        __syncthreads();
    }
    if (warp == kAllWarps - 1) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem) : "memory");
    }
    grid_wait();
}

// A row's parts: of each piece of its unit, its even tiles and its odd ones. Slices of the block take them in turns.
constexpr int kJoinSlices = 4, kJoinThreads = kTile * kJoinSlices;

__global__ void __launch_bounds__(kJoinThreads) k_weigh_tiles_join(AttnArgs p, WeighArgs a, TileWork work)
{
    __shared__ float2 slices[kJoinSlices][kTile];
    const int row = threadIdx.x % kTile, slice = threadIdx.x / kTile;
    grid_next();
    grid_wait();
    for (int at = blockIdx.x; at < work.cut[0]; at += gridDim.x) {
        const Piece &u = work.heads[at];
        const int n = 2 * u.parts;
        const float2 *parts = work.parts + (int64_t)u.item * 2 * kTile + row;
        float mx = kNone, l = 0.0f;
#pragma unroll 8
        for (int k = slice; k < n; k += kJoinSlices) {
            const float2 part = parts[(int64_t)k * kTile];
            const float up = fmaxf(mx, part.x);
            l = l * exp2_fast(mx - up) + part.y * exp2_fast(part.x - up);
            mx = up;
        }
        slices[slice][row] = make_float2(mx, l);
        __syncthreads();
        if (slice == 0 && row < (min(kTile, u.rows - u.row0) + 7) / 8 * 8) {
            for (int k = 1; k < kJoinSlices; ++k)
                mx = fmaxf(mx, slices[k][row].x);
            l = 0.0f;
            for (int k = 0; k < kJoinSlices; ++k)
                l = fmaf(slices[k][row].y, exp2_fast(slices[k][row].x - mx), l);
            a.stats[((int64_t)u.h * a.slots + first_slot(p, u.r, u.q_row0) + u.row0 / 8) * 8 + row] =
                u.row0 + row < u.rows ? row_stats_of(mx, l) : make_float2(0.0f, 0.0f);
        }
        __syncthreads();
    }
}

// The sums of the row tiles that see a token, in their order.
constexpr int kAddThreads = 128;

__global__ void __launch_bounds__(kAddThreads) k_weigh_add(AttnArgs p, WeighArgs a)
{
    grid_wait();
    Items items = {0, 0};
    for (int64_t item = blockIdx.x;; item += gridDim.x) {
        AttnRequest q;
        int r, h, t0;
        if (!find_item(p, item, [&](const AttnRequest &x) { return x.rows > p.few_rows ? kAddThreads : 0; }, &items, &q, &r,
                       &h, &t0))
            return;
        const int tok = t0 + threadIdx.x, blob = tok / 16;
        if (tok >= q.kv)
            continue;
        // Row tile i sees the blob from where its last row reaches position 16 blob on: row (16 blob - x0) ratio;
        // under a window, if the blob is not of the first tokens, up to where its first row leaves the blob's
        // last token behind: position 16 blob + 15 + window.
        const int64_t from = (16 * (int64_t)blob - q.x0) * p.ratio, tiles = (q.rows + kTile - 1) / kTile;
        const int64_t i0 = from > 0 ? from / kTile : 0;
        int64_t i1 = tiles;
        if (p.a.window > 0 && blob >= ((int64_t)p.a.sinks + 15) / 16) {
            const int64_t rows = (16 * (int64_t)blob + 15 + p.a.window - q.x0) * p.ratio;   // that begin before
            i1 = rows <= 0 ? 0 : min(i1, (rows + kTile - 1) / kTile);
        }
        const float *sums = a.sums + ((int64_t)h * a.tiles + first_tile(p, r, q.row0)) * a.tokens + tok;
        float total = 0.0f;
#pragma unroll 8
        for (int64_t i = i0; i < i1; ++i)
            total += sums[i * a.tokens];
        const float had = a.w.in == nullptr ? 0.0f : a.w.in[r * a.w.in_request_stride + h * a.w.in_head_stride + tok];
        a.w.out[r * a.w.out_request_stride + h * a.w.out_head_stride + tok] = had + total;
    }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

struct TileSizes {
    int32_t tiles;
    size_t cut, heads, parts, sums;
    size_t bytes() const { return cut + heads + parts + sums; }
};

TileSizes sizes_of(const cg_int4_cache *c, const cg_attention *a, int32_t tokens)
{
    TileSizes z;
    z.tiles = (int32_t)((int64_t)a->tokens * (a->q_heads / c->num_heads) / kTile + a->requests + 1);
    const int64_t units = (int64_t)z.tiles * c->num_heads, items = units > kMaxBlocks ? units : kMaxBlocks;
    z.cut = 256;
    z.heads = align256((size_t)units * sizeof(Piece));
    z.parts = align256((size_t)items * 2 * kTile * sizeof(float2));
    z.sums = align256((size_t)units * tokens * sizeof(float));
    return z;
}

}  // namespace

size_t weigh_many_workspace(const cg_int4_cache *c, const cg_attention *a, int32_t tokens)
{
    return sizes_of(c, a, tokens).bytes();
}

int32_t *weigh_many_taken(void *ws) { return static_cast<int32_t *>(ws) + 1; }

cudaError_t weigh_many_launch(const AttnArgs &p, WeighArgs a, const cg_int4_cache *c, void *ws, cudaStream_t s)
{
    const TileSizes z = sizes_of(c, &p.a, a.tokens);
    uint8_t *at = static_cast<uint8_t *>(ws);
    TileWork work;
    work.most = z.tiles * c->num_heads;   // (fits: their sums are within the bound on those)
    work.cut = reinterpret_cast<int32_t *>(at);
    work.heads = reinterpret_cast<Piece *>(at += z.cut);
    work.parts = reinterpret_cast<float2 *>(at += z.heads);
    a.sums = reinterpret_cast<float *>(at += z.parts);
    a.tiles = z.tiles;
    int sms = 0;
    cudaError_t err = attn_sm_count(&sms);
    if (err != cudaSuccess)
        return err;
    const int blocks = sms < kMaxBlocks ? sms : kMaxBlocks;
    return int4_dispatch(c->head_size, c->group, [&](auto blob) {
        using B = decltype(blob);
        const int smem = (int)sizeof(TileShared<B>);
        cudaError_t e = cudaFuncSetAttribute(k_weigh_tiles<B, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k_weigh_tiles<B, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess)
            e = launch_under(k_weigh_tiles<B, false>, dim3(blocks), kAllThreads, smem, s, p, a, work);
        if (e == cudaSuccess)
            e = launch_under(k_weigh_tiles_join, dim3(2 * blocks), kJoinThreads, 0, s, p, a, work);
        if (e == cudaSuccess)
            e = launch_under(k_weigh_tiles<B, true>, dim3(blocks), kAllThreads, smem, s, p, a, work);
        if (e == cudaSuccess)
            e = launch_under(k_weigh_add, dim3(8 * blocks), kAddThreads, 0, s, p, a);
        return e;
    });
}

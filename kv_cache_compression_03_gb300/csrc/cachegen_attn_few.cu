// Attention over the 4-bit cache for few query rows per KV head: single
// tokens and a few drafted ones (up to 32 rows: query heads of the KV head
// times new tokens). Bound by HBM: D + 8 D/G bytes per token and head are read
// once, and the work on them has to keep pace with that.
//
// Mathematics. With k^ = lo + s n, q.k^ = sum_g s_g (q.n)_g + lo_g (sum q)_g, and
// sum_t p_t v^_t = sum_t (p_t s_t) (n_t - 8) + sum_t p_t (lo_t + 8 s_t): the matrix
// instructions take the codes themselves as bf16, which hold them exactly, and
// the group's parameters meet one score or one probability, not every value.
// A code becomes bf16 by one mask: a bf16 whose bits are 0 .. 255 (a subnormal
// or the first binade) is those bits times 2^-133, so the codes of bits 0..3 are
// n 2^-133 and those of bits 4..7 are n 2^-129 where they lie. The powers of two
// come off exactly: queries are scaled per row (and by 1/16 at the channels
// of the upper codes) so that their largest is near 2^126, p by 2^ve: 2^90, less where
// a large s or lo would overflow. Results keep their factor through both joins, so that
// no sum of p times a value leaves fp32's range whatever the value, and lose it together
// with sum p. Downwards fp32 ends at 2^-149: p s n 2^(ve - 133) loses bits where s is below
// about 2^-90, an error of 2^-149 2^(133 - ve) a step of 16 tokens. What is summed
// beside the codes is summed by matrix instructions too: lo (sum q) with sum q
// in two or three bf16 parts (16 bits at least), sum p s, sum p lo, sum p and
// sum p s 8 as rows of one small accumulator, with p in two bf16 parts as well.
// The one rounding that is left is that of p s to bf16 (2^-8 relative), for which
// p s is put together from p's parts in one multiply-add; with p rounded first the
// error against 64 bits was 0.0028 of the result, with this 0.0023, and 0.0017 is
// what the rounding of the result makes of it anyway. Scores, sums and the running
// maximum stay in fp32.
//
// Tiles. mma.sync m16n8k16 with the tokens (K) or channels (V) as the 16 rows
// and 8 query rows as columns, so 4 or 8 query heads fill an instruction that
// is idle to 15/16 with queries as rows. One warp takes a blob of 16 tokens at
// a time, alone: its own ring of bulk copies, its own running maximum and sum,
// no block barrier in the loop. The cache's layout puts the words that a
// thread of the instruction needs side by side: a blob's codes come in 16-byte
// shared loads without bank conflicts.
//
// Split. The batch's blobs, in the order request, KV head, row tile, token,
// are one line that the blocks cut into equal pieces, whatever the lengths.
// A piece that holds a (request, head, tile) whole writes its output; cut ones
// write their maximum, sum and accumulator, and a second kernel joins them in
// the order of the tokens, so results do not depend on timing.
//
// Measured (8 KV heads of 128, 32 query heads, groups of 32): 64 requests of 6K tokens
// on average 111 us, 4.6 TB/s where a copy reaches 6.8 (a floor of 74 us); 32 requests
// under a window of 4096 tokens 47 us; one request of 128K 46 us; the smallest call 12.6 us, of which the two
// launches make most. Issue slots are busy for 53 % of the time with 12 warps on an SM (168
// registers each), which wait on the chain codes -> scores -> p -> values of their own blob
// most. Rows 9 to 16 take 16 columns and 8 warps an SM; a third or fourth such tile would read
// the tokens again, so more rows go to the other kernel.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cg_attention.h"

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRing = 4;         // blobs in a warp's ring
constexpr int kMinPiece = 4 * kWarps;   // blobs of a block, at least
constexpr float kNone = -3.0e38f;   // no maximum yet; finite, so that differences are numbers
constexpr int kStartExp = 90;       // p is taken times 2^90 at first

// ---------------------------------------------------------------- schedule

// The blobs that a request's rows can see: [0, sink) and [sink + skip, ..),
// nb of them (at least 1, so that every row gets its output).
struct Span {
    int32_t nb, sink, skip;
};

__device__ __forceinline__ Span span_of(const AttnArgs &p, const AttnRequest &q)
{
    const int32_t end = (q.kv + 15) / 16;
    Span s = {end, 0, 0};
    if (p.a.window > 0) {
        const int64_t low = (int64_t)q.kv - q.nq + 1 - p.a.window;   // the first row's
        if (low > 0) {
            const int32_t first = (int32_t)(low / 16);
            const int64_t sb = ((int64_t)p.a.sinks + 15) / 16;
            s.sink = sb < first ? (int32_t)sb : first;
            s.skip = first - s.sink;
            s.nb = end - s.skip;
        }
    }
    if (s.nb < 1)
        s.nb = 1;
    return s;
}

template <int RU>
__device__ __forceinline__ int64_t work_of(const AttnArgs &p, int r, AttnRequest *q, uint32_t *error)
{
    if (!attn_request(p, r, q, error) || q->rows > p.few_rows)
        return 0;
    return (int64_t)((q->rows + RU - 1) / RU) * p.heads * span_of(p, *q).nb;
}

struct Place {   // a point of the line
    int32_t r;        // request (requests: past the end)
    int64_t off;      // blobs from the request's start
    AttnRequest q;
};

__device__ __forceinline__ int64_t piece_of(int64_t total, int pieces)
{
    // (64-bit division is slow, and seldom needed)
    const int64_t up = total + pieces - 1;
    const int64_t chunk = up >> 32 ? up / pieces : (int64_t)((uint32_t)up / (uint32_t)pieces);
    return chunk < kMinPiece ? kMinPiece : chunk;
}

// Block-wide: the line's length, the blobs of a piece, and the place of
// piece `piece` plus `plus`. Block 0 of the main kernel reports bad requests.
template <int RU>
__device__ __forceinline__ Place schedule(const AttnArgs &p, int pieces, int piece, int plus, bool report,
                                          int64_t *total_out, int64_t *chunk_out)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto work_at = [&](int r, AttnRequest *q, bool say) -> int64_t {
        if (r >= p.a.requests)
            return 0;
        uint32_t error;
        const int64_t w = work_of<RU>(p, r, q, &error);
        if (say && error != CG_OK)
            int4_set_status(p.status, error);
        return w;
    };
    auto scan = [&](int64_t w) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, w, d);
            if (lane >= d)
                w += o;
        }
        return w;
    };
    if (p.a.requests <= 32) {   // each warp for itself
        Place at = {p.a.requests, 0, {0, 0, 0, 0}};
        const int64_t w = work_at(lane, &at.q, report && warp == 0), inc = scan(w);
        *total_out = __shfl_sync(0xFFFFFFFFu, inc, 31);
        *chunk_out = piece_of(*total_out, pieces);
        const int64_t want = piece * *chunk_out + plus, start = inc - w;
        const uint32_t mine = __ballot_sync(0xFFFFFFFFu, want >= start && want < start + w);
        if (mine) {
            const int src = __ffs(mine) - 1;
            at.r = src;
            at.off = __shfl_sync(0xFFFFFFFFu, want - start, src);
            at.q.row0 = __shfl_sync(0xFFFFFFFFu, at.q.row0, src);
            at.q.nq = __shfl_sync(0xFFFFFFFFu, at.q.nq, src);
            at.q.kv = __shfl_sync(0xFFFFFFFFu, at.q.kv, src);
            at.q.rows = __shfl_sync(0xFFFFFFFFu, at.q.rows, src);
        }
        return at;
    }
    __shared__ int64_t warp_sum[kWarps];
    __shared__ Place found;
    const bool once = p.a.requests <= kThreads;
    int64_t total = 0, chunk = 0, want = -1;
    if (tid == 0)
        found.r = p.a.requests;
    for (int pass = 0; pass < 2; ++pass) {
        int64_t carry = 0;
        for (int r0 = 0; r0 < p.a.requests; r0 += kThreads) {
            const int r = r0 + tid;
            AttnRequest q;
            const int64_t w = work_at(r, &q, report && pass == 0), inc = scan(w);
            if (lane == 31)
                warp_sum[warp] = inc;
            __syncthreads();
            int64_t before = carry;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                if (i < warp)
                    before += warp_sum[i];
                carry += warp_sum[i];
            }
            __syncthreads();
            if (pass == 0 && once) {
                total = carry;
                chunk = piece_of(total, pieces);
                want = piece * chunk + plus;
            }
            const int64_t start = before + inc - w;
            if (want >= start && want < start + w)
                found = {r, want - start, q};
        }
        if (pass == 0) {
            if (once)
                break;
            total = carry;
            chunk = piece_of(total, pieces);
            want = piece * chunk + plus;
        }
    }
    __syncthreads();
    *total_out = total;
    *chunk_out = chunk;
    return found;
}

// A (request, head, row tile) and the stretch of its blobs in this piece.
struct Unit {
    int32_t r, h, rt, tiles;
    AttnRequest q;
    Span span;
    int32_t b0, b1;
};

// Finds the unit at a place; `left` blobs of the piece remain.
template <int RU>
__device__ __forceinline__ void unit_at(const AttnArgs &p, const Place &at, int64_t left, Unit *u)
{
    u->q = at.q;
    u->r = at.r;
    u->span = span_of(p, u->q);
    u->tiles = (u->q.rows + RU - 1) / RU;
    const int32_t i = at.off >> 31 ? (int32_t)(at.off / u->span.nb) : (int32_t)at.off / u->span.nb;
    u->h = i / u->tiles;
    u->rt = i - u->h * u->tiles;
    u->b0 = (int32_t)(at.off - (int64_t)i * u->span.nb);
    const int64_t end = u->b0 + left;
    u->b1 = end < u->span.nb ? (int32_t)end : u->span.nb;
}

// The next unit of the line (the caller knows that there is one).
template <int RU>
__device__ __forceinline__ void unit_next(const AttnArgs &p, int64_t left, Unit *u)
{
    if (++u->rt == u->tiles) {
        u->rt = 0;
        if (++u->h == p.heads) {
            u->h = 0;
            uint32_t error;
            while (++u->r < p.a.requests && work_of<RU>(p, u->r, &u->q, &error) == 0)
                ;
            if (u->r >= p.a.requests) {   // not reached while blobs are left
                u->b0 = u->b1 = 0;
                return;
            }
            u->span = span_of(p, u->q);
            u->tiles = (u->q.rows + RU - 1) / RU;
        }
    }
    u->b0 = 0;
    u->b1 = left < u->span.nb ? (int32_t)left : u->span.nb;
}

// A warp's stretch of a unit's blobs in this piece.
__device__ __forceinline__ void warp_range(const Unit &u, int warp, int *b, int *e)
{
    const int n = u.b1 - u.b0;
    *b = u.b0 + (int)((int64_t)n * warp / kWarps);
    *e = u.b0 + (int)((int64_t)n * (warp + 1) / kWarps);
}

// ------------------------------------------------------------ instructions

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same into a fresh accumulator.
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Codes i and i + 4 of a word as a bf16 pair: n 2^-133 for even i, n 2^-129 for
// odd i (bf16 bits 0 .. 255 count in steps of 2^-133).
__device__ __forceinline__ uint32_t codes_of(uint32_t w, int i)
{
    return (i < 2 ? w : w >> 8) & (i & 1 ? 0x00F000F0u : 0x000F000Fu);
}
constexpr uint32_t kEight = 0x00080008u;   // 8 2^-133, twice

__device__ __forceinline__ float pow2(int e)   // -126 <= e <= 127
{
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// ---------------------------------------------------------------- workspace

// Partial results: [block][2] of { float o[RU][D]; float4 (m, l, ve, unused)[RU]; },
// o times 2^(ve - kRoom). Slot 0 of a block belongs to a unit that began in an earlier
// block, slot 1 to one that goes on in the next.
template <int D, int RU>
constexpr int kPartFloats = RU *(D + 4);

// A warp's sums stay below 2^128 (see where the maximum is raised); four warps and up to
// kFewMaxBlocks parts are added with factors of at most 1.
constexpr int kRoom = 16;

// ------------------------------------------------------------- main kernel

// HB: blobs that a warp takes in one step. Two give its schedulers two
// independent chains and halve what a step costs besides (waits, votes, the
// next copy); with 16 rows (NT = 2) there are registers for one.
template <typename B, int NT>
struct FewShared {
    static constexpr int RU = 8 * NT, HB = NT == 1 ? 2 : 1, kStages = kRing / HB;
    uint8_t ring[kWarps][kStages][HB * B::kBytes];
    float merge[kWarps][RU][B::kD / NT];   // one of NT parts of the channels
    float m[kWarps][RU], l[kWarps][RU];
    int32_t ve[kWarps];
    uint64_t full[kWarps][kStages];
};

template <typename B, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) k_attention_few(AttnArgs p, float *parts)
{
    using S = FewShared<B, NT>;
    constexpr int D = B::kD, NW = B::kWords, NG = B::kGroups, WPG = NW / NG, RU = S::RU;
    constexpr int HB = S::HB, kStages = S::kStages;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;

    // the joining kernel's blocks may come up as this one's leave
    grid_next();
    if (lane == 0)
        for (int i = 0; i < kStages; ++i)
            bar_init(&sm.full[warp][i], HB);   // one arrival per blob of the step
    bar_init_fence();
    int64_t total, chunk;
    const Place at = schedule<RU>(p, gridDim.x, blockIdx.x, 0, blockIdx.x == 0, &total, &chunk);
    const int64_t begin = blockIdx.x * chunk;
    if (begin >= total)
        return;
    const int64_t count = (begin + chunk < total ? begin + chunk : total) - begin;

    const int bpp = p.page_tokens / 16;
    // ---- the warp's feeder: copies some steps ahead of the warp, through the same units.
    // Up to 32 blobs of the stretch are looked up at once, one by each lane, which then
    // issues its own blob's copy.
    Unit first;
    unit_at<RU>(p, at, count, &first);
    Unit fu = first;
    int64_t f_pos = fu.b1 - fu.b0;   // blobs of the piece up to the end of the feeder's unit
    int f_b, f_e;                    // blobs of the stretch not looked up yet
    warp_range(fu, warp, &f_b, &f_e);
    int f_i = 0, f_n = 0;            // blobs issued and looked up of the current 32
    uint32_t f_off = 0, f_ok = 0;    // the lane's blob (in 128-byte units of the layer); valid lanes
    uint32_t issued = 0;
    uint32_t ahead = 0;              // which blobs of the steps in flight are there, HB bits a step
    auto feed = [&]() {
        ahead >>= HB;
        if (f_i >= f_n) {
            while (f_b >= f_e) {
                if (f_pos >= count)
                    return;
                unit_next<RU>(p, count - f_pos, &fu);
                f_pos += fu.b1 - fu.b0;
                warp_range(fu, warp, &f_b, &f_e);
            }
            f_i = 0;
            f_n = f_e - f_b < 32 ? f_e - f_b : 32;
            int id = -1;
            if (lane < f_n && fu.q.kv > 0) {
                const int vb = f_b + lane, ab = vb < fu.span.sink ? vb : vb + fu.span.skip;
                const int page = ab / bpp;
                id = p.a.block_table[fu.r * p.a.table_stride + page];
                if ((unsigned)id >= (unsigned)p.num_pages)
                    int4_set_status(p.status, CG_ERR_CORRUPT);
                // at most num_pages * heads * page_tokens / 16 blobs: below 2^32 such units (cg_int4.h)
                f_off = (((uint32_t)id * p.heads + fu.h) * bpp + (ab - page * bpp)) * (B::kBytes / 128);
            }
            f_ok = __ballot_sync(0xFFFFFFFFu, (unsigned)id < (unsigned)p.num_pages);
            f_b += f_n;
        }
        const int st = issued & (kStages - 1);
        if ((unsigned)(lane - f_i) < (unsigned)HB) {
            uint64_t *bar = &sm.full[warp][st];
            if (f_ok >> lane & 1) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                bar_expect(bar, B::kBytes);
                bulk_copy(sm.ring[warp][st] + (lane - f_i) * B::kBytes, p.layer + (uint64_t)f_off * 128,
                          B::kBytes, bar);
            } else {
                bar_arrive(bar);
            }
        }
        ahead |= (f_ok >> f_i & ((1u << HB) - 1)) << (HB * (kStages - 1));
        f_i += HB;
        ++issued;
    };
    __syncwarp();
    for (int i = 0; i < kStages; ++i)
        feed();

    bool alive = true;               // no wait has run out
    uint32_t used = 0;
    Unit u = first;
    int64_t pos = 0;
    for (;;) {
        // ---- queries: column g of row tile nt is row rt * RU + 8 nt + g
        const int row_base = u.rt * RU;
        uint32_t qf[NT][NW][4];
        uint32_t qs[NT][2];          // scale2 times the sum of q in group t % NG, as parts of
                                     // which the product with (s, lo) takes the lo half
        float rho[NT][2];            // scale2 over the power of two in qf
        int x[NT][2];                // positions of rows 2t and 2t + 1 (-1: no such row)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = row_base + 8 * nt + g;
            const bool there = row < u.q.rows;
            const int qt = there ? row / p.ratio : 0, qh = u.h * p.ratio + (there ? row - qt * p.ratio : 0);
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.a.q) +
                                     (int64_t)(u.q.row0 + qt) * p.a.q_token_stride + qh * p.a.q_head_stride;
            uint4 v[NW];
            uint32_t top = 0;        // largest |q| of the row (as bf16 bits, in both halves)
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                v[w] = there ? *reinterpret_cast<const uint4 *>(q + 32 * w + 8 * t) : make_uint4(0, 0, 0, 0);
                top = __vmaxu2(top, v[w].x & 0x7FFF7FFFu);
                top = __vmaxu2(top, v[w].y & 0x7FFF7FFFu);
                top = __vmaxu2(top, v[w].z & 0x7FFF7FFFu);
                top = __vmaxu2(top, v[w].w & 0x7FFF7FFFu);
            }
            top = max(top & 0xFFFFu, top >> 16);
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            // exact: |q| 2^fe stays below 2^127; small rows (and 0) take the largest factor
            int fe = 126 - ((int)(top >> 7) - 127);
            fe = fe < 127 ? fe : 127;
            const float up = pow2(fe), up16 = pow2(fe - 4);
            // scale2 2^(133 - fe) in two steps, both upwards: the power alone may pass 2^127, and what
            // lies between passes fp32's range only where the result does
            const float back = p.scale2 * pow2((133 - fe) >> 1) * pow2((134 - fe) >> 1);
            float sum[NG] = {};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const uint4 c = v[w];
                // channels i and i + 4 side by side, as the codes of a word come
                qf[nt][w][0] = pack_bf16(par_s(c.x) * up, par_s(c.z) * up);
                qf[nt][w][1] = pack_bf16(par_lo(c.x) * up16, par_lo(c.z) * up16);
                qf[nt][w][2] = pack_bf16(par_s(c.y) * up, par_s(c.w) * up);
                qf[nt][w][3] = pack_bf16(par_lo(c.y) * up16, par_lo(c.w) * up16);
                sum[w / WPG] += par_s(c.x) + par_lo(c.x) + par_s(c.y) + par_lo(c.y) + par_s(c.z) +
                                par_lo(c.z) + par_s(c.w) + par_lo(c.w);
            }
            rho[nt][0] = __shfl_sync(0xFFFFFFFFu, back, 8 * t);
            rho[nt][1] = __shfl_sync(0xFFFFFFFFu, back, 8 * t + 4);
            float mine = 0.0f;       // of group t % NG, whole row
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 1);
                sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 2);
                if (t % NG == i)
                    mine = p.scale2 * sum[i];
            }
            uint32_t part[4] = {0, 0, 0, 0};   // high halves: mine, in descending parts
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                part[i] = pack_bf16(0.0f, mine);
                mine -= par_lo(part[i]);
            }
            if (NG == 4) {
                qs[nt][0] = part[0];
                qs[nt][1] = part[1];
            } else {
                qs[nt][0] = part[0];
#pragma unroll
                for (int i = 1; i < 4; ++i)
                    if (t / NG == i)
                        qs[nt][0] = part[i];
                qs[nt][1] = NG == 2 && t < 2 ? part[2] : 0;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int rr = row_base + 8 * nt + 2 * t + j;
                x[nt][j] = rr < u.q.rows ? u.q.kv - u.q.nq + rr / p.ratio : -1;
            }
        }
        // positions of the tile's first and last row: blobs that both see whole need no mask
        const int last_row = (row_base + RU < u.q.rows ? row_base + RU : u.q.rows) - 1;
        const int x_lo = u.q.kv - u.q.nq + row_base / p.ratio;
        const int x_hi = u.q.kv - u.q.nq + last_row / p.ratio;
        const int window = p.a.window > 0 ? p.a.window : INT32_MAX;

        float o[NW * 2][NT][4] = {};
        // rows of 16: g < NG sum p s_g, NG + g sum p lo_g, 8 + g sum p s_g 8 2^-133, 15 sum p
        float aux[NT][4] = {};
        uint32_t eight[NG];          // the rows 8 + g
#pragma unroll
        for (int gi = 0; gi < NG; ++gi)
            eight[gi] = g == gi ? kEight : 0;
        const uint32_t ones = g == 7 ? 0x3F803F80u : 0;
        const uint32_t par_sel = g < NG ? 0x5410u : 0x7632u;   // s or lo of two words
        const uint32_t par_keep = g < 2 * NG ? 0xFFFFFFFFu : 0;
        const int par_at = B::kVParams + 2 * t * 4 * NG + (g % NG) * 4;
        float m[NT][2];              // running maximum of the scores, less ve
        int ve = kStartExp;          // p is taken times 2^ve
        float limit = 8.0f + kStartExp;
        uint32_t par_bias = 0x80008000u - ((96 - kStartExp + 127) << 7) * 0x10001u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            m[nt][0] = m[nt][1] = kNone;

        int b, e;
        warp_range(u, warp, &b, &e);
        for (; b < e; b += HB) {
            const int st = used & (kStages - 1);
            if (alive) {
                const bool give_up = kTestTimeout && used == 1;
                if (give_up || !__all_sync(0xFFFFFFFFu, bar_wait(&sm.full[warp][st], (used / kStages) & 1))) {
                    alive = false;   // `used` stays: the first step not waited for
                    int4_set_status(p.status, CG_ERR_TIMEOUT);
                } else {
                    ++used;
                }
            }
            const uint32_t there = ahead & ((1u << HB) - 1);
            if (alive && there) {
                const uint8_t *ring = sm.ring[warp][st];
                float z[HB][NT][4];
                uint32_t va[HB][2];
                int tok[HB];
                bool whole = true;
#pragma unroll
                for (int hb = 0; hb < HB; ++hb) {
                    const uint8_t *blob = ring + hb * B::kBytes;
                    // ---- scores of tokens g and g + 8 with rows 2t and 2t + 1
                    uint32_t k0[NW], k1[NW], kp0[NG], kp1[NG];
                    load_words(k0, blob + B::kKCodes + g * (D / 2) + t * (D / 8));
                    load_words(k1, blob + B::kKCodes + (g + 8) * (D / 2) + t * (D / 8));
                    load_words(kp0, blob + B::kKParams + g * 4 * NG);
                    load_words(kp1, blob + B::kKParams + (g + 8) * 4 * NG);
                    float zl[NT][4];
#pragma unroll
                    for (int gi = 0; gi < NG; ++gi) {
                        float acc[NT][4];
#pragma unroll
                        for (int w = gi * WPG; w < (gi + 1) * WPG; ++w)
#pragma unroll
                            for (int i = 0; i < 4; i += 2) {
                                const uint32_t a0 = codes_of(k0[w], i), a1 = codes_of(k1[w], i);
                                const uint32_t a2 = codes_of(k0[w], i + 1), a3 = codes_of(k1[w], i + 1);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    if (w == gi * WPG && i == 0)
                                        mma16816_first(acc[nt], a0, a1, a2, a3, qf[nt][w][i], qf[nt][w][i + 1]);
                                    else
                                        mma16816(acc[nt], a0, a1, a2, a3, qf[nt][w][i], qf[nt][w][i + 1]);
                            }
                        const float s0 = par_s(kp0[gi]), s1 = par_s(kp1[gi]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                z[hb][nt][j] = gi ? fmaf(s0, acc[nt][j], z[hb][nt][j]) : s0 * acc[nt][j];
                                z[hb][nt][2 + j] =
                                    gi ? fmaf(s1, acc[nt][2 + j], z[hb][nt][2 + j]) : s1 * acc[nt][2 + j];
                            }
                    }
                    const uint32_t a0 = *reinterpret_cast<const uint32_t *>(blob + B::kKParams +
                                                                            (g * NG + t % NG) * 4);
                    const uint32_t a1 = *reinterpret_cast<const uint32_t *>(blob + B::kKParams +
                                                                            ((g + 8) * NG + t % NG) * 4);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816_first(zl[nt], a0, a1, a0, a1, qs[nt][0], qs[nt][1]);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            z[hb][nt][j] = fmaf(z[hb][nt][j], rho[nt][j & 1], zl[nt][j]);
                    }
                    // rows of the V parameters: s or lo of tokens 2t, 2t + 1 and 2t + 8, 2t + 9
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint8_t *at = blob + par_at + i * 8 * 4 * NG;
                        va[hb][i] = __byte_perm(*reinterpret_cast<const uint32_t *>(at),
                                                *reinterpret_cast<const uint32_t *>(at + 4 * NG), par_sel);
                        if (NG < 4)
                            va[hb][i] &= par_keep;
                    }
                    // a blob that was not copied lies behind every row
                    const int vb = b + hb;
                    tok[hb] = there >> hb & 1 ? 16 * (vb < u.span.sink ? vb : vb + u.span.skip) : 0x7FFFFFC0;
                    whole &= tok[hb] + 15 <= x_lo && (x_hi - tok[hb] < window || tok[hb] + 15 < p.a.sinks);
                }
                if (!whole) {
#pragma unroll
                    for (int hb = 0; hb < HB; ++hb) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int at_tok = tok[hb] + g + (j >= 2 ? 8 : 0), xr = x[nt][j & 1];
                                const bool sees =
                                    at_tok <= xr && (xr - at_tok < window || at_tok < p.a.sinks);
                                z[hb][nt][j] = sees ? z[hb][nt][j] : -INFINITY;
                            }
                        // parameters behind the last token may be anything
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int first = tok[hb] + 2 * t + 8 * i;
                            va[hb][i] &= first + 1 < u.q.kv ? 0xFFFFFFFFu : first < u.q.kv ? 0xFFFFu : 0u;
                        }
                    }
                }
                // ---- the running maximum is raised only when a score exceeds it by 2^8: p stays
                // below 2^(ve + 8) and rescaling is rare. Sums of p s and p lo have to stay finite
                // too: s and |lo| below 2^(96 - ve), and 2^21 tokens of a warp reach 2^125. (What
                // 2^-ve would make of them is not formed before they are divided by sum p.)
                float over = z[0][0][0] - m[0][0];
                uint32_t va_top = 0;
#pragma unroll
                for (int hb = 0; hb < HB; ++hb) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            over = fmaxf(over, z[hb][nt][j] - m[nt][j & 1]);
                    va_top = __vmaxu2(va_top, __vmaxu2(va[hb][0] & 0x7FFF7FFFu, va[hb][1] & 0x7FFF7FFFu));
                }
                const bool raise = over > limit, large = (va_top + par_bias) & 0x80008000u;
                if (__any_sync(0xFFFFFFFFu, raise || large)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float mx = fmaxf(z[0][nt][j], z[0][nt][2 + j]);
                            if (HB == 2)
                                mx = fmaxf(mx, fmaxf(z[HB - 1][nt][j], z[HB - 1][nt][2 + j]));
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1)
                                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
                            mx = fmaxf(mx - (float)ve, m[nt][j]);
                            const float f = exp2_fast(m[nt][j] - mx);
                            m[nt][j] = mx;
#pragma unroll
                            for (int c = 0; c < NW * 2; ++c) {
                                o[c][nt][j] *= f;
                                o[c][nt][2 + j] *= f;
                            }
                            aux[nt][j] *= f;
                            aux[nt][2 + j] *= f;
                        }
                    if (__any_sync(0xFFFFFFFFu, large)) {
                        uint32_t top = max(va_top & 0xFFFFu, va_top >> 16);
#pragma unroll
                        for (int d = 1; d < 32; d <<= 1)
                            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                        const int e = 95 - ((int)(top >> 7) - 127);   // top < 2^(96 - e)
                        const float f = pow2(e - ve);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
#pragma unroll
                                for (int c = 0; c < NW * 2; ++c)
                                    o[c][nt][j] *= f;
                                aux[nt][j] *= f;
                            }
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                m[nt][j] += (float)(ve - e);
                        }
                        ve = e;
                        limit = 8.0f + (float)e;
                        par_bias = 0x80008000u - (uint32_t)min((96 - e + 127) << 7, 0x7F80) * 0x10001u;
                    }
                }
#pragma unroll
                for (int hb = 0; hb < HB; ++hb) {
                    const uint8_t *blob = ring + hb * B::kBytes;
                    // p as the other factor (row g, tokens 2t, 2t + 1 and 8 more), in two bf16 parts
                    uint32_t pf[NT][2], pr[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            z[hb][nt][j] = exp2_fast(z[hb][nt][j] - m[nt][j & 1]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t big = pack_bf16(z[hb][nt][2 * j], z[hb][nt][2 * j + 1]);
                            const uint32_t rest = pack_bf16(z[hb][nt][2 * j] - par_s(big),
                                                            z[hb][nt][2 * j + 1] - par_lo(big));
                            pf[nt][j] = transpose8x8(big);
                            pr[nt][j] = transpose8x8(rest);
                        }
                        mma16816(aux[nt], va[hb][0], ones, va[hb][1], ones, pf[nt][0], pf[nt][1]);
                        mma16816(aux[nt], va[hb][0], ones, va[hb][1], ones, pr[nt][0], pr[nt][1]);
                    }
                    // ---- values
                    uint32_t v0[NW], v1[NW];
                    load_words(v0, blob + B::kVCodes + t * D + g * (D / 8));
                    load_words(v1, blob + B::kVCodes + (t + 4) * D + g * (D / 8));
#pragma unroll
                    for (int gi = 0; gi < NG; ++gi) {
                        const uint32_t s0 = __shfl_sync(0xFFFFFFFFu, va[hb][0], 4 * gi + t);
                        const uint32_t s1 = __shfl_sync(0xFFFFFFFFu, va[hb][1], 4 * gi + t);
                        uint32_t ps[NT][2];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            ps[nt][0] = fma_bf16x2(pf[nt][0], s0, mul_bf16x2(pr[nt][0], s0));
                            ps[nt][1] = fma_bf16x2(pf[nt][1], s1, mul_bf16x2(pr[nt][1], s1));
                            mma16816(aux[nt], 0, eight[gi], 0, eight[gi], ps[nt][0], ps[nt][1]);
                        }
#pragma unroll
                        for (int w = gi * WPG; w < (gi + 1) * WPG; ++w)
#pragma unroll
                            for (int i = 0; i < 4; i += 2) {
                                const uint32_t a0 = codes_of(v0[w], i), a1 = codes_of(v0[w], i + 1);
                                const uint32_t a2 = codes_of(v1[w], i), a3 = codes_of(v1[w], i + 1);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816(o[w * 2 + i / 2][nt], a0, a1, a2, a3, ps[nt][0], ps[nt][1]);
                            }
                    }
                }
            }
            __syncwarp();   // every lane has read the stage
            if (alive)
                feed();
        }

        // ---- the warps' results of this unit, joined in shared memory
        const float down = pow2(-ve);
        float off[NT][NG][2], ex[NT][NG][2];   // sum p (lo + 8 s) 2^-kRoom; sum p s 8, as o counts it
        if (lane == 0)
            sm.ve[warp] = ve;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    const float ps = __shfl_sync(0xFFFFFFFFu, aux[nt][j], 4 * gi + t);
                    const float pl = __shfl_sync(0xFFFFFFFFu, aux[nt][j], 4 * (NG + gi) + t);
                    off[nt][gi][j] = fmaf(ps, pow2(3 - kRoom), pl * pow2(-kRoom));
                    ex[nt][gi][j] = __shfl_sync(0xFFFFFFFFu, aux[nt][2 + j], 4 * gi + t);
                }
                m[nt][j] += (float)ve;
                if (g == 7) {
                    sm.m[warp][8 * nt + 2 * t + j] = m[nt][j];
                    sm.l[warp][8 * nt + 2 * t + j] = aux[nt][2 + j] * down;
                }
            }
        __syncthreads();
        const bool from_before = u.b0 > 0, goes_on = u.b1 < u.span.nb;
        float *part = parts + ((size_t)blockIdx.x * 2 + (from_before ? 0 : 1)) * kPartFloats<D, RU>;
        const int rows_here = last_row - row_base + 1;
        // the warps' results come to the least of their factors
        int v_least = ve;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v_least = min(v_least, sm.ve[w]);
        const float level = pow2(v_least - ve);
        float f[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float mx = kNone;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    mx = fmaxf(mx, sm.m[w][8 * nt + 2 * t + j]);
                f[nt][j] = exp2_fast(m[nt][j] - mx) * level;
            }
        constexpr int kPartW = NW / NT;   // words (32 channels) of a pass
        const float up = pow2(133 - kRoom);
#pragma unroll
        for (int pass = 0; pass < NT; ++pass) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int w = 0; w < kPartW; ++w) {
                        const int ww = pass * kPartW + w, gi = ww / WPG;
                        const float e8 = ex[nt][gi][j], add = off[nt][gi][j];
                        float4 v;    // channels 4g .. 4g + 3; the upper codes counted 16-fold
                        v.x = (o[2 * ww][nt][j] - e8) * up;
                        v.y = (fmaf(o[2 * ww][nt][2 + j], 0.0625f, -e8)) * up;
                        v.z = (o[2 * ww + 1][nt][j] - e8) * up;
                        v.w = (fmaf(o[2 * ww + 1][nt][2 + j], 0.0625f, -e8)) * up;
                        v = make_float4((v.x + add) * f[nt][j], (v.y + add) * f[nt][j],
                                        (v.z + add) * f[nt][j], (v.w + add) * f[nt][j]);
                        *reinterpret_cast<float4 *>(&sm.merge[warp][8 * nt + 2 * t + j][32 * w + 4 * g]) = v;
                    }
            __syncthreads();
            constexpr int kQuads = D / NT / 4;   // float4 per row
            for (int i = tid; i < rows_here * kQuads; i += kThreads) {
                const int row = i / kQuads, c = (i - row * kQuads) * 4;
                float mx = kNone, ls = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    mx = fmaxf(mx, sm.m[w][row]);
                float4 sum = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 v = *reinterpret_cast<const float4 *>(&sm.merge[w][row][c]);
                    sum.x += v.x;
                    sum.y += v.y;
                    sum.z += v.z;
                    sum.w += v.w;
                    const float mw = sm.m[w][row];
                    ls += sm.l[w][row] * exp2_fast(mw - mx);
                }
                const int ch = pass * (D / NT) + c;
                if (from_before || goes_on) {
                    *reinterpret_cast<float4 *>(part + row * D + ch) = sum;
                    if (pass == 0 && c == 0) {
                        reinterpret_cast<float4 *>(part + RU * D)[row] = make_float4(mx, ls, (float)v_least, 0.0f);
                    }
                } else {
                    const float inv = ls == 0.0f ? 0.0f : pow2(kRoom - v_least) / ls;
                    const int rr = row_base + row, qt = rr / p.ratio, qh = u.h * p.ratio + rr - qt * p.ratio;
                    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) +
                                         (int64_t)(u.q.row0 + qt) * p.a.out_token_stride +
                                         qh * p.a.out_head_stride + ch;
                    *reinterpret_cast<uint2 *>(out) =
                        make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
                }
            }
            __syncthreads();
        }
        pos += u.b1 - u.b0;
        if (pos >= count)
            break;
        unit_next<RU>(p, count - pos, &u);
    }
    // a wait that ran out: the copies still in flight, of the steps from that one on, must
    // land before the block's memory goes
    if (!alive)
        for (; used < issued; ++used)
            bar_wait(&sm.full[warp][used & (kStages - 1)], (used / kStages) & 1);
}

// ------------------------------------------------------------------- joining

// Block c joins the unit that begins in block c of the main kernel and goes
// on behind it, if there is one.
template <int D, int RU>
__global__ void __launch_bounds__(kThreads, 8) k_attention_join(AttnArgs p, int pieces, const float *parts)
{
    grid_next();
    int64_t total, chunk;
    const int c = blockIdx.x;
    // where the next piece starts: inside the unit, if one goes on
    const Place at = schedule<RU>(p, pieces, c + 1, 0, false, &total, &chunk);
    const int64_t border = (c + 1) * chunk;
    Unit u;
    if (border < total)
        unit_at<RU>(p, at, 1, &u);
    grid_wait();   // for the main kernel's parts
    if (border >= total || u.b0 == 0 || u.b0 > chunk)
        return;   // nothing there, or begins at the border, or before block c
    const int64_t end = border - u.b0 + u.span.nb;
    const int last = (int)((end + chunk - 1) / chunk) - 1;   // the block that holds its end
    const int row_base = u.rt * RU;
    const int rows_here = (row_base + RU < u.q.rows ? row_base + RU : u.q.rows) - row_base;
    // weights of the parts: 2^(m - max m), to the least of their factors, and the sums that they give
    extern __shared__ float weight[];   // [RU][parts]
    __shared__ float inv[RU];
    const int n = last - c + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto stats = [&](int k, int row) {
        const float *part = parts + ((size_t)(c + k) * 2 + (k == 0)) * kPartFloats<D, RU>;
        return reinterpret_cast<const float4 *>(part + RU * D)[row];
    };
    for (int row = warp; row < rows_here; row += kWarps) {
        float mx = kNone, l = 0.0f, least = (float)kStartExp;
        for (int k = lane; k < n; k += 32) {
            const float4 part = stats(k, row);
            mx = fmaxf(mx, part.x);
            least = fminf(least, part.z);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
            least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, d));
        }
        for (int k = lane; k < n; k += 32) {
            const float4 part = stats(k, row);
            const float e = exp2_fast(part.x - mx);
            weight[row * n + k] = e * pow2((int)(least - part.z));
            l = fmaf(part.y, e, l);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
            l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        if (lane == 0)
            inv[row] = l == 0.0f ? 0.0f : pow2(kRoom - (int)least) / l;
    }
    __syncthreads();
    constexpr int kQuads = D / 4;
    for (int i = threadIdx.x; i < rows_here * kQuads; i += kThreads) {
        const int row = i / kQuads, ch = (i - row * kQuads) * 4;
        float4 sum = make_float4(0, 0, 0, 0);
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
            const float4 v = *reinterpret_cast<const float4 *>(
                parts + ((size_t)(c + k) * 2 + (k == 0)) * kPartFloats<D, RU> + row * D + ch);
            const float e = weight[row * n + k];
            sum.x = fmaf(v.x, e, sum.x);
            sum.y = fmaf(v.y, e, sum.y);
            sum.z = fmaf(v.z, e, sum.z);
            sum.w = fmaf(v.w, e, sum.w);
        }
        const float f = inv[row];
        const int rr = row_base + row, qt = rr / p.ratio, qh = u.h * p.ratio + rr - qt * p.ratio;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) +
                             (int64_t)(u.q.row0 + qt) * p.a.out_token_stride + qh * p.a.out_head_stride + ch;
        *reinterpret_cast<uint2 *>(out) =
            make_uint2(pack_bf16(sum.x * f, sum.y * f), pack_bf16(sum.z * f, sum.w * f));
    }
}

// Row tiles of 8 or 16 query rows, by the most rows that a request can have.
int tile_rows(int max_rows) { return max_rows <= 8 ? 8 : 16; }

template <typename B, int NT>
cudaError_t launch(const AttnArgs &p, float *parts, cudaStream_t s)
{
    using Sh = FewShared<B, NT>;
    int sms = 0;
    cudaError_t err = attn_sm_count(&sms);
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(k_attention_few<B, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)sizeof(Sh));
    if (err != cudaSuccess)
        return err;
    int blocks = (NT == 1 ? 3 : 2) * sms;
    if (blocks > kFewMaxBlocks)
        blocks = kFewMaxBlocks;
    k_attention_few<B, NT><<<blocks, kThreads, sizeof(Sh), s>>>(p, parts);
    err = cudaGetLastError();
    if (err != cudaSuccess)
        return err;
    // launched while the main kernel still runs: its own schedule is worked out
    // meanwhile, and it waits for the main kernel before it reads the parts
    return launch_under(k_attention_join<B::kD, 8 * NT>, dim3(blocks), kThreads, 8 * NT * blocks * sizeof(float), s,
                        p, blocks, parts);
}

}  // namespace

size_t attn_few_workspace(int head_size, int max_rows)
{
    const int ru = tile_rows(max_rows);
    return (size_t)kFewMaxBlocks * 2 * ru * (head_size + 4) * sizeof(float);
}

cudaError_t attn_few_launch(const AttnArgs &p, int head_size, int group, int max_rows, void *ws,
                            cudaStream_t s)
{
    float *parts = static_cast<float *>(ws);
    return int4_dispatch(head_size, group, [&](auto blob) {
        using B = decltype(blob);
        return tile_rows(max_rows) == 8 ? launch<B, 1>(p, parts, s) : launch<B, 2>(p, parts, s);
    });
}

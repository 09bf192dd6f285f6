// The kernels that take the tokens of the 4-bit cache on the 16-row side of mma.sync (few
// query rows in attention, and the attention weights of tokens): how a batch's blobs are cut
// into pieces, and the instructions on codes.
#pragma once

#include "cg_attention.h"

// (a namespace of each file: the kernels for many rows have units of their own)
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMinPiece = 4 * kWarps;   // blobs of a block, at least
constexpr float kNone = -3.0e38f;   // no maximum yet; finite, so that differences are numbers

// ---------------------------------------------------------------- schedule

// What a kernel's batch has besides: shared tokens (as attn_request has it), and units that have to count as
// more blobs than they have (p.least_unit). Known to the compiler: looked at when a call runs, the two cost attention
// that has neither up to 1 us of its smallest call and 1 % of a prompt of 8192 tokens (558 us, 554 so).
template <bool kSharedTokens, bool kLeastUnit>
struct BatchOf {
    static constexpr bool kShared = kSharedTokens, kLeast = kLeastUnit;
};

// The blobs that a request's rows can see: [0, sink) and [sink + skip, ..),
// nb of them (at least 1, so that every row gets its output). A unit counts as nb blobs of the line;
// where it has to count as more than it has, `real` of them are there and pieces of the
// unit take as large a part of those.
struct Span {
    int32_t nb, sink, skip, real;
};

template <typename K>
__device__ __forceinline__ Span span_of(const AttnArgs &p, const AttnRequest &q)
{
    const int32_t end = (q.kv + 15) / 16;
    Span s = {end, 0, 0, end};
    if (p.a.window > 0) {
        const int64_t low = (int64_t)q.x0 + 1 - p.a.window;   // the first row's
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
    s.real = s.nb;
    if (K::kLeast && s.nb < p.least_unit)
        s.nb = p.least_unit;
    return s;
}

template <int RU, typename K>
__device__ __forceinline__ int64_t work_of(const AttnArgs &p, int r, AttnRequest *q, uint32_t *error)
{
    if (!attn_request<K::kShared>(p, r, q, error) || q->rows > p.few_rows)
        return 0;
    return (int64_t)((q->rows + RU - 1) / RU) * p.heads * span_of<K>(p, *q).nb;
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
template <int RU, typename K>
__device__ __forceinline__ Place schedule(const AttnArgs &p, int pieces, int piece, int plus, bool report,
                                          int64_t *total_out, int64_t *chunk_out)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto work_at = [&](int r, AttnRequest *q, bool say) -> int64_t {
        if (r >= p.a.requests)
            return 0;
        uint32_t error;
        const int64_t w = work_of<RU, K>(p, r, q, &error);
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
            at.q.x0 = __shfl_sync(0xFFFFFFFFu, at.q.x0, src);
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
template <int RU, typename K>
__device__ __forceinline__ void unit_at(const AttnArgs &p, const Place &at, int64_t left, Unit *u)
{
    u->q = at.q;
    u->r = at.r;
    u->span = span_of<K>(p, u->q);
    u->tiles = (u->q.rows + RU - 1) / RU;
    const int32_t i = at.off >> 31 ? (int32_t)(at.off / u->span.nb) : (int32_t)at.off / u->span.nb;
    u->h = i / u->tiles;
    u->rt = i - u->h * u->tiles;
    u->b0 = (int32_t)(at.off - (int64_t)i * u->span.nb);
    const int64_t end = u->b0 + left;
    u->b1 = end < u->span.nb ? (int32_t)end : u->span.nb;
}

// The next unit of the line (the caller knows that there is one).
template <int RU, typename K>
__device__ __forceinline__ void unit_next(const AttnArgs &p, int64_t left, Unit *u)
{
    if (++u->rt == u->tiles) {
        u->rt = 0;
        if (++u->h == p.heads) {
            u->h = 0;
            uint32_t error;
            while (++u->r < p.a.requests && work_of<RU, K>(p, u->r, &u->q, &error) == 0)
                ;
            if (u->r >= p.a.requests) {   // not reached while blobs are left
                u->b0 = u->b1 = 0;
                return;
            }
            u->span = span_of<K>(p, u->q);
            u->tiles = (u->q.rows + RU - 1) / RU;
        }
    }
    u->b0 = 0;
    u->b1 = left < u->span.nb ? (int32_t)left : u->span.nb;
}

// A warp's stretch of a unit's blobs in this piece.
template <typename K>
__device__ __forceinline__ void warp_range(const Unit &u, int warp, int *b, int *e)
{
    int b0 = u.b0, b1 = u.b1;
    if (K::kLeast && u.span.real != u.span.nb) {
        b0 = (int)((int64_t)b0 * u.span.real / u.span.nb);
        b1 = (int)((int64_t)b1 * u.span.real / u.span.nb);
    }
    const int n = b1 - b0;
    *b = b0 + (int)((int64_t)n * warp / kWarps);
    *e = b0 + (int)((int64_t)n * (warp + 1) / kWarps);
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

// ------------------------------------------------------------------- scores

// The queries of 8 rows of a KV head as the second factor of the instruction: column g is row
// row0 + g (0 where the request has no such row).
//   qf   the row times a power of two, 1/16 of it at the channels of the upper codes
//   qs   scale2 times the sum of q in group t % NG, as parts of which the product with (s, lo)
//        takes the lo half
//   rho  scale2 over the power of two in qf, of rows 2t and 2t + 1
template <typename B>
__device__ __forceinline__ void load_queries(const AttnArgs &p, const AttnRequest &rq, int h, int row0,
                                             uint32_t (&qf)[B::kWords][4], uint32_t (&qs)[2], float (&rho)[2])
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
        qf[w][0] = pack_bf16(par_s(c.x) * up, par_s(c.z) * up);
        qf[w][1] = pack_bf16(par_lo(c.x) * up16, par_lo(c.z) * up16);
        qf[w][2] = pack_bf16(par_s(c.y) * up, par_s(c.w) * up);
        qf[w][3] = pack_bf16(par_lo(c.y) * up16, par_lo(c.w) * up16);
        sum[w / WPG] += par_s(c.x) + par_lo(c.x) + par_s(c.y) + par_lo(c.y) + par_s(c.z) +
                        par_lo(c.z) + par_s(c.w) + par_lo(c.w);
    }
    rho[0] = __shfl_sync(0xFFFFFFFFu, back, 8 * t);
    rho[1] = __shfl_sync(0xFFFFFFFFu, back, 8 * t + 4);
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
        qs[0] = part[0];
        qs[1] = part[1];
    } else {
        qs[0] = part[0];
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (t / NG == i)
                qs[0] = part[i];
        qs[1] = NG == 2 && t < 2 ? part[2] : 0;
    }
}

// The scores (in powers of two) of a blob's tokens g and g + 8 with rows 2t and 2t + 1 of NT row
// tiles: z[nt] = (g, 2t), (g, 2t + 1), (g + 8, 2t), (g + 8, 2t + 1).
template <typename B, int NT>
__device__ __forceinline__ void blob_scores(const uint8_t *blob, const uint32_t (&qf)[NT][B::kWords][4],
                                            const uint32_t (&qs)[NT][2], const float (&rho)[NT][2],
                                            float (&z)[NT][4])
{
    constexpr int D = B::kD, NW = B::kWords, NG = B::kGroups, WPG = NW / NG;
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
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
                z[nt][j] = gi ? fmaf(s0, acc[nt][j], z[nt][j]) : s0 * acc[nt][j];
                z[nt][2 + j] = gi ? fmaf(s1, acc[nt][2 + j], z[nt][2 + j]) : s1 * acc[nt][2 + j];
            }
    }
    const uint32_t a0 = *reinterpret_cast<const uint32_t *>(blob + B::kKParams + (g * NG + t % NG) * 4);
    const uint32_t a1 = *reinterpret_cast<const uint32_t *>(blob + B::kKParams + ((g + 8) * NG + t % NG) * 4);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        mma16816_first(zl[nt], a0, a1, a0, a1, qs[nt][0], qs[nt][1]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            z[nt][j] = fmaf(z[nt][j], rho[nt][j & 1], zl[nt][j]);
    }
}

}  // namespace

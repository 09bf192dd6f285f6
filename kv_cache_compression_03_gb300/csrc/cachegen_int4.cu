// Store and load of the 4-bit paged cache (cg_int4_store, cg_int4_load).
//
// Per (token, head) row and group of G channels, lo = min x, s = bf16((max x
// - lo) (1 / 15)), n = min(15, rne((x - lo) / s)); the value is lo + s n. Both are
// streams (4 D bytes of bf16 against D + 8 D / G in the cache per token and head)
// bound by HBM; what has to keep pace is the work per value.
//
// A block takes up to 16 tokens of one layer, all heads. Where each token lies
// is worked out once, in shared memory, so that the rest is adds.
//
// Measured (8 heads of 128, groups of 32): load of 16384 tokens x 32 layers 404 us, at the copy
// rate, 6.8 TB/s; store of as many 634 us, 4.4 TB/s, bound by instruction issue (3.2 of 4 a
// cycle): 149 instructions for 8 values. What took it there from 2.4 ms: no division per value
// or per row, pairs of fp32 in one instruction (820 -> 778 us), a head's K and V rows read at
// once by the same threads (-> 667), six blocks on an SM at 40 registers (-> 635; seven spill).
// 64 tokens of one layer: 4.9 us for store and load.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cg_int4.h"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 16;   // tokens of a block
constexpr int kEnoughBlocks = 304;   // two on each of 152 SMs

struct RowArgs {
    uint8_t *data;
    void *status;
    size_t layer_bytes;   // one layer of the cache
    int32_t num_slots, page_tokens, heads, tile;
    uint16_t *k, *v;      // bf16 bits
    int64_t kl, kt, vl, vt;
    int32_t kh, vh;
    const int32_t *slots;
    int64_t tokens;
};

// Where the block's tokens lie: their rows of head 0, the blob of head 0, and the
// token in it (-1: a slot that is skipped). Blobs of the next heads follow at
// head_bytes().
struct Tile {
    uint16_t *row[2][kMaxTile];   // K, V
    uint8_t *blob[kMaxTile];
    int32_t tok[kMaxTile];
};

template <typename B>
__device__ __forceinline__ uint32_t head_bytes(const RowArgs &a)
{
    return (uint32_t)(a.page_tokens / 16) * B::kBytes;
}

template <typename B>
__device__ __forceinline__ int find_tile(const RowArgs &a, Tile &tile)
{
    const int64_t first = (int64_t)blockIdx.x * a.tile;
    const int n = (int)(a.tokens - first < a.tile ? a.tokens - first : a.tile);
    if (threadIdx.x < n) {
        const int slot = a.slots[first + threadIdx.x];
        tile.row[0][threadIdx.x] = a.k + blockIdx.y * a.kl + (first + threadIdx.x) * a.kt;
        tile.row[1][threadIdx.x] = a.v + blockIdx.y * a.vl + (first + threadIdx.x) * a.vt;
        int tok = -1;
        if (slot >= 0 && slot < a.num_slots) {
            const int page = slot / a.page_tokens, in = slot - page * a.page_tokens;
            tok = in & 15;
            tile.blob[threadIdx.x] = a.data + blockIdx.y * a.layer_bytes +
                                     (size_t)page * a.heads * head_bytes<B>(a) + (in >> 4) * B::kBytes;
        } else if (slot != -1) {
            int4_set_status(a.status, CG_ERR_CORRUPT);
        }
        tile.tok[threadIdx.x] = tok;
    }
    __syncthreads();
    return n;
}

// A thread's walk over (token, row) pairs, `rows` rows to a token, a fixed
// number of pairs apart.
struct Walk {
    int token, row, step_token, step_row, rows;
    __device__ __forceinline__ Walk(int at, int step, int rows_)
    {
        rows = rows_;
        token = at / rows;
        row = at - token * rows;
        step_token = step / rows;
        step_row = step - step_token * rows;
    }
    __device__ __forceinline__ void next()
    {
        token += step_token;
        row += step_row;
        if (row >= rows) {
            row -= rows;
            ++token;
        }
    }
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b)
{
    uint32_t c;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    uint32_t c;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

// bf16(fp32(range (1 / 15))), 1 / 15 in fp32: the format takes the product, which every
// device rounds alike, and not the quotient. The two are within two last bits of fp32, so
// s is the same but for one range in about 2^14, next to a border of the rounding to bf16.
__device__ __forceinline__ float scale_of(float range)
{
    return __bfloat162float(__float2bfloat16_rn(__fmul_rn(range, 1.0f / 15.0f)));
}

// Codes of 8 values: n = rne(d / s), d = x - lo. n0 = rne(d (1 / s)) is n or, next
// to a tie, its neighbour; e = d - n0 s is exact (both are multiples of d's last
// bit and e is below s), so |e| against s / 2 decides, with n even where they are
// equal. (The fp32 quotient of the definition rounds to k + 1/2 only where d / s is
// k + 1/2: 2 d - (2 k + 1) s is 0 or at least two last bits of d, more than half a
// last bit of the quotient times s.) So no division per value: a handful of
// multiply-adds, and the correction only in warps that have a value at a tie.
__device__ __forceinline__ uint32_t codes_of_row(const float (&x)[8], float lo, float s)
{
    constexpr float kMagic = 12582912.0f;   // 1.5 2^23: adding it rounds to whole numbers
    constexpr uint32_t kMagicBits = 0x4B400000u;
    float inv;   // n0 may be off by one next to a tie, so this need not be exact
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const float h = 0.5f * s;
    float r[8], e[8], top = 0.0f;
    const float2 lo2 = make_float2(-lo, -lo), inv2 = make_float2(inv, inv), s2 = make_float2(s, s);
    const float2 magic2 = make_float2(kMagic, kMagic), one2 = make_float2(-1.0f, -1.0f);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 d = add2(make_float2(x[j], x[j + 1]), lo2), n = fma2(d, inv2, magic2);
        const float2 f = fma2(fma2(n, one2, magic2), s2, d);
        r[j] = n.x, r[j + 1] = n.y;
        e[j] = f.x, e[j + 1] = f.y;
        top = fmaxf(fmaxf(top, fabsf(f.x)), fabsf(f.y));
    }
    if (top >= 0.9999f * h) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // one to the side of e where |e| > h, or = h with n0 odd
            const uint32_t bits = __float_as_uint(r[j]);
            const bool off = fabsf(e[j]) > __uint_as_float(__float_as_uint(h) - (bits & 1u));
            const uint32_t side = 1u | (uint32_t)(__float_as_int(e[j]) >> 31);
            r[j] = __uint_as_float(bits + (off ? side : 0u));
        }
    }
    // each r's bits are kMagicBits + n
    uint32_t code = 0u - kMagicBits * 0x11111111u;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        code += __float_as_uint(r[j]) << (4 * j);
    return code;
}

// The same by division, where s is too small for the above (its last bit, or its
// reciprocal, would leave fp32's normal range).
__device__ __forceinline__ uint32_t codes_of_tiny_row(const float (&x)[8], float lo, float s)
{
    uint32_t code = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        code |= (uint32_t)min(15, __float2int_rn(__fdiv_rn(__fsub_rn(x[j], lo), s))) << (4 * j);
    return code;
}

// A thread's 8 channels (16 bytes of bf16, one word of codes) of a row; the G / 8
// threads of a group reduce its range with shuffles. tok < 0: no row.
template <typename B, bool kIsV>
__device__ __forceinline__ void store_row(const uint4 &w, int tok, int chunk, uint8_t *blob, void *status)
{
    const int w32 = chunk / 4, part = chunk % 4;
    const float x[8] = {bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y),
                        bf_lo(w.z), bf_hi(w.z), bf_lo(w.w), bf_hi(w.w)};
    // the range two channels at a time; a NaN stays one through both
    uint32_t lo2 = min2(min2(w.x, w.y), min2(w.z, w.w)), hi2 = max2(max2(w.x, w.y), max2(w.z, w.w));
#pragma unroll
    for (int m = 1; m < B::kG / 8; m <<= 1) {
        lo2 = min2(lo2, __shfl_xor_sync(0xFFFFFFFFu, lo2, m));
        hi2 = max2(hi2, __shfl_xor_sync(0xFFFFFFFFu, hi2, m));
    }
    if (tok < 0)
        return;
    lo2 = min2(lo2, __byte_perm(lo2, lo2, 0x1032));
    hi2 = max2(hi2, __byte_perm(hi2, hi2, 0x1032));
    float lo = bf_lo(lo2), s = scale_of(__fsub_rn(bf_lo(hi2), lo));
    // inf or NaN in the group, or hi - lo overflows, or the largest value would round to inf
    if (!(__fmaf_rn(15.0f, s, lo) < 0x1.FFp127f)) {
        int4_set_status(status, CG_ERR_NONFINITE);
        s = lo = 0.0f;
    }
    uint32_t code = 0;
    if (s >= 0x1p-100f && s <= 0x1p120f)
        code = codes_of_row(x, lo, s);
    else if (s > 0.0f)
        code = codes_of_tiny_row(x, lo, s);
    if (!kIsV) {
        *reinterpret_cast<uint32_t *>(blob + B::kKCodes + tok * (B::kD / 2) + part * (B::kD / 8) + w32 * 4) = code;
    } else {
        uint8_t *p = blob + B::kVCodes + (tok >> 1) * B::kD + 2 * part * (B::kD / 8) + w32 * 4 + 2 * (tok & 1);
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)code;
        *reinterpret_cast<uint16_t *>(p + B::kD / 8) = (uint16_t)(code >> 16);
    }
    if (chunk % (B::kG / 8) == 0)
        *reinterpret_cast<uint32_t *>(blob + (kIsV ? B::kVParams : B::kKParams) +
                                      (tok * B::kGroups + chunk / (B::kG / 8)) * 4) = pack_bf16(s, lo);
}

// D / 8 threads to a head's K row and then its V row, both read at once.
template <typename B>
__global__ void __launch_bounds__(kThreads, 6) k_int4_store(RowArgs a)
{
    __shared__ Tile tile;
    constexpr int kChunks = B::kD / 8, kRowsAtOnce = kThreads / kChunks;
    const int n = find_tile<B>(a, tile);
    const int chunk = threadIdx.x % kChunks;
    const uint32_t per_head = head_bytes<B>(a);
    const int total = n * a.heads;
    Walk at(threadIdx.x / kChunks, kRowsAtOnce, a.heads);
    for (int i = threadIdx.x / kChunks; i - threadIdx.x / kChunks < total; i += kRowsAtOnce, at.next()) {
        const int tok = i < total ? tile.tok[at.token] : -1;
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        uint8_t *blob = nullptr;
        if (tok >= 0) {
            k = __ldcs(reinterpret_cast<const uint4 *>(tile.row[0][at.token] + (int64_t)at.row * a.kh) + chunk);
            v = __ldcs(reinterpret_cast<const uint4 *>(tile.row[1][at.token] + (int64_t)at.row * a.vh) + chunk);
            blob = tile.blob[at.token] + at.row * per_head;
        }
        store_row<B, false>(k, tok, chunk, blob, a.status);
        store_row<B, true>(v, tok, chunk, blob, a.status);
    }
}

// Load expands codes with one rounding (expand). s n has 12 bits, and one rounding to bf16
// gives what the format's two (to fp32, then to bf16) give wherever fp32 holds the sum, and
// where s n is far below half a last bit of lo. What is left is a lo that fp32 drops next to
// an s n halfway between two bf16 values, which is then rounded to the even one: the rows
// with such a group, which data hardly has, are found by tiny_lo() and written once more by
// load_twice_rounded(). (Both roundings for every code: 254 -> 318 us for 32768 tokens, 40
// layers of 2 heads.)
//
// Not 0 where lo != 0 is at most half a last bit of fp32 at 15 s: 2^20 |lo| < s, for pairs.
__device__ __forceinline__ uint32_t tiny_lo(uint32_t s, uint32_t lo)
{
    const uint32_t size = lo & 0x7FFF7FFFu;
    uint32_t big, less;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(big) : "r"(size), "r"(0x49804980u));
    asm("set.lt.u32.bf16x2 %0, %1, %2;" : "=r"(less) : "r"(big), "r"(s));   // all bits of a half
    return less & size;
}

// The block's rows as k_int4_load writes them, by the same threads, with both roundings. A
// loop of few registers: it is there for correctness alone.
template <typename B>
__device__ __forceinline__ void load_twice_rounded(const RowArgs &a, const Tile &tile, int n)
{
#pragma unroll 1
    for (int v = 0; v < 2; ++v) {
        const int per_row = v ? 8 : 4, chan = v ? 4 : 8;   // threads of a row, channels of a word
        const int g = threadIdx.x % per_row;
        // V's threads take two tokens at a time
        Walk at(threadIdx.x / per_row, kThreads / per_row, a.heads);
#pragma unroll 1
        for (; (v + 1) * at.token < n; at.next())
#pragma unroll 1
            for (int t = (v + 1) * at.token; t < (v + 1) * (at.token + 1) && t < n; ++t) {
                const int tok = tile.tok[t];
                if (tok < 0)
                    continue;
                const uint8_t *blob = tile.blob[t] + at.row * head_bytes<B>(a);
                const uint8_t *codes = blob + (v ? B::kVCodes + (tok >> 1) * B::kD + 2 * (tok & 1)
                                                 : B::kKCodes + tok * (B::kD / 2)) + g * (B::kD / 8);
                const uint8_t *pars = blob + (v ? B::kVParams : B::kKParams) + tok * 4 * B::kGroups;
                uint16_t *to = tile.row[v][t] + (int64_t)at.row * (v ? a.vh : a.kh) + chan * g;
#pragma unroll 1
                for (int i = 0; i < B::kWords * chan; ++i) {
                    const int w = i / chan, c = i - w * chan;
                    const uint32_t code = codes[4 * w + c / 2] >> (4 * (c & 1)) & 15u;
                    const uint32_t q = *reinterpret_cast<const uint32_t *>(pars + 4 * (32 * w / B::kG));
                    to[32 * w + c] = (uint16_t)pack_bf16(__fmaf_rn((float)code, par_s(q), par_lo(q)), 0.0f);
                }
            }
    }
}

// K: four threads to a row, each the words of its eighth channels (16 bytes of
// codes at D = 128, 16-byte stores). V: eight threads to a row and two tokens at
// a time, since the cache keeps pairs of tokens in one word; where the tokens are
// no pair each reads its own half.
template <typename B>
__global__ void __launch_bounds__(kThreads) k_int4_load(RowArgs a)
{
    __shared__ Tile tile;
    constexpr int NW = B::kWords, NG = B::kGroups, WPG = NW / NG;
    const int n = find_tile<B>(a, tile);
    const uint32_t per_head = head_bytes<B>(a);
    uint32_t tiny = 0;
    {
        const int t = threadIdx.x & 3;
        Walk at(threadIdx.x / 4, kThreads / 4, a.heads);
        for (; at.token < n; at.next()) {
            const int tok = tile.tok[at.token];
            uint16_t *dst = tile.row[0][at.token] + (int64_t)at.row * a.kh + 8 * t;
            if (tok < 0) {
#pragma unroll
                for (int w = 0; w < NW; ++w)
                    __stcs(reinterpret_cast<uint4 *>(dst + 32 * w), make_uint4(0, 0, 0, 0));
                continue;
            }
            const uint8_t *blob = tile.blob[at.token] + at.row * per_head;
            uint32_t code[NW], par[NG];
            load_words(code, blob + B::kKCodes + tok * (B::kD / 2) + t * (B::kD / 8));
            load_words(par, blob + B::kKParams + tok * 4 * NG);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const uint32_t q = par[w / WPG], s = __byte_perm(q, q, 0x1010), lo = __byte_perm(q, q, 0x3232);
                tiny |= tiny_lo(s, lo);
                const uint32_t y0 = expand(code[w], 0, s, lo), y1 = expand(code[w], 1, s, lo);
                const uint32_t y2 = expand(code[w], 2, s, lo), y3 = expand(code[w], 3, s, lo);
                __stcs(reinterpret_cast<uint4 *>(dst + 32 * w),
                       make_uint4(__byte_perm(y0, y1, 0x5410), __byte_perm(y2, y3, 0x5410),
                                  __byte_perm(y0, y1, 0x7632), __byte_perm(y2, y3, 0x7632)));
            }
        }
    }
    {
        const int g = threadIdx.x & 7;
        Walk at(threadIdx.x / 8, kThreads / 8, a.heads);
        for (; 2 * at.token < n; at.next()) {
            const int t0 = 2 * at.token, t1 = t0 + 1 < n ? t0 + 1 : t0;
            const int tok0 = tile.tok[t0], tok1 = tile.tok[t1];
            const bool pair = t1 > t0 && tok0 >= 0 && !(tok0 & 1) && tok1 == tok0 + 1 && tile.blob[t0] == tile.blob[t1];
            const int64_t in_row = (int64_t)at.row * a.vh + 4 * g;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (e == 1 && (pair || t1 == t0))
                    break;
                const int tok = e ? tok1 : tok0;
                uint16_t *to = tile.row[1][e ? t1 : t0] + in_row;
                if (tok < 0) {
#pragma unroll
                    for (int w = 0; w < NW; ++w)
                        __stcs(reinterpret_cast<uint2 *>(to + 32 * w), make_uint2(0, 0));
                    continue;
                }
                const uint8_t *blob = tile.blob[e ? t1 : t0] + at.row * per_head;
                uint32_t code[NW], par0[NG], par1[NG];
                load_words(code, blob + B::kVCodes + (tok >> 1) * B::kD + g * (B::kD / 8));
                load_words(par0, blob + B::kVParams + (tok & ~1) * 4 * NG);
                load_words(par1, blob + B::kVParams + (tok | 1) * 4 * NG);
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const uint32_t s = __byte_perm(par0[w / WPG], par1[w / WPG], 0x5410);
                    const uint32_t lo = __byte_perm(par0[w / WPG], par1[w / WPG], 0x7632);
                    tiny |= tiny_lo(s, lo);
                    const uint32_t y0 = expand(code[w], 0, s, lo), y1 = expand(code[w], 1, s, lo);
                    const uint32_t y2 = expand(code[w], 2, s, lo), y3 = expand(code[w], 3, s, lo);
                    const uint2 even = make_uint2(__byte_perm(y0, y1, 0x5410), __byte_perm(y2, y3, 0x5410));
                    const uint2 odd = make_uint2(__byte_perm(y0, y1, 0x7632), __byte_perm(y2, y3, 0x7632));
                    __stcs(reinterpret_cast<uint2 *>(to + 32 * w), tok & 1 ? odd : even);
                    if (pair)
                        __stcs(reinterpret_cast<uint2 *>(tile.row[1][t1] + in_row + 32 * w), odd);
                }
            }
        }
    }
    if (tiny)
        load_twice_rounded<B>(a, tile, n);
}

__global__ void k_int4_take_error(uint32_t *status, uint4 *result)
{
    *result = make_uint4(atomicExch(status, 0u), 0, 0, 0);
}

// Checks of both calls; *work is false where there is nothing to do.
cg_status check_rows(const cg_int4_cache *c, int32_t first_layer, int32_t layers,
                     const cg_kv_rows *rows, const int32_t *slots, int64_t tokens, RowArgs *a,
                     bool *work)
{
    const cg_status st = int4_check(c);
    if (st != CG_OK)
        return st;
    if (first_layer < 0 || layers < 0 || first_layer > c->num_layers ||
        layers > c->num_layers - first_layer || tokens < 0 || rows == nullptr)
        return CG_ERR_INVALID_ARG;
    *work = layers > 0 && tokens > 0;
    if (!*work)
        return CG_OK;
    const int64_t strides[6] = {rows->k_layer_stride, rows->k_token_stride, rows->k_head_stride,
                                rows->v_layer_stride, rows->v_token_stride, rows->v_head_stride};
    for (int64_t s : strides)
        if (s < 0 || s % 8 != 0)
            return CG_ERR_INVALID_ARG;
    if (rows->k == nullptr || rows->v == nullptr || slots == nullptr ||
        !int4_aligned(rows->k, 16) || !int4_aligned(rows->v, 16) || !int4_aligned(slots, 4))
        return CG_ERR_INVALID_ARG;
    if (tokens >= ((int64_t)1 << 31) || layers > 65535)   // the grid's limits
        return CG_ERR_UNSUPPORTED;
    // 16 tokens to a block, fewer where that would leave SMs idle
    a->tile = kMaxTile;
    while (a->tile > 1 && (tokens + a->tile - 1) / a->tile * layers < kEnoughBlocks)
        a->tile /= 2;
    a->layer_bytes = (size_t)c->num_pages * int4_page_bytes(c);
    a->data = static_cast<uint8_t *>(c->data) + (size_t)first_layer * a->layer_bytes;
    a->status = c->status;
    a->num_slots = c->num_pages * c->page_tokens;
    a->page_tokens = c->page_tokens;
    a->heads = c->num_heads;
    a->k = static_cast<uint16_t *>(rows->k);
    a->v = static_cast<uint16_t *>(rows->v);
    if (strides[2] > INT32_MAX || strides[5] > INT32_MAX)
        return CG_ERR_UNSUPPORTED;
    a->kl = strides[0];
    a->kt = strides[1];
    a->kh = (int32_t)strides[2];
    a->vl = strides[3];
    a->vt = strides[4];
    a->vh = (int32_t)strides[5];
    a->slots = slots;
    a->tokens = tokens;
    return CG_OK;
}

dim3 row_grid(const RowArgs &a, int32_t layers)
{
    return dim3((unsigned)((a.tokens + a.tile - 1) / a.tile), (unsigned)layers);
}

}  // namespace

extern "C" cg_status cg_int4_cache_bytes(const cg_int4_cache *c, size_t *bytes)
{
    if (c == nullptr || bytes == nullptr)
        return CG_ERR_INVALID_ARG;
    const cg_status st = int4_check_shape(c);
    if (st != CG_OK)
        return st;
    *bytes = (size_t)c->num_layers * c->num_pages * int4_page_bytes(c);
    return CG_OK;
}

extern "C" cg_status cg_int4_take_error(const cg_int4_cache *c, void *result, cg_stream_t stream)
{
    const cg_status st = int4_check(c);
    if (st != CG_OK)
        return st;
    if (result == nullptr || !int4_aligned(result, 16))
        return CG_ERR_INVALID_ARG;
    k_int4_take_error<<<1, 1, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        static_cast<uint32_t *>(c->status), static_cast<uint4 *>(result));
    return cudaGetLastError() == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

extern "C" cg_status cg_int4_store(const cg_int4_cache *c, int32_t first_layer, int32_t layers,
                                   const cg_kv_rows *rows, const int32_t *slots, int64_t tokens,
                                   cg_stream_t stream)
{
    RowArgs a;
    bool work = false;
    const cg_status st = check_rows(c, first_layer, layers, rows, slots, tokens, &a, &work);
    if (st != CG_OK || !work)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid = row_grid(a, layers);
    const cudaError_t err = int4_dispatch(c->head_size, c->group, [&](auto blob) {
        k_int4_store<decltype(blob)><<<grid, kThreads, 0, s>>>(a);
        return cudaGetLastError();
    });
    return err == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

extern "C" cg_status cg_int4_load(const cg_int4_cache *c, int32_t first_layer, int32_t layers,
                                  const cg_kv_rows *rows, const int32_t *slots, int64_t tokens,
                                  cg_stream_t stream)
{
    RowArgs a;
    bool work = false;
    const cg_status st = check_rows(c, first_layer, layers, rows, slots, tokens, &a, &work);
    if (st != CG_OK || !work)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid = row_grid(a, layers);
    const cudaError_t err = int4_dispatch(c->head_size, c->group, [&](auto blob) {
        k_int4_load<decltype(blob)><<<grid, kThreads, 0, s>>>(a);
        return cudaGetLastError();
    });
    return err == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

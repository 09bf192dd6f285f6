// Store and load of the 4-bit paged cache (cg_int4_store, cg_int4_load).
//
// Per (token, head) row and group of G channels, lo = min x, s = bf16((max x
// - lo) / 15), n = min(15, rne((x - lo) / s)); the value is lo + s n.
// A thread owns 8 channels (16 bytes of bf16, one word of codes); the G / 8
// threads of a group reduce its range with shuffles.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cg_int4.h"

namespace {

constexpr int kThreads = 256;

struct RowArgs {
    uint8_t *data;
    void *status;
    size_t layer_bytes;   // one layer of the cache
    int32_t num_slots, page_tokens, heads;
    uint16_t *k, *v;      // bf16 bits
    int64_t kl, kt, kh, vl, vt, vh;
    const int32_t *slots;
    int64_t tokens;
};

// Address of the blob that holds a slot of head h, and the token in it.
template <typename B>
__device__ __forceinline__ uint8_t *blob_of(const RowArgs &a, int layer, int slot, int h, int *tok)
{
    const int page = slot / a.page_tokens, in = slot - page * a.page_tokens;
    *tok = in & 15;
    const size_t blobs = a.page_tokens / 16;
    return a.data + (size_t)layer * a.layer_bytes +
           (((size_t)page * a.heads + h) * blobs + (in >> 4)) * B::kBytes;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <typename B>
__global__ void __launch_bounds__(kThreads) k_int4_store(RowArgs a)
{
    constexpr int kChunks = B::kD / 8;   // threads of a row
    const int64_t per_token = (int64_t)2 * a.heads * kChunks;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t tok_i = i / per_token;
    const int r = (int)(i - tok_i * per_token);
    const int chunk = r % kChunks, h = r / kChunks % a.heads, is_v = r / kChunks / a.heads;
    const int layer = blockIdx.y;
    const bool there = tok_i < a.tokens;
    const int slot = there ? a.slots[tok_i] : -1;
    const bool ok = slot >= 0 && slot < a.num_slots;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (ok) {
        const uint16_t *src = is_v ? a.v + layer * a.vl + tok_i * a.vt + h * a.vh
                                   : a.k + layer * a.kl + tok_i * a.kt + h * a.kh;
        w = __ldcs(reinterpret_cast<const uint4 *>(src) + chunk);
    } else if (slot < -1 || slot >= a.num_slots) {
        int4_set_status(a.status, CG_ERR_CORRUPT);
    }
    const float x[8] = {bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y),
                        bf_lo(w.z), bf_hi(w.z), bf_lo(w.w), bf_hi(w.w)};
    float lo = x[0], hi = x[0], any = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        lo = fminf(lo, x[j]);
        hi = fmaxf(hi, x[j]);
        any = fmaf(x[j], 0.0f, any);   // NaN once a value is inf or NaN
    }
#pragma unroll
    for (int m = 1; m < B::kG / 8; m <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, m));
        any += __shfl_xor_sync(0xFFFFFFFFu, any, m);
    }
    if (!ok)
        return;
    float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f)));
    if (any != 0.0f || isinf(s)) {     // any is 0 or NaN
        int4_set_status(a.status, CG_ERR_NONFINITE);
        s = lo = 0.0f;
    }
    uint32_t code = 0;
    if (s > 0.0f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int n = min(15, __float2int_rn(__fdiv_rn(__fsub_rn(x[j], lo), s)));
            code |= (uint32_t)n << (4 * j);
        }
    }
    int tok;
    uint8_t *blob = blob_of<B>(a, layer, slot, h, &tok);
    const int w32 = chunk / 4, part = chunk % 4;
    if (!is_v) {
        *reinterpret_cast<uint32_t *>(blob + B::kKCodes + tok * (B::kD / 2) +
                                      part * (B::kD / 8) + w32 * 4) = code;
    } else {
        uint8_t *p = blob + B::kVCodes + (tok >> 1) * B::kD + 2 * part * (B::kD / 8) + w32 * 4 +
                     2 * (tok & 1);
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)code;
        *reinterpret_cast<uint16_t *>(p + B::kD / 8) = (uint16_t)(code >> 16);
    }
    if (chunk % (B::kG / 8) == 0) {
        const int g = chunk / (B::kG / 8);
        *reinterpret_cast<uint32_t *>(blob + (is_v ? B::kVParams : B::kKParams) +
                                      (tok * B::kGroups + g) * 4) = pack_bf16(s, lo);
    }
}

template <typename B>
__global__ void __launch_bounds__(kThreads) k_int4_load(RowArgs a)
{
    constexpr int kChunks = B::kD / 8;
    const int64_t per_token = (int64_t)2 * a.heads * kChunks;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t tok_i = i / per_token;
    if (tok_i >= a.tokens)
        return;
    const int r = (int)(i - tok_i * per_token);
    const int chunk = r % kChunks, h = r / kChunks % a.heads, is_v = r / kChunks / a.heads;
    const int layer = blockIdx.y;
    const int slot = a.slots[tok_i];
    uint4 out = make_uint4(0, 0, 0, 0);
    if (slot >= 0 && slot < a.num_slots) {
        int tok;
        const uint8_t *blob = blob_of<B>(a, layer, slot, h, &tok);
        const int w32 = chunk / 4, part = chunk % 4;
        uint32_t code;
        if (!is_v) {
            code = *reinterpret_cast<const uint32_t *>(blob + B::kKCodes + tok * (B::kD / 2) +
                                                       part * (B::kD / 8) + w32 * 4);
        } else {
            const uint8_t *p = blob + B::kVCodes + (tok >> 1) * B::kD + 2 * part * (B::kD / 8) +
                               w32 * 4 + 2 * (tok & 1);
            code = *reinterpret_cast<const uint16_t *>(p) |
                   (uint32_t)*reinterpret_cast<const uint16_t *>(p + B::kD / 8) << 16;
        }
        const uint32_t par = *reinterpret_cast<const uint32_t *>(
            blob + (is_v ? B::kVParams : B::kKParams) +
            (tok * B::kGroups + chunk / (B::kG / 8)) * 4);
        const float s = par_s(par), lo = par_lo(par);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = __fadd_rn(lo, __fmul_rn(s, (float)((code >> (4 * j)) & 15u)));
        out = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                         pack_bf16(y[6], y[7]));
    } else if (slot != -1) {
        int4_set_status(a.status, CG_ERR_CORRUPT);
    }
    uint16_t *dst = is_v ? a.v + layer * a.vl + tok_i * a.vt + h * a.vh
                         : a.k + layer * a.kl + tok_i * a.kt + h * a.kh;
    __stcs(reinterpret_cast<uint4 *>(dst) + chunk, out);
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
    // the grid's limits: 2^31 - 1 blocks, 65,535 layers
    const int64_t threads = tokens * 2 * c->num_heads * (c->head_size / 8);
    if (tokens >= ((int64_t)1 << 31) || (threads + kThreads - 1) / kThreads >= ((int64_t)1 << 31) ||
        layers > 65535)
        return CG_ERR_UNSUPPORTED;
    a->layer_bytes = (size_t)c->num_pages * int4_page_bytes(c);
    a->data = static_cast<uint8_t *>(c->data) + (size_t)first_layer * a->layer_bytes;
    a->status = c->status;
    a->num_slots = c->num_pages * c->page_tokens;
    a->page_tokens = c->page_tokens;
    a->heads = c->num_heads;
    a->k = static_cast<uint16_t *>(rows->k);
    a->v = static_cast<uint16_t *>(rows->v);
    a->kl = strides[0];
    a->kt = strides[1];
    a->kh = strides[2];
    a->vl = strides[3];
    a->vt = strides[4];
    a->vh = strides[5];
    a->slots = slots;
    a->tokens = tokens;
    return CG_OK;
}

dim3 row_grid(const cg_int4_cache *c, int32_t layers, int64_t tokens)
{
    const int64_t threads = tokens * 2 * c->num_heads * (c->head_size / 8);
    return dim3((unsigned)((threads + kThreads - 1) / kThreads), (unsigned)layers);
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
    const dim3 grid = row_grid(c, layers, tokens);
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
    const dim3 grid = row_grid(c, layers, tokens);
    const cudaError_t err = int4_dispatch(c->head_size, c->group, [&](auto blob) {
        k_int4_load<decltype(blob)><<<grid, kThreads, 0, s>>>(a);
        return cudaGetLastError();
    });
    return err == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

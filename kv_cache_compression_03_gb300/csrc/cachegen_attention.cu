// cg_int4_attention: attention of new tokens over one layer of the 4-bit
// paged cache, out_i = sum_j p_ij v^_j with p_i = softmax_j(scale q_i . k^_j)
// over the visible tokens j, in one pass over them with the running maximum
// and sum of the softmax.
//
// The simplest form: one warp per (query row, query head), a token at a time.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cg_attention.h"

namespace {

constexpr int kThreads = 128;

// The request of a query row: last r with cu[r] <= t. False where cu does
// not place t in one valid request.
__device__ __forceinline__ bool request_of(const AttnArgs &p, int t, int *r, int *n, int *i)
{
    const int32_t *cu = p.a.cu_q;
    int lo = 0, hi = p.a.requests;
    if (hi == 0 || cu[0] > t)
        return false;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    *r = lo;
    *n = cu[lo + 1] - cu[lo];
    *i = t - cu[lo];
    return cu[lo + 1] > t && cu[lo + 1] <= p.a.tokens && cu[lo] >= 0;
}

template <typename B>
__global__ void __launch_bounds__(kThreads) k_attention_rows(AttnArgs p)
{
    constexpr int kCh = B::kD / 32;   // channels of a lane: kCh lane ..
    const cg_attention &a = p.a;
    const int lane = threadIdx.x & 31;
    for (int64_t r = (int64_t)blockIdx.x * kThreads + threadIdx.x; r < a.requests;
         r += (int64_t)gridDim.x * kThreads)
        if (a.cu_q[r] < 0 || a.cu_q[r + 1] < a.cu_q[r] || a.cu_q[r + 1] > a.tokens)
            int4_set_status(p.status, CG_ERR_CORRUPT);
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= (int64_t)a.tokens * a.q_heads)
        return;
    const int t = (int)(row / a.q_heads), qh = (int)(row % a.q_heads);
    const int h = qh / (a.q_heads / p.heads);
    int r, n, i;
    if (!request_of(p, t, &r, &n, &i) || n * p.ratio <= p.few_rows)
        return;
    const int kv = a.kv_lens[r];
    if (kv < 0 || (int64_t)kv > (int64_t)a.table_width * p.page_tokens) {
        int4_set_status(p.status, CG_ERR_CORRUPT);
        return;
    }
    if (a.max_q_len > 0 && n > a.max_q_len) {
        int4_set_status(p.status, CG_ERR_INVALID_ARG);
        return;
    }
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + t * a.q_token_stride +
                             qh * a.q_head_stride;
    float qf[kCh], o[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        qf[c] = __bfloat162float(q[lane * kCh + c]);
        o[c] = 0.0f;
    }
    const int c0 = lane * kCh, w32 = c0 / 32;
    const int koff = (c0 % 32) / 8 * (B::kD / 8) + w32 * 4 + (c0 % 8) / 2;
    const int voff = (c0 % 32) / 4 * (B::kD / 8) + w32 * 4 + (c0 % 4) / 2;
    const int g = c0 / B::kG;
    const int64_t x = (int64_t)kv - n + i;
    const int end = (int)(x + 1 < kv ? (x + 1 > 0 ? x + 1 : 0) : kv);
    const int64_t low = a.window > 0 ? x + 1 - a.window : 0;
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j < end; ++j) {
        if (j < low && j >= a.sinks) {
            j = (int)low - 1;
            continue;
        }
        const int page = a.block_table[r * a.table_stride + j / p.page_tokens];
        if (page < 0 || page >= p.num_pages) {
            int4_set_status(p.status, CG_ERR_CORRUPT);
            continue;
        }
        const int in = j % p.page_tokens, tok = in & 15;
        const uint8_t *blob = p.layer + (((size_t)page * p.heads + h) * (p.page_tokens / 16) +
                                         (in >> 4)) * B::kBytes;
        const uint32_t kp = *reinterpret_cast<const uint32_t *>(blob + B::kKParams +
                                                                (tok * B::kGroups + g) * 4);
        const uint32_t vp = *reinterpret_cast<const uint32_t *>(blob + B::kVParams +
                                                                (tok * B::kGroups + g) * 4);
        const uint8_t *kc = blob + B::kKCodes + tok * (B::kD / 2) + koff;
        const uint8_t *vc = blob + B::kVCodes + (tok >> 1) * B::kD + 2 * (tok & 1) + voff;
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < kCh; ++c)
            dot = fmaf(qf[c], fmaf(par_s(kp), (float)(kc[c / 2] >> (4 * (c & 1)) & 15), par_lo(kp)),
                       dot);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
        const float score = dot * a.scale * 1.4426950408889634f;   // in powers of two
        const float mn = fmaxf(m, score);
        const float f = exp2f(m - mn), e = exp2f(score - mn);
        m = mn;
        l = l * f + e;
#pragma unroll
        for (int c = 0; c < kCh; ++c)
            o[c] = o[c] * f +
                   e * fmaf(par_s(vp), (float)(vc[c / 2] >> (4 * (c & 1)) & 15), par_lo(vp));
    }
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + t * a.out_token_stride +
                         qh * a.out_head_stride;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int c = 0; c < kCh; c += 2)
        *reinterpret_cast<uint32_t *>(out + c0 + c) = pack_bf16(o[c] * inv, o[c + 1] * inv);
}

// The call's sizes (not its pointers).
cg_status check_sizes(const cg_int4_cache *c, const cg_attention *a)
{
    const cg_status st = int4_check_shape(c);
    if (st != CG_OK)
        return st;
    if (a->requests < 0 || a->tokens < 0 || a->q_heads <= 0 || a->q_heads % c->num_heads != 0 ||
        a->max_q_len < 0 || a->window < 0 || a->sinks < 0 || a->table_width < 0 ||
        a->table_stride < a->table_width || !isfinite(a->scale))
        return CG_ERR_INVALID_ARG;
    if (a->requests > CG_MAX_REQUESTS ||
        (int64_t)a->table_width * c->page_tokens >= ((int64_t)1 << 31) ||
        (int64_t)a->tokens * a->q_heads >= ((int64_t)1 << 31))
        return CG_ERR_UNSUPPORTED;
    return CG_OK;
}

constexpr int kFewRows = 64;

// Most rows of one KV head that a request can have (query heads times tokens).
int64_t max_rows(const cg_int4_cache *c, const cg_attention *a)
{
    const int n = a->max_q_len > 0 && a->max_q_len < a->tokens ? a->max_q_len : a->tokens;
    return (int64_t)n * (a->q_heads / c->num_heads);
}

}  // namespace

extern "C" cg_status cg_int4_attention_workspace(const cg_int4_cache *c, const cg_attention *a,
                                                 size_t *bytes)
{
    if (c == nullptr || a == nullptr || bytes == nullptr)
        return CG_ERR_INVALID_ARG;
    const cg_status st = check_sizes(c, a);
    if (st != CG_OK)
        return st;
    const int64_t rows = max_rows(c, a);
    *bytes = attn_few_workspace(c->head_size, (int)(rows < kFewRows ? rows : kFewRows));
    return CG_OK;
}

extern "C" cg_status cg_int4_attention(const cg_int4_cache *c, int32_t layer,
                                       const cg_attention *a, void *workspace,
                                       size_t workspace_bytes, cg_stream_t stream)
{
    cg_status st = int4_check(c);
    if (st != CG_OK)
        return st;
    size_t need = 0;
    st = cg_int4_attention_workspace(c, a, &need);
    if (st != CG_OK)
        return st;
    if (layer < 0 || layer >= c->num_layers)
        return CG_ERR_INVALID_ARG;
    if (a->requests == 0 || a->tokens == 0)
        return CG_OK;
    if (a->q == nullptr || a->out == nullptr || a->cu_q == nullptr || a->kv_lens == nullptr ||
        (a->block_table == nullptr && a->table_width > 0) || !int4_aligned(a->q, 16) ||
        !int4_aligned(a->out, 16) || !int4_aligned(a->cu_q, 4) || !int4_aligned(a->kv_lens, 4) ||
        !int4_aligned(a->block_table, 4) || !int4_aligned(workspace, 256))
        return CG_ERR_INVALID_ARG;
    const int64_t strides[4] = {a->q_token_stride, a->q_head_stride, a->out_token_stride,
                                a->out_head_stride};
    for (int64_t s : strides)
        if (s < 0 || s % 8 != 0)
            return CG_ERR_INVALID_ARG;
    if (workspace_bytes < need || (need > 0 && workspace == nullptr))
        return CG_ERR_CAPACITY;
    AttnArgs p;
    p.layer = static_cast<const uint8_t *>(c->data) +
              (size_t)layer * c->num_pages * int4_page_bytes(c);
    p.status = c->status;
    p.num_pages = c->num_pages;
    p.page_tokens = c->page_tokens;
    p.heads = c->num_heads;
    p.ratio = a->q_heads / c->num_heads;
    p.few_rows = kFewRows;
    p.scale2 = a->scale * 1.4426950408889634f;
    p.a = *a;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t most = max_rows(c, a);
    cudaError_t err = attn_few_launch(p, c->head_size, c->group,
                                      (int)(most < kFewRows ? most : kFewRows), workspace, s);
    if (err == cudaSuccess && most > kFewRows) {
        const int64_t rows = (int64_t)a->tokens * a->q_heads;
        const unsigned grid = (unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32));
        err = int4_dispatch(c->head_size, c->group, [&](auto blob) {
            k_attention_rows<decltype(blob)><<<grid, kThreads, 0, s>>>(p);
            return cudaGetLastError();
        });
    }
    return err == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

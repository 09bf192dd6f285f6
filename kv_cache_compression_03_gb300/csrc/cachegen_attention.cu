// cg_int4_attention: attention of new tokens over one layer of the 4-bit
// paged cache, out_i = sum_j p_ij v^_j with p_i = softmax_j(scale q_i . k^_j)
// over the visible tokens j. Checks, and the choice between the kernel for few
// rows (bound by reading the cache) and the one for many (bound by the products).

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "cg_attention.h"

namespace {

constexpr float kLog2E = 1.4426950408889634f;   // scores are taken in powers of two

// The call's sizes (not its pointers).
cg_status check_sizes(const cg_int4_cache *c, const cg_attention *a)
{
    const cg_status st = int4_check_shape(c);
    if (st != CG_OK)
        return st;
    if (a->requests < 0 || a->tokens < 0 || a->q_heads <= 0 || a->q_heads % c->num_heads != 0 ||
        a->max_q_len < 0 || a->window < 0 || a->sinks < 0 || a->table_width < 0 ||
        a->table_stride < a->table_width || !isfinite(a->scale * kLog2E))
        return CG_ERR_INVALID_ARG;
    if (a->requests > CG_MAX_REQUESTS ||
        (int64_t)a->table_width * c->page_tokens >= ((int64_t)1 << 31) ||
        (int64_t)a->tokens * a->q_heads >= ((int64_t)1 << 31))
        return CG_ERR_UNSUPPORTED;
    return CG_OK;
}

// Requests with up to this many rows per KV head go to the kernel for few rows,
// which works on 16 at a time and reads the tokens again for each 16; the other
// expands them once for up to 256. Here and there, 8 KV heads of 128: 20 rows,
// eight requests at 16K, 116 us and 127 us; 32 rows, four at 128K, 389 and 427,
// 64 at 1K, 86 and 82; 48 rows, four at 128K, 569 and 428, 16 at 2K, 62 and 44.
constexpr int kFewRows = 32;

// Most rows of one KV head that a request can have (query heads times tokens).
int64_t max_rows(const cg_int4_cache *c, const cg_attention *a)
{
    const int n = a->max_q_len > 0 && a->max_q_len < a->tokens ? a->max_q_len : a->tokens;
    return (int64_t)n * (a->q_heads / c->num_heads);
}

// The workspace's part for the kernel for few rows.
size_t few_bytes(const cg_int4_cache *c, int64_t rows)
{
    const size_t n = attn_few_workspace(c->head_size, (int)(rows < kFewRows ? rows : kFewRows));
    return (n + 255) / 256 * 256;
}

}  // namespace

cudaError_t attn_sm_count(int *sms)
{
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    const bool keep = dev >= 0 && dev < 64;
    *sms = keep ? known[dev].load(std::memory_order_relaxed) : 0;
    if (*sms == 0) {
        err = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
        if (err == cudaSuccess && keep)
            known[dev].store(*sms, std::memory_order_relaxed);
    }
    return err;
}

extern "C" cg_status cg_int4_attention_workspace(const cg_int4_cache *c, const cg_attention *a,
                                                 size_t *bytes)
{
    if (c == nullptr || a == nullptr || bytes == nullptr)
        return CG_ERR_INVALID_ARG;
    const cg_status st = check_sizes(c, a);
    if (st != CG_OK)
        return st;
    // a part each: the two kernels may run side by side
    const int64_t rows = max_rows(c, a);
    *bytes = few_bytes(c, rows);
    if (rows > kFewRows)
        *bytes += attn_many_workspace(c->head_size);
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
    p.scale2 = a->scale * kLog2E;
    p.a = *a;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t most = max_rows(c, a);
    cudaError_t err = attn_few_launch(p, c->head_size, c->group,
                                      (int)(most < kFewRows ? most : kFewRows), workspace, s);
    if (err == cudaSuccess && most > kFewRows)
        err = attn_many_launch(p, c->head_size, c->group,
                               static_cast<uint8_t *>(workspace) + few_bytes(c, most), s);
    return err == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

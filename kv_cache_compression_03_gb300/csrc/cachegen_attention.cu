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

// And all of a batch's rows of one KV head.
int64_t all_rows(const cg_int4_cache *c, const cg_attention *a)
{
    return (int64_t)a->tokens * (a->q_heads / c->num_heads);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// The workspace's part for the kernel for few rows.
size_t few_bytes(const cg_int4_cache *c, int64_t rows)
{
    return align256(attn_few_workspace(c->head_size, (int)(rows < kFewRows ? rows : kFewRows)));
}

size_t pass_bytes(const cg_int4_cache *c, int64_t rows, bool first)
{
    if (rows <= kFewRows)
        return few_bytes(c, rows);
    // a part each: the two kernels may run side by side
    if (first)
        return align256(attn_many_workspace(c->head_size, attn_many_items(rows, c->num_heads)));
    return few_bytes(c, rows) + align256(attn_many_workspace(c->head_size, 0));
}

// Shared tokens: whether a pass of their own pays. Each request reading them costs instructions and the L2's
// rate, not memory's, and what it costs more than two passes' launches, joins, starts and ends must be there
// first. Estimates in us, from measurements (152 SMs; 32 query heads of 128, 500 tokens of a request's own):
//   requests, queries, KV heads    shared    one pass    two
//   32, 1, 8                         2048        35       43
//                                    8192        80       49
//   8, 1, 8                          8192        33       45
//                                   32768        76       64
//   16, 4, 2 (64 rows)               8192        51       68
//                                   32768       119       88
//   8, 100, 8 (400 rows)             8192       157      192
//                                   32768       531      481
#ifdef CG_TEST_SHARED_TWO
constexpr bool kTestTwoPasses = true;   // test builds: whatever the sizes
#else
constexpr bool kTestTwoPasses = kTestTimeout;
#endif

bool two_passes(const cg_int4_cache *c, const cg_attention *a, int32_t shared)
{
    if (kTestTwoPasses)
        return true;
    const int64_t requests = a->requests > 0 ? a->requests : 1, all = all_rows(c, a), heads = c->num_heads;
    const int64_t most = max_rows(c, a), each = most < all / requests + 1 ? most : all / requests + 1;
    const int64_t tiles = (shared + 127) / 128;   // of 128 tokens; rows come in units of 256
    const double bytes = (double)shared * heads * (int4_blob_bytes(c->head_size, c->group) / 16);
    // bytes a us out of the L2, of blobs that take as many instructions with half the channels
    const double rate = c->head_size == 128 ? 5.8e6 : 3.9e6, tile = c->head_size == 128 ? 2.25 : 1.35;
    auto by_few = [&](int64_t rows) { return rows <= 8 ? bytes / rate : (double)((rows + 15) / 16) * bytes / (0.53 * rate); };
    auto by_many = [&](int64_t units, int64_t split, double ends) {
        return (double)((units * split + 151) / 152) * ((double)((tiles + split - 1) / split) + ends) * tile;
    };
    double one, two;    // what the shared tokens cost in one pass, and in two
    if (each <= kFewRows) {
        one = (double)requests * by_few(each);
        two = all <= kFewRows ? 20.0 : 10.0;
    } else {
        const int64_t units = (all / 256 + requests < requests * ((most + 255) / 256) ? all / 256 + requests
                                                                                      : requests * ((most + 255) / 256)) * heads;
        one = by_many(units, units <= 76 ? 152 / units : 1, 0.0) * (each <= 128 ? 0.7 : 1.0);
        two = 35.0;
    }
    if (all <= kFewRows)
        return two + by_few(all) < one;
    const int64_t units = (all + 255) / 256 * heads, items = attn_many_items(all, c->num_heads);
    double first = by_many(units, 1, 3.0);
    for (int64_t split = 2; split <= 31 && split <= tiles / 2 && units * split <= items; ++split) {
        const double cut = by_many(units, split, 3.0);
        first = cut < first ? cut : first;
    }
    return two + first < one;
}

cg_status launch_pass(const cg_int4_cache *c, const AttnArgs &p, uint8_t *workspace, cudaStream_t s)
{
    const int64_t most = max_rows(c, &p.a);
    cudaError_t err = cudaSuccess;
    if (most <= kFewRows || !p.first) {
        err = attn_few_launch(p, c->head_size, c->group, (int)(most < kFewRows ? most : kFewRows), workspace, s);
        workspace += few_bytes(c, most);
    }
    if (err == cudaSuccess && most > kFewRows)
        err = attn_many_launch(p, c->head_size, c->group, workspace, s);
    return err == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

}  // namespace

cg_status attn_check_sizes(const cg_int4_cache *c, const cg_attention *a)
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

AttnArgs attn_args(const cg_int4_cache *c, int32_t layer, const cg_attention *a)
{
    AttnArgs p = {};
    p.layer = static_cast<const uint8_t *>(c->data) +
              (size_t)layer * c->num_pages * int4_page_bytes(c);
    p.status = c->status;
    p.num_pages = c->num_pages;
    p.page_tokens = c->page_tokens;
    p.heads = c->num_heads;
    p.ratio = p.pos_ratio = a->q_heads / c->num_heads;
    p.few_rows = kFewRows;
    p.scale2 = a->scale * kLog2E;
    p.kv_limit = (int64_t)a->table_width * c->page_tokens;
    p.a = *a;
    return p;
}

cg_status attn_check_arrays(const cg_attention *a, bool with_out)
{
    if ((a->q == nullptr && a->tokens > 0) || a->cu_q == nullptr || a->kv_lens == nullptr ||
        (a->block_table == nullptr && a->table_width > 0) || !int4_aligned(a->q, 16) ||
        !int4_aligned(a->cu_q, 4) || !int4_aligned(a->kv_lens, 4) || !int4_aligned(a->block_table, 4) ||
        (with_out && (a->out == nullptr || !int4_aligned(a->out, 16))))
        return CG_ERR_INVALID_ARG;
    const int64_t strides[4] = {a->q_token_stride, a->q_head_stride, with_out ? a->out_token_stride : 0,
                                with_out ? a->out_head_stride : 0};
    for (int64_t s : strides)
        if (s < 0 || s % 8 != 0)
            return CG_ERR_INVALID_ARG;
    return CG_OK;
}

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
    const cg_status st = attn_check_sizes(c, a);
    if (st != CG_OK)
        return st;
    *bytes = pass_bytes(c, max_rows(c, a), false);
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
    if (!int4_aligned(workspace, 256))
        return CG_ERR_INVALID_ARG;
    st = attn_check_arrays(a, true);
    if (st != CG_OK)
        return st;
    if (workspace_bytes < need || (need > 0 && workspace == nullptr))
        return CG_ERR_CAPACITY;
    const AttnArgs p = attn_args(c, layer, a);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launch_pass(c, p, static_cast<uint8_t *>(workspace), s);
}

// Shared tokens, where they are many: one pass takes them for all rows of the batch, as one request's
// that all see every token, and leaves its results and their sums in fp32; the other takes each
// request's own tokens as ever and joins the two where it writes a row (o = sum of l_i 2^(m_i - m) o_i
// over the sum of l_i 2^(m_i - m)). Where they are few, one pass in which every request reads
// them itself, out of the L2.
//
// 64 requests with a token each and 4 query heads to a KV head are 256 rows to the shared tokens:
// they are read once, by the kernel for many rows, where each request would read
// them itself, 64 times. 16384 shared and up to 1024 own tokens, 8 KV heads: 80 us and 268 (36 the first
// pass, 13 its join, 30 the second, 8 its join; of the floor of 10 us the shared tokens are 3). 8 requests of 300
// queries, 32 query and 2 KV heads, 32768 shared: 880 and 1046.

extern "C" cg_status cg_int4_attention_shared_workspace(const cg_int4_cache *c, const cg_attention *a,
                                                        int32_t shared, size_t *bytes)
{
    const cg_status st = cg_int4_attention_workspace(c, a, bytes);   // of the pass over own tokens
    if (st != CG_OK)
        return st;
    if (shared < 0 || shared % c->page_tokens != 0 || shared / c->page_tokens > a->table_width ||
        (shared > 0 && a->window > 0))
        return CG_ERR_INVALID_ARG;
    if (shared == 0 || !two_passes(c, a, shared))
        return CG_OK;
    // and that of the other, whose last kernels may still run when this one's first come up
    *bytes += pass_bytes(c, all_rows(c, a), true);
    const size_t rows = (size_t)a->tokens * a->q_heads;
    *bytes += align256(rows * c->head_size * sizeof(float)) + align256(rows * sizeof(float2));
    return CG_OK;
}

extern "C" cg_status cg_int4_attention_shared(const cg_int4_cache *c, int32_t layer, const cg_attention *a,
                                              int32_t shared, void *workspace, size_t workspace_bytes,
                                              cg_stream_t stream)
{
    cg_status st = int4_check(c);
    if (st != CG_OK)
        return st;
    size_t need = 0;
    st = cg_int4_attention_shared_workspace(c, a, shared, &need);
    if (st != CG_OK)
        return st;
    if (shared == 0)
        return cg_int4_attention(c, layer, a, workspace, workspace_bytes, stream);
    if (layer < 0 || layer >= c->num_layers)
        return CG_ERR_INVALID_ARG;
    if (a->requests == 0 || a->tokens == 0)
        return CG_OK;
    if (!int4_aligned(workspace, 256))
        return CG_ERR_INVALID_ARG;
    st = attn_check_arrays(a, true);
    if (st != CG_OK)
        return st;
    if (workspace_bytes < need || (need > 0 && workspace == nullptr))
        return CG_ERR_CAPACITY;
    const size_t rows = (size_t)a->tokens * a->q_heads;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    AttnArgs p = attn_args(c, layer, a);
    // a block begins and ends a unit for as long as it reads some 16 blobs: short ones are not strung
    // together (4 requests of 7 to 65 tokens, 12 heads: 54 us with, 14 without)
    p.least_unit = 16;
    if (!two_passes(c, a, shared)) {
        p.front = shared;
        return launch_pass(c, p, ws, s);
    }
    p.shared = shared;
    p.row_stats = reinterpret_cast<float2 *>(ws + need - align256(rows * sizeof(float2)));
    p.rows = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(p.row_stats) -
                                       align256(rows * c->head_size * sizeof(float)));
    AttnArgs first = p;
    first.first = true;
    first.items = attn_many_items(all_rows(c, a), c->num_heads);
    first.pos_ratio = INT32_MAX;
    first.a.cu_q += a->requests;
    first.a.requests = 1;
    first.a.max_q_len = 0;
    // however many rows there are, they go to one kernel
    first.few_rows = all_rows(c, a) <= kFewRows ? kFewRows : 0;
    p.a.block_table += shared / c->page_tokens;
    p.a.table_width -= shared / c->page_tokens;
    st = launch_pass(c, first, ws, s);
    return st == CG_OK ? launch_pass(c, p, ws + pass_bytes(c, all_rows(c, a), true), s) : st;
}

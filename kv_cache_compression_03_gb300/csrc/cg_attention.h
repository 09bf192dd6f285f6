// Shared by the attention kernels of the 4-bit cache.
#pragma once

#include "cg_int4.h"

struct AttnArgs {
    const uint8_t *layer;   // the cache's bytes of one layer
    void *status;
    int32_t num_pages, page_tokens, heads, ratio;   // ratio: query heads per KV head
    int32_t few_rows;       // requests with up to this many rows per KV head go to the
                            // kernel for few rows
    float scale2;           // scale * log2(e)
    int64_t kv_limit;       // most tokens of a request
    int32_t least_unit;     // few rows, shared tokens and weights: blobs that a request and head count as at least
    // Where all requests begin with the same tokens, either each of them reads those, the first
    // `front`, by way of the table's first row; or one pass takes the first `shared`, all rows
    // of the batch as one request's, and leaves its results in rows, and the other takes the
    // tokens behind them (the table and the lengths begin there) and joins the two.
    int32_t front;          // 0: none
    int32_t shared;         // 0: none
    bool first;             // the pass over the shared tokens
    int32_t items;          // its items that the workspace holds
    int32_t pos_ratio;      // rows to a position: ratio; more than there are where all rows see alike
    float *rows;            // [tokens * q_heads][head_size], normalised; nullptr: no shared tokens
    float2 *row_stats;      // [tokens * q_heads]: maximum of the scores, sum
    cg_attention a;
};

// One request's rows and tokens.
struct AttnRequest {
    int32_t row0, x0, kv;   // first query row, its position, cached tokens
    int32_t rows;           // new tokens * ratio: rows of one KV head
};

// False for a request without rows and for an invalid one, which *error
// then names. kShared: there may be shared tokens (p.first, p.shared, p.front).
template <bool kShared>
__device__ __forceinline__ bool attn_request(const AttnArgs &p, int r, AttnRequest *q,
                                             uint32_t *error)
{
    // in the pass over the shared tokens cu_q points at its last entry, the batch's rows (all that
    // there can be where it is beyond them: the other pass, whose requests lie before it, reports it)
    const bool first = kShared && p.first;
    const int32_t c0 = first ? 0 : p.a.cu_q[r];
    const int32_t c1 = first ? min(p.a.cu_q[0], p.a.tokens) : p.a.cu_q[r + 1];
    const bool shares = kShared && !first && p.shared + p.front > 0;
    // (of rows from there on the pass over the shared tokens left nothing)
    const int32_t most = shares ? min(p.a.cu_q[p.a.requests], p.a.tokens) : p.a.tokens;
    const int32_t kv = first ? p.shared : p.a.kv_lens[r];
    *error = CG_OK;
    if (c0 < 0 || c1 < c0 || c1 > most || kv < 0 || kv > p.kv_limit)
        *error = CG_ERR_CORRUPT;
    else if (p.a.max_q_len > 0 && c1 - c0 > p.a.max_q_len)
        *error = CG_ERR_INVALID_ARG;
    else if (shares && c1 > c0 && kv - (p.shared + p.front) < c1 - c0)
        *error = CG_ERR_INVALID_ARG;
    q->row0 = c0;
    q->kv = first || !kShared ? kv : kv - p.shared;
    q->x0 = first ? kv - 1 : q->kv - (c1 - c0);
    q->rows = (c1 - c0) * p.ratio;   // at most tokens * q_heads, which fits
    return *error == CG_OK && c1 > c0;
}

// ------------------------------------------------------------- instructions

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Row (token * q_heads + head) of the pass behind the shared tokens: the factors of its own
// normalised result, whose scores had maximum m and sum l, and of the shared tokens'.
__device__ __forceinline__ float2 join_factors(const AttnArgs &p, int64_t row, float m, float l)
{
    const float2 before = p.row_stats[row];
    const float mx = fmaxf(m, before.x);
    const float a = l * exp2_fast(m - mx), b = before.y * exp2_fast(before.x - mx), sum = a + b;
    return sum == 0.0f ? make_float2(0.0f, 0.0f) : make_float2(a / sum, b / sum);
}

// Product of bf16 pairs, rounded to bf16.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t c;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

// ------------------------------------------------------ barriers and copies

__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void bar_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count)
                 : "memory");
}

__device__ __forceinline__ void bar_init_fence()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void bar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void bar_expect(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void bulk_copy(void *dst, const void *src, uint32_t bytes,
                                          uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(smem_addr(dst)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar))
        : "memory");
}

// A wait gives up after a second. *leave (if given) is looked at as well: set,
// the wait ends at once. Each poll may suspend the thread for a while.
constexpr uint64_t kBarWaitNs = 1000000000ull;

// Test builds (CG_TEST_ATTN_TIMEOUT) give up chosen waits at once, with copies and
// products in flight that are all valid and complete: what a block does then must be
// right in the product build too, where no test can make a wait run out.
#ifdef CG_TEST_ATTN_TIMEOUT
constexpr bool kTestTimeout = true;
#else
constexpr bool kTestTimeout = false;
#endif

__device__ __forceinline__ bool bar_poll(uint32_t at, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(at), "r"(parity)
        : "memory");
    return done;
}

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ bool bar_wait_long(uint32_t at, uint32_t parity, volatile uint32_t *leave)
{
    uint64_t start = 0;
    for (uint32_t i = 0;; ++i) {
        if (bar_poll(at, parity))
            return true;
        if ((i & 63) != 63)   // the clock is looked at now and then
            continue;
        if (leave != nullptr && *leave)
            return false;
        const uint64_t now = now_ns();
        if (start == 0)
            start = now;
        else if (now - start > kBarWaitNs)
            return false;
    }
}

__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity)
{
    const uint32_t at = smem_addr(bar);
    return bar_poll(at, parity) || bar_wait_long(at, parity, nullptr);
}

// ------------------------------------------------------------------ launches

// A call's kernels come up under one another (programmatic stream serialization). The
// next one may start from here on.
__device__ __forceinline__ void grid_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Waits until the one before has ended and its results are there. Every kernel that was
// launched so waits before it ends, in every block, so that what follows the call in the
// stream follows all of its kernels.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_under(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                         Args... args)
{
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Checks of a call's sizes, and of its pointers and strides (out's where it has one); its
// arguments for the kernels, without shared tokens.
cg_status attn_check_sizes(const cg_int4_cache *c, const cg_attention *a);
cg_status attn_check_arrays(const cg_attention *a, bool with_out);
AttnArgs attn_args(const cg_int4_cache *c, int32_t layer, const cg_attention *a);

// SM count of the current device, looked up once per device.
cudaError_t attn_sm_count(int *sms);

// Most blocks of the kernel for few rows, whose partial results the
// workspace holds.
constexpr int kFewMaxBlocks = 480;

size_t attn_few_workspace(int head_size, int max_rows);
cudaError_t attn_few_launch(const AttnArgs &p, int head_size, int group, int max_rows, void *ws,
                            cudaStream_t s);
// Items that the shared tokens of `rows` rows of each KV head may be cut into; bytes for so many (0: for a
// pass over own tokens).
int attn_many_items(int64_t rows, int heads);
size_t attn_many_workspace(int head_size, int items);
cudaError_t attn_many_launch(const AttnArgs &p, int head_size, int group, void *ws, cudaStream_t s);

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
    cg_attention a;
};

// One request's rows and tokens.
struct AttnRequest {
    int32_t row0, nq, kv;   // first query row, query rows, cached tokens
    int32_t rows;           // nq * ratio: rows of one KV head
};

// False for a request without rows and for an invalid one, which *error
// then names.
__device__ __forceinline__ bool attn_request(const AttnArgs &p, int r, AttnRequest *q,
                                             uint32_t *error)
{
    const int32_t c0 = p.a.cu_q[r], c1 = p.a.cu_q[r + 1], kv = p.a.kv_lens[r];
    *error = CG_OK;
    if (c0 < 0 || c1 < c0 || c1 > p.a.tokens || kv < 0 ||
        (int64_t)kv > (int64_t)p.a.table_width * p.page_tokens)
        *error = CG_ERR_CORRUPT;
    else if (p.a.max_q_len > 0 && c1 - c0 > p.a.max_q_len)
        *error = CG_ERR_INVALID_ARG;
    q->row0 = c0;
    q->nq = c1 - c0;
    q->kv = kv;
    q->rows = q->nq * p.ratio;   // at most tokens * q_heads, which fits
    return *error == CG_OK && c1 > c0;
}

// ------------------------------------------------------------- instructions

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

// SM count of the current device, looked up once per device.
cudaError_t attn_sm_count(int *sms);

// Most blocks of the kernel for few rows, whose partial results the
// workspace holds.
constexpr int kFewMaxBlocks = 480;

size_t attn_few_workspace(int head_size, int max_rows);
cudaError_t attn_few_launch(const AttnArgs &p, int head_size, int group, int max_rows, void *ws,
                            cudaStream_t s);
size_t attn_many_workspace(int head_size);
cudaError_t attn_many_launch(const AttnArgs &p, int head_size, int group, void *ws, cudaStream_t s);

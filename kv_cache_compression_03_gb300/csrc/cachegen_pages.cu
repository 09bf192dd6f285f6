// cg_pages_grow: pages and slots of a batch's new tokens from the requests'
// lengths, on the GPU.
//
// Two prefix sums over the requests (new tokens, pages needed) place every
// new token and page. The sums run in one block, so nothing waits on another
// block and the in-place outputs have one writer; that block also hands out
// the pages. Slots of small batches are filled by the same block, those of
// larger ones by a second launch over the tokens. The call is bound by
// launch and barrier latency, not by its few bytes.

#include <cuda_runtime.h>
#include <stdint.h>

#include "cg_int4.h"

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kSlotThreads = 256;
constexpr int kFewTokens = 8192;   // slots that the first block fills itself

struct Sum {
    int64_t tokens, pages;
};

__device__ __forceinline__ Sum warp_scan(Sum v, int lane)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t t = __shfl_up_sync(0xFFFFFFFFu, v.tokens, d);
        const int64_t p = __shfl_up_sync(0xFFFFFFFFu, v.pages, d);
        if (lane >= d) {
            v.tokens += t;
            v.pages += p;
        }
    }
    return v;
}

// Last r in [0, n) with at[r] <= x, for ascending at with at[0] <= x.
__device__ __forceinline__ int last_at_most(const int32_t *at, int n, int32_t x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int slot_of(const cg_page_batch &b, int32_t page, int32_t x)
{
    if (page < 0 || page >= b.num_pages) {
        int4_set_status(b.status, CG_ERR_CORRUPT);
        return -1;
    }
    return page * b.page_tokens + x % b.page_tokens;
}

// Dynamic shared memory: cu[requests + 1], base[requests + 1] (exclusive
// sums of the new tokens and of the pages needed).
__global__ void __launch_bounds__(kThreads) k_pages_grow(cg_page_batch b)
{
    extern __shared__ int32_t smem[];
    int32_t *cu = smem, *base = smem + b.requests + 1;
    __shared__ Sum warp_sum[kWarps];
    __shared__ uint32_t error;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t P = b.page_tokens;
    const int32_t nfree = *b.free_count;
    if (tid == 0) {
        error = CG_OK;
        static_cast<uint4 *>(b.status)[0] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    if (tid == 0 && (nfree < 0 || nfree > b.free_capacity))
        atomicCAS(&error, 0u, (uint32_t)CG_ERR_CORRUPT);
    Sum carry = {0, 0};
    for (int r0 = 0; r0 < b.requests; r0 += kThreads) {
        const int r = r0 + tid;
        Sum v = {0, 0};
        if (r < b.requests) {
            const int64_t len = b.lens[r], n = b.counts[r];
            if (len < 0 || n < 0) {
                atomicCAS(&error, 0u, (uint32_t)CG_ERR_INVALID_ARG);
            } else {
                const int64_t all = (len + n + P - 1) / P;
                if (all > b.table_width || len + n > INT32_MAX)
                    atomicCAS(&error, 0u, (uint32_t)CG_ERR_CAPACITY);
                v.tokens = n;
                v.pages = all - (len + P - 1) / P;
            }
        }
        const Sum own = v;
        v = warp_scan(v, lane);
        if (lane == 31)
            warp_sum[warp] = v;
        __syncthreads();
        Sum before = carry, total = carry;
        for (int i = 0; i < kWarps; ++i) {
            const Sum s = warp_sum[i];
            if (i < warp) {
                before.tokens += s.tokens;
                before.pages += s.pages;
            }
            total.tokens += s.tokens;
            total.pages += s.pages;
        }
        __syncthreads();
        if (r < b.requests) {   // past an int the call fails below
            cu[r] = (int32_t)(before.tokens + v.tokens - own.tokens);
            base[r] = (int32_t)(before.pages + v.pages - own.pages);
        }
        carry = total;
    }
    if (tid == 0) {
        cu[b.requests] = (int32_t)carry.tokens;
        base[b.requests] = (int32_t)carry.pages;
        if (carry.tokens > b.tokens || carry.pages > nfree)
            atomicCAS(&error, 0u, (uint32_t)CG_ERR_CAPACITY);
    }
    __syncthreads();
    const uint32_t err = error;
    const int32_t ntok = err ? 0 : cu[b.requests], npage = err ? 0 : base[b.requests];
    // pages taken
    for (int32_t k = tid; k < npage; k += kThreads) {
        const int r = last_at_most(base, b.requests, k);
        const int32_t held = (b.lens[r] + P - 1) / P;
        const int32_t id = b.free_pages[nfree - 1 - k];
        if (id < 0 || id >= b.num_pages)
            int4_set_status(b.status, CG_ERR_CORRUPT);
        b.block_table[r * b.table_stride + held + (k - base[r])] = id;
    }
    // slots, where this block fills them
    if (b.tokens <= kFewTokens)
        for (int32_t t = tid; t < b.tokens; t += kThreads) {
            int slot = -1;
            if (t < ntok) {
                const int r = last_at_most(cu, b.requests, t);
                const int32_t len = b.lens[r], x = len + (t - cu[r]);
                const int32_t held = (len + P - 1) / P, at = x / P;
                const int32_t page = at < held ? b.block_table[r * b.table_stride + at]
                                               : b.free_pages[nfree - 1 - (base[r] + at - held)];
                slot = slot_of(b, page, x);
            }
            b.slots_out[t] = slot;
        }
    __syncthreads();   // lens_out may be lens, free_count_out free_count
    for (int r = tid; r < b.requests; r += kThreads) {
        const int32_t len = b.lens[r];
        b.lens_out[r] = err ? len : len + b.counts[r];
        b.cu_out[r] = err ? 0 : cu[r];
    }
    if (tid == 0) {
        b.cu_out[b.requests] = ntok;
        *b.free_count_out = nfree - npage;
        if (err)
            static_cast<uint32_t *>(b.status)[0] = err;
    }
}

// Slots of a large batch, once the tables are complete; lens_out is lens +
// counts (cu_out all zero after an error, so nothing is read then).
__global__ void __launch_bounds__(kSlotThreads) k_page_slots(cg_page_batch b)
{
    const int64_t t = (int64_t)blockIdx.x * kSlotThreads + threadIdx.x;
    if (t >= b.tokens)
        return;
    int slot = -1;
    if (t < b.cu_out[b.requests]) {
        const int r = last_at_most(b.cu_out, b.requests, (int32_t)t);
        const int32_t x = b.lens_out[r] - (b.cu_out[r + 1] - (int32_t)t);
        slot = slot_of(b, b.block_table[r * b.table_stride + x / b.page_tokens], x);
    }
    b.slots_out[t] = slot;
}

}  // namespace

extern "C" cg_status cg_pages_grow(const cg_page_batch *b, cg_stream_t stream)
{
    if (b == nullptr || b->requests < 0 || b->tokens < 0 || b->table_width < 0 ||
        b->table_stride < b->table_width || b->free_capacity < 0 || b->num_pages <= 0 ||
        b->page_tokens <= 0)
        return CG_ERR_INVALID_ARG;
    if (b->page_tokens % 16 != 0 || b->page_tokens > 1024 ||
        (int64_t)b->num_pages * b->page_tokens >= ((int64_t)1 << 31) ||
        b->requests > CG_MAX_REQUESTS || b->tokens >= ((int64_t)1 << 31))
        return CG_ERR_UNSUPPORTED;
    if (b->status == nullptr || !int4_aligned(b->status, 16) || b->free_count == nullptr ||
        b->cu_out == nullptr || b->free_count_out == nullptr)
        return CG_ERR_INVALID_ARG;
    if ((b->requests > 0 && (b->lens == nullptr || b->counts == nullptr ||
                             b->lens_out == nullptr)) ||
        (b->requests > 0 && b->table_width > 0 && b->block_table == nullptr) ||
        (b->free_capacity > 0 && b->free_pages == nullptr) ||
        (b->tokens > 0 && b->slots_out == nullptr))
        return CG_ERR_INVALID_ARG;
    const void *words[] = {b->block_table, b->lens, b->counts, b->free_pages, b->free_count,
                           b->cu_out, b->lens_out, b->free_count_out, b->slots_out};
    for (const void *p : words)
        if (!int4_aligned(p, 4))
            return CG_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int smem = 2 * (b->requests + 1) * (int)sizeof(int32_t);
    if (smem > 48 * 1024 - 2048 &&
        cudaFuncSetAttribute(k_pages_grow, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
            cudaSuccess)
        return CG_ERR_CUDA;
    k_pages_grow<<<1, kThreads, smem, s>>>(*b);
    if (b->tokens > kFewTokens)
        k_page_slots<<<(unsigned)((b->tokens + kSlotThreads - 1) / kSlotThreads), kSlotThreads, 0,
                       s>>>(*b);
    return cudaGetLastError() == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

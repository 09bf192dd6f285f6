// cg_pages_grow: pages and slots of a batch's new tokens from the requests'
// lengths, on the GPU; cg_pages_release: the pages behind shorter lengths back to the list.
//
// Growing. Two prefix sums over the requests (new tokens, pages needed) place every
// new token and page. The sums run in one block, so nothing waits on another
// block and the in-place outputs have one writer. Pages and slots of small
// batches are filled by the same block; larger ones take two more launches, over
// the pages and over the slots, with the sums of pages left for them in the slot
// map. The call is bound by launch and barrier latency, not by its few bytes: 4.6 us for
// 64 requests with a token each (one launch), 20 us for 4096 with 128 on average (2.5 MB, three
// launches).

#include <cuda_runtime.h>
#include <stdint.h>

#include "cg_int4.h"

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kSlotThreads = 256;
constexpr int kSlotTile = 4 * kSlotThreads;   // slots of a block of the second launch
constexpr int kFewTokens = CG_MAX_REQUESTS;   // slots that the first block fills itself

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
// sums of the new tokens and of the pages needed), held[requests] (pages).
__global__ void __launch_bounds__(kThreads) k_pages_grow(cg_page_batch b)
{
    extern __shared__ int32_t smem[];
    int32_t *cu = smem, *base = cu + b.requests + 1, *held = base + b.requests + 1;
    __shared__ Sum warp_sum[kWarps];
    __shared__ uint32_t error;   // the greatest code of several, whichever is found first
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t P = b.page_tokens;
    const int32_t nfree = *b.free_count;
    if (tid == 0) {
        error = CG_OK;
        static_cast<uint4 *>(b.status)[0] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    if (tid == 0 && (nfree < 0 || nfree > b.free_capacity))
        atomicMax(&error, (uint32_t)CG_ERR_CORRUPT);
    // a thread's requests lie together: one scan over the threads places them all
    constexpr int kMost = (CG_MAX_REQUESTS + kThreads - 1) / kThreads;
    const int each = (b.requests + kThreads - 1) / kThreads;
    int32_t tokens[kMost], pages[kMost];
    Sum v = {0, 0};
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int r = tid * each + i;
        tokens[i] = pages[i] = 0;
        if (i < each && r < b.requests) {
            const int64_t len = b.lens[r], n = b.counts[r];
            if (len < 0 || n < 0) {
                atomicMax(&error, (uint32_t)CG_ERR_INVALID_ARG);
            } else {
                const int64_t all = (len + n + P - 1) / P, have = (len + P - 1) / P;
                if (all > b.table_width || len + n > INT32_MAX)
                    atomicMax(&error, (uint32_t)CG_ERR_CAPACITY);
                tokens[i] = (int32_t)n;
                pages[i] = (int32_t)(all - have);
                held[r] = (int32_t)have;
                v.tokens += n;
                v.pages += all - have;
            }
        }
    }
    const Sum own = v;
    v = warp_scan(v, lane);
    if (lane == 31)
        warp_sum[warp] = v;
    __syncthreads();
    const Sum warps = warp_scan(warp_sum[lane], lane);   // every warp for itself
    Sum total = {__shfl_sync(0xFFFFFFFFu, warps.tokens, 31), __shfl_sync(0xFFFFFFFFu, warps.pages, 31)};
    const int64_t wt = __shfl_sync(0xFFFFFFFFu, warps.tokens, (warp + 31) & 31);
    const int64_t wp = __shfl_sync(0xFFFFFFFFu, warps.pages, (warp + 31) & 31);
    int64_t tok = v.tokens - own.tokens + (warp ? wt : 0), page = v.pages - own.pages + (warp ? wp : 0);
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int r = tid * each + i;
        if (i < each && r < b.requests) {   // past an int the call fails below
            cu[r] = (int32_t)tok;
            base[r] = (int32_t)page;
            tok += tokens[i];
            page += pages[i];
        }
    }
    if (tid == 0) {
        cu[b.requests] = (int32_t)total.tokens;
        base[b.requests] = (int32_t)total.pages;
        if (total.tokens > b.tokens || total.pages > nfree)
            atomicMax(&error, (uint32_t)CG_ERR_CAPACITY);
    }
    __syncthreads();
    const uint32_t err = error;
    const int32_t ntok = err ? 0 : cu[b.requests], npage = err ? 0 : base[b.requests];
    if (b.tokens <= kFewTokens) {
        for (int32_t k = tid; k < npage; k += kThreads) {
            const int32_t id = b.free_pages[nfree - 1 - k];
            const int r = last_at_most(base, b.requests, k);
            if (id < 0 || id >= b.num_pages)
                int4_set_status(b.status, CG_ERR_CORRUPT);
            b.block_table[r * b.table_stride + held[r] + (k - base[r])] = id;
        }
        for (int32_t t = tid; t < b.tokens; t += kThreads) {
            int slot = -1;
            if (t < ntok) {
                const int r = last_at_most(cu, b.requests, t);
                const int32_t x = b.lens[r] + (t - cu[r]), at = x / P;
                const int32_t id = at < held[r] ? b.block_table[r * b.table_stride + at]
                                                : b.free_pages[nfree - 1 - (base[r] + at - held[r])];
                slot = slot_of(b, id, x);
            }
            b.slots_out[t] = slot;
        }
    } else {   // more slots than requests: room for the sums
        for (int r = tid; r <= b.requests; r += kThreads)
            b.slots_out[r] = err ? 0 : base[r];
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

// Pages of a large batch: the sums stand in slots_out, the lengths are the new
// ones, and the list ends where it did before the pages were taken.
__global__ void __launch_bounds__(kSlotThreads) k_page_ids(cg_page_batch b)
{
    const int32_t *base = b.slots_out;
    const int32_t npage = base[b.requests], nfree = *b.free_count_out + npage;
    for (int64_t k = (int64_t)blockIdx.x * kSlotThreads + threadIdx.x; k < npage;
         k += (int64_t)gridDim.x * kSlotThreads) {
        const int32_t id = b.free_pages[nfree - 1 - k];
        const int r = last_at_most(base, b.requests, (int32_t)k);
        const int32_t len = b.lens_out[r] - (b.cu_out[r + 1] - b.cu_out[r]);
        const int32_t held = (len + b.page_tokens - 1) / b.page_tokens;
        if (id < 0 || id >= b.num_pages)
            int4_set_status(b.status, CG_ERR_CORRUPT);
        b.block_table[r * b.table_stride + held + (k - base[r])] = id;
    }
}

// Slots of a large batch, once the tables are complete; lens_out is lens +
// counts (cu_out all zero after an error, so nothing is read then). A block's
// slots belong to few requests: two searches find the first and the last.
__global__ void __launch_bounds__(kSlotThreads) k_page_slots(cg_page_batch b)
{
    __shared__ int range[2];
    const int64_t t0 = (int64_t)blockIdx.x * kSlotTile;
    const int32_t ntok = b.cu_out[b.requests];
    const int64_t end = t0 + kSlotTile < b.tokens ? t0 + kSlotTile : b.tokens;
    if (threadIdx.x < 64 && (threadIdx.x & 31) == 0 && t0 < ntok)
        range[threadIdx.x >> 5] =
            last_at_most(b.cu_out, b.requests, threadIdx.x ? (int32_t)(end < ntok ? end - 1 : ntok - 1) : (int32_t)t0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSlotTile / kSlotThreads; ++i) {
        const int64_t t = t0 + i * kSlotThreads + threadIdx.x;
        if (t >= end)
            break;
        int slot = -1;
        if (t < ntok) {
            const int r = range[0] + last_at_most(b.cu_out + range[0], range[1] - range[0] + 1, (int32_t)t);
            const int32_t x = b.lens_out[r] - (b.cu_out[r + 1] - (int32_t)t);
            slot = slot_of(b, b.block_table[r * b.table_stride + x / b.page_tokens], x);
        }
        b.slots_out[t] = slot;
    }
}

// ------------------------------------------------------------------ release

// A block of 1024 threads sums the pages that the requests release, in their order, and
// writes all that is one to a request.
__global__ void __launch_bounds__(kThreads) k_pages_release(cg_page_release b)
{
    __shared__ int64_t warp_sum[kWarps];
    __shared__ uint32_t error;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t P = b.page_tokens, nfree = *b.free_count;
    if (tid == 0) {
        error = CG_OK;
        static_cast<uint4 *>(b.status)[0] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    if (tid == 0 && (nfree < 0 || nfree > b.free_capacity))
        atomicMax(&error, (uint32_t)CG_ERR_CORRUPT);
    constexpr int kMost = (CG_MAX_REQUESTS + kThreads - 1) / kThreads;
    const int each = (b.requests + kThreads - 1) / kThreads;
    int32_t len[kMost], kept[kMost], pages[kMost];
    int64_t own = 0;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int r = tid * each + i;
        len[i] = kept[i] = pages[i] = 0;
        if (i < each && r < b.requests) {
            len[i] = b.lens[r];
            kept[i] = b.new_lens[r];
            if (kept[i] < 0 || kept[i] > len[i]) {
                atomicMax(&error, (uint32_t)CG_ERR_INVALID_ARG);
            } else {
                const int64_t held = ((int64_t)len[i] + P - 1) / P;
                if (held > b.table_width)
                    atomicMax(&error, (uint32_t)CG_ERR_CAPACITY);
                pages[i] = (int32_t)(held - ((int64_t)kept[i] + P - 1) / P);
                own += pages[i];
            }
        }
    }
    int64_t inc = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d)
            inc += o;
    }
    if (lane == 31)
        warp_sum[warp] = inc;
    __syncthreads();
    int64_t before = inc - own, total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp)
            before += warp_sum[i];
        total += warp_sum[i];
    }
    if (tid == 0 && total > (int64_t)b.free_capacity - nfree)
        atomicMax(&error, (uint32_t)CG_ERR_CAPACITY);
    __syncthreads();
    const uint32_t err = error;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int r = tid * each + i;
        if (i < each && r < b.requests) {
            b.cu_out[r] = err ? 0 : (int32_t)before;
            before += pages[i];
            b.lens_out[r] = err ? len[i] : kept[i];
        }
    }
    if (tid == 0) {
        b.cu_out[b.requests] = err ? 0 : (int32_t)total;
        *b.free_count_out = err ? nfree : nfree + (int32_t)total;
        if (err)
            static_cast<uint32_t *>(b.status)[0] = err;
    }
}

// The page ids, a warp to a request: a load and two stores a page, whose latency is what it takes (4096
// requests, 450 thousand pages: 19 us with the sums; 64 requests 8.6).
__global__ void __launch_bounds__(kSlotThreads) k_release_ids(cg_page_release b)
{
    const int lane = threadIdx.x & 31, r = (int)((blockIdx.x * kSlotThreads + threadIdx.x) >> 5);
    if (r >= b.requests)
        return;
    const int32_t first = b.cu_out[r], n = b.cu_out[r + 1] - first;
    if (n == 0)   // after an error too
        return;
    const int32_t nfree = *b.free_count_out - b.cu_out[b.requests];
    const int32_t stays = (int32_t)(((int64_t)b.lens_out[r] + b.page_tokens - 1) / b.page_tokens);
    int32_t *table = b.block_table + r * b.table_stride + stays;
    bool bad = false;
    for (int32_t i = lane; i < n; i += 32) {
        const int32_t id = table[i];
        bad |= id < 0 || id >= b.num_pages;
        b.free_pages[nfree + first + i] = id;
        table[i] = -1;
    }
    // one of a warp tells (a batch of bad ids, each for itself: 289 us where 14 do)
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0)
        int4_set_status(b.status, CG_ERR_CORRUPT);
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
    const int smem = (3 * b->requests + 2) * (int)sizeof(int32_t);
    if (smem > 48 * 1024 - 2048 &&
        cudaFuncSetAttribute(k_pages_grow, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
            cudaSuccess)
        return CG_ERR_CUDA;
    k_pages_grow<<<1, kThreads, smem, s>>>(*b);
    if (b->tokens > kFewTokens) {
        // pages that there can be, two to a thread
        const int64_t pages = b->tokens / b->page_tokens + b->requests;
        k_page_ids<<<(unsigned)(pages / (2 * kSlotThreads) + 1), kSlotThreads, 0, s>>>(*b);
        k_page_slots<<<(unsigned)((b->tokens + kSlotTile - 1) / kSlotTile), kSlotThreads, 0,
                       s>>>(*b);
    }
    return cudaGetLastError() == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

extern "C" cg_status cg_pages_release(const cg_page_release *b, cg_stream_t stream)
{
    if (b == nullptr || b->requests < 0 || b->table_width < 0 || b->table_stride < b->table_width ||
        b->free_capacity < 0 || b->num_pages <= 0 || b->page_tokens <= 0)
        return CG_ERR_INVALID_ARG;
    if (b->page_tokens % 16 != 0 || b->page_tokens > 1024 ||
        (int64_t)b->num_pages * b->page_tokens >= ((int64_t)1 << 31) || b->requests > CG_MAX_REQUESTS)
        return CG_ERR_UNSUPPORTED;
    if (b->status == nullptr || !int4_aligned(b->status, 16) || b->free_count == nullptr ||
        b->cu_out == nullptr || b->free_count_out == nullptr)
        return CG_ERR_INVALID_ARG;
    if ((b->requests > 0 && (b->lens == nullptr || b->new_lens == nullptr || b->lens_out == nullptr)) ||
        (b->requests > 0 && b->table_width > 0 && b->block_table == nullptr) ||
        (b->free_capacity > 0 && b->free_pages == nullptr))
        return CG_ERR_INVALID_ARG;
    const void *words[] = {b->block_table, b->lens, b->new_lens, b->free_pages, b->free_count,
                           b->cu_out, b->lens_out, b->free_count_out};
    for (const void *p : words)
        if (!int4_aligned(p, 4))
            return CG_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    k_pages_release<<<1, kThreads, 0, s>>>(*b);
    if (b->requests > 0)
        k_release_ids<<<(b->requests * 32 + kSlotThreads - 1) / kSlotThreads, kSlotThreads, 0, s>>>(*b);
    return cudaGetLastError() == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

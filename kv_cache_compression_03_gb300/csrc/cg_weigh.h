// Attention weights of tokens: what its kernels for few and for many rows share.
#pragma once

#include "cg_few.h"

struct WeighArgs {
    cg_token_weights w;
    float2 *parts;       // [block][2][rows of a tile]: m, l of pieces; slot 0 began in an earlier block
    float2 *stats;       // [heads][slots][8]: m, 1 / l (0, 0: no such row, or it sees nothing)
    int32_t slots;       // row tiles of 8 of all requests
    // what the second pass works from, either
    uint4 *queries;      // [heads][slots][words][32]: the second factor, as a lane of the warp has it
    float *factors;      // [heads][slots][groups + 1][8]: rho, sq
    // or
    float *scores;       // [requests][heads][rows][tokens]
    int32_t rows, tokens;
    // requests with more rows than p.few_rows: their sums by row tiles of 128
    float *sums;         // [heads][tiles][tokens]
    int32_t tiles;
    int32_t *taken;      // [2], which the first kernel sets to 0; nullptr where there are no such requests
};

namespace {

using WeighBatch = BatchOf<false, true>;

// Row tiles of 8 of request r lie from here on. (Of a rows before it and b of its own, ceil(b / 8)
// is at most floor((a + b) / 8) - floor(a / 8) + 1.)
__device__ __forceinline__ int32_t first_slot(const AttnArgs &p, int r, int32_t row0)
{
    return (int32_t)((int64_t)row0 * p.ratio / 8) + r;
}

// The lane, read once: kept, not read again wherever it is used.
__device__ __forceinline__ int lane_once()
{
    int lane;
    asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));
    return lane;
}

// Codes i and i + 4 of a word, less c (8), as a bf16 pair: exact out of the mantissa of 128 + n. `from` is 128 + c,
// twice.
__device__ __forceinline__ uint32_t centred(uint32_t w, int i, uint32_t from = 0x43084308u)
{
    const uint32_t x = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    uint32_t y;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(from));
    return y;
}

__device__ __forceinline__ float2 row_stats_of(float m, float l)
{
    return l == 0.0f ? make_float2(0.0f, 0.0f) : make_float2(m, 1.0f / l);
}

// Items of each(q) tokens of a (request, KV head), those of all heads of the first tokens first. One
// warp finds its item, going on from where the last call stood (32 requests from r0 on, `before`
// items ahead of them): false when there are no more. Requests without rows have items too;
// those of which each() makes 0 have none.
struct Items {
    int r0;
    int64_t before;
};

template <typename F>
__device__ __forceinline__ bool find_item(const AttnArgs &p, int64_t item, F each, Items *at, AttnRequest *q, int *r,
                                          int *h, int *tok)
{
    const int lane = threadIdx.x & 31;
    for (;; at->r0 += 32) {
        if (at->r0 >= p.a.requests)
            return false;
        uint32_t error;
        int64_t w = 0;
        if (at->r0 + lane < p.a.requests) {
            attn_request<WeighBatch::kShared>(p, at->r0 + lane, q, &error);
            if (error == CG_OK && each(*q) > 0)
                w = (int64_t)((q->kv + each(*q) - 1) / each(*q)) * p.heads;
        }
        int64_t inc = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
            if (lane >= d)
                inc += o;
        }
        const int64_t start = at->before + inc - w;
        const uint32_t mine = __ballot_sync(0xFFFFFFFFu, item >= start && item < start + w);
        if (mine == 0) {
            at->before += __shfl_sync(0xFFFFFFFFu, inc, 31);
            continue;
        }
        const int src = __ffs(mine) - 1;
        const int64_t off = __shfl_sync(0xFFFFFFFFu, item - start, src);
        *r = at->r0 + src;
        attn_request<WeighBatch::kShared>(p, *r, q, &error);
        const int i = (int)(off / p.heads);
        *h = (int)(off - (int64_t)i * p.heads);
        *tok = i * each(*q);
        return true;
    }
}

}  // namespace

// The kernels for many rows: bytes that they need besides the others' (for `rows` rows of a request's KV head
// at most), and the launch behind those.
size_t weigh_many_workspace(const cg_int4_cache *c, const cg_attention *a, int32_t tokens);
int32_t *weigh_many_taken(void *ws);
cudaError_t weigh_many_launch(const AttnArgs &p, WeighArgs a, const cg_int4_cache *c, void *ws, cudaStream_t s);

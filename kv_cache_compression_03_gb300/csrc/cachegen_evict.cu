// Eviction from the 4-bit paged cache: which tokens of a head stay (cg_choose_tokens), and
// their move to the front of their request's pages (cg_int4_compact).

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cg_int4.h"

namespace {

// ---------------------------------------------------------------- the choice

constexpr int kChooseThreads = 1024, kChooseWarps = kChooseThreads / 32;

// Ascending as the weights are: NaN first, -0 and +0 alike.
__device__ __forceinline__ uint32_t key_of(float w)
{
    const uint32_t bits = __float_as_uint(w + 0.0f);
    return isnan(w) ? 0u : bits & 0x80000000u ? ~bits : bits | 0x80000000u;
}

// A block to a row: the threshold is found eight bits at a time, then the tokens above it, and
// of those at it the lowest, are written in order.
__global__ void __launch_bounds__(kChooseThreads) k_choose_tokens(cg_token_choice c)
{
    __shared__ int32_t count[256];
    __shared__ int32_t sums[2][kChooseWarps];
    __shared__ int32_t found[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x;
    const int h = (int)(row % c.heads), r = (int)(row / c.heads % c.requests);
    const int64_t l = row / c.heads / c.requests;
    const int32_t m = c.lens[r];
    int32_t *kept = c.kept + row * c.budget;
    const bool bad = m < 0 || m > c.width;
    if (bad || m <= c.budget) {
        if (bad && tid == 0)
            int4_set_status(c.status, CG_ERR_CORRUPT);
        for (int i = tid; i < c.budget; i += kChooseThreads)
            kept[i] = !bad && i < m ? i : -1;
        return;
    }
    const float *w = c.weights + l * c.layer_stride + r * c.request_stride + h * c.head_stride;
    // the choice is among [sinks, end), of which `pick` stay
    const int32_t end = m - c.recent, pick = c.budget - c.sinks - c.recent;
    uint32_t prefix = 0;      // of the threshold's key
    int32_t left = pick;      // to be taken at or below the prefix's end
    if (pick > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256)
                count[tid] = 0;
            __syncthreads();
            const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
            for (int j = c.sinks + tid; j < end; j += kChooseThreads) {
                const uint32_t key = key_of(w[j]);
                if ((key & mask) == prefix)
                    atomicAdd(&count[key >> shift & 255], 1);
            }
            __syncthreads();
            if (warp == 0) {   // lane i: the bins 8 i .. 8 i + 7, from the top
                int32_t own = 0;
                for (int k = 0; k < 8; ++k)
                    own += count[255 - 8 * lane - k];
                int32_t inc = own;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int32_t o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
                    if (lane >= d)
                        inc += o;
                }
                int32_t above = inc - own;
                if (above < left && inc >= left) {
                    int b = 255 - 8 * lane;
                    while (above + count[b] < left)
                        above += count[b--];
                    found[0] = b;
                    found[1] = left - above;
                }
            }
            __syncthreads();
            prefix |= (uint32_t)found[0] << shift;
            left = found[1];
            __syncthreads();
        }
    }
    // prefix is the threshold; `left` of the tokens at it are taken. A warp has a stretch.
    const int32_t total = end - c.sinks, each = (total + kChooseWarps - 1) / kChooseWarps;
    const int32_t b0 = c.sinks + min(warp * each, total), b1 = c.sinks + min((warp + 1) * each, total);
    int32_t over = 0, at = 0;
    if (pick > 0)
        for (int j = b0 + lane; j < b1; j += 32) {
            const uint32_t key = key_of(w[j]);
            over += key > prefix;
            at += key == prefix;
        }
    over = __reduce_add_sync(0xFFFFFFFFu, over);
    at = __reduce_add_sync(0xFFFFFFFFu, at);
    if (lane == 0) {
        sums[0][warp] = over;
        sums[1][warp] = at;
    }
    __syncthreads();
    int32_t pos = c.sinks, taken = 0;    // where the warp's first goes; tokens at the threshold before
    for (int i = 0; i < warp; ++i) {
        pos += sums[0][i];
        taken += sums[1][i];
    }
    pos += min(taken, left);
    if (pick > 0)
        for (int j0 = b0; j0 < b1; j0 += 32) {
            const int j = j0 + lane;
            const uint32_t key = j < b1 ? key_of(w[j]) : 0u;
            const uint32_t eq = __ballot_sync(0xFFFFFFFFu, j < b1 && key == prefix);
            const int rank = taken + __popc(eq & ((1u << lane) - 1));
            const bool stays = j < b1 && (key > prefix || (key == prefix && rank < left));
            const uint32_t all = __ballot_sync(0xFFFFFFFFu, stays);
            if (stays)
                kept[pos + __popc(all & ((1u << lane) - 1))] = j;
            pos += __popc(all);
            taken += __popc(eq);
        }
    for (int i = tid; i < c.sinks; i += kChooseThreads)
        kept[i] = i;
    for (int i = tid; i < c.recent; i += kChooseThreads)
        kept[c.budget - c.recent + i] = end + i;
}

__global__ void __launch_bounds__(256) k_choose_lens(cg_token_choice c)
{
    const int r = blockIdx.x * 256 + threadIdx.x;
    if (r < c.requests) {
        const int32_t m = c.lens[r];
        c.lens_out[r] = m <= c.width && m > c.budget ? c.budget : m;
    }
}

// ------------------------------------------------------------------ the move

constexpr int kMoveThreads = 256;
constexpr int kWave = 64;   // tokens moved at a time

struct MoveArgs {
    uint8_t *data;        // the first layer
    void *status;
    size_t layer_bytes;
    int32_t num_pages, page_tokens, heads;
    cg_compaction c;
};

// A block to a (layer, request, head). Tokens move to lower places, in ascending order: a wave of
// places is read whole, then written, and what later waves read lies behind it.
template <typename B>
__global__ void __launch_bounds__(kMoveThreads) k_int4_compact(MoveArgs a)
{
    constexpr int D = B::kD, NG = B::kGroups;
    constexpr int kKUnits = D / 2, kUnits = 2 * kKUnits + 32;   // of a blob: K, V codes, parameters
    constexpr int kMost = (kUnits * (kWave / 16) + kMoveThreads - 1) / kMoveThreads;
    __shared__ const uint8_t *src[kWave];   // the blob of head h that holds the token
    __shared__ uint8_t src_tok[kWave];
    __shared__ uint8_t *dst[kWave / 16];
    __shared__ int32_t first_moved;
    const cg_compaction &c = a.c;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const int h = (int)(row % a.heads), r = (int)(row / a.heads % c.requests);
    const int64_t l = row / a.heads / c.requests;
    const int32_t n = c.new_lens[r], m = c.lens[r];
    if (n == m && n >= 0)
        return;
    const int32_t *kept = c.kept + l * c.kept_layer_stride + r * c.kept_request_stride + h * c.kept_head_stride;
    const bool fits = n >= 0 && n < m && n <= c.budget && (int64_t)m <= (int64_t)c.table_width * a.page_tokens &&
                      (c.weights == nullptr || m <= c.weights_width);
    if (tid == 0)
        first_moved = n;
    __syncthreads();
    bool bad = !fits;
    if (fits)
        for (int i = tid; i < n; i += kMoveThreads) {
            const int32_t j = kept[i], before = i ? kept[i - 1] : -1;
            bad |= j <= before || j < 0 || j >= m;
            if (j != i)
                atomicMin(&first_moved, i);
        }
    if (__syncthreads_or(bad)) {
        if (tid == 0)
            int4_set_status(a.status, CG_ERR_CORRUPT);
        return;
    }
    const int32_t *table = c.block_table + r * c.table_stride;
    float *w = c.weights == nullptr ? nullptr
                                    : c.weights + l * c.weights_layer_stride + r * c.weights_request_stride +
                                          h * c.weights_head_stride;
    const int bpp = a.page_tokens / 16;
    auto blob_of = [&](int32_t token) -> uint8_t * {
        const int page = token / a.page_tokens, id = table[page];
        if ((unsigned)id >= (unsigned)a.num_pages) {
            int4_set_status(a.status, CG_ERR_CORRUPT);
            return nullptr;
        }
        return a.data + l * a.layer_bytes +
               (((size_t)id * a.heads + h) * bpp + (token - page * a.page_tokens) / 16) * B::kBytes;
    };
    for (int32_t p0 = first_moved & ~15; p0 < n; p0 += kWave) {
        float weight = 0.0f;
        if (tid < kWave) {
            const int32_t p = p0 + tid, j = p < n ? kept[p] : p;
            // a place behind the last shares its pair's bytes, and one whose token cannot be read keeps
            // its own: both are read where they are written
            const uint8_t *from = p < n ? blob_of(j) : nullptr;
            uint8_t *to = p <= n ? blob_of(p) : nullptr;
            src[tid] = from != nullptr ? from : to;
            src_tok[tid] = from != nullptr ? j & 15 : p & 15;
            if (tid % 16 == 0)
                dst[tid / 16] = to;
            if (w != nullptr && p < n)
                weight = w[j];
        }
        __syncthreads();
        uint4 x[kMost];
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
            const int u = tid + k * kMoveThreads, blob = u / kUnits, v = u - blob * kUnits;
            x[k] = make_uint4(0, 0, 0, 0);
            if (blob >= kWave / 16)
                continue;
            if (v < kKUnits) {
                const int t = 16 * blob + v / (D / 32);
                if (src[t] != nullptr)
                    x[k] = *reinterpret_cast<const uint4 *>(src[t] + B::kKCodes + src_tok[t] * (D / 2) +
                                                            v % (D / 32) * 16);
            } else if (v < 2 * kKUnits) {
                const int t = 16 * blob + (v - kKUnits) / (D / 16) * 2, part = (v - kKUnits) % (D / 16) * 16;
                uint4 y[2];
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    y[b] = src[t + b] != nullptr ? *reinterpret_cast<const uint4 *>(src[t + b] + B::kVCodes +
                                                                                    (src_tok[t + b] >> 1) * D + part)
                                                 : make_uint4(0, 0, 0, 0);
                const uint32_t sel = (src_tok[t] & 1 ? 0x0032u : 0x0010u) | (src_tok[t + 1] & 1 ? 0x7600u : 0x5400u);
                x[k] = make_uint4(__byte_perm(y[0].x, y[1].x, sel), __byte_perm(y[0].y, y[1].y, sel),
                                  __byte_perm(y[0].z, y[1].z, sel), __byte_perm(y[0].w, y[1].w, sel));
            } else {
                const int t = 16 * blob + (v & 15), is_v = (v - 2 * kKUnits) >> 4;
                if (src[t] != nullptr) {
                    uint32_t par[NG];
                    load_words(par, src[t] + (is_v ? B::kVParams : B::kKParams) + src_tok[t] * 4 * NG);
                    x[k].x = par[0];
                    x[k].y = par[NG > 1 ? 1 : 0];
                    x[k].z = par[NG > 2 ? 2 : 0];
                    x[k].w = par[NG > 2 ? 3 : 0];
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
            const int u = tid + k * kMoveThreads, blob = u / kUnits, v = u - blob * kUnits;
            if (blob >= kWave / 16 || dst[blob] == nullptr)
                continue;
            uint8_t *to = dst[blob];
            if (v < kKUnits) {
                const int in = v / (D / 32), t = 16 * blob + in;
                if (p0 + t < n && src[t] != nullptr)
                    *reinterpret_cast<uint4 *>(to + B::kKCodes + in * (D / 2) + v % (D / 32) * 16) = x[k];
            } else if (v < 2 * kKUnits) {
                const int pair = (v - kKUnits) / (D / 16), t = 16 * blob + 2 * pair;
                if (p0 + t < n && src[t] != nullptr && src[t + 1] != nullptr)
                    *reinterpret_cast<uint4 *>(to + B::kVCodes + pair * D + (v - kKUnits) % (D / 16) * 16) = x[k];
            } else {
                const int in = v & 15, t = 16 * blob + in, is_v = (v - 2 * kKUnits) >> 4;
                if (p0 + t < n && src[t] != nullptr) {
                    uint8_t *par = to + (is_v ? B::kVParams : B::kKParams) + in * 4 * NG;
                    if constexpr (NG == 4)
                        *reinterpret_cast<uint4 *>(par) = x[k];
                    else if constexpr (NG == 2)
                        *reinterpret_cast<uint2 *>(par) = make_uint2(x[k].x, x[k].y);
                    else
                        *reinterpret_cast<uint32_t *>(par) = x[k].x;
                }
            }
        }
        if (w != nullptr && tid < kWave && p0 + tid < n)
            w[p0 + tid] = weight;
        __syncthreads();
    }
    if (w != nullptr)
        for (int32_t i = n + tid; i < m; i += kMoveThreads)
            w[i] = 0.0f;
}

}  // namespace

extern "C" cg_status cg_choose_tokens(const cg_token_choice *c, cg_stream_t stream)
{
    if (c == nullptr || c->layers < 0 || c->requests < 0 || c->heads < 0 || c->width < 0 || c->budget < 0 ||
        c->recent < 0 || c->sinks < 0 || (int64_t)c->sinks + c->recent > c->budget || c->layer_stride < 0 ||
        c->request_stride < 0 || c->head_stride < 0)
        return CG_ERR_INVALID_ARG;
    const int64_t limit = (int64_t)1 << 31, lists = (int64_t)c->layers * c->requests;
    if (c->requests > CG_MAX_REQUESTS || lists >= limit || lists * c->heads >= limit)
        return CG_ERR_UNSUPPORTED;
    if (c->status == nullptr || !int4_aligned(c->status, 16) ||
        (c->requests > 0 && (c->lens == nullptr || c->lens_out == nullptr)) ||
        (lists * c->heads > 0 && ((c->width > 0 && c->weights == nullptr) || (c->budget > 0 && c->kept == nullptr))) ||
        !int4_aligned(c->weights, 4) || !int4_aligned(c->lens, 4) || !int4_aligned(c->kept, 4) ||
        !int4_aligned(c->lens_out, 4))
        return CG_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(c->status, 0, 16, s) != cudaSuccess)
        return CG_ERR_CUDA;
    if (lists * c->heads > 0)
        k_choose_tokens<<<(unsigned)(lists * c->heads), kChooseThreads, 0, s>>>(*c);
    if (c->requests > 0)
        k_choose_lens<<<(c->requests + 255) / 256, 256, 0, s>>>(*c);
    return cudaGetLastError() == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

extern "C" cg_status cg_int4_compact(const cg_int4_cache *cache, int32_t first_layer, const cg_compaction *c,
                                     cg_stream_t stream)
{
    const cg_status st = int4_check(cache);
    if (st != CG_OK)
        return st;
    if (c == nullptr || c->layers < 0 || c->requests < 0 || c->budget < 0 || c->table_width < 0 || first_layer < 0 ||
        (int64_t)first_layer + c->layers > cache->num_layers || c->table_stride < c->table_width ||
        c->kept_layer_stride < 0 || c->kept_request_stride < 0 || c->kept_head_stride < 0 ||
        (c->weights != nullptr && (c->weights_width < 0 || c->weights_layer_stride < 0 ||
                                   c->weights_request_stride < 0 || c->weights_head_stride < 0)))
        return CG_ERR_INVALID_ARG;
    const int64_t limit = (int64_t)1 << 31, lists = (int64_t)c->layers * c->requests;
    if (c->requests > CG_MAX_REQUESTS || (int64_t)c->table_width * cache->page_tokens >= limit || lists >= limit ||
        lists * cache->num_heads >= limit)
        return CG_ERR_UNSUPPORTED;
    if (lists == 0)
        return CG_OK;
    if (c->lens == nullptr || c->new_lens == nullptr || (c->budget > 0 && c->kept == nullptr) ||
        (c->table_width > 0 && c->block_table == nullptr) || !int4_aligned(c->kept, 4) ||
        !int4_aligned(c->weights, 4) || !int4_aligned(c->lens, 4) || !int4_aligned(c->new_lens, 4) ||
        !int4_aligned(c->block_table, 4))
        return CG_ERR_INVALID_ARG;
    MoveArgs a;
    a.layer_bytes = (size_t)cache->num_pages * int4_page_bytes(cache);
    a.data = static_cast<uint8_t *>(cache->data) + first_layer * a.layer_bytes;
    a.status = cache->status;
    a.num_pages = cache->num_pages;
    a.page_tokens = cache->page_tokens;
    a.heads = cache->num_heads;
    a.c = *c;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = int4_dispatch(cache->head_size, cache->group, [&](auto blob) {
        k_int4_compact<decltype(blob)><<<(unsigned)(lists * cache->num_heads), kMoveThreads, 0, s>>>(a);
        return cudaGetLastError();
    });
    return err == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

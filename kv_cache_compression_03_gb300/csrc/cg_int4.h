// The 4-bit paged cache: its layout, checks and device helpers, shared by
// the store/load kernels and the attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cg_internal.h"

// Byte offsets inside a blob of 16 tokens (one head), cachegen.h has the map.
template <int D, int G>
struct Int4Blob {
    static constexpr int kD = D;
    static constexpr int kG = G;
    static constexpr int kGroups = D / G;
    static constexpr int kWords = D / 32;          // 32-bit words of codes per thread and token
    static constexpr int kKCodes = 0;
    static constexpr int kKParams = 8 * D;
    static constexpr int kVCodes = kKParams + 64 * kGroups;
    static constexpr int kVParams = kVCodes + 8 * D;
    static constexpr int kBytes = kVParams + 64 * kGroups;
};

__host__ __device__ constexpr int int4_blob_bytes(int D, int G) { return 16 * (D + 8 * (D / G)); }

__device__ __forceinline__ void int4_set_status(void *st, uint32_t code)
{
    atomicCAS(static_cast<uint32_t *>(st), 0u, code);
}

// The two halves of a parameter word: s in the low half, lo in the high one.
__device__ __forceinline__ float par_s(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float par_lo(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Pairs of fp32 in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// lo + s n for the codes i and i + 4 of a word, rounded once: n comes exact out
// of the mantissa of 128 + n.
__device__ __forceinline__ uint32_t expand(uint32_t w, int i, uint32_t s, uint32_t lo)
{
    const uint32_t x = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    uint32_t n, y;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(n) : "r"(x), "r"(0x43004300u));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(n), "r"(s), "r"(lo));
    return y;
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t *p)
{
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
}

inline bool int4_aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Shape checks of a cache (not its pointers).
inline cg_status int4_check_shape(const cg_int4_cache *c)
{
    if (c->num_layers <= 0 || c->num_pages <= 0 || c->num_heads <= 0 || c->page_tokens <= 0 ||
        c->head_size <= 0 || c->group <= 0)
        return CG_ERR_INVALID_ARG;
    if (c->page_tokens % 16 != 0 || c->page_tokens > 1024)
        return CG_ERR_UNSUPPORTED;
    if (c->head_size != 64 && c->head_size != 128)
        return CG_ERR_UNSUPPORTED;
    if ((c->group != 32 && c->group != 64 && c->group != 128) || c->group > c->head_size)
        return CG_ERR_UNSUPPORTED;
    const int64_t limit = (int64_t)1 << 31;
    if ((int64_t)c->num_pages * c->page_tokens >= limit ||
        (int64_t)c->num_layers * c->num_pages >= limit ||
        (int64_t)c->num_layers * c->num_pages * c->num_heads >= limit)
        return CG_ERR_UNSUPPORTED;
    // one layer in 128-byte units (every blob is whole ones) counts in 32 bits: below 512 GiB
    if ((int64_t)c->num_pages * c->num_heads >= 2 * limit / (c->page_tokens / 16) /
                                                   (int4_blob_bytes(c->head_size, c->group) / 128))
        return CG_ERR_UNSUPPORTED;
    // so do the bytes of a page
    if ((int64_t)c->num_heads * (c->page_tokens / 16) * int4_blob_bytes(c->head_size, c->group) >= 2 * limit)
        return CG_ERR_UNSUPPORTED;
    return CG_OK;
}

inline cg_status int4_check(const cg_int4_cache *c)
{
    if (c == nullptr)
        return CG_ERR_INVALID_ARG;
    const cg_status st = int4_check_shape(c);
    if (st != CG_OK)
        return st;
    if (c->data == nullptr || c->status == nullptr || !int4_aligned(c->data, 256) ||
        !int4_aligned(c->status, 16))
        return CG_ERR_INVALID_ARG;
    return CG_OK;
}

inline size_t int4_page_bytes(const cg_int4_cache *c)  // one page of one layer, all heads
{
    return (size_t)c->num_heads * (c->page_tokens / 16) * int4_blob_bytes(c->head_size, c->group);
}

// Calls f(Int4Blob<D, G>()) for the cache's head size and group.
template <typename F>
cudaError_t int4_dispatch(int D, int G, F f)
{
    if (D == 64)
        return G == 32 ? f(Int4Blob<64, 32>()) : f(Int4Blob<64, 64>());
    return G == 32 ? f(Int4Blob<128, 32>())
                   : G == 64 ? f(Int4Blob<128, 64>()) : f(Int4Blob<128, 128>());
}

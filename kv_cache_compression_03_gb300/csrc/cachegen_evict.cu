// Eviction from the 4-bit paged cache: which tokens of a head stay (cg_choose_tokens), and
// their move to the front of their request's pages (cg_int4_compact).

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cg_attention.h"

namespace {

// ---------------------------------------------------------------- the choice

constexpr int kChooseThreads = 1024, kChooseWarps = kChooseThreads / 32;

// Ascending as the weights are, above 0: NaN first, -0 and +0 alike.
__device__ __forceinline__ uint32_t key_of(float w)
{
    const uint32_t bits = __float_as_uint(w + 0.0f);
    return w != w ? 1u : bits ^ ((uint32_t)((int32_t)bits >> 31) | 0x80000000u);
}

// One more at a place in shared memory, without a branch.
__device__ __forceinline__ void count_if(bool yes, int32_t *at)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p red.shared.add.u32 [%1], 1;\n\t}" ::"r"((uint32_t)yes),
                 "r"((uint32_t)__cvta_generic_to_shared(at))
                 : "memory");
}

// Bit j of lane i to bit i of lane j.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x)
{
    const int lane = threadIdx.x & 31;
    uint32_t m = 0x0000FFFFu;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1, m ^= m << s) {
        const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, x, s);
        x = lane & s ? (x & ~m) | ((y >> s) & m) : (x & m) | ((y & m) << s);
    }
    return x;
}

__device__ __forceinline__ int32_t warp_before(int32_t v, int lane)   // exclusive sum
{
    int32_t inc = v;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int32_t o = __shfl_up_sync(0xFFFFFFFFu, inc, s);
        if (lane >= s)
            inc += o;
    }
    return inc - v;
}

// A warp's tokens that stay, from kept[0] on: of its token 32 e + lane, counted from `first` on, bit e of `stays`
// says that it does, and of `same` that it is at the threshold, where the lowest `take` stay.
__device__ __forceinline__ void put_kept(int32_t *kept, uint32_t stays, uint32_t same, bool any_same, int32_t take,
                                         int32_t first, int32_t per_lane, int lane)
{
    // lane e: the tokens 32 e .. 32 e + 31 of the warp's
    uint32_t word = transpose_bits(stays);
    if (any_same) {
        uint32_t eq = transpose_bits(same);
        take = min(max(take - warp_before(__popc(eq), lane), 0), 32);
        for (; take > 0 && eq != 0; --take, eq &= eq - 1)
            word |= eq & (0u - eq);
    }
    const int32_t here = __popc(word), before = warp_before(here, lane);
    if (__reduce_add_sync(0xFFFFFFFFu, here) < 8 * per_lane) {   // few: each lane its own
        kept += before;
        for (; word != 0; word &= word - 1)
            *kept++ = first + 32 * lane + __ffs(word) - 1;
    } else {   // 32 tokens at a time, so that neighbours are written together
        for (int e = 0; e < per_lane; ++e) {
            const uint32_t all = __shfl_sync(0xFFFFFFFFu, word, e);
            const int32_t at_e = __shfl_sync(0xFFFFFFFFu, before, e);
            if (all >> lane & 1)
                kept[at_e + __popc(all & ((1u << lane) - 1))] = first + 32 * e + lane;
        }
    }
}

// ---- a row in the registers of a warp or a block

// W warps to a row, each with an equal part of the tokens that are chosen among, up to E a lane (token
// 32 e + lane of the warp's). The threshold is the largest key that `pick` tokens reach; its bits are found
// from the top, by counting the tokens that reach each candidate, until exactly `pick` do: some 20 steps of
// 2 instructions a token, whose sums go through shared memory and one barrier each.
//
// What bounds it: those instructions where there are many rows, the steps' chain where there are few. Against digits
// counted in shared memory, as below, whose places cost a block 5000 instructions however short its row is: 4352
// rows of 7 tokens 8 us and 37, 3456 of 117 8 and 31, 6144 of 1308 43 and 58; 60 rows of 3669 10 and 14, 56 of
// 6306 12 and 14. But 512 rows of 4608 17 and 14, 1440 of 7361 42 and 29: from 152 rows on, more than 2048 tokens go
// by digits.
constexpr int kBitsThreads = 128;   // where a warp has a row

template <int W, int E>
__global__ void __launch_bounds__(W == 1 ? kBitsThreads : 32 * W, W == 1 ? 8 : 32 / W) k_choose_bits(cg_token_choice c)
{
    __shared__ int32_t sums[2][W], over[W], at[W];
    const int lane = threadIdx.x & 31, warp = W == 1 ? 0 : threadIdx.x >> 5, tid = 32 * warp + lane;
    const int64_t row = W == 1 ? (int64_t)blockIdx.x * (kBitsThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (W == 1 && row >= (int64_t)c.layers * c.requests * c.heads)
        return;
    const int h = (int)(row % c.heads), r = (int)(row / c.heads % c.requests);
    const int64_t l = row / c.heads / c.requests;
    const int32_t m = c.lens[r];
    int32_t *kept = c.kept + row * c.budget;
    const bool bad = m < 0 || m > c.width;
    if (bad || m <= c.budget) {   // all of the row's warps
        for (int64_t i = tid; i < c.budget; i += 32 * W)
            kept[i] = !bad && i < m ? (int32_t)i : -1;
        return;
    }
    const float *w = c.weights + l * c.layer_stride + r * c.request_stride + h * c.head_stride;
    // the choice is among [sinks, end), of which `pick` stay
    const int32_t end = m - c.recent, pick = c.budget - c.sinks - c.recent, n = end - c.sinks;
    const int32_t per_lane = (n + 32 * W - 1) / (32 * W);            // at most E
    const int32_t first = c.sinks + warp * per_lane * 32;            // the warp's
    w += first;
    const int32_t mine = min(per_lane, (end - first - lane + 31) >> 5);   // tokens of the lane
    uint32_t key[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        key[e] = e < mine ? __float_as_uint(__ldg(w + 32 * e + lane)) : 0u;
    for (int i = tid; i < c.sinks; i += 32 * W)
        kept[i] = i;
    for (int i = tid; i < c.recent; i += 32 * W)
        kept[c.budget - c.recent + i] = end + i;
    if (pick == 0)
        return;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (e % 4 == 0 && e >= per_lane)   // for all lanes
            break;
        key[e] = e < mine ? key_of(__uint_as_float(key[e])) : 0u;   // 0: no token
    }
    uint32_t threshold = 0;
    int32_t reach = n;        // tokens at or above it, always `pick` at least
    for (int bit = 31; bit >= 0 && reach != pick; --bit) {
        const uint32_t tried = threshold | 1u << bit;
        int32_t count = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (e % 4 == 0 && e >= per_lane)
                break;
            count += key[e] >= tried;
        }
        count = __reduce_add_sync(0xFFFFFFFFu, count);
        if (W > 1) {
            if (lane == 0)
                sums[bit & 1][warp] = count;
            __syncthreads();
            count = __reduce_add_sync(0xFFFFFFFFu, lane < W ? sums[bit & 1][lane] : 0);
        }
        if (count >= pick) {
            threshold = tried;
            reach = count;
        }
    }
    const bool exact = reach == pick;   // all of them stay, else those above the threshold and the first at it
    uint32_t stays = 0, same = 0;       // bit e: of the lane's token
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (e % 4 == 0 && e >= per_lane)
            break;
        if (key[e] > threshold)
            stays |= 1u << e;
        if (key[e] == threshold && key[e] != 0u)
            same |= 1u << e;
    }
    if (exact) {
        stays |= same;
        same = 0;
    }
    const int32_t above = __reduce_add_sync(0xFFFFFFFFu, __popc(stays)), level = __reduce_add_sync(0xFFFFFFFFu, __popc(same));
    int32_t pos = c.sinks, taken = 0, left = pick - above;
    if (W > 1) {
        if (lane == 0) {
            over[warp] = above;
            at[warp] = level;
        }
        __syncthreads();
        const int32_t o = lane < W ? over[lane] : 0, a = lane < W ? at[lane] : 0;
        left = pick - __reduce_add_sync(0xFFFFFFFFu, o);
        pos += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? o : 0);
        taken = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? a : 0);
    }
    put_kept(kept + pos + min(taken, left), stays, same, level > 0, left - taken, first, per_lane, lane);
}

// ---- a row in the registers of a block or a cluster

constexpr int kDigits = 2048;                 // 11, 11 and 10 bits of a key
constexpr int kMostCluster = 8;

template <int T>
struct ChooseShared {
    int32_t count[3][kDigits];
    int32_t coarse[3][kDigits / 32];          // sums of 32
    int32_t found[2];
    int32_t over[T / 32], at[T / 32];         // of each warp
    int32_t all[2];                           // of the block
};

__device__ __forceinline__ void cluster_sync(int size)
{
    if (size == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The value at `p`, a place in this block's shared memory, in that of the cluster's block `rank`.
__device__ __forceinline__ int32_t cluster_load(const int32_t *p, int rank)
{
    uint32_t at;
    int32_t v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at)
                 : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// The digit of d's count that the threshold has, where `left` tokens are to be taken from above: by one
// warp, which leaves it and what is left of them in sm.found. The sums of 32 places of all blocks are looked
// at first (a load from another block's memory goes lane by lane: all places of all blocks were 180 us of 190
// for 256 rows of 65536), all blocks' at once.
template <int T>
__device__ __forceinline__ void find_digit(ChooseShared<T> &sm, int d, int32_t left, int size)
{
    const int lane = threadIdx.x & 31;
    auto sum_of = [&](const int32_t *from) {
        if (size == 1)
            return *from;
        int32_t v[kMostCluster], sum = 0;
#pragma unroll
        for (int k = 0; k < kMostCluster; ++k)
            v[k] = k < size ? cluster_load(from, k) : 0;
#pragma unroll
        for (int k = 0; k < kMostCluster; ++k)
            sum += v[k];
        return sum;
    };
    // lane i: sums i and i + 32 from the top
    const int32_t upper = sum_of(&sm.coarse[d][kDigits / 32 - 1 - lane]), lower = sum_of(&sm.coarse[d][31 - lane]);
    const int32_t up_before = warp_before(upper, lane), up_all = __shfl_sync(0xFFFFFFFFu, up_before + upper, 31);
    const bool in_upper = up_all >= left;
    const int32_t own = in_upper ? upper : lower, before = in_upper ? up_before : up_all + warp_before(lower, lane);
    const int at = __ffs(__ballot_sync(0xFFFFFFFFu, before + own >= left)) - 1;
    const int group = (in_upper ? kDigits / 32 - 1 : 31) - at;
    const int32_t above = __shfl_sync(0xFFFFFFFFu, before, at);
    const int32_t place = sum_of(&sm.count[d][32 * group + 31 - lane]), place_before = above + warp_before(place, lane);
    const int digit = __ffs(__ballot_sync(0xFFFFFFFFu, place_before + place >= left)) - 1;
    if (lane == digit) {
        sm.found[0] = 32 * group + 31 - lane;
        sm.found[1] = left - place_before;
    }
}

// A block or a cluster of `size` blocks to a row, each with an equal part of the tokens that are chosen among, and of
// that each warp, up to E tokens a lane (token 32 e + lane of the warp's), so the weights are read once. The
// threshold's key is found in three digits, counted in shared memory. The first has sign, exponent and two
// bits, so that weights of a few octaves fall into many places; what is above it stays, and only the few
// tokens that share it (read again) are counted by the others. Every warp then knows how many stay before
// its own.
//
// What bounds it: 56 instructions for a token (7 make its key, 5 count it, 5 tell whether it stays, the rest
// are what a block does for its 2048 places and its barriers), of which 1.7 a cycle are issued since blocks
// wait for one another four times; the weights are read at 1.1 TB/s. 256 rows of 65536: 60 us, 512 rows of
// 4608: 11. (All three digits over all tokens, each token placed by a vote: 90, 82 us instead of 60.)
template <int T, int E>
__global__ void __launch_bounds__(T, 1024 / T) k_choose_tokens(cg_token_choice c, int size)
{
    constexpr int kRowThreads = T, kRowWarps = T / 32;
    __shared__ ChooseShared<T> sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / size;
    const int rank = blockIdx.x % size;
    const int h = (int)(row % c.heads), r = (int)(row / c.heads % c.requests);
    const int64_t l = row / c.heads / c.requests;
    const int32_t m = c.lens[r];
    int32_t *kept = c.kept + row * c.budget;
    const bool bad = m < 0 || m > c.width;
    if (bad || m <= c.budget) {   // the whole cluster
        for (int64_t i = rank * kRowThreads + tid; i < c.budget; i += size * kRowThreads)
            kept[i] = !bad && i < m ? (int32_t)i : -1;
        return;
    }
    const float *w = c.weights + l * c.layer_stride + r * c.request_stride + h * c.head_stride;
    // the choice is among [sinks, end), of which `pick` stay
    const int32_t end = m - c.recent, pick = c.budget - c.sinks - c.recent, n = end - c.sinks;
    const int32_t per_lane = (n + size * kRowThreads - 1) / (size * kRowThreads);   // at most E
    const int32_t first = c.sinks + (rank * kRowWarps + warp) * per_lane * 32;      // the warp's
    w += first;
    const int32_t mine = min(per_lane, (end - first - lane + 31) >> 5);             // tokens of the lane
    uint32_t key[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        key[e] = e < mine ? __float_as_uint(__ldg(w + 32 * e + lane)) : 0u;
    for (int i = tid; i < 3 * kDigits / 4; i += kRowThreads)
        reinterpret_cast<int4 *>(sm.count[0])[i] = make_int4(0, 0, 0, 0);
    for (int i = rank * kRowThreads + tid; i < c.sinks; i += size * kRowThreads)
        kept[i] = i;
    for (int i = rank * kRowThreads + tid; i < c.recent; i += size * kRowThreads)
        kept[c.budget - c.recent + i] = end + i;
    if (pick == 0)
        return;
    __syncthreads();
    // ---- the first digit of all tokens
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (e % 4 == 0 && e >= per_lane)   // for all lanes
            break;
        key[e] = e < mine ? key_of(__uint_as_float(key[e])) : 0u;   // 0: no token
        count_if(key[e] != 0u, &sm.count[0][key[e] >> 21]);
    }
    uint32_t prefix = 0;      // of the threshold's key
    int32_t left = pick;      // to be taken from the tokens that begin with it
    uint32_t stays = 0, same = 0;   // bit e: the lane's token is above the threshold, begins as it does
#pragma unroll
    for (int d = 0; d < 3; ++d) {
        __syncthreads();
        for (int k = warp; k < (d == 2 ? 1024 : kDigits) / 32; k += kRowWarps) {
            const int32_t sum = __reduce_add_sync(0xFFFFFFFFu, sm.count[d][32 * k + lane]);
            if (lane == 0)
                sm.coarse[d][k] = sum;
        }
        if (d == 2 && tid < 32)
            sm.coarse[d][32 + tid] = 0;
        cluster_sync(size);
        if (warp == 0)
            find_digit(sm, d, left, size);
        __syncthreads();
        const uint32_t digit = (uint32_t)sm.found[0];
        left = sm.found[1];
        prefix = prefix << (d == 2 ? 10 : 11) | digit;
        if (d == 0) {
            // its keys: from .. below, and not 0
            const uint32_t from = max(prefix << 21, 1u), below = prefix << 21 | ((1u << 21) - 1);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (e % 4 == 0 && e >= per_lane)
                    break;
                if (key[e] > below)
                    stays |= 1u << e;
                if (key[e] >= from)
                    same |= 1u << e;
            }
            same &= ~stays;
        }
        // the tokens that share the digits so far
        for (uint32_t rest = same; rest != 0; rest &= rest - 1) {
            const int e = __ffs(rest) - 1;
            const uint32_t k = key_of(__ldg(w + 32 * e + lane));
            const uint32_t here = d == 0 ? prefix : d == 1 ? k >> 10 : k;
            if (here == prefix) {
                if (d < 2)
                    atomicAdd(&sm.count[d + 1][d == 0 ? k >> 10 & 2047u : k & 1023u], 1);
            } else {
                same ^= 1u << e;
                stays |= (uint32_t)(here > prefix) << e;
            }
        }
    }
    // ---- how many stay before each warp's
    const int32_t over = __reduce_add_sync(0xFFFFFFFFu, __popc(stays)), at = __reduce_add_sync(0xFFFFFFFFu, __popc(same));
    if (lane == 0) {
        sm.over[warp] = over;
        sm.at[warp] = at;
    }
    __syncthreads();
    if (tid < 2) {
        const int32_t *from = tid ? sm.at : sm.over;
        int32_t sum = 0;
        for (int k = 0; k < kRowWarps; ++k)
            sum += from[k];
        sm.all[tid] = sum;
    }
    cluster_sync(size);
    int32_t pos = c.sinks, taken = 0;
    for (int k = 0; k < rank; ++k) {
        pos += cluster_load(&sm.all[0], k);
        taken += cluster_load(&sm.all[1], k);
    }
    for (int k = 0; k < warp; ++k) {
        pos += sm.over[k];
        taken += sm.at[k];
    }
    if (size > 1)   // no block's shared memory goes while another one reads it
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    put_kept(kept + pos + min(taken, left), stays, same, at > 0, left - taken, first, per_lane, lane);
    if (size > 1)
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Rows too long for the registers of a cluster (more than 131072 tokens): a block to a row, which it reads from
// memory for each of four digits of 8 bits, to count what stays before each warp, and to write.
__global__ void __launch_bounds__(kChooseThreads) k_choose_long(cg_token_choice c)
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
        for (int64_t i = tid; i < c.budget; i += kChooseThreads)
            kept[i] = !bad && i < m ? (int32_t)i : -1;
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
            for (int64_t j = c.sinks + tid; j < end; j += kChooseThreads) {
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
    const int64_t total = end - c.sinks, each = (total + kChooseWarps - 1) / kChooseWarps;
    const int64_t b0 = c.sinks + min(warp * each, total), b1 = c.sinks + min((warp + 1) * each, total);
    int32_t over = 0, at = 0;
    if (pick > 0)
        for (int64_t j = b0 + lane; j < b1; j += 32) {
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
        for (int64_t j0 = b0; j0 < b1; j0 += 32) {
            const int64_t j = j0 + lane;
            const uint32_t key = j < b1 ? key_of(w[j]) : 0u;
            const uint32_t eq = __ballot_sync(0xFFFFFFFFu, j < b1 && key == prefix);
            const int rank = taken + __popc(eq & ((1u << lane) - 1));
            const bool stays = j < b1 && (key > prefix || (key == prefix && rank < left));
            const uint32_t all = __ballot_sync(0xFFFFFFFFu, stays);
            if (stays)
                kept[pos + __popc(all & ((1u << lane) - 1))] = (int32_t)j;
            pos += __popc(all);
            taken += __popc(eq);
        }
    for (int64_t i = tid; i < c.sinks; i += kChooseThreads)
        kept[i] = (int32_t)i;
    for (int64_t i = tid; i < c.recent; i += kChooseThreads)
        kept[c.budget - c.recent + i] = (int32_t)(end + i);
}

// The lengths, once every row's kernel has read the old ones (they may be overwritten), and the status.
constexpr int kLensThreads = 1024;

__global__ void __launch_bounds__(kLensThreads) k_choose_lens(cg_token_choice c)
{
    bool bad = false;
    grid_wait();
    for (int r = threadIdx.x; r < c.requests; r += kLensThreads) {
        const int32_t m = c.lens[r];
        bad |= m < 0 || m > c.width;
        c.lens_out[r] = m <= c.width && m > c.budget ? c.budget : m;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0)
        *static_cast<uint4 *>(c.status) = make_uint4(bad ? CG_ERR_CORRUPT : CG_OK, 0, 0, 0);
}

template <int T, int E>
cudaError_t launch_choice(const cg_token_choice &c, int64_t rows, int size, cudaStream_t s)
{
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * size));
    cfg.blockDim = dim3(T);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_choose_tokens<T, E>, c, size);
}

template <int W, int E>
cudaError_t launch_bits(const cg_token_choice &c, int64_t rows, cudaStream_t s)
{
    constexpr int kRows = W == 1 ? kBitsThreads / 32 : 1;
    k_choose_bits<W, E><<<(unsigned)((rows + kRows - 1) / kRows), W == 1 ? kBitsThreads : 32 * W, 0, s>>>(c);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ the move

constexpr int kMoveThreads = 256;
constexpr int kWave = 128;    // tokens moved at a time
constexpr int kStages = 3;    // waves read ahead

struct MoveArgs {
    uint8_t *data;        // the first layer
    void *status;
    size_t layer_bytes;
    int32_t num_pages, page_tokens, heads;
    cg_compaction c;
};

// A wave's tokens in shared memory: of V the whole pair of which a token is half.
template <typename B>
struct alignas(16) MoveStage {
    uint8_t k[kWave][B::kD / 2];
    uint8_t v[kWave][B::kD];
    uint8_t par[2][kWave][4 * B::kGroups];
    const uint8_t *src[kWave];     // the blob that holds the token (nullptr: none)
    uint8_t *dst[kWave / 16];
    float weight[kWave];
    uint8_t tok[kWave];            // in its blob
};

template <int N>
__device__ __forceinline__ void copy_async(void *to, const void *from)
{
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(N) : "memory");
}

// Bytes move: codes and parameters as they are, no token is unpacked. What bounds it is how much is under way:
// three waves of 30 KB a block, two blocks to an SM, whose barriers stop the loads at each wave. All 32 layers of a
// request, 8192 of 16384 tokens each: 180 us for 567 MB read (a token's V comes with that of its pair) and 336
// written, 5.0 TB/s; one layer of 16 requests, 2048 of 2304 tokens: 19.5 us, the caches' lines in L2.
//
// A cluster to a (layer, request, head); its blocks take waves of places in turns. Tokens move to lower
// places in ascending order, so the tokens of a wave lie at its own places or behind: a wave is written
// once it and all before it have been read (a cluster barrier), and the next ones may be read long before.
template <typename B>
__global__ void __launch_bounds__(kMoveThreads, 2) k_int4_compact(MoveArgs a, int size)
{
    constexpr int D = B::kD, NG = B::kGroups;
    using Stage = MoveStage<B>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Stage *stages = reinterpret_cast<Stage *>(smem_raw);
    __shared__ int32_t first_moved;
    const cg_compaction &c = a.c;
    const int tid = threadIdx.x, rank = blockIdx.x % size;
    const int64_t row = blockIdx.x / size;
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
    // every block looks at the whole list
    bool bad = !fits;
    int32_t moved = n;
    if (fits)
#pragma unroll 4
        for (int64_t i = tid; i < n; i += kMoveThreads) {
            const int32_t j = kept[i], before = i ? kept[i - 1] : -1;
            bad |= j <= before || j >= m;
            if (j != i)
                moved = min(moved, (int32_t)i);
        }
    moved = __reduce_min_sync(0xFFFFFFFFu, moved);
    if ((tid & 31) == 0 && moved < n)
        atomicMin(&first_moved, moved);
    if (__syncthreads_or(bad)) {   // in every block of the cluster
        if (tid == 0 && rank == 0)
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
    const int32_t start = first_moved < n ? first_moved & ~15 : n;   // blobs before it stay as they are
    const int waves = (int)(((int64_t)n - start + kWave - 1) / kWave);
    // Of this block's wave i, in steps that a dependent load each ends: the token that comes to a thread's
    // place, where both lie, and its bytes.
    auto place_of = [&](int i) { return start + ((int64_t)i * size + rank) * kWave + tid; };
    auto token_of = [&](int i) {
        const int64_t p = place_of(i);
        return tid < kWave && p < n ? kept[p] : -1;
    };
    struct Found {
        const uint8_t *from;
        uint8_t *to;
        float weight;
    };
    auto find = [&](int i, int32_t j) -> Found {
        const int64_t p = place_of(i);
        Found f = {nullptr, nullptr, 0.0f};
        if (tid < kWave && p <= n && p - tid < n) {
            f.from = j >= 0 ? blob_of(j) : nullptr;
            f.to = blob_of((int32_t)p);
            f.weight = w != nullptr && j >= 0 ? w[j] : 0.0f;
        }
        return f;
    };
    auto fetch = [&](int i, int32_t j, const Found &f) {
        const int64_t p0 = place_of(i) - tid;
        Stage &st = stages[i % kStages];
        if (p0 < n && tid < kWave) {
            // a place behind the last shares its pair's bytes, and one whose token cannot be read keeps
            // its own: both are read where they are written
            st.src[tid] = f.from != nullptr ? f.from : f.to;
            st.tok[tid] = f.from != nullptr ? j & 15 : tid & 15;
            if (tid % 16 == 0)
                st.dst[tid / 16] = p0 + tid < n ? f.to : nullptr;
            st.weight[tid] = f.weight;
        }
        __syncthreads();
        if (p0 < n) {
            constexpr int kKParts = D / 32, kVParts = D / 16;
#pragma unroll 4
            for (int u = tid; u < kWave * kKParts; u += kMoveThreads) {
                const int t = u / kKParts, part = u % kKParts * 16;
                if (st.src[t] != nullptr)
                    copy_async<16>(&st.k[t][part], st.src[t] + B::kKCodes + st.tok[t] * (D / 2) + part);
            }
#pragma unroll 4
            for (int u = tid; u < kWave * kVParts; u += kMoveThreads) {
                const int t = u / kVParts, part = u % kVParts * 16;
                if (st.src[t] != nullptr)
                    copy_async<16>(&st.v[t][part], st.src[t] + B::kVCodes + (st.tok[t] >> 1) * D + part);
            }
            for (int u = tid; u < 2 * kWave; u += kMoveThreads) {
                const int t = u % kWave, v = u / kWave;
                if (st.src[t] != nullptr)
                    copy_async<4 * NG>(&st.par[v][t], st.src[t] + (v ? B::kVParams : B::kKParams) + st.tok[t] * 4 * NG);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int rounds = (waves + size - 1) / size;
    for (int i = 0; i < kStages; ++i) {
        const int32_t j = token_of(i);
        fetch(i, j, find(i, j));
    }
    int32_t ahead = token_of(kStages);   // of the wave that is fetched next
    for (int i = 0; i < rounds; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        cluster_sync(size);   // this round's waves have been read, by all threads of all blocks
        const int32_t j = ahead;
        const Found found = find(i + kStages, j);   // (its loads end under the writes)
        ahead = token_of(i + kStages + 1);
        const int64_t p0 = place_of(i) - tid;
        const Stage &st = stages[i % kStages];
        if (p0 < n) {
            const int there = (int)min((int64_t)kWave, n - p0);   // places of the wave
            constexpr int kUnits = D / 2;                         // 16 bytes each, of a blob's K or V codes
#pragma unroll 4
            for (int u = tid; u < kWave / 16 * kUnits; u += kMoveThreads) {
                const int blob = u / kUnits, in = u % kUnits, t = 16 * blob + in / (D / 32);
                if (t < there && st.dst[blob] != nullptr)
                    *reinterpret_cast<uint4 *>(st.dst[blob] + B::kKCodes + in * 16) =
                        *reinterpret_cast<const uint4 *>(&st.k[t][in % (D / 32) * 16]);
            }
#pragma unroll 4
            for (int u = tid; u < kWave / 16 * kUnits; u += kMoveThreads) {
                const int blob = u / kUnits, in = u % kUnits, t = 16 * blob + in / (D / 16) * 2, part = in % (D / 16) * 16;
                if (t < there && st.dst[blob] != nullptr) {
                    // halves of two tokens' words
                    const uint4 x = *reinterpret_cast<const uint4 *>(&st.v[t][part]);
                    const uint4 y = *reinterpret_cast<const uint4 *>(&st.v[t + 1][part]);
                    const uint32_t sel = (st.tok[t] & 1 ? 0x0032u : 0x0010u) | (st.tok[t + 1] & 1 ? 0x7600u : 0x5400u);
                    *reinterpret_cast<uint4 *>(st.dst[blob] + B::kVCodes + in * 16) =
                        make_uint4(__byte_perm(x.x, y.x, sel), __byte_perm(x.y, y.y, sel), __byte_perm(x.z, y.z, sel),
                                   __byte_perm(x.w, y.w, sel));
                }
            }
            for (int u = tid; u < 2 * kWave; u += kMoveThreads) {
                const int t = u % kWave, v = u / kWave;
                if (t < there && st.dst[t / 16] != nullptr) {
                    uint32_t par[NG];
                    load_words(par, st.par[v][t]);
                    uint8_t *to = st.dst[t / 16] + (v ? B::kVParams : B::kKParams) + t % 16 * 4 * NG;
                    if constexpr (NG == 4)
                        *reinterpret_cast<uint4 *>(to) = make_uint4(par[0], par[1], par[2], par[3]);
                    else if constexpr (NG == 2)
                        *reinterpret_cast<uint2 *>(to) = make_uint2(par[0], par[1]);
                    else
                        *reinterpret_cast<uint32_t *>(to) = par[0];
                }
            }
            if (w != nullptr && tid < there)
                w[p0 + tid] = st.weight[tid];
        }
        __syncthreads();   // the stage is free
        fetch(i + kStages, j, found);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (w != nullptr)   // read by no wave any more
        for (int64_t i = n + rank * kMoveThreads + tid; i < m; i += size * kMoveThreads)
            w[i] = 0.0f;
}

template <typename B>
cudaError_t launch_move(const MoveArgs &a, int64_t lists, cudaStream_t s)
{
    const size_t smem = kStages * sizeof(MoveStage<B>);
    const cudaError_t err = cudaFuncSetAttribute(k_int4_compact<B>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess)
        return err;
    // Two blocks to an SM. Lists that do not fill the SMs are shared by the blocks of a cluster (128 lists of
    // 2048: 28 us with two, 20 with four); more are not, a barrier of the cluster to each wave costs more
    // than it gives (256 of 8192: 179 us, with two blocks 228).
    int size = 1;
    while (size < kMostCluster && lists < 152 && lists * size < 400)
        size *= 2;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(lists * size));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_int4_compact<B>, a, size);
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
    const int64_t rows = lists * c->heads;
    cudaError_t err = cudaSuccess;
    if (rows > 0) {
        // Blocks to a row that go by digits: as many as hold it, and more while there are SMs for them. Small blocks,
        // four on an SM, where they do: what bounds them is each block's chain of barriers.
        // It goes by the rows' room, lengths being known to the GPU alone: 512 rows of 4608 tokens with room for as many
        // 14 us, for 32768 30, for 131072 98 (clusters of eight large blocks, most of which find no token), for
        // 140000 21 (the kernel that reads from memory).
        constexpr int kSmall = 256, kLarge = 512, kMost = 32;   // threads; tokens of one
        int size = 1;
        while (size < kMostCluster && c->width > kMost * kSmall * size)
            size *= 2;
        while (size < kMostCluster && rows * size < 152 && c->width > 8 * kSmall * size)
            size *= 2;
        const int64_t per_block = ((int64_t)c->width + size - 1) / size;
        const bool small = per_block <= kMost * kSmall;
        const int64_t each = (per_block + (small ? kSmall : kLarge) - 1) / (small ? kSmall : kLarge);
        if (c->width <= 2048)
            err = c->width <= 128   ? launch_bits<1, 4>(*c, rows, s)
                  : c->width <= 512 ? launch_bits<1, 16>(*c, rows, s)
                                    : launch_bits<4, 16>(*c, rows, s);
        else if (c->width <= 8192 && rows < 152)
            err = c->width <= 5120 ? launch_bits<8, 20>(*c, rows, s) : launch_bits<8, 32>(*c, rows, s);
        else if (rows * size >= limit || each > kMost)
            k_choose_long<<<(unsigned)rows, kChooseThreads, 0, s>>>(*c);
        else if (!small)
            err = each <= 24 ? launch_choice<kLarge, 24>(*c, rows, size, s) : launch_choice<kLarge, 32>(*c, rows, size, s);
        else
            err = each <= 8    ? launch_choice<kSmall, 8>(*c, rows, size, s)
                  : each <= 20 ? launch_choice<kSmall, 20>(*c, rows, size, s)
                               : launch_choice<kSmall, 32>(*c, rows, size, s);
    }
    if (err == cudaSuccess)
        err = cudaGetLastError();
    if (err == cudaSuccess)
        err = launch_under(k_choose_lens, dim3(1), kLensThreads, 0, s, *c);
    return err == cudaSuccess ? CG_OK : CG_ERR_CUDA;
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
        return launch_move<decltype(blob)>(a, lists * cache->num_heads, s);
    });
    return err == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

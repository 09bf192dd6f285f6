/*
 * cachegen.h: C ABI of the GB300 CacheGen KV-cache codec.
 *
 * The codec compresses a bf16 KV cache kv[L][2][T][H][D] (layers, K/V,
 * tokens, heads, head size; C = H*D channels) into
 *   - one fp32 scale per (K/V, layer, token): a = max_c |x|,
 *   - one 16-bit integer CDF per (token group, K/V, layer, channel),
 *   - one arithmetic-coded bitstream per (K/V, layer, token),
 * and decodes it back to bf16. The operation follows
 *   "LMCache 中的 KV Cache 压缩：CacheGen 编解码原理、配置方式与源码解析"
 *   (0539edu.com/news/4720135), cited below as [CG-LMCache]:
 *   §1 QuantizationSpec (per-layer bin counts), §2 Quantization,
 *   §3 CDF estimation and normalisation, §4 arithmetic coding in batches
 *   of at most 256 tokens, §5 decoding (prefix sum of stream lengths) and
 *   dequantisation;
 * with the 32-bit low/high arithmetic coder of Witten, Neal and Cleary
 * ("Arithmetic coding for data compression", CACM 30(6), 1987).
 *
 * Exact definitions (all integer results are bit-exact across runs):
 *   bins_l     bin count of layer l (from the K or V spec list); N = bins,
 *              MAX = bins/2 - 1; symbols lie in [0, 2*MAX].
 *   quantise   a = max_c |x_c|; f = MAX / a (fp32, f = 0 when a = 0);
 *              q = round_half_even(fp32(fp32(x * f) + MAX))  [CG-LMCache §2]
 *   groups     the T tokens form objects of chunk_tokens tokens (the last
 *              may be shorter); each object is cut into groups of at most
 *              256 tokens                                    [CG-LMCache §4]
 *   CDF        per (group, K/V, layer, channel), over the group's n tokens:
 *              cdf[i] = floor(cum[i] * (65536 - N) / n) + i, i = 0..N,
 *              cum[i] = number of symbols < i                [CG-LMCache §3]
 *   streams    one per (K/V, layer, token), holding the C symbols in
 *              channel order, coded with the channel's CDF: for r =
 *              high - low + 1, high = low + floor(r*cdf[s+1]/2^16) - 1,
 *              low = low + floor(r*cdf[s]/2^16), then the usual halving with
 *              pending bits; terminated by one more pending bit and then 0
 *              if low < 2^30 else 1, followed by the pending bits; bits MSB
 *              first, last byte zero-padded
 *   order      streams (and their lengths) are ordered group, then K/V,
 *              then layer, then token within the group; the byte stream is
 *              their concatenation; the decoder finds each stream by the
 *              exclusive prefix sum of the lengths           [CG-LMCache §5]
 *   dequantise y = bf16_rne(fp32(fp32((q - MAX) / MAX) * a))  [CG-LMCache §5]
 *
 * Buffers, layouts, ownership:
 *   The caller allocates every device buffer (kv, outputs, workspace) and
 *   keeps ownership; the library allocates only the host-side plan. All
 *   device pointers are plain device addresses. Calls that take a
 *   cudaStream_t enqueue work on it and return without waiting unless the
 *   comment says otherwise.
 *     kv         bf16 [L][2][T][H*D], 16-byte aligned
 *     amax       fp32 [2][L][T] (the scale a of each K/V, layer, token)
 *     lengths    int32 [2*L*T] stream lengths in bytes, stream order
 *     cdf        uint16 [cdf_entries]: per group, K/V, layer, channel the
 *                N+1 entries cdf[0..N] (cdf[N] = 65536 is stored as 0),
 *                16-byte aligned
 *     bytestream uint8, the concatenated streams, 16-byte aligned
 *
 * Threads: a plan holds two side streams and two events with which
 * cg_encode and cg_decode fork work onto a second stream and join it back
 * (cg_encode's side stream has the device's greatest stream priority, so
 * its smaller bin-count classes, whose tiles take longer, are dispatched
 * before the largest class and before lower-priority work). Calls that
 * use the same plan must therefore come from one host thread at a time (use
 * one plan per thread); calls on different plans are independent. Device
 * work of two calls may overlap only if they use different workspaces.
 *
 * Errors: argument and configuration errors are returned synchronously.
 * Errors found on the device (capacity exceeded, non-finite input, a
 * corrupt container) set a status word in the workspace; read it with
 * cg_last_device_error after the stream's work. Kernels never trap and
 * never wait on other blocks.
 */
#ifndef CACHEGEN_H
#define CACHEGEN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *cg_stream_t; /* a cudaStream_t; NULL = legacy default stream */

/* Layer range [start_layer, end_layer) with one bin count [CG-LMCache §1].
 * Per K and per V the ranges must cover [0, num_layers) exactly once;
 * bins must be even and in [4, 64]. */
typedef struct cg_quant_spec {
    int32_t start_layer;
    int32_t end_layer;
    int32_t bins;
} cg_quant_spec;

/* Shape of the KV blob and the codec configuration. num_heads*head_size
 * (C) must be a positive multiple of 8; chunk_tokens > 0 is the object
 * size in tokens [CG-LMCache §4: chunk_size]. */
typedef struct cg_config {
    int32_t num_layers;
    int32_t num_tokens;
    int32_t num_heads;
    int32_t head_size;
    int32_t chunk_tokens;
    const cg_quant_spec *kspecs;
    int32_t n_kspecs;
    const cg_quant_spec *vspecs;
    int32_t n_vspecs;
} cg_config;

typedef enum cg_status {
    CG_OK = 0,
    CG_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size */
    CG_ERR_SPEC = 2,        /* spec ranges do not tile [0, L) or bad bins */
    CG_ERR_CAPACITY = 3,    /* an output buffer is too small */
    CG_ERR_NONFINITE = 4,   /* the input holds inf or NaN, or a row too
                               small for a finite scale factor */
    CG_ERR_CORRUPT = 5,     /* a container or its tables are inconsistent */
    CG_ERR_TIMEOUT = 6,     /* a bounded device wait gave up (the decoder's
                               wait for a CDF table's bulk copy) */
    CG_ERR_CUDA = 7,        /* a CUDA runtime call failed */
    CG_ERR_UNSUPPORTED = 8  /* the shape exceeds this build's limits */
} cg_status;

typedef struct cg_plan cg_plan;

/* Sizes derived from a plan. */
typedef struct cg_sizes {
    size_t workspace_bytes;   /* device scratch that cg_encode/cg_decode need */
    size_t max_stream_bytes;  /* a bytestream capacity that can never overflow */
    size_t cdf_entries;       /* uint16 entries of the cdf buffer */
    size_t num_streams;       /* int32 entries of lengths (= 2*L*T) */
    size_t num_scales;        /* fp32 entries of amax (= 2*L*T) */
    size_t raw_bytes;         /* bytes of the bf16 KV blob (= 2*L*T*C*2) */
    int32_t num_groups;       /* token groups of at most 256 tokens */
    int32_t num_tiles;        /* groups * 2 * L */
    int32_t encode_launches;  /* kernels one cg_encode enqueues */
    int32_t decode_launches;  /* kernels one cg_decode enqueues */
    int32_t num_objects;      /* objects of chunk_tokens tokens (cg_object_range) */
} cg_sizes;

/* Device buffers of one encoded blob (all caller-owned). */
typedef struct cg_encoded {
    uint8_t *bytestream;
    size_t bytestream_capacity;
    int32_t *lengths;
    uint16_t *cdf;
    float *amax;
} cg_encoded;

/* Validate a configuration and build a plan (host memory only).
 * Returns CG_ERR_INVALID_ARG for null pointers or non-positive sizes,
 * CG_ERR_SPEC for spec lists that do not tile the layers or bad bins,
 * CG_ERR_UNSUPPORTED when the shape exceeds the kernels' limits
 * (L <= 256; C <= 4096 and C*(max bins+1)*2 bytes of CDF table must fit
 * in shared memory). [CG-LMCache §1] */
cg_status cg_plan_create(const cg_config *cfg, cg_plan **plan_out);

/* Free a plan (NULL is ignored). */
void cg_plan_destroy(cg_plan *plan);

/* Fill *out with the buffer sizes of a plan. Host only. */
cg_status cg_plan_sizes(const cg_plan *plan, cg_sizes *out);

/* The configuration a plan was built from (for a plan from
 * cg_container_open: the shape, chunk_tokens and spec lists recorded in the
 * container, which from_bytes of [CG-LMCache §5] must recover). Host only.
 * out gets the five sizes and n_kspecs / n_vspecs; its kspecs / vspecs
 * point at the caller's arrays kspecs[kcap] and vspecs[vcap], which receive
 * the spec triples in the order they were given. If kcap < n_kspecs or
 * vcap < n_vspecs nothing is copied and CG_ERR_CAPACITY is returned (the
 * counts are still set, so a caller can size its arrays and call again);
 * a NULL array is allowed with a capacity of 0. */
cg_status cg_plan_config(const cg_plan *plan, cg_config *out, cg_quant_spec *kspecs,
                         int32_t kcap, cg_quant_spec *vspecs, int32_t vcap);

/* Encode kv (device, bf16 [L][2][T][H*D]) into out's device buffers
 * [CG-LMCache §2-§4]. workspace (device, >= workspace_bytes, 256-byte
 * aligned) is scratch; its first 256 bytes receive the device status and
 * the total stream length, read back with cg_last_device_error. A
 * bytestream_capacity below the encoded size sets CG_ERR_CAPACITY on the
 * device and leaves the bytestream incomplete (never written out of
 * bounds); max_stream_bytes never overflows. Asynchronous on stream. */
cg_status cg_encode(const cg_plan *plan, const void *kv, void *workspace, size_t workspace_bytes,
                    const cg_encoded *out, cg_stream_t stream);

/* Decode in (device buffers written by cg_encode or cg_deserialize, with
 * stream_bytes bytes of streams; bytestream_capacity must be at least
 * stream_bytes rounded up to 16; stream_bytes below the number of
 * streams is CG_ERR_CORRUPT) into kv_out (device, bf16
 * [L][2][T][H*D], 16-byte aligned) [CG-LMCache §5]. With kv_out 32-byte
 * aligned and H*D a multiple of 16 every row is written in whole 32-byte
 * sectors (faster); otherwise in 16-byte pieces, with the same result.
 * Invalid CDF rows or lengths that do not add up to stream_bytes set
 * CG_ERR_CORRUPT on the device; a bounded wait inside the decoder that
 * runs out sets CG_ERR_TIMEOUT. Decoding of a corrupt stream still ends
 * after C symbols per stream and never reads outside the buffers.
 * Asynchronous on stream. */
cg_status cg_decode(const cg_plan *plan, const cg_encoded *in, uint64_t stream_bytes,
                    void *workspace, size_t workspace_bytes, void *kv_out, cg_stream_t stream);

/* Wait for stream, then read the device status word and the total stream
 * bytes of the last cg_encode/cg_decode that used this workspace (or the
 * status block of cg_encode_noalloc or cg_int8_encode; plan may be NULL,
 * the block's layout does not depend on it). Either output may be NULL.
 * Returns CG_ERR_CUDA if the copy fails. */
cg_status cg_last_device_error(const cg_plan *plan, const void *workspace, cg_status *status,
                               uint64_t *stream_bytes, cg_stream_t stream);

/* Bytes of the flat container for stream_bytes bytes of streams. The
 * container (little-endian) is: "CGKV", u32 version 1, i32 L, T, H, D,
 * chunk_tokens, n_kspecs, n_vspecs, num_groups, u64 stream_bytes; the
 * specs (K then V) as i32 triples; amax f32[2LT]; lengths i32[2LT]; cdf
 * u16[cdf_entries]; the streams. It replaces the pickled object of
 * [CG-LMCache §4]. */
cg_status cg_container_size(const cg_plan *plan, uint64_t stream_bytes, size_t *bytes);

/* Write the container of an encoded blob into host memory (pinned memory
 * copies fastest): header on the host, sections copied device-to-host.
 * Waits for stream before returning. */
cg_status cg_serialize(const cg_plan *plan, const cg_encoded *enc, uint64_t stream_bytes,
                       void *host_out, size_t host_capacity, size_t *written, cg_stream_t stream);

/* Read a container header from host memory and build its plan.
 * *stream_bytes gets the stream length. CG_ERR_CORRUPT for a bad magic,
 * version or inconsistent sizes. */
cg_status cg_container_open(const void *host_in, size_t len, cg_plan **plan_out,
                            uint64_t *stream_bytes);

/* Copy a container's sections from host memory into device buffers for
 * cg_decode. The plan must come from cg_container_open on the same bytes.
 * Waits for stream before returning. */
cg_status cg_deserialize(const cg_plan *plan, const void *host_in, size_t len,
                         const cg_encoded *dev_out, cg_stream_t stream);

/* Objects. LMCache keeps a KV cache as objects of chunk_tokens tokens
 * [CG-LMCache §4: chunk_size] (the last may be shorter). One cg_encode
 * codes every object of a plan in the same launches; since token groups
 * never span two objects, an object's CDF blocks, lengths and streams are
 * exactly those of encoding its tokens alone. The calls below cut an
 * encoded blob into one container per object, and put the containers of
 * all objects back into device buffers for one cg_decode.
 *
 * cg_object_range: first token and token count of object (0 <= object <
 * num_objects of cg_plan_sizes). Host only; CG_ERR_INVALID_ARG for an
 * object out of range.
 *
 * cg_object_streams: after a cg_encode (or cg_decode) that used this
 * workspace, the byte offset and length of the object's streams within the
 * bytestream, read from the workspace. Waits for stream.
 *
 * cg_object_container_size: bytes of the object's container for
 * stream_bytes bytes of streams. Host only.
 *
 * cg_serialize_object: write the object's container into host memory. It is
 * the container format of cg_serialize for a plan with the same L, H, D,
 * chunk_tokens and specs and T = the object's token count; its sections are
 * the object's amax columns [2][L][n], lengths, CDF blocks and streams, so it
 * is byte-identical to encoding and serialising the object's tokens alone.
 * Waits for stream.
 *
 * cg_deserialize_objects: copy the containers of all num_objects objects,
 * in object order (hosts[i] holds lens[i] bytes), into device buffers laid
 * out as cg_encode writes them for the whole plan; *stream_bytes gets the
 * total stream length to pass to cg_decode. Every header is checked before
 * anything is copied: CG_ERR_CORRUPT if a container is not object i of this
 * plan (shape, specs, tokens, groups, length), CG_ERR_CAPACITY if the
 * streams do not fit, CG_ERR_INVALID_ARG if num_objects differs from the
 * plan's. Waits for stream. */
cg_status cg_object_range(const cg_plan *plan, int32_t object, int32_t *first_token,
                          int32_t *num_tokens);
cg_status cg_object_streams(const cg_plan *plan, const void *workspace, int32_t object,
                            uint64_t *offset, uint64_t *bytes, cg_stream_t stream);
cg_status cg_object_container_size(const cg_plan *plan, int32_t object, uint64_t stream_bytes,
                                   size_t *bytes);
cg_status cg_serialize_object(const cg_plan *plan, const cg_encoded *enc, const void *workspace,
                              int32_t object, void *host_out, size_t host_capacity,
                              size_t *written, cg_stream_t stream);
cg_status cg_deserialize_objects(const cg_plan *plan, int32_t num_objects,
                                 const void *const *hosts, const size_t *lens,
                                 const cg_encoded *dev_out, uint64_t *stream_bytes,
                                 cg_stream_t stream);

/* Bytes of the fixed scratch array that cg_encode_noalloc uses (64 MiB). */
#define CG_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)

/* Encode like cg_encode, but without a workspace argument and without any
 * device allocation: for callers that cannot allocate device memory when
 * they encode, such as a serving engine that has already reserved nearly
 * all of the GPU for its KV cache pool, or a latency-critical path where
 * cudaMalloc/cudaFree (which may synchronise the device) is not allowed.
 * The pages describe no such call; it is an addition of this library.
 * The scratch is one array of CG_NOALLOC_SCRATCH_BYTES bytes inside the
 * library, which every GPU that loads the library keeps until the process
 * exits. A plan whose workspace_bytes exceed it is rejected with
 * CG_ERR_UNSUPPORTED before anything is enqueued. The caller still passes
 * kv and the output buffers (same rules as cg_encode) and status_out, a
 * device buffer of at least 16 bytes that receives the device status word
 * and the total stream bytes (read it with cg_last_device_error, passing
 * status_out as the workspace). Every call looks up the array's device
 * address in the current device's context (nothing is cached, so a device
 * reset leaves no stale address); the first call on each device also loads
 * the library's device code there, so make that first call before any
 * stream capture. All calls share the one array and it keeps the last
 * call's contents (each call clears what must start at zero): calls that
 * can overlap on the GPU, from any stream or thread, race on it, so
 * serialise them. status_out is not a workspace: the object calls
 * (cg_object_streams, cg_serialize_object) read tile offsets that only a
 * cg_encode workspace holds, so they must not be given status_out; encode
 * with cg_encode when per-object containers are needed. Asynchronous on
 * stream. */
cg_status cg_encode_noalloc(const cg_plan *plan, const void *kv, const cg_encoded *out,
                            void *status_out, cg_stream_t stream);

/* Int8 baseline codec, the comparison point for the ratio and throughput
 * of the codec above. "CacheGen复现项目：面向大模型服务的高效KV缓存压缩与流式传输
 * 方案" (§编解码器模块) quantises KV to 8-bit integers with scale factors
 * and gives no formula; this library reads it as the symmetric scaling of
 * [CG-LMCache §2] with MAX = 127 and no offset, one scale per row:
 *   a = max_c |x_c|; f = 127 / a (fp32, f = 0 when a = 0);
 *   q = round_half_even(fp32(x * f)) in [-127, 127]  (int8)
 *   y = bf16_rne(fp32(fp32(q / 127) * a))
 * A row is C = channels bf16 values; for a KV cache, rows are the
 * (layer, K/V, token) rows of kv[L][2][T][H*D] in memory order, so
 * rows = 2*L*T and channels = H*D.
 *
 * cg_int8_encode: kv (device, bf16 [rows][channels], 16-byte aligned) into
 * q_out (device, int8 [rows][channels], 8-byte aligned) and scales_out
 * (device, fp32 [rows], the a of each row). status_out (device, 16 bytes,
 * 16-byte aligned) is cleared by the call; a row holding inf/NaN, or one
 * so small (a below about 2^-121) that 127 / a overflows fp32, sets its
 * first word to CG_ERR_NONFINITE (that row's q are then meaningless); read
 * it with cg_last_device_error(NULL, status_out, ...). channels is a
 * multiple of 8 up to 4096 (CG_ERR_INVALID_ARG, CG_ERR_UNSUPPORTED above);
 * rows = 0 only clears the status. Asynchronous on stream.
 *
 * cg_int8_decode: q and scales (device, as written by cg_int8_encode) into
 * kv_out (device, bf16 [rows][channels], 16-byte aligned). Every byte value
 * decodes (0x80, never written by the encoder, gives -128/127 * a).
 * Asynchronous on stream. */
cg_status cg_int8_encode(const void *kv, int64_t rows, int32_t channels, void *q_out,
                         float *scales_out, void *status_out, cg_stream_t stream);
cg_status cg_int8_decode(const void *q, const float *scales, int64_t rows, int32_t channels,
                         void *kv_out, cg_stream_t stream);

/* A KV cache held in 4 bits, in pages, that attention reads directly: for
 * serving from a cache that stays compressed on the GPU. It takes the rows
 * that cg_decode restores (kv[l][0] and kv[l][1] are its k and v) or that a
 * model has just computed, and gives them back for cg_encode. These calls
 * are additions of this library; the pages describe none of them.
 *
 *   quantise   per (token, head) row of head_size channels and group of
 *              `group` channels: lo = min x, hi = max x,
 *              s = bf16_rne(fp32(fp32(hi - lo) * fp32(1 / 15)));
 *              n = min(15, round_half_even(fp32(fp32(x - lo) / s))),
 *              n = 0 where s = 0                        (4 bits, s and lo bf16)
 *   value      x^ = lo + s n; cg_int4_load gives bf16_rne(fp32(lo + fp32(s n)))
 *   attention  out_i = sum_j p_ij v^_j, p_i = softmax over the visible j of
 *              scale q_i . k^_j. Query i of a request with n queries and m
 *              cached tokens (its own among them) stands at position
 *              x = m - n + i and sees j when j <= x and (window == 0 or
 *              x - j < window or j < sinks). A query that sees nothing gets 0.
 *
 * Layout. data is [num_layers][num_pages][num_heads][page_tokens / 16] blobs
 * of 16 tokens; a blob of head size D with g = D / group is 16 (D + 8 g) bytes:
 *   K codes   [16 tokens][D/2]: channel c in byte c%32/8 * D/8 + c/32 * 4 + c%8/2
 *   K params  [16 tokens][g] of (s, lo), two bf16
 *   V codes   [8 token pairs][D]: channel c of token 2p + b in byte
 *             c%32/4 * D/8 + c/32 * 4 + 2 b + c%4/2
 *   V params  as K params
 * with the even channel of a byte in its low half: the words that one thread
 * of a matrix instruction needs lie side by side, and a head's tokens of a
 * page come in one bulk copy. Slot s of a layer is token s % page_tokens of
 * page s / page_tokens.
 *
 * status: 16 bytes (16-byte aligned) that the caller clears once; a call sets
 * the first word when it meets an error on the device and it has none yet.
 * Read it with cg_last_device_error(NULL, status, ...). Calls never clear it,
 * so it costs a call nothing and one read covers many calls;
 * cg_int4_take_error reads and clears it in one step.
 *
 * Limits (CG_ERR_UNSUPPORTED): head_size 64 or 128, group 32, 64 or 128 and
 * at most head_size, page_tokens a multiple of 16 up to 1024, num_layers *
 * num_pages * num_heads and num_pages * page_tokens below 2^31, one layer's
 * bytes below 2^39, a page's below 2^32. data must be
 * 256-byte aligned. */
typedef struct cg_int4_cache {
    void *data;
    void *status;
    int32_t num_layers;
    int32_t num_pages;
    int32_t page_tokens;
    int32_t num_heads;
    int32_t head_size;
    int32_t group;
} cg_int4_cache;

/* Bytes of a cache's data (its data and status pointers are not looked at).
 * Host only. */
cg_status cg_int4_cache_bytes(const cg_int4_cache *cache, size_t *bytes);

/* Moves the error in the cache's status, if any, to result (device, 16 bytes,
 * 16-byte aligned; read it with cg_last_device_error(NULL, result, ...)) and
 * leaves none, in one step on the device: an error that a call on another
 * stream meets meanwhile is in this result or stays for the next.
 * Asynchronous on stream. */
cg_status cg_int4_take_error(const cg_int4_cache *cache, void *result, cg_stream_t stream);

/* K and V rows: bf16 [layers][tokens][num_heads][head_size] with strides in
 * elements, channels contiguous; both pointers 16-byte aligned and every
 * stride a multiple of 8 (the head strides below 2^31). A layer of
 * cg_decode's output has k = kv[l][0], v = kv[l][1], a layer stride of 2*T*C, a
 * token stride of C and a head stride of head_size. */
typedef struct cg_kv_rows {
    void *k;
    void *v;
    int64_t k_layer_stride, k_token_stride, k_head_stride;
    int64_t v_layer_stride, v_token_stride, v_head_stride;
} cg_kv_rows;

/* cg_int4_store: quantise rows of `layers` layers into layers [first_layer,
 * first_layer + layers) of the cache: token t goes to slot slots[t] (device,
 * int32 [tokens]) of every layer. Slot -1 skips the token (padding); any
 * other slot outside the cache is skipped with CG_ERR_CORRUPT in status. Two
 * tokens of one call must not have the same slot (which of their parts stay
 * is then undefined). A group with inf or NaN, or whose hi - lo or largest
 * value lo + 15 s overflows, sets CG_ERR_NONFINITE and is stored as zeros.
 *
 * cg_int4_load: the other way, into rows. Slot -1 gives zeros, any other slot
 * outside the cache zeros and CG_ERR_CORRUPT. The same slot may occur often.
 *
 * Both are asynchronous on stream, in one launch. */
cg_status cg_int4_store(const cg_int4_cache *cache, int32_t first_layer, int32_t layers,
                        const cg_kv_rows *rows, const int32_t *slots, int64_t tokens,
                        cg_stream_t stream);
cg_status cg_int4_load(const cg_int4_cache *cache, int32_t first_layer, int32_t layers,
                       const cg_kv_rows *rows, const int32_t *slots, int64_t tokens,
                       cg_stream_t stream);

/* Most requests of one cg_pages_grow or cg_int4_attention call. */
#define CG_MAX_REQUESTS 8192

/* Pages and slots for the new tokens of a batch, worked out on the GPU from
 * the requests' lengths, so that a serving loop (or a captured graph) needs
 * no host round trip. Request r holds lens[r] tokens in ceil(lens[r] /
 * page_tokens) pages, whose ids stand in row r of block_table (int32, rows
 * table_stride elements apart, table_width entries); counts[r] tokens are new.
 * The pages that they need beyond those are taken from the end of the list
 * free_pages[0 .. *free_count): the k-th page needed, by request and then by
 * position, is free_pages[*free_count - 1 - k]. The call writes
 *   block_table  the ids of the pages taken; no other entry
 *   cu_out       int32 [requests + 1]: exclusive prefix sum of counts
 *   lens_out     int32 [requests]: lens + counts (may be lens itself)
 *   free_count_out  int32 [1]: pages left (may be free_count itself)
 *   slots_out    int32 [tokens]: the slot of each new token, requests one
 *                after the other; -1 from cu_out[requests] on
 *   status       16 bytes, 16-byte aligned, always written: CG_OK, or
 *                CG_ERR_INVALID_ARG   a negative length or count
 *                CG_ERR_CAPACITY      too few free pages, a table row or
 *                                     slots_out too short
 *                CG_ERR_CORRUPT       free_count outside [0, free_capacity]
 *                                     or a page id outside [0, num_pages)
 *                of several the greatest code (a page id counts where there
 *                is no other error)
 * With an error nothing is taken: block_table is as it was, lens_out and
 * free_count_out repeat their inputs, cu_out is 0 and slots_out is -1 (a page
 * id outside the cache, in block_table or taken from free_pages, is the
 * exception: only its tokens' slots are -1). No other two arrays may overlap. Asynchronous on stream. */
typedef struct cg_page_batch {
    int32_t *block_table;
    int64_t table_stride;
    int32_t table_width;
    int32_t requests;
    const int32_t *lens;
    const int32_t *counts;
    const int32_t *free_pages;
    const int32_t *free_count;
    int32_t free_capacity;
    int32_t num_pages;
    int32_t page_tokens;
    int32_t *cu_out;
    int32_t *lens_out;
    int32_t *free_count_out;
    int32_t *slots_out;
    int64_t tokens;
    void *status;
} cg_page_batch;

cg_status cg_pages_grow(const cg_page_batch *batch, cg_stream_t stream);

/* Attention of new tokens over one layer of the cache (the formula above).
 * Their K and V must have been stored before. q and out are bf16 [tokens]
 * [q_heads][head_size] with strides in elements (multiples of 8, pointers
 * 16-byte aligned); query head h reads KV head h / (q_heads / num_heads).
 * cu_q (int32 [requests + 1]), kv_lens (int32 [requests]) and block_table
 * are device arrays as cg_pages_grow leaves them: request r owns the rows
 * [cu_q[r], cu_q[r+1]) of q and out, which may be none; rows from
 * cu_q[requests] on are left as they were. max_q_len: no request has more
 * rows of q than this (0: not known). Give it for batches of single and drafted
 * tokens: without it a call launches the kernel for many rows as well, and takes
 * the wider form of the one for few (64 single tokens at 4-8K, 4 query heads to a
 * KV head: 188 us, with it 111).
 * Table entries of pages in which no query of the request sees a token are
 * not read.
 *
 * Errors found on the device, in the cache's status: CG_ERR_CORRUPT for a
 * cu_q that is not ascending within [0, tokens], a negative kv_len or one
 * beyond table_width pages (the request's rows are left as they were), and
 * for a page id outside the cache (its tokens count as not visible);
 * CG_ERR_INVALID_ARG for a request with more than max_q_len rows (left as
 * they were); CG_ERR_TIMEOUT when a bounded wait ran out.
 *
 * out must not overlap q or the cache. Sums are in fp32: q, k and scale q
 * have to stay below 2^120, scores (and the sums of their terms' sizes) below
 * 2^100, and V values below 2^96 where a request has more than 32 rows per KV
 * head (query heads of it times new tokens), below 2^126 where it has fewer.
 * There, codes are summed in units that end at 2^-106 of 1, or of the KV head's
 * largest value v where that is above 32: small V values have an error of up to
 * 2^-108 max(1, v) times the tokens besides that of the roundings.
 *
 * workspace (device, 256-byte aligned, the size that
 * cg_int4_attention_workspace gives from the cache's shape, tokens, q_heads and
 * max_q_len; it looks at no pointer) is scratch: calls that may
 * overlap need one each. Asynchronous on stream. */
typedef struct cg_attention {
    const void *q;
    int64_t q_token_stride, q_head_stride;
    void *out;
    int64_t out_token_stride, out_head_stride;
    const int32_t *cu_q;
    const int32_t *kv_lens;
    const int32_t *block_table;
    int64_t table_stride;
    int32_t table_width;
    int32_t requests;
    int32_t tokens;
    int32_t q_heads;
    int32_t max_q_len;
    int32_t window;
    int32_t sinks;
    float scale;
} cg_attention;

cg_status cg_int4_attention_workspace(const cg_int4_cache *cache, const cg_attention *args,
                                      size_t *bytes);
cg_status cg_int4_attention(const cg_int4_cache *cache, int32_t layer, const cg_attention *args,
                            void *workspace, size_t workspace_bytes, cg_stream_t stream);

/* The same where every request begins with the same cached tokens (an instruction
 * or a document that a batch shares): the first shared_tokens of each request's tokens
 * lie in the same pages, the first shared_tokens / page_tokens entries of its row of
 * block_table. They are read by way of the first row of block_table (the other rows' entries
 * there are not read), and where there are enough of them once for all queries. kv_lens
 * counts the shared tokens too.
 *
 * Limits and roundings are those of cg_int4_attention for requests with more than 32 rows per KV
 * head, however few a request has: where the shared tokens are read for all queries at once, those
 * may be taken by the kernel for many rows. So V values have to stay below 2^96 (small ones may have
 * the error that they have for few rows all the same), and k, v and the
 * probabilities may each be rounded to bf16 (2^-8 relative at most), where for few rows
 * cg_int4_attention rounds the probabilities' products with the groups' steps alone. 64 requests of one
 * token each and 16384 shared ones: the result is off by 0.0028 of its norm, by 0.0019 in a call without
 * shared tokens, and by 0.0016 where nothing but itself is rounded.
 *
 * shared_tokens is a multiple of page_tokens and window is 0 (CG_ERR_INVALID_ARG; what
 * of the first tokens is in a window depends on the query); shared_tokens = 0 is
 * cg_int4_attention. A request whose new tokens do not all lie behind the shared ones
 * sets CG_ERR_INVALID_ARG in the cache's status, and one whose rows do not all lie before
 * cu_q[requests] CG_ERR_CORRUPT (their rows are left as they were).
 * A page id outside the cache among the shared ones hides its tokens from every query.
 * The workspace's size depends on requests and shared_tokens too, and is at most tokens * q_heads *
 * (head_size + 2) floats and 86 MB larger. */
cg_status cg_int4_attention_shared_workspace(const cg_int4_cache *cache, const cg_attention *args,
                                             int32_t shared_tokens, size_t *bytes);
cg_status cg_int4_attention_shared(const cg_int4_cache *cache, int32_t layer,
                                   const cg_attention *args, int32_t shared_tokens,
                                   void *workspace, size_t workspace_bytes, cg_stream_t stream);

/* Eviction: a cache that is kept to a budget by the attention that its tokens get.
 * cg_int4_weigh sums the attention weights of every token, cg_choose_tokens picks the
 * tokens of each head that stay, cg_int4_compact moves them to the front of their
 * request's pages, and cg_pages_release gives the pages behind them back to the list
 * that cg_pages_grow takes from. A request's heads (and layers) may keep different
 * tokens, but equally many. Positions count what is in the cache: what attention and
 * its masks call token j is from then on the j-th token that stayed.
 *
 * cg_int4_weigh, over one layer:
 *   out[r][h][j] = in[r][h][j] + sum_i sum_g p_igj   for j < kv_lens[r],
 * where p_ig is the softmax of cg_int4_attention for query i of request r and query head
 * g, over the request's new tokens i and the query heads g of KV head h. A token that a
 * query does not see gets 0 from it. Elements from kv_lens[r] on are left as they were.
 * p is computed in fp32, the sum over i and g in an order that does not depend on timing.
 *
 * args are those of cg_int4_attention (out and its strides are not looked at), with
 * the same limits and device errors (and tokens of a row, or width, at most 2^31 - 2^16); a
 * kv_len beyond width is CG_ERR_CORRUPT. Where cu_q is not ascending (which is reported) and the rows of the
 * requests that it leaves do not follow one another, all of the call's weights are undefined. in (NULL:
 * zeros) and out have rows of width floats, elements adjacent, strides in elements; in
 * may be out (with the same strides) and otherwise must not overlap it. Rows of out must not
 * overlap, nor out q or the cache. workspace as for attention; its size depends on the
 * cache's shape, tokens, requests, q_heads, max_q_len, table_width and width: room for the
 * scores where they are below 256 MB, for the queries again where they are not; and where a
 * request may have more than 64 rows (query heads of a KV head times new tokens), for sums of each 128
 * rows, a float a token, where those are below 1 GB. */
typedef struct cg_token_weights {
    const float *in;
    float *out;
    int64_t in_request_stride, in_head_stride;
    int64_t out_request_stride, out_head_stride;
    int32_t width;
} cg_token_weights;

cg_status cg_int4_weigh_workspace(const cg_int4_cache *cache, const cg_attention *args,
                                  const cg_token_weights *weights, size_t *bytes);
cg_status cg_int4_weigh(const cg_int4_cache *cache, int32_t layer, const cg_attention *args,
                        const cg_token_weights *weights, void *workspace, size_t workspace_bytes,
                        cg_stream_t stream);

/* cg_choose_tokens: of each row of weights (float [layers][requests][heads], rows of
 * width floats, elements adjacent, strides in elements) the tokens that stay. Of a request
 * with m = lens[r] tokens the first `sinks` and the last `recent` stay, and of the
 * others those with the greatest weights, min(m, budget) in all; of equal weights the
 * lower token, and NaN is below every other weight.
 *   kept      int32 [layers][requests][heads][budget], contiguous: the tokens that
 *             stay, ascending; -1 behind the last
 *   lens_out  int32 [requests]: min(m, budget) (may be lens itself; cg_int4_compact
 *             wants both)
 *   status    16 bytes, 16-byte aligned, always written: CG_OK, or CG_ERR_CORRUPT for a
 *             length that is negative or beyond width (its row of kept is -1,
 *             lens_out repeats it)
 * sinks + recent must not exceed budget (CG_ERR_INVALID_ARG). No other two arrays may
 * overlap. Limits (CG_ERR_UNSUPPORTED): CG_MAX_REQUESTS requests, layers * requests *
 * heads below 2^31. Asynchronous on stream. */
typedef struct cg_token_choice {
    const float *weights;
    int64_t layer_stride, request_stride, head_stride;
    int32_t layers, requests, heads, width;
    const int32_t *lens;
    int32_t budget, recent, sinks;
    int32_t *kept;
    int32_t *lens_out;
    void *status;
} cg_token_choice;

cg_status cg_choose_tokens(const cg_token_choice *choice, cg_stream_t stream);

/* cg_int4_compact: in layers [first_layer, first_layer + layers) of the cache, token
 * kept[l][r][h][i] of request r (its place in head h) goes to place i, for i <
 * new_lens[r]. kept is int32 [layers][requests][num_heads], rows of budget entries,
 * adjacent, strides in elements, as cg_choose_tokens writes it. weights (NULL: none;
 * float [layers][requests][num_heads], rows of weights_width floats) move along, and
 * those from new_lens[r] to lens[r] become 0. The places from new_lens[r] on keep their
 * bytes. A request with new_lens[r] = lens[r] is left as it is, whatever kept holds.
 * Tokens whose place does not change are not written where a whole blob of 16 stays
 * as it is, so pages that requests share may stand at the front of their tables as
 * long as all of their tokens stay; no other page may belong to two requests.
 *
 * Errors in the cache's status, CG_ERR_CORRUPT: a length that is negative or beyond
 * table_width pages or weights_width, new_lens[r] above lens[r] or (below it) above budget,
 * entries of kept that do not ascend within [0, lens[r]) (that head's tokens, of that
 * layer, or the whole request are left as they were); a page id outside the cache (what
 * would be read or written there is not moved). Table entries from lens[r] on are not read.
 * No two arrays may overlap. Asynchronous on stream. */
typedef struct cg_compaction {
    const int32_t *kept;
    int64_t kept_layer_stride, kept_request_stride, kept_head_stride;
    float *weights;
    int64_t weights_layer_stride, weights_request_stride, weights_head_stride;
    int32_t weights_width;
    int32_t budget;
    int32_t layers, requests;
    const int32_t *lens;
    const int32_t *new_lens;
    const int32_t *block_table;
    int64_t table_stride;
    int32_t table_width;
} cg_compaction;

cg_status cg_int4_compact(const cg_int4_cache *cache, int32_t first_layer,
                          const cg_compaction *args, cg_stream_t stream);

/* cg_pages_release: the counterpart of cg_pages_grow. Request r holds lens[r] tokens and
 * keeps new_lens[r] of them (0: the request ends); the pages behind those go to the
 * end of the list free_pages[0 .. *free_count), by request and then by position, and
 * their entries of block_table become -1. The call writes
 *   free_pages      the ids released, from *free_count on
 *   block_table     -1 for the pages released; no other entry
 *   cu_out          int32 [requests + 1]: exclusive prefix sum of the pages released
 *   lens_out        int32 [requests]: new_lens (may be lens or new_lens itself)
 *   free_count_out  int32 [1]: pages on the list (may be free_count itself)
 *   status          16 bytes, 16-byte aligned, always written: CG_OK, or
 *                   CG_ERR_INVALID_ARG   a negative length, or new_lens[r] above lens[r]
 *                   CG_ERR_CAPACITY      the list, or a table row, is too short
 *                   CG_ERR_CORRUPT       free_count outside [0, free_capacity]
 *                   or a released page id outside [0, num_pages)
 *                   of several the greatest code (a page id counts where there is no
 *                   other error)
 * With an error nothing is released: block_table and free_pages are as they were, lens_out
 * and free_count_out repeat lens and free_count, cu_out is 0 (a page id outside the cache
 * is the exception: it goes to the list as it is, where cg_pages_grow will find it). A
 * page that several requests share must not be released by more than one of them. No
 * other two arrays may overlap. Limits as for cg_pages_grow. Asynchronous on stream. */
typedef struct cg_page_release {
    int32_t *block_table;
    int64_t table_stride;
    int32_t table_width;
    int32_t requests;
    const int32_t *lens;
    const int32_t *new_lens;
    int32_t *free_pages;
    const int32_t *free_count;
    int32_t free_capacity;
    int32_t num_pages;
    int32_t page_tokens;
    int32_t *cu_out;
    int32_t *lens_out;
    int32_t *free_count_out;
    void *status;
} cg_page_release;

cg_status cg_pages_release(const cg_page_release *batch, cg_stream_t stream);

/* Per-kernel timing, for profiling. When enabled, each kernel that
 * cg_encode/cg_decode enqueue is bracketed by two CUDA events on the launch
 * stream (up to max_launches kernels are recorded; later ones are not).
 * cg_profile_read waits for the recorded events, reports per kernel name
 * the launches and the summed event time, and clears the record.
 * max_launches = 0 disables and frees the events. Not thread-safe: one
 * host thread per plan while profiling. */
typedef struct cg_kernel_profile {
    const char *kernel; /* static string */
    int64_t launches;
    double total_ms;
} cg_kernel_profile;

cg_status cg_profile_enable(cg_plan *plan, int32_t max_launches);
cg_status cg_profile_read(cg_plan *plan, cg_kernel_profile *out, int32_t capacity,
                          int32_t *count);

/* Human-readable name of a status code (static string). */
const char *cg_status_string(cg_status status);

#ifdef __cplusplus
}
#endif

#endif /* CACHEGEN_H */

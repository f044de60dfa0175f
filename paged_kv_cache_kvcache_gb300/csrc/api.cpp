// C ABI of libpagedattn: argument validation on the host, then kernel launches.
// No entry point allocates, synchronises or reads device memory on the host
// (except pa_read_device_error, a debugging aid).
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include <cuda_runtime.h>

#include "internal.h"

namespace pa {

static thread_local char g_err[512] = "";

void set_error(const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
}

int fail(int code, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

int check_dims(const pa_dims *dims)
{
    if (!dims)
        return fail(PA_ERR_INVALID_ARG, "dims is NULL");
    const pa_dims &d = *dims;
    if (d.num_blocks < 0 || d.block_size <= 0 || d.num_heads <= 0 || d.num_kv_heads <= 0 || d.head_dim <= 0)
        return fail(PA_ERR_INVALID_ARG, "dims must be positive (num_blocks may be 0)");
    if (d.num_heads % d.num_kv_heads != 0)
        return fail(PA_ERR_UNSUPPORTED, "num_heads (%d) is not a multiple of num_kv_heads (%d)", d.num_heads,
                    d.num_kv_heads);
    if (d.num_heads / d.num_kv_heads > kMaxGroup)
        return fail(PA_ERR_UNSUPPORTED, "group size %d > %d", d.num_heads / d.num_kv_heads, kMaxGroup);
    if (d.head_dim != 64 && d.head_dim != 128)
        return fail(PA_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}", d.head_dim);
    if (d.block_size < 16 || d.block_size > 1024 || (d.block_size & (d.block_size - 1)))
        return fail(PA_ERR_UNSUPPORTED, "block_size %d is not a power of two in [16, 1024]", d.block_size);
    if ((int64_t)d.num_blocks * d.block_size > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "num_blocks*block_size exceeds int32");
    return PA_OK;
}

static bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

} // namespace pa

using namespace pa;

extern "C" const char *pa_last_error_string(void) { return g_err; }

extern "C" int pa_version(void) { return 0x000500; }

extern "C" int pa_upload(void *dev_dst, const void *host_src, size_t bytes, pa_stream_t stream)
{
    if (bytes == 0)
        return PA_OK;
    if (!dev_dst || !host_src)
        return fail(PA_ERR_INVALID_ARG, "pa_upload: NULL pointer");
    cudaError_t e = cudaMemcpyAsync(dev_dst, host_src, bytes, cudaMemcpyHostToDevice, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail(PA_ERR_CUDA, "cudaMemcpyAsync: %s", cudaGetErrorString(e));
    return PA_OK;
}

extern "C" int pa_store_kvcache(const pa_dims *dims, const void *k, const void *v, void *k_cache, void *v_cache,
                                const int32_t *slot_mapping, int32_t num_tokens, pa_stream_t stream)
{
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (num_tokens < 0)
        return fail(PA_ERR_INVALID_ARG, "num_tokens < 0");
    if (num_tokens == 0)
        return PA_OK;
    if (!k || !v || !k_cache || !v_cache || !slot_mapping)
        return fail(PA_ERR_INVALID_ARG, "pa_store_kvcache: NULL pointer");
    if (misaligned(k) || misaligned(v) || misaligned(k_cache) || misaligned(v_cache))
        return fail(PA_ERR_INVALID_ARG, "pa_store_kvcache: tensors must be 16-byte aligned");
    return launch_store_kvcache(*dims, k, v, k_cache, v_cache, slot_mapping, num_tokens, stream);
}

// Host-side checks of pa_rope_store(_int8), then the launch.
static int rope_store(const char *fn, const pa_dims *dims, const pa_rope *rope, const void *q, const void *k,
                      const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t *positions,
                      const int32_t *slot_mapping, int32_t num_tokens, void *q_out, void *k_cache, void *v_cache,
                      bool int8, void *k_scale, void *v_scale, pa_stream_t stream)
{
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (!rope)
        return fail(PA_ERR_INVALID_ARG, "%s: rope is NULL", fn);
    const pa_rope &r = *rope;
    if (r.rotary_dim < 16 || r.rotary_dim > dims->head_dim || r.rotary_dim % 16 != 0)
        return fail(PA_ERR_UNSUPPORTED, "%s: rotary_dim %d is not a multiple of 16 in [16, head_dim]", fn, r.rotary_dim);
    if (r.num_axes < 1 || r.num_axes > 4)
        return fail(PA_ERR_UNSUPPORTED, "%s: num_axes %d not in [1, 4]", fn, r.num_axes);
    for (int i = 0; i < r.rotary_dim / 2; ++i)
        if (r.pair_axis[i] >= r.num_axes)
            return fail(PA_ERR_INVALID_ARG, "%s: pair %d turns on axis %d of %d", fn, i, r.pair_axis[i], r.num_axes);
    if ((r.interleaved != 0 && r.interleaved != 1) || r.max_position < 1 || !(r.eps >= 0.f) || !std::isfinite(r.eps))
        return fail(PA_ERR_INVALID_ARG, "%s: interleaved must be 0 or 1, max_position positive, eps finite and >= 0", fn);
    if (num_tokens < 0)
        return fail(PA_ERR_INVALID_ARG, "num_tokens < 0");
    if ((int64_t)num_tokens * (dims->num_heads + 2 * dims->num_kv_heads) > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "%s: %d tokens of %d heads exceed an int32", fn, num_tokens,
                    dims->num_heads + 2 * dims->num_kv_heads);
    if (num_tokens == 0)
        return PA_OK;
    if (!r.cos_sin || !q || !k || !v || !positions || !slot_mapping || !q_out || !k_cache || !v_cache ||
        (int8 && (!k_scale || !v_scale)))
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (misaligned(r.cos_sin) || misaligned(r.q_weight) || misaligned(r.k_weight) || misaligned(q) || misaligned(k) ||
        misaligned(v) || misaligned(q_out) || misaligned(k_cache) || misaligned(v_cache) || misaligned(k_scale) ||
        misaligned(v_scale))
        return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
    const int64_t qrow = (int64_t)dims->num_heads * dims->head_dim, krow = (int64_t)dims->num_kv_heads * dims->head_dim;
    if (q_stride < qrow || k_stride < krow || v_stride < krow || q_stride % 8 || k_stride % 8 || v_stride % 8)
        return fail(PA_ERR_INVALID_ARG, "%s: strides must be multiples of 8 of at least a token's values", fn);
    if (q_out == q && q_stride != qrow)
        return fail(PA_ERR_INVALID_ARG, "%s: q_out may only be q where q's tokens are contiguous", fn);
    if (dims->num_blocks == 0)
        return fail(PA_ERR_INVALID_ARG, "empty KV pool");
    return launch_rope_store({*dims, r, q, k, v, q_stride, k_stride, v_stride, positions, slot_mapping, num_tokens, q_out,
                              k_cache, v_cache, k_scale, v_scale},
                             stream);
}

extern "C" int pa_rope_store(const pa_dims *dims, const pa_rope *rope, const void *q, const void *k, const void *v,
                             int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t *positions,
                             const int32_t *slot_mapping, int32_t num_tokens, void *q_out, void *k_cache,
                             void *v_cache, pa_stream_t stream)
{
    return rope_store("pa_rope_store", dims, rope, q, k, v, q_stride, k_stride, v_stride, positions, slot_mapping,
                      num_tokens, q_out, k_cache, v_cache, false, nullptr, nullptr, stream);
}

extern "C" int pa_rope_store_int8(const pa_dims *dims, const pa_rope *rope, const void *q, const void *k,
                                  const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                  const int32_t *positions, const int32_t *slot_mapping, int32_t num_tokens,
                                  void *q_out, void *k_cache, void *v_cache, void *k_scale, void *v_scale,
                                  pa_stream_t stream)
{
    return rope_store("pa_rope_store_int8", dims, rope, q, k, v, q_stride, k_stride, v_stride, positions, slot_mapping,
                      num_tokens, q_out, k_cache, v_cache, true, k_scale, v_scale, stream);
}

// Host-side checks shared by pa_prefill_varlen and pa_prefill_varlen_int8;
// fills `a`.  Sets *nothing when the plan has no work (then no launch happens).
static int prepare_prefill(const char *fn, const pa_dims *dims, const void *q, const void *k_cache,
                           const void *v_cache, const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                           const int32_t *block_tables, float scale, void *out, const pa_prefill_meta *meta,
                           const int32_t *tiles, PrefillArgs *a, bool *nothing)
{
    *nothing = false;
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (!meta)
        return fail(PA_ERR_INVALID_ARG, "meta is NULL");
    if (meta->num_tiles < 0 || meta->total_q < 0 || meta->num_seqs < 0 || meta->max_blocks_per_seq < 1)
        return fail(PA_ERR_INVALID_ARG, "malformed prefill meta");
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(PA_ERR_INVALID_ARG, "scale must be finite and > 0");
    const int group = dims->num_heads / dims->num_kv_heads;
    if (meta->rows_per_tile != (kPrefillRows / group > 0 ? kPrefillRows / group : 1))
        return fail(PA_ERR_INVALID_ARG, "prefill meta was packed for other dims");
    if (meta->num_tiles == 0 || meta->total_q == 0) {
        *nothing = true;
        return PA_OK;
    }
    if (!q || !k_cache || !v_cache || !cu_seqlens_q || !cu_seqlens_k || !block_tables || !out || !tiles)
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(out))
        return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
    if (dims->num_blocks == 0)
        return fail(PA_ERR_INVALID_ARG, "empty KV pool");
    *a = PrefillArgs{};
    a->dims = *dims;
    a->q = q;
    a->k_cache = k_cache;
    a->v_cache = v_cache;
    a->cu_seqlens_q = cu_seqlens_q;
    a->cu_seqlens_k = cu_seqlens_k;
    a->block_tables = block_tables;
    a->tiles = tiles;
    a->out = out;
    a->scale = scale;
    a->num_tiles = meta->num_tiles;
    a->total_q = meta->total_q;
    a->max_blocks_per_seq = meta->max_blocks_per_seq;
    a->rows_per_tile = meta->rows_per_tile;
    return PA_OK;
}

extern "C" int pa_prefill_varlen(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                                 const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                 const int32_t *block_tables, float scale, void *out, const pa_prefill_meta *meta,
                                 const int32_t *tiles, pa_stream_t stream)
{
    PrefillArgs a;
    bool nothing = false;
    int rc = prepare_prefill("pa_prefill_varlen", dims, q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k,
                             block_tables, scale, out, meta, tiles, &a, &nothing);
    if (rc != PA_OK || nothing)
        return rc;
    return launch_prefill(a, stream);
}

extern "C" int pa_prefill_varlen_fused(const pa_dims *dims, const void *q, const void *k, const void *v,
                                       void *k_cache, void *v_cache, const int32_t *cu_seqlens_q,
                                       const int32_t *cu_seqlens_k, const int32_t *block_tables,
                                       const int32_t *slot_mapping, float scale, void *out,
                                       const pa_prefill_meta *meta, const int32_t *tiles, pa_stream_t stream)
{
    PrefillArgs a;
    bool nothing = false;
    int rc = prepare_prefill("pa_prefill_varlen_fused", dims, q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k,
                             block_tables, scale, out, meta, tiles, &a, &nothing);
    if (rc != PA_OK || nothing)
        return rc;
    if (!k || !v || !slot_mapping)
        return fail(PA_ERR_INVALID_ARG, "pa_prefill_varlen_fused: NULL pointer");
    if (misaligned(k) || misaligned(v))
        return fail(PA_ERR_INVALID_ARG, "pa_prefill_varlen_fused: tensors must be 16-byte aligned");
    a.k_in = k;
    a.v_in = v;
    a.slot_mapping = slot_mapping;
    a.small_boxes = !meta->prefix_aligned;
    return launch_prefill(a, stream);
}

// INT8 prefill (plain and with the quantising store): the gather launch fills the
// plan's bf16 scratch cache from the INT8 cache (k_in set: after quantising the new
// rows into it), then the bf16 prefill kernel attends over the scratch cache through
// the scratch tables (128-token blocks).
static int prefill_int8(const char *fn, bool store, const pa_dims *dims, const void *q, const void *k, const void *v,
                        const void *k_cache, const void *v_cache, const void *k_scale, const void *v_scale,
                        const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, const int32_t *block_tables,
                        const int32_t *slot_mapping, const int32_t *scratch_tables, const int32_t *scratch_items,
                        float scale, void *out, const pa_prefill_meta *meta, const int32_t *tiles, void *workspace,
                        size_t workspace_bytes, pa_stream_t stream, int32_t window = 0, int32_t sinks = 0)
{
    PrefillArgs a;
    bool nothing = false;
    int rc = prepare_prefill(fn, dims, q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, block_tables, scale, out,
                             meta, tiles, &a, &nothing);
    if (rc != PA_OK || nothing)
        return rc;
    const pa_dims &d = *dims;
    if (!k_scale || !v_scale || !scratch_tables || !scratch_items || !workspace)
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (misaligned(k_scale) || misaligned(v_scale) || misaligned(workspace) || misaligned(scratch_items))
        return fail(PA_ERR_INVALID_ARG, "%s: scales, scratch items and workspace must be 16-byte aligned", fn);
    if (meta->scratch_blocks < 1 || meta->scratch_pitch < 1 ||
        meta->workspace_bytes != (uint64_t)meta->scratch_blocks * kPrefillKeyTile * d.num_kv_heads * d.head_dim * 4)
        return fail(PA_ERR_INVALID_ARG, "%s: prefill meta was packed for other dims", fn);
    if (workspace_bytes < meta->workspace_bytes)
        return fail(PA_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %llu", fn, workspace_bytes,
                    (unsigned long long)meta->workspace_bytes);
    if (store) {
        if (!k || !v || !slot_mapping)
            return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
        if (misaligned(k) || misaligned(v))
            return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
    }
    const size_t half = (size_t)meta->scratch_blocks * kPrefillKeyTile * d.num_kv_heads * d.head_dim;
    GatherArgs g{};
    g.num_kv_heads = d.num_kv_heads;
    g.head_dim = d.head_dim;
    g.block_size = d.block_size;
    g.max_blocks = meta->max_blocks_per_seq;
    g.scratch_blocks = meta->scratch_blocks;
    g.num_slots = (int64_t)d.num_blocks * d.block_size;
    g.k_codes = static_cast<const int8_t *>(k_cache);
    g.v_codes = static_cast<const int8_t *>(v_cache);
    g.k_scale = static_cast<const uint16_t *>(k_scale);
    g.v_scale = static_cast<const uint16_t *>(v_scale);
    g.block_tables = block_tables;
    g.scratch_items = scratch_items;
    g.k_out = static_cast<uint16_t *>(workspace);
    g.v_out = g.k_out + half;
    g.out_v8 = (reinterpret_cast<uintptr_t>(workspace) & 31u) == 0 ? 1 : 0;
    if (store) {
        g.k_in = static_cast<const uint16_t *>(k);
        g.v_in = static_cast<const uint16_t *>(v);
        g.slot_mapping = slot_mapping;
        g.k_codes_w = static_cast<int8_t *>(const_cast<void *>(k_cache));
        g.v_codes_w = static_cast<int8_t *>(const_cast<void *>(v_cache));
        g.k_scale_w = static_cast<uint16_t *>(const_cast<void *>(k_scale));
        g.v_scale_w = static_cast<uint16_t *>(const_cast<void *>(v_scale));
    }
    g.window = window;
    g.sinks = sinks;
    if ((rc = launch_int8_gather(g, stream)) != PA_OK)
        return rc;
    a.window = window;
    a.sinks = sinks;
    a.dims.num_blocks = meta->scratch_blocks;
    a.dims.block_size = kPrefillKeyTile;
    a.k_cache = g.k_out;
    a.v_cache = g.v_out;
    a.block_tables = scratch_tables;
    a.max_blocks_per_seq = meta->scratch_pitch;
    a.scratch_cache = true;
    return launch_prefill(a, stream);
}

extern "C" int pa_prefill_varlen_int8(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                                      const void *k_scale, const void *v_scale, const int32_t *cu_seqlens_q,
                                      const int32_t *cu_seqlens_k, const int32_t *block_tables,
                                      const int32_t *scratch_tables, const int32_t *scratch_items, float scale,
                                      void *out, const pa_prefill_meta *meta, const int32_t *tiles, void *workspace,
                                      size_t workspace_bytes, pa_stream_t stream)
{
    return prefill_int8("pa_prefill_varlen_int8", false, dims, q, nullptr, nullptr, k_cache, v_cache, k_scale, v_scale,
                        cu_seqlens_q, cu_seqlens_k, block_tables, nullptr, scratch_tables, scratch_items, scale, out,
                        meta, tiles, workspace, workspace_bytes, stream);
}

extern "C" int pa_prefill_varlen_int8_fused(const pa_dims *dims, const void *q, const void *k, const void *v,
                                            void *k_cache, void *v_cache, void *k_scale, void *v_scale,
                                            const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                            const int32_t *block_tables, const int32_t *slot_mapping,
                                            const int32_t *scratch_tables, const int32_t *scratch_items, float scale,
                                            void *out, const pa_prefill_meta *meta, const int32_t *tiles,
                                            void *workspace, size_t workspace_bytes, pa_stream_t stream)
{
    return prefill_int8("pa_prefill_varlen_int8_fused", true, dims, q, k, v, k_cache, v_cache, k_scale, v_scale,
                        cu_seqlens_q, cu_seqlens_k, block_tables, slot_mapping, scratch_tables, scratch_items, scale,
                        out, meta, tiles, workspace, workspace_bytes, stream);
}

// The window of a windowed prefill, cut to the batch's longest sequence (no further key is there to be seen).
static int check_window(const char *fn, const pa_prefill_meta *meta, int32_t *window, int32_t *sinks)
{
    if (*window < 1 || *sinks < 0)
        return fail(PA_ERR_INVALID_ARG, "%s: window must be at least 1, sinks at least 0", fn);
    const int32_t longest = meta && meta->max_seqlen_k > 0 ? meta->max_seqlen_k : 1;
    *window = *window < longest ? *window : longest;
    *sinks = *sinks < longest ? *sinks : longest;
    return PA_OK;
}

extern "C" int pa_prefill_window(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                                 const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                 const int32_t *block_tables, int32_t window, int32_t sinks, float scale, void *out,
                                 const pa_prefill_meta *meta, const int32_t *tiles, pa_stream_t stream)
{
    PrefillArgs a;
    bool nothing = false;
    int rc = check_window("pa_prefill_window", meta, &window, &sinks);
    if (rc == PA_OK)
        rc = prepare_prefill("pa_prefill_window", dims, q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, block_tables,
                             scale, out, meta, tiles, &a, &nothing);
    if (rc != PA_OK || nothing)
        return rc;
    a.window = window;
    a.sinks = sinks;
    return launch_prefill(a, stream);
}

extern "C" int pa_prefill_window_int8(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                                      const void *k_scale, const void *v_scale, const int32_t *cu_seqlens_q,
                                      const int32_t *cu_seqlens_k, const int32_t *block_tables,
                                      const int32_t *scratch_tables, const int32_t *scratch_items, int32_t window,
                                      int32_t sinks, float scale, void *out, const pa_prefill_meta *meta,
                                      const int32_t *tiles, void *workspace, size_t workspace_bytes,
                                      pa_stream_t stream)
{
    if (int rc = check_window("pa_prefill_window_int8", meta, &window, &sinks))
        return rc;
    return prefill_int8("pa_prefill_window_int8", false, dims, q, nullptr, nullptr, k_cache, v_cache, k_scale, v_scale,
                        cu_seqlens_q, cu_seqlens_k, block_tables, nullptr, scratch_tables, scratch_items, scale, out,
                        meta, tiles, workspace, workspace_bytes, stream, window, sinks);
}

// Host-side checks shared by pa_decode and pa_decode_int8; fills `a`.  Sets
// *nothing when the plan has no work (then no launch happens).
static int prepare_decode(const char *fn, const pa_dims *dims, const void *q, const void *k_cache,
                          const void *v_cache, const int32_t *context_lens, const int32_t *block_tables, float scale,
                          void *out, const pa_decode_meta *meta, const int32_t *items, const int32_t *seq_items,
                          void *workspace, size_t workspace_bytes, DecodeArgs *a, bool *nothing)
{
    *nothing = false;
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (!meta)
        return fail(PA_ERR_INVALID_ARG, "meta is NULL");
    if (meta->num_items < 0 || meta->num_seqs < 0 || meta->max_blocks_per_seq < 1 || meta->max_splits < 1)
        return fail(PA_ERR_INVALID_ARG, "malformed decode meta");
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(PA_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (meta->num_items == 0) {
        *nothing = true;
        return PA_OK;
    }
    if (!q || !k_cache || !v_cache || !context_lens || !block_tables || !out || !items || !seq_items)
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(out))
        return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
    if (workspace_bytes < meta->workspace_bytes)
        return fail(PA_ERR_WORKSPACE, "decode workspace has %zu bytes, needs %llu", workspace_bytes,
                    (unsigned long long)meta->workspace_bytes);
    if (meta->workspace_bytes > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return fail(PA_ERR_INVALID_ARG, "decode workspace must be non-NULL and 256-byte aligned");
    *a = DecodeArgs{};
    a->dims = *dims;
    a->q = q;
    a->k_cache = k_cache;
    a->v_cache = v_cache;
    a->context_lens = context_lens;
    a->block_tables = block_tables;
    a->items = items;
    a->seq_items = seq_items;
    a->out = out;
    if (meta->num_partials < 0)
        return fail(PA_ERR_INVALID_ARG, "malformed decode meta");
    if (meta->num_partials > 0) {
        size_t per = (size_t)dims->num_heads * dims->head_dim * 4;
        size_t need = align_up((size_t)meta->num_partials * per, 256) +
                      align_up((size_t)meta->num_partials * dims->num_heads * 4, 256);
        if (need > meta->workspace_bytes)
            return fail(PA_ERR_INVALID_ARG, "decode meta workspace size inconsistent with its partial count");
        a->part_o = static_cast<float *>(workspace);
        a->part_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                                align_up((size_t)meta->num_partials * per, 256));
    }
    a->scale = scale;
    a->num_seqs = meta->num_seqs;
    a->num_items = meta->num_items;
    a->max_blocks_per_seq = meta->max_blocks_per_seq;
    a->max_splits = meta->max_splits;
    return PA_OK;
}

extern "C" int pa_decode(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                         const int32_t *context_lens, const int32_t *block_tables, float scale, void *out,
                         const pa_decode_meta *meta, const int32_t *items, const int32_t *seq_items, void *workspace,
                         size_t workspace_bytes, pa_stream_t stream)
{
    DecodeArgs a;
    bool nothing = false;
    int rc = prepare_decode("pa_decode", dims, q, k_cache, v_cache, context_lens, block_tables, scale, out, meta,
                            items, seq_items, workspace, workspace_bytes, &a, &nothing);
    if (rc != PA_OK || nothing)
        return rc;
    return launch_decode(a, stream);
}

extern "C" int pa_decode_fused(const pa_dims *dims, const void *q, const void *k, const void *v, void *k_cache,
                               void *v_cache, const int32_t *slot_mapping, const int32_t *context_lens,
                               const int32_t *block_tables, float scale, void *out, const pa_decode_meta *meta,
                               const int32_t *items, const int32_t *seq_items, void *workspace,
                               size_t workspace_bytes, pa_stream_t stream)
{
    DecodeArgs a;
    bool nothing = false;
    int rc = prepare_decode("pa_decode_fused", dims, q, k_cache, v_cache, context_lens, block_tables, scale, out,
                            meta, items, seq_items, workspace, workspace_bytes, &a, &nothing);
    if (rc != PA_OK || nothing)
        return rc;
    if (!k || !v || !slot_mapping)
        return fail(PA_ERR_INVALID_ARG, "pa_decode_fused: NULL pointer");
    if (misaligned(k) || misaligned(v))
        return fail(PA_ERR_INVALID_ARG, "pa_decode_fused: tensors must be 16-byte aligned");
    a.k_new = k;
    a.v_new = v;
    a.slot_mapping = slot_mapping;
    return launch_decode(a, stream);
}

extern "C" int pa_decode_int8_fused(const pa_dims *dims, const void *q, const void *k, const void *v,
                                    void *k_cache, void *v_cache, void *k_scale, void *v_scale,
                                    const int32_t *slot_mapping, const int32_t *context_lens,
                                    const int32_t *block_tables, float scale, void *out, const pa_decode_meta *meta,
                                    const int32_t *items, const int32_t *seq_items, void *workspace,
                                    size_t workspace_bytes, pa_stream_t stream)
{
    DecodeArgs a;
    bool nothing = false;
    int rc = prepare_decode("pa_decode_int8_fused", dims, q, k_cache, v_cache, context_lens, block_tables, scale,
                            out, meta, items, seq_items, workspace, workspace_bytes, &a, &nothing);
    if (rc != PA_OK || nothing)
        return rc;
    if (!k || !v || !slot_mapping || !k_scale || !v_scale)
        return fail(PA_ERR_INVALID_ARG, "pa_decode_int8_fused: NULL pointer");
    if (misaligned(k) || misaligned(v) || misaligned(k_scale) || misaligned(v_scale))
        return fail(PA_ERR_INVALID_ARG, "pa_decode_int8_fused: tensors must be 16-byte aligned");
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.k_new = k;
    a.v_new = v;
    a.slot_mapping = slot_mapping;
    return launch_decode_int8(a, stream);
}

extern "C" int pa_store_kvcache_int8(const pa_dims *dims, const void *k, const void *v, void *k_cache,
                                     void *v_cache, void *k_scale, void *v_scale, const int32_t *slot_mapping,
                                     int32_t num_tokens, pa_stream_t stream)
{
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (num_tokens < 0)
        return fail(PA_ERR_INVALID_ARG, "num_tokens < 0");
    if (num_tokens == 0)
        return PA_OK;
    if (!k || !v || !k_cache || !v_cache || !k_scale || !v_scale || !slot_mapping)
        return fail(PA_ERR_INVALID_ARG, "pa_store_kvcache_int8: NULL pointer");
    if (misaligned(k) || misaligned(v) || misaligned(k_cache) || misaligned(v_cache) || misaligned(k_scale) ||
        misaligned(v_scale))
        return fail(PA_ERR_INVALID_ARG, "pa_store_kvcache_int8: tensors must be 16-byte aligned");
    return launch_store_kvcache_int8(*dims, k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, num_tokens,
                                     stream);
}

extern "C" int pa_decode_int8(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                              const void *k_scale, const void *v_scale, const int32_t *context_lens,
                              const int32_t *block_tables, float scale, void *out, const pa_decode_meta *meta,
                              const int32_t *items, const int32_t *seq_items, void *workspace,
                              size_t workspace_bytes, pa_stream_t stream)
{
    DecodeArgs a;
    bool nothing = false;
    int rc = prepare_decode("pa_decode_int8", dims, q, k_cache, v_cache, context_lens, block_tables, scale, out,
                            meta, items, seq_items, workspace, workspace_bytes, &a, &nothing);
    if (rc != PA_OK || nothing)
        return rc;
    if (!k_scale || !v_scale)
        return fail(PA_ERR_INVALID_ARG, "pa_decode_int8: NULL scale pointer");
    if (misaligned(k_scale) || misaligned(v_scale))
        return fail(PA_ERR_INVALID_ARG, "pa_decode_int8: scales must be 16-byte aligned");
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    return launch_decode_int8(a, stream);
}

// Host-side checks of a shared-prefix decode; fills `a`.  Sets *nothing when there is no work.
static int prepare_shared(const char *fn, bool int8, const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                          const int32_t *block_tables, float scale, void *out, const pa_shared_meta *meta,
                          const int32_t *items, const int32_t *cta_items, const int32_t *seq_parts,
                          const int32_t *direct_items, const int32_t *table_rows, const int32_t *single_items,
                          void *workspace, size_t workspace_bytes, SharedArgs *a, bool *nothing)
{
    *nothing = false;
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (!meta)
        return fail(PA_ERR_INVALID_ARG, "meta is NULL");
    if (meta->num_seqs < 0 || meta->num_items < 0 || meta->num_ctas < 0 || meta->num_ctas > meta->num_items ||
        (meta->num_items > 0 && meta->num_ctas < 1) || meta->num_partials < 0 || meta->max_blocks_per_seq < 1)
        return fail(PA_ERR_INVALID_ARG, "malformed shared decode meta");
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(PA_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (meta->num_seqs == 0) {
        *nothing = true;
        return PA_OK;
    }
    const int group = dims->num_heads / dims->num_kv_heads;
    if (meta->num_heads != dims->num_heads || meta->num_kv_heads != dims->num_kv_heads ||
        meta->head_dim != dims->head_dim || meta->block_size != dims->block_size ||
        meta->rows_per_tile != (kPrefillRows / group > 0 ? kPrefillRows / group : 1))
        return fail(PA_ERR_INVALID_ARG, "%s: meta was packed for other dims", fn);
    if (!q || !k_cache || !v_cache || !block_tables || !out || !items || !cta_items || !seq_parts ||
        !direct_items || !table_rows || !single_items)
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(out) || misaligned(items) ||
        misaligned(direct_items) || misaligned(single_items))
        return fail(PA_ERR_INVALID_ARG, "%s: tensors and items must be 16-byte aligned", fn);
    if ((reinterpret_cast<uintptr_t>(seq_parts) & 7u) || misaligned(cta_items) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(table_rows) & 3u))
        return fail(PA_ERR_INVALID_ARG, "%s: misaligned plan array or block table", fn);
    if (meta->num_items > 0 && dims->num_blocks == 0)
        return fail(PA_ERR_INVALID_ARG, "empty KV pool");
    if (meta->num_scratch_tiles < 0 || meta->num_single_items < 0 || meta->num_shared_items < 0 ||
        meta->num_shared_items > meta->num_items)
        return fail(PA_ERR_INVALID_ARG, "malformed shared decode meta");
    const bool direct = (meta->direct & (int8 ? 2 : 1)) != 0;
    const size_t word_at = shared_part_bytes(*dims, meta->num_partials);
    const size_t part_bytes = word_at + shared_go_bytes(*meta);
    const uint64_t need = direct ? 0
                          : int8 ? part_bytes + shared_scratch_bytes(*dims, meta->num_scratch_tiles, meta->num_seqs)
                                 : part_bytes;
    if (need != (int8 ? meta->workspace_bytes_int8 : meta->workspace_bytes))
        return fail(PA_ERR_INVALID_ARG, "%s: meta was packed for other dims", fn);
    if (workspace_bytes < need)
        return fail(PA_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %llu", fn, workspace_bytes,
                    (unsigned long long)need);
    if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return fail(PA_ERR_INVALID_ARG, "%s: workspace must be non-NULL and 256-byte aligned", fn);
    *a = SharedArgs{};
    a->dims = *dims;
    a->q = q;
    a->k_cache = k_cache;
    a->v_cache = v_cache;
    a->block_tables = block_tables;
    a->items = items;
    a->cta_items = cta_items;
    a->seq_parts = seq_parts;
    a->table_rows = table_rows;
    a->direct_items = direct ? direct_items : nullptr;
    a->out = out;
    if (need > 0) {
        a->part_o = static_cast<float *>(workspace);
        a->part_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                                shared_part_o_bytes(*dims, meta->num_partials));
        if (shared_beside(*meta))
            a->go_word = reinterpret_cast<uint64_t *>(static_cast<char *>(workspace) + word_at);
        a->scratch = static_cast<char *>(workspace) + part_bytes;
    }
    a->num_scratch_tiles = meta->num_scratch_tiles;
    a->scale = scale;
    a->num_seqs = meta->num_seqs;
    // parts of single sequences: in the CTAs' lists, or apart in the decode kernels
    a->single_items = single_items;
    a->num_items = meta->num_items;
    a->num_single_items = meta->apart ? meta->num_single_items : 0;
    a->num_ctas = meta->num_ctas;
    a->rows_per_tile = meta->rows_per_tile;
    a->max_blocks_per_seq = meta->max_blocks_per_seq;
    a->max_parts = meta->max_parts;
    a->merge = meta->merge != 0;
    return PA_OK;
}

extern "C" int pa_decode_shared(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                                const int32_t *block_tables, float scale, void *out, const pa_shared_meta *meta,
                                const int32_t *items, const int32_t *cta_items, const int32_t *seq_parts,
                                const int32_t *direct_items, const int32_t *table_rows, const int32_t *single_items,
                                void *workspace, size_t workspace_bytes, pa_stream_t stream)
{
    SharedArgs a;
    bool nothing = false;
    int rc = prepare_shared("pa_decode_shared", false, dims, q, k_cache, v_cache, block_tables, scale, out, meta, items,
                            cta_items, seq_parts, direct_items, table_rows, single_items, workspace, workspace_bytes, &a,
                            &nothing);
    if (rc != PA_OK || nothing)
        return rc;
    return launch_decode_shared(a, stream);
}

extern "C" int pa_decode_shared_int8(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                                     const void *k_scale, const void *v_scale, const int32_t *block_tables, float scale,
                                     void *out, const pa_shared_meta *meta, const int32_t *items,
                                     const int32_t *cta_items, const int32_t *seq_parts, const int32_t *direct_items,
                                     const int32_t *table_rows, const int32_t *single_items,
                                     const int32_t *scratch_tiles, void *workspace, size_t workspace_bytes,
                                     pa_stream_t stream)
{
    SharedArgs a;
    bool nothing = false;
    int rc = prepare_shared("pa_decode_shared_int8", true, dims, q, k_cache, v_cache, block_tables, scale, out, meta, items,
                            cta_items, seq_parts, direct_items, table_rows, single_items, workspace, workspace_bytes, &a,
                            &nothing);
    if (rc != PA_OK || nothing)
        return rc;
    if (!k_scale || !v_scale || !scratch_tiles)
        return fail(PA_ERR_INVALID_ARG, "pa_decode_shared_int8: NULL pointer");
    if (misaligned(k_scale) || misaligned(v_scale) || misaligned(scratch_tiles))
        return fail(PA_ERR_INVALID_ARG, "pa_decode_shared_int8: scales and items must be 16-byte aligned");
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.scratch_tiles = scratch_tiles;
    return launch_decode_shared(a, stream);
}

extern "C" int pa_copy_blocks(const pa_dims *dims, void *k_cache, void *v_cache, const int32_t *triples,
                              int32_t num_triples, pa_stream_t stream)
{
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (num_triples < 0)
        return fail(PA_ERR_INVALID_ARG, "num_triples < 0");
    if (num_triples == 0)
        return PA_OK;
    if (!k_cache || !v_cache || !triples)
        return fail(PA_ERR_INVALID_ARG, "pa_copy_blocks: NULL pointer");
    if (misaligned(k_cache) || misaligned(v_cache) || (reinterpret_cast<uintptr_t>(triples) & 3u))
        return fail(PA_ERR_INVALID_ARG, "pa_copy_blocks: misaligned pointer");
    return launch_copy_blocks(*dims, k_cache, v_cache, triples, num_triples, stream);
}

extern "C" int pa_copy_blocks_int8(const pa_dims *dims, void *k_cache, void *v_cache, void *k_scale, void *v_scale,
                                   const int32_t *triples, int32_t num_triples, pa_stream_t stream)
{
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (num_triples < 0)
        return fail(PA_ERR_INVALID_ARG, "num_triples < 0");
    if (num_triples == 0)
        return PA_OK;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !triples)
        return fail(PA_ERR_INVALID_ARG, "pa_copy_blocks_int8: NULL pointer");
    if (misaligned(k_cache) || misaligned(v_cache) || misaligned(k_scale) || misaligned(v_scale) ||
        (reinterpret_cast<uintptr_t>(triples) & 3u))
        return fail(PA_ERR_INVALID_ARG, "pa_copy_blocks_int8: misaligned pointer");
    return launch_copy_blocks(*dims, k_cache, v_cache, triples, num_triples, stream, k_scale, v_scale);
}

// Host-side checks of the pa_pool calls; fills `a`.
static int prepare_pool(const char *fn, const pa_dims *dims, const pa_pool *pool, const void *workspace,
                        size_t workspace_bytes, bool needs_workspace, bool needs_pages, PoolArgs *a)
{
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (!pool)
        return fail(PA_ERR_INVALID_ARG, "%s: pool is NULL", fn);
    const pa_pool &o = *pool;
    if (o.num_rows < 1 || o.max_blocks < 1 || o.num_layers < 1)
        return fail(PA_ERR_INVALID_ARG, "%s: num_rows, max_blocks and num_layers must be positive", fn);
    if ((int64_t)o.num_rows * o.max_blocks > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "%s: num_rows * max_blocks exceeds int32", fn);
    if (dims->num_blocks == 0)
        return fail(PA_ERR_INVALID_ARG, "empty KV pool");
    if (!o.block_tables || !o.context_lens || !o.ref_counts)
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pool array", fn);
    auto unaligned = [](const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
    if (unaligned(o.block_tables, 4) || unaligned(o.context_lens, 4) || unaligned(o.ref_counts, 16))
        return fail(PA_ERR_INVALID_ARG, "%s: misaligned pool array (ref_counts: 16 bytes)", fn);
    if (needs_pages) {
        if (!o.k_cache || !o.v_cache || !o.k_scale != !o.v_scale)
            return fail(PA_ERR_INVALID_ARG, "%s: k_cache and v_cache, and both scales or neither, must be given", fn);
        const uint64_t scales = (uint64_t)dims->num_blocks * dims->block_size * dims->num_kv_heads * 2;
        const uint64_t layer = scales / 2 * dims->head_dim * (o.k_scale ? 1 : 2);
        if (misaligned(o.k_cache) || misaligned(o.v_cache) || misaligned(o.k_scale) || misaligned(o.v_scale))
            return fail(PA_ERR_INVALID_ARG, "%s: caches and scales must be 16-byte aligned", fn);
        if (o.num_layers > 1 && (o.layer_stride % 16 != 0 || o.layer_stride < layer))
            return fail(PA_ERR_INVALID_ARG, "%s: layer_stride must be a multiple of 16 of at least a layer's %llu bytes",
                        fn, (unsigned long long)layer);
        if (o.num_layers > 1 && o.k_scale && (o.scale_layer_stride % 2 != 0 || o.scale_layer_stride < scales))
            return fail(PA_ERR_INVALID_ARG, "%s: scale_layer_stride must be even and at least a layer's %llu bytes", fn,
                        (unsigned long long)scales);
    }
    if (needs_workspace) {
        const size_t need = pool_workspace_bytes(o.num_rows, dims->num_blocks);
        if (workspace_bytes < need)
            return fail(PA_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn, workspace_bytes, need);
        if (!workspace || unaligned(workspace, 256))
            return fail(PA_ERR_INVALID_ARG, "%s: workspace must be non-NULL and 256-byte aligned", fn);
    }
    a->dims = *dims;
    a->pool = o;
    a->workspace = const_cast<void *>(workspace);
    return PA_OK;
}

extern "C" int pa_pool_workspace(const pa_dims *dims, const pa_pool *pool, uint64_t *bytes)
{
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (!pool || !bytes || pool->num_rows < 1)
        return fail(PA_ERR_INVALID_ARG, "pa_pool_workspace: NULL pointer or num_rows < 1");
    *bytes = pool_workspace_bytes(pool->num_rows, dims->num_blocks);
    return PA_OK;
}

extern "C" int pa_pool_append(const pa_dims *dims, const pa_pool *pool, const int32_t *rows, const int32_t *cu_new,
                              int32_t n, int32_t *slot_mapping, int32_t num_tokens, void *workspace,
                              size_t workspace_bytes, pa_stream_t stream)
{
    PoolArgs a;
    int rc = prepare_pool("pa_pool_append", dims, pool, workspace, workspace_bytes, true, false, &a);
    if (rc != PA_OK)
        return rc;
    if (n < 0 || n > pool->num_rows || num_tokens < 0 || (n == 0 && num_tokens > 0))
        return fail(PA_ERR_INVALID_ARG, "pa_pool_append: %d rows, %d tokens (the pool has %d rows)", n, num_tokens,
                    pool->num_rows);
    if (n == 0)
        return PA_OK;
    if (!rows || !cu_new || (!slot_mapping && num_tokens > 0))
        return fail(PA_ERR_INVALID_ARG, "pa_pool_append: NULL pointer");
    return launch_pool_append(a, rows, cu_new, n, slot_mapping, num_tokens, stream);
}

extern "C" int pa_pool_fork(const pa_dims *dims, const pa_pool *pool, const int32_t *parents, const int32_t *children,
                            int32_t n, void *workspace, size_t workspace_bytes, pa_stream_t stream)
{
    PoolArgs a;
    int rc = prepare_pool("pa_pool_fork", dims, pool, workspace, workspace_bytes, true, true, &a);
    if (rc != PA_OK)
        return rc;
    if (n < 0 || n > pool->num_rows)
        return fail(PA_ERR_INVALID_ARG, "pa_pool_fork: %d children (the pool has %d rows)", n, pool->num_rows);
    if (n == 0)
        return PA_OK;
    if (!parents || !children)
        return fail(PA_ERR_INVALID_ARG, "pa_pool_fork: NULL pointer");
    return launch_pool_fork(a, parents, children, n, stream);
}

extern "C" int pa_pool_free(const pa_dims *dims, const pa_pool *pool, const int32_t *rows, int32_t n,
                            pa_stream_t stream)
{
    PoolArgs a;
    int rc = prepare_pool("pa_pool_free", dims, pool, nullptr, 0, false, false, &a);
    if (rc != PA_OK)
        return rc;
    if (n < 0)
        return fail(PA_ERR_INVALID_ARG, "pa_pool_free: n < 0");
    if (n == 0)
        return PA_OK;
    if (!rows)
        return fail(PA_ERR_INVALID_ARG, "pa_pool_free: NULL pointer");
    return launch_pool_free(a, rows, n, stream);
}

extern "C" int pa_pool_compact(const pa_dims *dims, const pa_pool *pool, int32_t *remap, int32_t *block_tables_out,
                               int32_t *ref_counts_out, void *workspace, size_t workspace_bytes, pa_stream_t stream)
{
    PoolArgs a;
    int rc = prepare_pool("pa_pool_compact", dims, pool, workspace, workspace_bytes, true, true, &a);
    if (rc != PA_OK)
        return rc;
    if (!remap || !block_tables_out || !ref_counts_out)
        return fail(PA_ERR_INVALID_ARG, "pa_pool_compact: NULL pointer");
    if (remap == pool->ref_counts || remap == ref_counts_out || remap == pool->block_tables || remap == block_tables_out)
        return fail(PA_ERR_INVALID_ARG, "pa_pool_compact: remap must be an array of its own");
    return launch_pool_compact(a, remap, block_tables_out, ref_counts_out, stream);
}

extern "C" int pa_pool_evict(const pa_dims *dims, const pa_pool *pool, const int32_t *rows, int32_t n,
                             const float *scores, float *scores_out, int32_t budget, int32_t first, int32_t last,
                             int32_t *kept, void *workspace, size_t workspace_bytes, pa_stream_t stream)
{
    PoolArgs a;
    int rc = prepare_pool("pa_pool_evict", dims, pool, workspace, workspace_bytes, true, true, &a);
    if (rc != PA_OK)
        return rc;
    if (n < 0 || n > pool->num_rows)
        return fail(PA_ERR_INVALID_ARG, "pa_pool_evict: %d rows (the pool has %d)", n, pool->num_rows);
    if (budget < 1 || first < 0 || last < 0 || (int64_t)first + last > budget)
        return fail(PA_ERR_INVALID_ARG, "pa_pool_evict: budget %d must be positive and hold the first %d and last %d tokens",
                    budget, first, last);
    // (the choice counts past a row's end, and past the budget's)
    if ((int64_t)pool->max_blocks * dims->block_size > INT32_MAX - 4096 || budget > INT32_MAX - 4096)
        return fail(PA_ERR_UNSUPPORTED, "pa_pool_evict: max_blocks * block_size or the budget exceeds int32");
    if (n == 0)
        return PA_OK;
    if (!rows || !scores || !scores_out || !kept)
        return fail(PA_ERR_INVALID_ARG, "pa_pool_evict: NULL pointer");
    return launch_pool_evict(a, rows, n, scores, scores_out, budget, first, last, kept, stream);
}

// Host-side checks of the decodes over a bounded cache, then the launch.
static int decode_bounded(const char *fn, const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                          bool int8, const void *k_scale, const void *v_scale, const int32_t *context_lens,
                          const int32_t *block_tables, const int32_t *table_rows, int32_t num_seqs, int32_t num_rows,
                          int32_t max_blocks, int32_t window, int32_t sinks, float scale, void *out, bool weights,
                          float decay, const float *scores, float *scores_out, void *workspace, size_t workspace_bytes,
                          pa_stream_t stream)
{
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(PA_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (window < 1 || sinks < 0)
        return fail(PA_ERR_INVALID_ARG, "%s: window must be at least 1, sinks at least 0", fn);
    if (num_seqs < 0 || num_rows < 1 || max_blocks < 1 || (!table_rows && num_seqs > num_rows))
        return fail(PA_ERR_INVALID_ARG, "%s: %d sequences, %d rows of %d blocks", fn, num_seqs, num_rows, max_blocks);
    if ((int64_t)max_blocks * dims->block_size > INT32_MAX - 16)
        return fail(PA_ERR_UNSUPPORTED, "%s: max_blocks_per_seq * block_size exceeds int32", fn);
    if ((int64_t)num_seqs * dims->num_kv_heads > INT32_MAX / 8)
        return fail(PA_ERR_UNSUPPORTED, "%s: num_seqs * num_kv_heads exceeds the grid", fn);
    if (weights && !(decay >= 0.f && decay <= 1.f))
        return fail(PA_ERR_INVALID_ARG, "%s: decay must be in [0, 1]", fn);
    if (num_seqs == 0)
        return PA_OK;
    if (!q || !k_cache || !v_cache || !context_lens || !block_tables || !out || (int8 && (!k_scale || !v_scale)) ||
        (weights && (!scores || !scores_out)))
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(k_scale) || misaligned(v_scale) ||
        misaligned(out) || misaligned(scores) || misaligned(scores_out))
        return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
    if (dims->num_blocks == 0)
        return fail(PA_ERR_INVALID_ARG, "empty KV pool");
    if (weights) {
        uint64_t need = 0;
        if ((rc = pa_decode_weights_workspace(dims, num_seqs, max_blocks, &need)) != PA_OK)
            return rc;
        if (workspace_bytes < need)
            return fail(PA_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %llu", fn, workspace_bytes,
                        (unsigned long long)need);
        if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
            return fail(PA_ERR_INVALID_ARG, "%s: workspace must be non-NULL and 256-byte aligned", fn);
    }
    return launch_decode_window({*dims, q, k_cache, v_cache, k_scale, v_scale, context_lens, block_tables, table_rows,
                                 num_seqs, num_rows, max_blocks, window, sinks, scale, out,
                                 weights ? static_cast<float *>(workspace) : nullptr, decay, scores, scores_out},
                                stream);
}

extern "C" int pa_decode_window(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                                const int32_t *context_lens, const int32_t *block_tables, const int32_t *table_rows,
                                int32_t num_seqs, int32_t num_rows, int32_t max_blocks_per_seq, int32_t window,
                                int32_t sinks, float scale, void *out, pa_stream_t stream)
{
    return decode_bounded("pa_decode_window", dims, q, k_cache, v_cache, false, nullptr, nullptr, context_lens,
                          block_tables, table_rows, num_seqs, num_rows, max_blocks_per_seq, window, sinks, scale, out,
                          false, 0.f, nullptr, nullptr, nullptr, 0, stream);
}

extern "C" int pa_decode_window_int8(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                                     const void *k_scale, const void *v_scale, const int32_t *context_lens,
                                     const int32_t *block_tables, const int32_t *table_rows, int32_t num_seqs,
                                     int32_t num_rows, int32_t max_blocks_per_seq, int32_t window, int32_t sinks,
                                     float scale, void *out, pa_stream_t stream)
{
    return decode_bounded("pa_decode_window_int8", dims, q, k_cache, v_cache, true, k_scale, v_scale, context_lens,
                          block_tables, table_rows, num_seqs, num_rows, max_blocks_per_seq, window, sinks, scale, out,
                          false, 0.f, nullptr, nullptr, nullptr, 0, stream);
}

extern "C" int pa_decode_weights_workspace(const pa_dims *dims, int32_t num_seqs, int32_t max_blocks_per_seq,
                                           uint64_t *bytes)
{
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (!bytes || num_seqs < 0 || max_blocks_per_seq < 1)
        return fail(PA_ERR_INVALID_ARG, "pa_decode_weights_workspace: NULL pointer, num_seqs < 0 or no blocks");
    const uint64_t units = (uint64_t)num_seqs * dims->num_kv_heads, room = (uint64_t)max_blocks_per_seq * dims->block_size;
    const uint64_t key = (uint64_t)window_raw_heads(*dims) * 4;
    if (units > INT32_MAX / 8 || room > INT32_MAX - 16 || units * room > UINT64_MAX / key) // (the decode's limits)
        return fail(PA_ERR_UNSUPPORTED, "pa_decode_weights_workspace: %d sequences of %d blocks are too many", num_seqs,
                    max_blocks_per_seq);
    *bytes = units * room * key;
    return PA_OK;
}

extern "C" int pa_decode_weights(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                                 const int32_t *context_lens, const int32_t *block_tables, const int32_t *table_rows,
                                 int32_t num_seqs, int32_t num_rows, int32_t max_blocks_per_seq, float scale,
                                 float decay, const float *scores, float *scores_out, void *out, void *workspace,
                                 size_t workspace_bytes, pa_stream_t stream)
{
    return decode_bounded("pa_decode_weights", dims, q, k_cache, v_cache, false, nullptr, nullptr, context_lens,
                          block_tables, table_rows, num_seqs, num_rows, max_blocks_per_seq, INT32_MAX, 0, scale, out,
                          true, decay, scores, scores_out, workspace, workspace_bytes, stream);
}

extern "C" int pa_decode_weights_int8(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                                      const void *k_scale, const void *v_scale, const int32_t *context_lens,
                                      const int32_t *block_tables, const int32_t *table_rows, int32_t num_seqs,
                                      int32_t num_rows, int32_t max_blocks_per_seq, float scale, float decay,
                                      const float *scores, float *scores_out, void *out, void *workspace,
                                      size_t workspace_bytes, pa_stream_t stream)
{
    return decode_bounded("pa_decode_weights_int8", dims, q, k_cache, v_cache, true, k_scale, v_scale, context_lens,
                          block_tables, table_rows, num_seqs, num_rows, max_blocks_per_seq, INT32_MAX, 0, scale, out,
                          true, decay, scores, scores_out, workspace, workspace_bytes, stream);
}

// pa_decode for callers that cannot allocate: the workspace is the library's
// own scratch array (see the header for its limit, set-up and sharing rules).
extern "C" int pa_decode_static(const pa_dims *dims, const void *q, const void *k_cache, const void *v_cache,
                                const int32_t *context_lens, const int32_t *block_tables, float scale, void *out,
                                const pa_decode_meta *meta, const int32_t *items, const int32_t *seq_items,
                                pa_stream_t stream)
{
    if (!meta)
        return fail(PA_ERR_INVALID_ARG, "meta is NULL");
    if (meta->workspace_bytes > PA_DECODE_STATIC_SCRATCH_BYTES)
        return fail(PA_ERR_WORKSPACE,
                    "pa_decode_static: plan needs %llu bytes of scratch, the library array holds %u; "
                    "use pa_decode with a workspace or pack with larger splits",
                    (unsigned long long)meta->workspace_bytes, PA_DECODE_STATIC_SCRATCH_BYTES);
    void *scratch = nullptr;
    int rc = decode_static_scratch(&scratch);
    if (rc != PA_OK)
        return rc;
    DecodeArgs a;
    bool nothing = false;
    rc = prepare_decode("pa_decode_static", dims, q, k_cache, v_cache, context_lens, block_tables, scale, out, meta,
                        items, seq_items, scratch, PA_DECODE_STATIC_SCRATCH_BYTES, &a, &nothing);
    if (rc != PA_OK || nothing)
        return rc;
    return launch_decode(a, stream);
}

extern "C" int pa_read_device_error(uint32_t *code, pa_stream_t stream)
{
    if (!code)
        return fail(PA_ERR_INVALID_ARG, "code is NULL");
    cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail(PA_ERR_CUDA, "cudaStreamSynchronize: %s", cudaGetErrorString(e));
    *code = 0;
    int rc = read_store_error(code);
    if (rc == PA_OK)
        rc = read_prefill_error(code);
    if (rc == PA_OK)
        rc = read_copy_error(code);
    if (rc == PA_OK)
        rc = read_decode_error(code);
    if (rc == PA_OK)
        rc = read_fused_error(code);
    if (rc == PA_OK)
        rc = read_fused8_error(code);
    if (rc == PA_OK)
        rc = read_selftest_error(code);
    if (rc == PA_OK)
        rc = read_shared_error(code);
    if (rc == PA_OK)
        rc = read_pool_error(code);
    if (rc == PA_OK)
        rc = read_rope_error(code);
    if (rc == PA_OK)
        rc = read_window_error(code);
    if (rc == PA_OK)
        rc = read_evict_error(code);
    return rc;
}

extern "C" int pa_stream_read(const void *src, size_t bytes, uint32_t *sink, pa_stream_t stream)
{
    if (bytes && !src)
        return fail(PA_ERR_INVALID_ARG, "pa_stream_read: src is NULL");
    if (!sink)
        return fail(PA_ERR_INVALID_ARG, "pa_stream_read: sink is NULL");
    if ((reinterpret_cast<uintptr_t>(src) & 15u) || (bytes & 15u) || (reinterpret_cast<uintptr_t>(sink) & 3u))
        return fail(PA_ERR_INVALID_ARG, "pa_stream_read: src and bytes must be 16-byte aligned, sink 4-byte aligned");
    return launch_stream_read(src, bytes, sink, stream);
}

extern "C" int pa_selftest_bounded_wait(uint32_t timeout_us, int arrive_first, pa_stream_t stream)
{
    if (timeout_us < 1 || timeout_us > 10000000u)
        return fail(PA_ERR_INVALID_ARG, "timeout_us (%u) must be in [1, 10000000]", timeout_us);
    return launch_selftest_wait(timeout_us, arrive_first ? 1 : 0, stream);
}

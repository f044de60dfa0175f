// Norm and rotation of the queries' and keys' heads, and the store of the new keys and values into the
// paged cache, in one pass.
//
// Formulas: for each head row x of D values, y = x * rsqrt(mean(x^2) + eps) * w (if there is a norm), then
// the pairs of the first R values are turned by the angle of the token's position on the pair's axis:
//   (a, b) -> (a cos - b sin, b cos + a sin),  pair i = (i, i + R/2) or (2i, 2i + 1).
// Everything in fp32 from the bf16 inputs; one rounding, to bf16 (or, in an INT8 cache, to the code: the
// quantiser of quant.cuh on the fp32 row, so a key is not rounded to bf16 in between).
//
// Sources (page title, section): "手搓 vLLM 推理引擎" (LLM-101-CN nano-vllm walkthrough), Step 4
// (Attention.forward stores the new K/V before it attends), Step 5 (positions and slots of the new
// tokens); "面试问答准备: nano-vLLM 推理引擎优化", Q3 (the INT8 quantiser).
//
// Work: D / 16 adjacent lanes per head row, 16 values each: lane j has pairs 8j .. 8j + 7 whole, so a turn
// needs no shuffle, and a row's sum of squares (or its max|x|) log2(D / 16) of them.  A warp takes a few
// rows (the same heads, so that its lanes do not part) of 512 / D tokens, whose cos and sin it loads once.
// Bound: HBM for prompts (each row read and written once: 16384 tokens of 28 + 2 x 4 heads of 128 in 52.4 us, 5.8 TB/s),
// the loads' latency and the codes' instructions into an INT8 cache (5000 tokens of 16 + 2 x 8 heads 17.8 us of inputs that
// L2 holds, 21.5 of others, 3.4 TB/s), the latency of one launch for decode steps (8 tokens 1.8 us in a graph).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace pa {

__device__ uint32_t g_rope_error; // bit 0: a slot outside [-1, num_slots); bit 1: a position outside the table

namespace {

constexpr int kThreads = 128;

struct RopeParams {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride; // values between tokens
    const int32_t *positions;             // [axes][num_tokens]
    const int32_t *slots;
    __nv_bfloat16 *q_out;
    void *k_cache, *v_cache; // bf16, or int8 codes
    __half *k_scale, *v_scale;
    const float *cos_sin;
    const __nv_bfloat16 *q_weight, *k_weight; // NULL: no norm
    uint64_t axis_bits[2];                    // two bits per pair: its axis
    float eps;
    int32_t num_tokens, num_heads, num_kv_heads, block_size;
    int32_t num_axes, max_position, pairs; // pairs: R / 2
    int32_t heads_per_unit;                // a token's rows are cut into units of so many at most
    int32_t units, q_units, kv_units;
    int64_t num_slots;
};

__device__ __forceinline__ void unpack8(const uint4 &u, float *x)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float *x)
{
    return make_uint4(ptx::pack_bf16(x[0], x[1]), ptx::pack_bf16(x[2], x[3]), ptx::pack_bf16(x[4], x[5]),
                      ptx::pack_bf16(x[6], x[7]));
}

// The lane's two pieces of 8 values of a row: of a turned part its 8 pairs, of the rest 16 consecutive values.
struct Place {
    int c0, c1;
    bool turn;
};

template <int D>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *src, int h, const Place &at, uint4 (&x)[2])
{
    x[0] = ptx::ld_once_v4(src + h * D + at.c0);
    x[1] = ptx::ld_once_v4(src + h * D + at.c1);
}

// count rows from src on (a token's, D values apart; raw: the first kRows) to dst; every lane of the warp is here,
// `write` is its token's.  kKind: 0 queries, 1 keys, 2 values.  w: the norm's weight or NULL.
template <int D, bool kInt8, bool kNext, int kRows, int kKind>
__device__ __forceinline__ void turn_rows(const __nv_bfloat16 *src, uint4 (&raw)[kRows][2], int count, const Place &at, const float (&cs)[8],
                                          const float (&sn)[8], const __nv_bfloat16 *w, float eps, void *dst_rows,
                                          __half *scales, int scale_step, bool write)
{
    constexpr int kLanes = D / 16;
    constexpr bool kCodes = kInt8 && kKind != 0;
    uint4 wt[2];
    if (kKind != 2 && w) {
        wt[0] = *reinterpret_cast<const uint4 *>(w + at.c0);
        wt[1] = *reinterpret_cast<const uint4 *>(w + at.c1);
    }
    auto finish = [&](int h, const uint4(&in)[2]) {
        if constexpr (kKind == 2 && !kCodes) { // a value's row goes as it is
            if (write) {
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(dst_rows) + h * D;
                *reinterpret_cast<uint4 *>(dst + at.c0) = in[0];
                *reinterpret_cast<uint4 *>(dst + at.c1) = in[1];
            }
            return;
        }
        float x[16];
        unpack8(in[0], x);
        unpack8(in[1], x + 8);
        if (kKind != 2 && w) {
            uint64_t two[8], sum2[2] = {ptx::f2(0.f, 0.f), ptx::f2(0.f, 0.f)};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                two[i] = ptx::f2(x[2 * i], x[2 * i + 1]);
                sum2[i & 1] = ptx::f2_fma(two[i], two[i], sum2[i & 1]);
            }
            float s0, s1;
            ptx::f2_split(ptx::f2_add(sum2[0], sum2[1]), s0, s1);
            float sum = s0 + s1;
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float r = rsqrtf(sum * (1.f / D) + eps);
            float y[16];
            unpack8(wt[0], y);
            unpack8(wt[1], y + 8);
            const uint64_t r2 = ptx::f2(r, r);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ptx::f2_split(ptx::f2_mul(ptx::f2_mul(two[i], r2), ptx::f2(y[2 * i], y[2 * i + 1])), x[2 * i], x[2 * i + 1]);
        }
        if (kKind != 2 && at.turn) {
            if constexpr (kNext) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float a = x[2 * i], b = x[2 * i + 1];
                    x[2 * i] = a * cs[i] - b * sn[i];
                    x[2 * i + 1] = b * cs[i] + a * sn[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const uint64_t a = ptx::f2(x[i], x[i + 1]), b = ptx::f2(x[i + 8], x[i + 9]);
                    const uint64_t c2 = ptx::f2(cs[i], cs[i + 1]), s2 = ptx::f2(sn[i], sn[i + 1]);
                    const uint64_t minus = ptx::f2(-x[i + 8], -x[i + 9]);
                    ptx::f2_split(ptx::f2_fma(minus, s2, ptx::f2_mul(a, c2)), x[i], x[i + 1]);
                    ptx::f2_split(ptx::f2_fma(a, s2, ptx::f2_mul(b, c2)), x[i + 8], x[i + 9]);
                }
            }
        }
        if constexpr (!kCodes) {
            if (write) {
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(dst_rows) + h * D;
                *reinterpret_cast<uint4 *>(dst + at.c0) = pack8(x);
                *reinterpret_cast<uint4 *>(dst + at.c1) = pack8(x + 8);
            }
        } else {
            float a = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                a = fmaxf(a, fabsf(x[i]));
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1)
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            const float scale = fmaxf(__fdiv_rn(a, 127.0f), 1e-8f);
            uint32_t c[4];
            quant::codes_of_16(x, scale, __frcp_rn(scale), c);
            if (write) {
                int8_t *dst = static_cast<int8_t *>(dst_rows) + h * D;
                *reinterpret_cast<uint2 *>(dst + at.c0) = make_uint2(c[0], c[1]);
                *reinterpret_cast<uint2 *>(dst + at.c1) = make_uint2(c[2], c[3]);
                if ((threadIdx.x & (kLanes - 1)) == 0)
                    scales[h * scale_step] = __float2half_rn(scale);
            }
        }
    };
#pragma unroll 1
    for (int h = 0; h < count; ++h) {
        const uint4 now[2] = {raw[0][0], raw[0][1]};
#pragma unroll
        for (int u = 0; u + 1 < kRows; ++u) {
            raw[u][0] = raw[u + 1][0];
            raw[u][1] = raw[u + 1][1];
        }
        if (h + kRows < count)
            load_row<D>(src, h + kRows, at, raw[kRows - 1]);
        finish(h, now);
    }
}

// kNext: pairs (2i, 2i + 1).  kAxes: more than one position per token.  kRows: rows in flight.
template <int D, bool kInt8, bool kNext, bool kAxes, int kRows>
__global__ void __launch_bounds__(kThreads, kRows > 1 ? 5 : 6) rope_store_kernel(const RopeParams p)
{
    constexpr int kLanes = D / 16; // of a row
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x & 31, j = lane % kLanes;
    const uint32_t warp = blockIdx.x * (uint32_t)(kThreads / 32) + (threadIdx.x >> 5);
    const uint32_t tokens = warp / (uint32_t)p.units;
    int unit = (int)(warp - tokens * (uint32_t)p.units);
    // every lane stays to the end: the groups of a warp shuffle together
    const uint32_t token = tokens * (32 / kLanes) + lane / kLanes;
    const int t = (int)min(token, (uint32_t)p.num_tokens - 1u);
    bool live = token < (uint32_t)p.num_tokens;
    const bool first = live && j == 0 && unit == 0; // flags a token's errors
    // the unit's rows: heads h0 .. h0 + count - 1 of the queries, the keys or the values
    const int kind = unit < p.q_units ? 0 : unit < p.q_units + p.kv_units ? 1 : 2;
    unit -= kind == 0 ? 0 : kind == 1 ? p.q_units : p.q_units + p.kv_units;
    const int h0 = unit * p.heads_per_unit;
    const int count = min(p.heads_per_unit, (kind == 0 ? p.num_heads : p.num_kv_heads) - h0);

    const int half = p.pairs;
    Place at;
    at.turn = 8 * j < half;
    at.c0 = kNext || !at.turn ? 16 * j : 8 * j;
    at.c1 = kNext || !at.turn ? at.c0 + 8 : at.c0 + half;

    const int32_t slot = p.slots[t];
    int pos[4];
#pragma unroll
    for (int a = 0; a < (kAxes ? 4 : 1); ++a)
        pos[a] = a == 0 || a < p.num_axes ? p.positions[(int64_t)a * p.num_tokens + t] : 0;
    // the first rows are on their way before the position is known
    const __nv_bfloat16 *src = (kind == 0   ? p.q + (int64_t)t * p.q_stride
                                : kind == 1 ? p.k + (int64_t)t * p.k_stride
                                            : p.v + (int64_t)t * p.v_stride) +
                               h0 * D;
    uint4 raw[kRows][2];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
        if (u < count)
            load_row<D>(src, u, at, raw[u]);

    bool inside = true;
#pragma unroll
    for (int a = 0; a < (kAxes ? 4 : 1); ++a)
        inside = inside && (uint32_t)pos[a] < (uint32_t)p.max_position;
    if (!inside && first)
        atomicOr(&g_rope_error, 2u);
    live = live && inside;
    float cs[8], sn[8];
    if constexpr (!kAxes) {
        if (at.turn && inside && kind != 2) {
            const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + (int64_t)pos[0] * 2 * half + 8 * j);
            *reinterpret_cast<float4 *>(cs) = row[0], *reinterpret_cast<float4 *>(cs + 4) = row[1];
            *reinterpret_cast<float4 *>(sn) = row[half / 4], *reinterpret_cast<float4 *>(sn + 4) = row[half / 4 + 1];
        }
    } else {
        if (at.turn && inside && kind != 2) {
            // the rows of the axes that the lane's pairs turn on, 16 bytes at a time (one axis for most lanes)
            const uint32_t bits = (uint32_t)(p.axis_bits[j >> 2] >> (16 * (j & 3))) & 0xffffu;
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const uint32_t x = bits ^ (0x5555u * a);
                const uint32_t off = x | (x >> 1); // bit 2i is clear where pair i turns on axis a
                if ((~off & 0x5555u) == 0u)
                    continue;
                const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + (int64_t)pos[a] * 2 * half + 8 * j);
                float c8[8], s8[8];
                *reinterpret_cast<float4 *>(c8) = row[0], *reinterpret_cast<float4 *>(c8 + 4) = row[1];
                *reinterpret_cast<float4 *>(s8) = row[half / 4], *reinterpret_cast<float4 *>(s8 + 4) = row[half / 4 + 1];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool mine = ((off >> (2 * i)) & 1u) == 0u;
                    cs[i] = mine ? c8[i] : cs[i];
                    sn[i] = mine ? s8[i] : sn[i];
                }
            }
        }
    }
    const bool stored = slot >= 0 && slot < p.num_slots;
    if (!stored && slot != -1 && first && live)
        atomicOr(&g_rope_error, 1u);

    if (kind == 0) {
        turn_rows<D, kInt8, kNext, kRows, 0>(src, raw, count, at, cs, sn, p.q_weight, p.eps,
                                             p.q_out + ((int64_t)t * p.num_heads + h0) * D, nullptr, 0, live);
        return;
    }
    const int64_t to = ((int64_t)(stored ? slot : 0) * p.num_kv_heads + h0) * D * (kInt8 ? 1 : 2);
    const int64_t st = kInt8 && stored ? ((int64_t)(slot / p.block_size) * p.num_kv_heads + h0) * p.block_size +
                                             slot % p.block_size
                                       : 0;
    if (kind == 1)
        turn_rows<D, kInt8, kNext, kRows, 1>(src, raw, count, at, cs, sn, p.k_weight, p.eps,
                                             static_cast<char *>(p.k_cache) + to, p.k_scale + st, p.block_size,
                                             live && stored);
    else
        turn_rows<D, kInt8, kNext, kRows, 2>(src, raw, count, at, cs, sn, nullptr, p.eps,
                                             static_cast<char *>(p.v_cache) + to, p.v_scale + st, p.block_size,
                                             live && stored);
    // Only now: at the start the next launch's CTAs would take this one's places (16384 tokens and a prefill of them over a
    // window 228.5 us, 227.5 here).
    ptx::launch_dependents();
}

template <int D, bool kInt8, bool kNext, bool kAxes, int kRows>
int launch(const RopeParams &p0, int heads_per_unit, cudaStream_t stream)
{
    constexpr int kTokens = 512 / D; // of a warp
    RopeParams p = p0;
    p.heads_per_unit = heads_per_unit;
    p.q_units = (p.num_heads + heads_per_unit - 1) / heads_per_unit;
    p.kv_units = (p.num_kv_heads + heads_per_unit - 1) / heads_per_unit;
    p.units = p.q_units + 2 * p.kv_units;
    const int64_t warps = ((int64_t)p.num_tokens + kTokens - 1) / kTokens * p.units; // (fewer than heads: an int32)
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rope_store_kernel<D, kInt8, kNext, kAxes, kRows>, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(PA_ERR_CUDA, "rope store launch: %s", cudaGetErrorString(e));
    }
    return PA_OK;
}

template <int D, bool kInt8, bool kNext, bool kAxes>
int launch_heads(const RopeParams &p, cudaStream_t stream)
{
    // A prompt's tokens are many: four heads share their cos and sin.  bf16 is bound by the loads' latency and keeps all
    // four rows in flight (16384 tokens of 28 + 8 heads: 52.6 us, 59.8 with one), INT8 by instructions, and has more warps
    // with one (5000 tokens of 16 + 16, in L2: 17.8 us, 20.0 with four).  A decode step's rows each have a warp's lanes at
    // once (8 tokens of 16 + 16: 1.8 us, 2.3 with four heads a warp).
    const int64_t rows = (int64_t)p.num_tokens * (p.num_heads + 2 * p.num_kv_heads);
    return rows >= 65536 ? launch<D, kInt8, kNext, kAxes, kInt8 ? 1 : 4>(p, 4, stream)
                         : launch<D, kInt8, kNext, kAxes, 1>(p, 1, stream);
}

template <int D, bool kInt8>
int launch_kind(const RopeParams &p, bool next, cudaStream_t stream)
{
    const bool axes = p.num_axes > 1;
    if (next)
        return axes ? launch_heads<D, kInt8, true, true>(p, stream) : launch_heads<D, kInt8, true, false>(p, stream);
    return axes ? launch_heads<D, kInt8, false, true>(p, stream) : launch_heads<D, kInt8, false, false>(p, stream);
}

} // namespace

int launch_rope_store(const RopeArgs &a, void *stream)
{
    RopeParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.k = static_cast<const __nv_bfloat16 *>(a.k);
    p.v = static_cast<const __nv_bfloat16 *>(a.v);
    p.q_stride = a.q_stride, p.k_stride = a.k_stride, p.v_stride = a.v_stride;
    p.positions = a.positions;
    p.slots = a.slot_mapping;
    p.q_out = static_cast<__nv_bfloat16 *>(a.q_out);
    p.k_cache = a.k_cache, p.v_cache = a.v_cache;
    p.k_scale = static_cast<__half *>(a.k_scale), p.v_scale = static_cast<__half *>(a.v_scale);
    p.cos_sin = a.rope.cos_sin;
    p.q_weight = static_cast<const __nv_bfloat16 *>(a.rope.q_weight);
    p.k_weight = static_cast<const __nv_bfloat16 *>(a.rope.k_weight);
    p.eps = a.rope.eps;
    p.num_tokens = a.num_tokens;
    p.num_heads = a.dims.num_heads, p.num_kv_heads = a.dims.num_kv_heads, p.block_size = a.dims.block_size;
    p.num_axes = a.rope.num_axes, p.max_position = a.rope.max_position, p.pairs = a.rope.rotary_dim / 2;
    p.num_slots = (int64_t)a.dims.num_blocks * a.dims.block_size;
    for (int i = 0; i < p.pairs; ++i)
        p.axis_bits[i >> 5] |= (uint64_t)(a.rope.pair_axis[i] & 3) << (2 * (i & 31));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool next = a.rope.interleaved != 0;
    if (a.dims.head_dim == 128)
        return a.k_scale ? launch_kind<128, true>(p, next, s) : launch_kind<128, false>(p, next, s);
    return a.k_scale ? launch_kind<64, true>(p, next, s) : launch_kind<64, false>(p, next, s);
}

int read_rope_error(uint32_t *code)
{
    uint32_t v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_rope_error, sizeof v);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbol(g_rope_error, &zero, sizeof zero);
    if (e != cudaSuccess)
        return fail(PA_ERR_CUDA, "reading rope error word: %s", cudaGetErrorString(e));
    *code |= v & 1u;        // the store's bit 0
    *code |= (v & 2u) << 8; // bit 9
    return PA_OK;
}

} // namespace pa

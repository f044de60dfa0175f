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
// needs no shuffle, and a row's sum of squares (or its max|x|) log2(D / 16) of them.  A group takes
// kHeads rows of one token, whose cos and sin it loads once.  Bound: HBM for prompts (each row read and
// written once), the latency of one launch for decode steps.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace pa {

__device__ uint32_t g_rope_error; // bit 0: a slot outside [-1, num_slots); bit 1: a position outside the table

namespace {

constexpr int kThreads = 256;

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
    int32_t units;                         // groups per token
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

// kNext: pairs (2i, 2i + 1).  kAxes: more than one position per token.
template <int D, bool kInt8, bool kNext, bool kAxes, int kHeads>
__global__ void __launch_bounds__(kThreads) rope_store_kernel(const RopeParams p)
{
    constexpr int kLanes = D / 16; // of a row
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const uint32_t group = blockIdx.x * (uint32_t)(kThreads / kLanes) + threadIdx.x / kLanes;
    const int j = threadIdx.x % kLanes;
    const uint32_t token = group / (uint32_t)p.units;
    const int h0 = (int)(group - token * (uint32_t)p.units) * kHeads;
    const int heads = p.num_heads + 2 * p.num_kv_heads;
    // every lane stays to the end: the groups of a warp shuffle together
    const int t = (int)min(token, (uint32_t)p.num_tokens - 1u);
    bool live = token < (uint32_t)p.num_tokens;

    // the lane's two pieces of 8 values: of a turned part its 8 pairs, of the rest 16 consecutive values
    const int half = p.pairs;
    const bool turn = 8 * j < half;
    const int c0 = kNext || !turn ? 16 * j : 8 * j;
    const int c1 = kNext || !turn ? c0 + 8 : c0 + half;

    uint4 raw[kHeads][2];
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
        const int h = h0 + u;
        raw[u][0] = raw[u][1] = make_uint4(0u, 0u, 0u, 0u);
        if (live && h < heads) {
            const __nv_bfloat16 *row =
                h < p.num_heads ? p.q + (int64_t)t * p.q_stride + (int64_t)h * D
                : h < p.num_heads + p.num_kv_heads
                    ? p.k + (int64_t)t * p.k_stride + (int64_t)(h - p.num_heads) * D
                    : p.v + (int64_t)t * p.v_stride + (int64_t)(h - p.num_heads - p.num_kv_heads) * D;
            raw[u][0] = ptx::ld_once_v4(row + c0);
            raw[u][1] = ptx::ld_once_v4(row + c1);
        }
    }
    const int32_t slot = p.slots[t];
    float cs[8], sn[8];
    if constexpr (!kAxes) {
        const int pos = p.positions[t];
        const bool inside = (uint32_t)pos < (uint32_t)p.max_position;
        if (!inside && live && j == 0 && h0 == 0)
            atomicOr(&g_rope_error, 2u);
        live = live && inside;
        if (turn && inside) {
            const float4 *at = reinterpret_cast<const float4 *>(p.cos_sin + (int64_t)pos * 2 * half + 8 * j);
            const float4 *as = reinterpret_cast<const float4 *>(p.cos_sin + (int64_t)pos * 2 * half + half + 8 * j);
            *reinterpret_cast<float4 *>(cs) = at[0], *reinterpret_cast<float4 *>(cs + 4) = at[1];
            *reinterpret_cast<float4 *>(sn) = as[0], *reinterpret_cast<float4 *>(sn + 4) = as[1];
        }
    } else {
        int pos[4];
        bool inside = true;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            pos[a] = a < p.num_axes ? p.positions[(int64_t)a * p.num_tokens + t] : 0;
            inside = inside && (uint32_t)pos[a] < (uint32_t)p.max_position;
        }
        if (!inside && live && j == 0 && h0 == 0)
            atomicOr(&g_rope_error, 2u);
        live = live && inside;
        if (turn && inside) {
            const uint32_t bits = (uint32_t)(p.axis_bits[j >> 2] >> (16 * (j & 3)));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int a = (bits >> (2 * i)) & 3;
                const int at = a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3];
                const float *row = p.cos_sin + (int64_t)at * 2 * half + 8 * j + i;
                cs[i] = row[0];
                sn[i] = row[half];
            }
        }
    }
    const bool stored = slot >= 0 && slot < p.num_slots;
    if (!stored && slot != -1 && live && j == 0 && h0 == 0)
        atomicOr(&g_rope_error, 1u);

#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
        const int h = h0 + u;
        const bool is_q = h < p.num_heads, is_v = h >= p.num_heads + p.num_kv_heads;
        const bool write = live && h < heads && (is_q || stored);
        float x[16];
        unpack8(raw[u][0], x);
        unpack8(raw[u][1], x + 8);
        const __nv_bfloat16 *w = is_q ? p.q_weight : p.k_weight;
        if (p.q_weight != nullptr || p.k_weight != nullptr) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sum = fmaf(x[i], x[i], sum);
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (!is_v && w != nullptr) {
                const float r = rsqrtf(sum * (1.f / D) + p.eps);
                float y[16];
                unpack8(*reinterpret_cast<const uint4 *>(w + c0), y);
                unpack8(*reinterpret_cast<const uint4 *>(w + c1), y + 8);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    x[i] = x[i] * r * y[i];
            }
        }
        if (turn && !is_v) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int ia = kNext ? 2 * i : i, ib = kNext ? 2 * i + 1 : i + 8;
                const float a = x[ia], b = x[ib];
                x[ia] = a * cs[i] - b * sn[i];
                x[ib] = b * cs[i] + a * sn[i];
            }
        }
        const int g = is_v ? h - p.num_heads - p.num_kv_heads : h - p.num_heads; // KV head, if it is one
        if (write && (!kInt8 || is_q)) { // a value's row goes as it is
            __nv_bfloat16 *dst = is_q ? p.q_out + ((int64_t)t * p.num_heads + h) * D
                                      : static_cast<__nv_bfloat16 *>(is_v ? p.v_cache : p.k_cache) +
                                            ((int64_t)slot * p.num_kv_heads + g) * D;
            *reinterpret_cast<uint4 *>(dst + c0) = is_v ? raw[u][0] : pack8(x);
            *reinterpret_cast<uint4 *>(dst + c1) = is_v ? raw[u][1] : pack8(x + 8);
        }
        if constexpr (kInt8) {
            float a = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                a = fmaxf(a, fabsf(x[i]));
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1)
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            if (!is_q && write) {
                const float scale = fmaxf(__fdiv_rn(a, 127.0f), 1e-8f);
                const float rcp = __frcp_rn(scale);
                uint32_t c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    c[i] = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        c[i] |= (uint32_t)(quant::code_of(x[4 * i + e], scale, rcp) & 0xff) << (8 * e);
                }
                int8_t *dst = static_cast<int8_t *>(is_v ? p.v_cache : p.k_cache) + ((int64_t)slot * p.num_kv_heads + g) * D;
                *reinterpret_cast<uint2 *>(dst + c0) = make_uint2(c[0], c[1]);
                *reinterpret_cast<uint2 *>(dst + c1) = make_uint2(c[2], c[3]);
                if (j == 0)
                    (is_v ? p.v_scale : p.k_scale)[((int64_t)(slot / p.block_size) * p.num_kv_heads + g) * p.block_size +
                                                   slot % p.block_size] = __float2half_rn(scale);
            }
        }
    }
}

template <int D, bool kInt8, bool kNext, bool kAxes, int kHeads>
int launch(const RopeParams &p0, cudaStream_t stream)
{
    RopeParams p = p0;
    p.units = (p.num_heads + 2 * p.num_kv_heads + kHeads - 1) / kHeads;
    const int64_t groups = (int64_t)p.num_tokens * p.units, per = kThreads / (D / 16);
    if (groups > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "rope store: %d tokens of %d heads are too many for one call", p.num_tokens,
                    p.num_heads + 2 * p.num_kv_heads);
    const int64_t blocks = (groups + per - 1) / per;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rope_store_kernel<D, kInt8, kNext, kAxes, kHeads>, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(PA_ERR_CUDA, "rope store launch: %s", cudaGetErrorString(e));
    }
    return PA_OK;
}

template <int D, bool kInt8, bool kNext, bool kAxes>
int launch_heads(const RopeParams &p, cudaStream_t stream)
{
    // a prompt's tokens are many: four rows per group, whose loads are in flight together and share cos and sin
    const int64_t rows = (int64_t)p.num_tokens * (p.num_heads + 2 * p.num_kv_heads);
    return rows >= 65536 ? launch<D, kInt8, kNext, kAxes, 4>(p, stream) : launch<D, kInt8, kNext, kAxes, 1>(p, stream);
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

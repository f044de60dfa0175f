// Single-token decode over a bounded cache, from tables and lengths on the device: with a window and first
// tokens that stay visible (pa_decode_window), or over whole contexts with each key's attention weight
// added to a score that is kept for it (pa_decode_weights).  bf16 and INT8 caches.
//
// Formulas, for sequence b of context n and query head h of KV head g, s_j = scale q . k_j over the keys seen:
//   window:  j in [max(0, n - window), n) or j < sinks;       out = sum_j 2^(s'_j - M) v_j / L
//   weights: all j < n;   score[g][j] <- decay score[g][j] + sum_{h of g} 2^(s'_{h,j} - M_h) / L_h
// with s' = s log2 e, M = max s', L = sum 2^(s' - M).
//
// Sources (page title, section): "手搓 vLLM 推理引擎" (LLM-101-CN nano-vllm walkthrough), Step 4 (decode
// through block tables); "推理系统", "瓶颈不是算力，是带宽" (decode time = bytes read / bandwidth);
// "面试问答准备: nano-vLLM 推理引擎优化" (Split-K: local max, sum and accumulator per part, merged by
// log-sum-exp; Q3: the INT8 cache).
//
// The keys a query sees are cut into aligned chunks of 16 (the first tokens', then the window's: at most two
// runs).  A cluster of CTAs takes one (sequence, KV head), its warps every n-th chunk, each through a ring of
// cp.async stages as in the other decode kernels; the CTAs' partial results meet in distributed shared
// memory, so there is one launch and no workspace, and the sums' order is fixed.  What a chunk holds of keys
// that are not seen is not read: those rows are zeros in shared memory, whatever the cache has there.  Two stages and
// three CTAs on an SM (bf16) hide more than three stages and two did (64 x 4160 keys 86.6 -> 84.5 us, 6.5 TB/s).  INT8 codes
// come by cp.async too: TMA boxes took a quarter fewer instructions and no less time (200 x 1004 keys 49 us against
// 47.5, now 45.7, 4.4 TB/s), and five or six CTAs of two stages took 46 to 48: what is left above the bytes is the ramp, three
// dependent look-ups and the merge of 1.3 waves, about 7 us each.  The merges take four values a thread, with every
// part's maximum, sum and values on their way together (8 x 600 keys with weights 8.1 -> 6.7 us; with one value a
// thread, and the maxima first, a pair of CTAs of 16 heads spent 4 us there).
// Weights need M and L before any of them can be formed: the scores s' wait in the workspace (16 keys of one
// head group are 512 contiguous bytes) until the cluster has met; keys and values leave L2 first, so they wait there.
// 64 contexts of 4096 to 8192 keys take 150 to 155 us (5.4 to 5.5 TB/s), over INT8 111 (3.9), 121 without weights: writing
// s' costs 10 of that, the second pass over them, latency for the most part, 20.
#include <algorithm>
#include <type_traits>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cta_count.h"
#include "internal.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace pa {

// bit 0: a block id outside the pool, a table row outside the table, or a context longer than its row
__device__ uint32_t g_window_error;

namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int NT, bool kInt8>
struct WinLayout {
    static constexpr int kStages = kInt8 ? 3 : 2;
    static constexpr int kRowBytes = kInt8 ? D : D * 2;  // one head's row of one token
    static constexpr int kChunkBytes = 16 * kRowBytes;   // 16 tokens of K (or V)
    static constexpr int kStageBytes = 2 * kChunkBytes;
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kScaleOff = kWarps * kWarpBytes; // INT8: [warp][stage] 16 K + 16 V fp16 scales
    static constexpr int kSmemBytes = kScaleOff + (kInt8 ? kWarps * kStages * 64 : 0);
    // behind the last chunk the ring holds the warps' results and the CTA's
    static constexpr int kHeads = 8 * NT;
    static constexpr int kRow = D + 4; // padded, in floats
    static constexpr int kMergeM = 0;
    static constexpr int kMergeL = kMergeM + kWarps * kHeads;
    static constexpr int kMergeO = kMergeL + kWarps * kHeads;
    static constexpr int kPartM = kMergeO + kWarps * kHeads * kRow; // the CTA's, read by the cluster
    static constexpr int kPartL = kPartM + kHeads;
    static constexpr int kPartO = kPartL + kHeads;
    static constexpr int kAllM = kPartO + kHeads * D; // the cluster's
    static constexpr int kAllL = kAllM + kHeads;
    static_assert((kAllL + kHeads) * 4 <= kWarps * kWarpBytes, "merge area");
};

struct WinParams {
    const __nv_bfloat16 *q;
    const void *k_cache;
    const void *v_cache;
    const __half *k_scale;
    const __half *v_scale;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *table_rows; // NULL: row b
    __nv_bfloat16 *out;
    float scale_log2;
    int32_t num_heads, num_kv_heads, group, block_size, num_blocks;
    int32_t num_rows, max_blocks;
    int32_t window, sinks;
    // weights
    float decay;
    const float *scores;
    float *scores_out;
    float *raw;        // [sequence][KV head][max_blocks * block_size][raw_heads]
    int32_t raw_heads; // the group, rounded up to 4, 8 or 16
};

constexpr uint32_t kFlip = 0x80808080u;  // int8 -> offset binary (x + 128), per byte
constexpr uint32_t kLoPair = 0x4140u;    // prmt: bytes 0, 1 under 0x64 high bytes
constexpr uint32_t kHiPair = 0x4342u;    // prmt: bytes 2, 3 under 0x64 high bytes
constexpr uint32_t kMagic = 0x64806480u; // f16x2 (1152, 1152)

// Two offset-binary codes of u (chosen by sel) -> f16x2 of the signed codes, exact.
__device__ __forceinline__ uint32_t codes_to_f16x2(uint32_t u, uint32_t sel)
{
    return ptx::sub_f16x2(ptx::prmt(u, 0x64646464u, sel), kMagic);
}

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w)
{
    return ptx::pack_f16(ptx::clamp_f16_nan(__uint_as_float(w << 16)), ptx::clamp_f16_nan(__uint_as_float(w & 0xffff0000u)));
}

__device__ __forceinline__ float lds_half(uint32_t addr) { return __half2float(__ushort_as_half(ptx::lds_u16(addr))); }

// Byte offset of 16-byte vector v of token t in a staged chunk: rows of 256, 128 or 64 bytes.
template <int kRowBytes>
__device__ __forceinline__ uint32_t swz(int t, int v)
{
    if constexpr (kRowBytes == 64)
        return (uint32_t)(t * 64 + ((v ^ ((t >> 1) & 3)) << 4));
    else
        return (uint32_t)(t * kRowBytes + ((v ^ (t & 7)) << 4));
}

template <int D, int NT, bool kInt8, bool kWeights>
__global__ void __launch_bounds__(kThreads, (kInt8 ? 5 : 4) - NT)
    decode_window_kernel(const WinParams p)
{
    using L = WinLayout<D, NT, kInt8>;
    constexpr int kStages = L::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int unit = (int)blockIdx.x / ctas;
    const int b = unit / p.num_kv_heads, g = unit - b * p.num_kv_heads;
    const int G = p.group, Hq = p.num_heads, Hkv = p.num_kv_heads, bs = p.block_size;
    ptx::grid_dependency_wait();

    // the row and its chunks
    const int row = p.table_rows ? p.table_rows[b] : b;
    const bool row_ok = (uint32_t)row < (uint32_t)p.num_rows;
    int ctx = row_ok ? max(p.context_lens[row], 0) : 0;
    const int room = p.max_blocks * bs;
    if ((!row_ok || ctx > room) && threadIdx.x == 0 && g == 0 && rank == 0)
        atomicOr(&g_window_error, 1u);
    ctx = min(ctx, room);
    const int32_t *bt_row = p.block_tables + (size_t)(row_ok ? row : 0) * p.max_blocks;
    const int lo = kWeights ? 0 : max(0, ctx - p.window);
    const int sink_end = kWeights ? 0 : min(p.sinks, lo);
    const int sink_chunks = min((sink_end + 15) >> 4, lo >> 4);
    const int skip = (lo >> 4) - sink_chunks; // chunks between the first tokens' and the window's
    const int chunks = ((ctx + 15) >> 4) - skip;
    const int w0 = rank * kWarps + warp, step = ctas * kWarps; // this warp's chunks: w0, w0 + step, ...
    const int my_n = chunks > w0 ? (chunks - w0 + step - 1) / step : 0;
    auto first_key = [&](int i) {
        const int v = w0 + i * step;
        return 16 * (v < sink_chunks ? v : v + skip);
    };
    auto seen = [&](int key) { return (key >= lo && key < ctx) || key < sink_end; };
    auto whole = [&](int key0) { return (key0 >= lo && key0 + 16 <= ctx) || key0 + 16 <= sink_end; };

    const uint32_t wbase = ptx::smem_u32(smem) + warp * L::kWarpBytes;
    const uint32_t sc_base = ptx::smem_u32(smem) + L::kScaleOff + warp * kStages * 64;
    int blk_cache = 0;
    // the keys and values of a step are read once: of L2, what waits there for the weights goes last
    const uint64_t once = ptx::policy_evict_first();

    // Chunk i of this warp into stage st.  A lane copies vector v0 of the rows t0, t0 + kRowsPer, ...
    constexpr int kVec = L::kRowBytes / 16;     // 16-byte vectors per row
    constexpr int kRowsPer = 32 / kVec;         // rows per instruction
    const int t0 = lane / kVec, v0 = lane % kVec;
    const size_t token_bytes = (size_t)Hkv * L::kRowBytes;
    const size_t lane_off = t0 * token_bytes + (size_t)g * L::kRowBytes + v0 * 16;
    const char *k_lane = static_cast<const char *>(p.k_cache) + lane_off;
    const char *v_lane = static_cast<const char *>(p.v_cache) + lane_off;
    auto copy = [&](uint32_t dst, const char *src, uint32_t bytes) {
        if constexpr (kWeights)
            ptx::cp_async_16_hint(dst, src, bytes, once);
        else
            ptx::cp_async_16(dst, src, bytes);
    };
    auto issue = [&](int i, int st) {
        if ((i & 31) == 0) { // the block ids of chunks i .. i + 31, one per lane
            blk_cache = 0;
            if (i + lane < my_n) {
                blk_cache = bt_row[first_key(i + lane) / bs];
                if ((uint32_t)blk_cache >= (uint32_t)p.num_blocks) {
                    blk_cache = -1;
                    atomicOr(&g_window_error, 1u);
                }
            }
        }
        const int phys = __shfl_sync(0xffffffffu, blk_cache, i & 31);
        const int key0 = first_key(i);
        const uint32_t sbase = wbase + st * L::kStageBytes;
        const int64_t row0 = (int64_t)phys * bs + (key0 & (bs - 1));
        const char *kp = k_lane + row0 * token_bytes, *vp = v_lane + row0 * token_bytes;
        if (phys >= 0 && whole(key0)) {
#pragma unroll
            for (int x = 0; x < 16 / kRowsPer; ++x) {
                const uint32_t dst = sbase + swz<L::kRowBytes>(x * kRowsPer + t0, v0);
                copy(dst, kp + x * kRowsPer * token_bytes, 16u);
                copy(dst + L::kChunkBytes, vp + x * kRowsPer * token_bytes, 16u);
            }
        } else { // rows that are not seen, or of a block outside the pool, are zeros
#pragma unroll
            for (int x = 0; x < 16 / kRowsPer; ++x) {
                const int t = x * kRowsPer + t0;
                const bool valid = phys >= 0 && seen(key0 + t);
                const uint32_t dst = sbase + swz<L::kRowBytes>(t, v0);
                ptx::cp_async_16(dst, valid ? kp + x * kRowsPer * token_bytes : static_cast<const char *>(p.k_cache),
                                 valid ? 16u : 0u);
                ptx::cp_async_16(dst + L::kChunkBytes,
                                 valid ? vp + x * kRowsPer * token_bytes : static_cast<const char *>(p.v_cache),
                                 valid ? 16u : 0u);
            }
        }
        if constexpr (kInt8) {
            if (lane < 4) { // 16 fp16 scales of K, 16 of V (a block outside the pool: zeros)
                const size_t si = ((size_t)max(phys, 0) * Hkv + g) * bs + (key0 & (bs - 1)) + (lane & 1) * 8;
                ptx::cp_async_16(sc_base + st * 64 + lane * 16, (lane < 2 ? p.k_scale : p.v_scale) + si,
                                 phys >= 0 ? 16u : 0u);
            }
        }
    };

#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        if (s < my_n)
            issue(s, s);
        ptx::cp_async_commit();
    }

    // Q^T fragments: B operand (k = d, n = head) of the score product.  INT8: f16, k-step kk of lane c covers
    // d = c * D/4 + 4 kk + {0 .. 3}, so that a lane's codes for all steps are one run of its token's row.
    uint32_t qf[NT][D / 16][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int hl = nt * 8 + r;
        const bool valid = hl < G;
        const __nv_bfloat16 *qrow = p.q + ((size_t)b * Hq + (size_t)g * G + (valid ? hl : 0)) * D;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            if constexpr (kInt8) {
                const uint2 w = valid ? reinterpret_cast<const uint2 *>(qrow + c * (D / 4))[kk] : make_uint2(0u, 0u);
                qf[nt][kk][0] = bf16x2_to_f16x2(w.x);
                qf[nt][kk][1] = bf16x2_to_f16x2(w.y);
            } else {
                const uint32_t *at = reinterpret_cast<const uint32_t *>(qrow) + kk * 8 + c;
                qf[nt][kk][0] = valid ? at[0] : 0u;
                qf[nt][kk][1] = valid ? at[4] : 0u;
            }
        }
    }

    float acc[NT][D / 16][4];
    float m_r[NT][2], l_r[NT][2];
    float by = quant::kProductsBy; // INT8: acc is this many times the sums
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m_r[nt][0] = m_r[nt][1] = -INFINITY;
        l_r[nt][0] = l_r[nt][1] = 0.f;
#pragma unroll
        for (int mi = 0; mi < D / 16; ++mi)
            acc[nt][mi][0] = acc[nt][mi][1] = acc[nt][mi][2] = acc[nt][mi][3] = 0.f;
    }

    // ldmatrix row addressing (per lane) inside a bf16 chunk
    const int a_tok = (lane & 7) + ((lane >> 3) & 1) * 8; // K: A = K[tok][d]
    const int a_hi = lane >> 4;
    const int v_tok = (lane & 7) + (lane >> 4) * 8;       // V: A = V^T via .trans
    const int v_hi = (lane >> 3) & 1;

    float *raw = kWeights ? p.raw + (size_t)unit * room * p.raw_heads : nullptr;

    for (int i = 0, st = 0; i < my_n; ++i, st = st + 1 < kStages ? st + 1 : 0) {
        __syncwarp();
        if (i + kStages - 1 < my_n)
            issue(i + kStages - 1, st > 0 ? st - 1 : kStages - 1);
        ptx::cp_async_commit();
        ptx::cp_async_wait<kStages - 1>();
        __syncwarp();

        const uint32_t kb = wbase + st * L::kStageBytes;
        const uint32_t vb = kb + L::kChunkBytes;
        const int key0 = first_key(i);

        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
        float ks0 = p.scale_log2, ks1 = p.scale_log2, vs0 = 1.f, vs1 = 1.f;
        if constexpr (kInt8) {
            uint32_t kw[2][D / 16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int x = 0; x < D / 64; ++x) {
                    const uint4 u = ptx::lds_v4(kb + swz<D>(r + 8 * h, (D / 64) * c + x));
                    kw[h][4 * x] = u.x, kw[h][4 * x + 1] = u.y, kw[h][4 * x + 2] = u.z, kw[h][4 * x + 3] = u.w;
                }
            }
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t u0 = kw[0][kk] ^ kFlip, u1 = kw[1][kk] ^ kFlip;
                const uint32_t a0 = codes_to_f16x2(u0, kLoPair), a2 = codes_to_f16x2(u0, kHiPair);
                const uint32_t a1 = codes_to_f16x2(u1, kLoPair), a3 = codes_to_f16x2(u1, kHiPair);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    ptx::mma_16816_f16(sc[nt], a0, a1, a2, a3, qf[nt][kk][0], qf[nt][kk][1]);
            }
            const uint32_t sb = sc_base + st * 64;
            ks0 *= lds_half(sb + 2 * r);
            ks1 *= lds_half(sb + 2 * (r + 8));
            vs0 = lds_half(sb + 32 + 2 * r);
            vs1 = lds_half(sb + 32 + 2 * (r + 8));
        } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t a0, a1, a2, a3;
                ptx::ldmatrix_x4(kb + swz<L::kRowBytes>(a_tok, 2 * kk + a_hi), a0, a1, a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    ptx::mma_16816(sc[nt], a0, a1, a2, a3, qf[nt][kk][0], qf[nt][kk][1]);
            }
        }

        const bool all = whole(key0), seen0 = all || seen(key0 + r), seen1 = all || seen(key0 + r + 8);
        if constexpr (kInt8) { // the scales of keys that are not seen may be anything
            vs0 = seen0 ? vs0 : 0.f;
            vs1 = seen1 ? vs1 : 0.f;
            quant::fit_products(vs0, vs1, by, acc);
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float s0 = seen0 ? sc[nt][0] * ks0 : -INFINITY;
            const float s1 = seen0 ? sc[nt][1] * ks0 : -INFINITY;
            const float s2 = seen1 ? sc[nt][2] * ks1 : -INFINITY;
            const float s3 = seen1 ? sc[nt][3] * ks1 : -INFINITY;
            if constexpr (kWeights) {
                const int h0 = nt * 8 + 2 * c;
                if (h0 < p.raw_heads) {
                    float *at = raw + (size_t)(key0 + r) * p.raw_heads + h0;
                    *reinterpret_cast<float2 *>(at) = make_float2(s0, s1);
                    *reinterpret_cast<float2 *>(at + (size_t)8 * p.raw_heads) = make_float2(s2, s3);
                }
            }
            float mx0 = fmaxf(s0, s2), mx1 = fmaxf(s1, s3);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
            }
            const float mn0 = fmaxf(m_r[nt][0], mx0), mn1 = fmaxf(m_r[nt][1], mx1);
            // a maximum of -inf (every score so far -inf or NaN) is no reference: -inf - -inf is NaN
            const float rf0 = mn0 == -INFINITY ? 0.f : mn0, rf1 = mn1 == -INFINITY ? 0.f : mn1;
            const float al0 = ptx::ex2(m_r[nt][0] - rf0), al1 = ptx::ex2(m_r[nt][1] - rf1);
            m_r[nt][0] = mn0;
            m_r[nt][1] = mn1;
            const float p0 = ptx::ex2(s0 - rf0), p1 = ptx::ex2(s1 - rf1);
            const float p2 = ptx::ex2(s2 - rf0), p3 = ptx::ex2(s3 - rf1);
            l_r[nt][0] = l_r[nt][0] * al0 + p0 + p2;
            l_r[nt][1] = l_r[nt][1] * al1 + p1 + p3;
            if (__any_sync(0xffffffffu, (al0 != 1.f) | (al1 != 1.f))) { // not while no row's maximum moves
#pragma unroll
                for (int mi = 0; mi < D / 16; ++mi) {
                    acc[nt][mi][0] *= al0;
                    acc[nt][mi][1] *= al1;
                    acc[nt][mi][2] *= al0;
                    acc[nt][mi][3] *= al1;
                }
            }
            // weights in the products' type: bf16 (2^-8), over INT8, with the value's scale and a factor that keeps them
            // among fp16's normal numbers, f16 (2^-11), both within the result's rounding
            if constexpr (kInt8) {
                pb[nt][0] = ptx::movmatrix_trans(ptx::pack_f16(p0 * vs0, p1 * vs0));
                pb[nt][1] = ptx::movmatrix_trans(ptx::pack_f16(p2 * vs1, p3 * vs1));
            } else {
                pb[nt][0] = ptx::movmatrix_trans(ptx::pack_bf16(p0, p1));
                pb[nt][1] = ptx::movmatrix_trans(ptx::pack_bf16(p2, p3));
            }
        }

        if constexpr (kInt8) {
            // V codes of tokens 2c, 2c+1, 2c+8, 2c+9: bytes [r*D/8, (r+1)*D/8) of each row; byte 2*mi + hi of
            // that run is d-row (mi, r + 8*hi) of O^T tile mi
            uint32_t vw[4][D / 32];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 2 * c + (j & 1) + 8 * (j >> 1);
                if constexpr (D == 128) {
                    const uint4 u = ptx::lds_v4(vb + swz<D>(t, r));
                    vw[j][0] = u.x, vw[j][1] = u.y, vw[j][2] = u.z, vw[j][3] = u.w;
                } else {
                    const uint2 u = ptx::lds_v2(vb + swz<D>(t, r >> 1) + (r & 1) * 8);
                    vw[j][0] = u.x, vw[j][1] = u.y;
                }
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint32_t x01 = ptx::prmt(vw[0][w], vw[1][w], 0x5140u) ^ kFlip; // tile 2w
                const uint32_t y01 = ptx::prmt(vw[0][w], vw[1][w], 0x7362u) ^ kFlip; // tile 2w + 1
                const uint32_t x89 = ptx::prmt(vw[2][w], vw[3][w], 0x5140u) ^ kFlip;
                const uint32_t y89 = ptx::prmt(vw[2][w], vw[3][w], 0x7362u) ^ kFlip;
                const uint32_t a0 = codes_to_f16x2(x01, kLoPair), a1 = codes_to_f16x2(x01, kHiPair);
                const uint32_t a2 = codes_to_f16x2(x89, kLoPair), a3 = codes_to_f16x2(x89, kHiPair);
                const uint32_t b0 = codes_to_f16x2(y01, kLoPair), b1 = codes_to_f16x2(y01, kHiPair);
                const uint32_t b2 = codes_to_f16x2(y89, kLoPair), b3 = codes_to_f16x2(y89, kHiPair);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    ptx::mma_16816_f16(acc[nt][2 * w], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    ptx::mma_16816_f16(acc[nt][2 * w + 1], b0, b1, b2, b3, pb[nt][0], pb[nt][1]);
                }
            }
        } else {
#pragma unroll
            for (int mi = 0; mi < D / 16; ++mi) {
                uint32_t a0, a1, a2, a3;
                ptx::ldmatrix_x4_trans(vb + swz<L::kRowBytes>(v_tok, 2 * mi + v_hi), a0, a1, a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    ptx::mma_16816(acc[nt][mi], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
            }
        }
    }
    ptx::cp_async_wait<0>();
    // Only now: the next launch's CTAs would take the places that this one leaves on some SMs and not on others, and keep
    // that lopsided order (64 x 4096 keys in a stream: 98 us with this at the start, 86 here).
    ptx::launch_dependents();

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
                l_r[nt][j] += __shfl_xor_sync(0xffffffffu, l_r[nt][j], o);

    if constexpr (kInt8) {
        const float x = __fdiv_rn(1.f, by);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mi = 0; mi < D / 16; ++mi)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[nt][mi][e] *= x;
    }

    // the warps' results meet in the ring
    __syncthreads();
    constexpr int H8 = L::kHeads;
    float *f = reinterpret_cast<float *>(smem);
    float *mrg_m = f + L::kMergeM, *mrg_l = f + L::kMergeL, *mrg_o = f + L::kMergeO;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int h0 = nt * 8 + 2 * c;
        if (lane < 4) {
            mrg_m[warp * H8 + h0] = m_r[nt][0];
            mrg_m[warp * H8 + h0 + 1] = m_r[nt][1];
            mrg_l[warp * H8 + h0] = l_r[nt][0];
            mrg_l[warp * H8 + h0 + 1] = l_r[nt][1];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float *o = mrg_o + (size_t)(warp * H8 + h0 + j) * L::kRow;
            if constexpr (kInt8) {
#pragma unroll
                for (int v = 0; v < D / 32; ++v)
                    *reinterpret_cast<float4 *>(o + r * (D / 8) + 4 * v) =
                        make_float4(acc[nt][2 * v][j], acc[nt][2 * v][j + 2], acc[nt][2 * v + 1][j], acc[nt][2 * v + 1][j + 2]);
            } else {
#pragma unroll
                for (int mi = 0; mi < D / 16; ++mi) {
                    o[mi * 16 + r] = acc[nt][mi][j];
                    o[mi * 16 + r + 8] = acc[nt][mi][j + 2];
                }
            }
        }
    }
    __syncthreads();
    // four values of the output per thread and turn
    float *part_m = f + L::kPartM, *part_l = f + L::kPartL, *part_o = f + L::kPartO;
    __nv_bfloat16 *out = p.out + ((size_t)b * Hq + (size_t)g * G) * D;
    auto put = [&](int idx, float sum, float4 o) { // no weight at all: 0, or NaN where a value is
        const float x = sum != 0.f ? 1.f / sum : 1.f;
        *reinterpret_cast<uint2 *>(out + idx) = make_uint2(ptx::pack_bf16(o.x * x, o.y * x), ptx::pack_bf16(o.z * x, o.w * x));
    };
    auto add = [](float4 &o, float e, float4 v) {
        o = make_float4(fmaf(e, v.x, o.x), fmaf(e, v.y, o.y), fmaf(e, v.z, o.z), fmaf(e, v.w, o.w));
    };
    for (int idx = 4 * (int)threadIdx.x; idx < G * D; idx += 4 * kThreads) {
        const int hl = idx / D, d = idx % D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            M = fmaxf(M, mrg_m[w * H8 + hl]);
        const float rf = M == -INFINITY ? 0.f : M;
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float e = ptx::ex2(mrg_m[w * H8 + hl] - rf);
            sum += e * mrg_l[w * H8 + hl];
            add(o, e, *reinterpret_cast<const float4 *>(mrg_o + (size_t)(w * H8 + hl) * L::kRow + d));
        }
        if (ctas == 1)
            put(idx, sum, o);
        else
            *reinterpret_cast<float4 *>(part_o + idx) = o;
        if (d == 0) {
            part_m[hl] = M;
            part_l[hl] = sum;
        }
    }
    if (ctas > 1)
        cluster.sync();
    else if (kWeights)
        __syncthreads();
    else
        return;

    // the cluster's: each CTA a share of the output.  Eight CTAs' results are on their way at once (16: a microsecond less
    // for a cluster of 16, one more for one of five).
    constexpr int kAtOnce = 8;
    auto of = [&](float *at, int cta) { return ctas > 1 ? cluster.map_shared_rank(at, cta) : at; };
    // the sums of 2^(m - M) l and 2^(m - M) o, in the CTAs' order
    auto totals = [&](auto with, int hl, int idx, float &M, float &sum, float4 &o) {
        M = -INFINITY, sum = 0.f, o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x0 = 0; x0 < ctas; x0 += kAtOnce) {
            float m[kAtOnce], l[kAtOnce];
            float4 v[kAtOnce];
#pragma unroll
            for (int x = 0; x < kAtOnce; ++x) {
                m[x] = -INFINITY, l[x] = 0.f, v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (x0 + x < ctas) {
                    m[x] = of(part_m, x0 + x)[hl];
                    l[x] = of(part_l, x0 + x)[hl];
                    if constexpr (with.value)
                        v[x] = *reinterpret_cast<const float4 *>(of(part_o, x0 + x) + idx);
                }
            }
            const float before = M;
#pragma unroll
            for (int x = 0; x < kAtOnce; ++x)
                M = fmaxf(M, m[x]);
            const float rf = M == -INFINITY ? 0.f : M, al = ptx::ex2(before - rf);
            sum *= al;
            o = make_float4(o.x * al, o.y * al, o.z * al, o.w * al);
#pragma unroll
            for (int x = 0; x < kAtOnce; ++x) {
                const float e = ptx::ex2(m[x] - rf);
                sum += e * l[x];
                add(o, e, v[x]);
            }
        }
    };
    for (int idx = 4 * (rank * kThreads + (int)threadIdx.x); ctas > 1 && idx < G * D; idx += 4 * ctas * kThreads) {
        float M, sum;
        float4 o;
        totals(std::true_type{}, idx / D, idx, M, sum, o);
        put(idx, sum, o);
    }
    if constexpr (kWeights) {
        float *all_m = f + L::kAllM, *all_l = f + L::kAllL;
        if (threadIdx.x < (unsigned)G) {
            float M, sum;
            float4 o;
            totals(std::false_type{}, threadIdx.x, 0, M, sum, o);
            all_m[threadIdx.x] = M == -INFINITY ? 0.f : M;
            all_l[threadIdx.x] = sum != 0.f ? 1.f / sum : 0.f; // (every weight is 0 then)
        }
        __syncthreads();
        // a key per lane and 16 of a chunk, kKeys loads of each in flight
        constexpr int kKeys = 8;
        const size_t srow = ((size_t)row * Hkv + g) * room;
        const bool keep = p.decay != 0.f;
        for (int i0 = lane >> 4; i0 < my_n; i0 += 2 * kKeys) {
            float4 x[kKeys][2 * NT];
            float old[kKeys];
#pragma unroll
            for (int u = 0; u < kKeys; ++u) {
                const int i = i0 + 2 * u, key = i < my_n ? first_key(i) + (lane & 15) : ctx;
                if (key < ctx) {
                    const float4 *at = reinterpret_cast<const float4 *>(raw + (size_t)key * p.raw_heads);
#pragma unroll
                    for (int e = 0; e < 2 * NT; ++e)
                        if (4 * e < p.raw_heads)
                            x[u][e] = at[e];
                    old[u] = keep ? p.scores[srow + key] : 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < kKeys; ++u) {
                const int i = i0 + 2 * u, key = i < my_n ? first_key(i) + (lane & 15) : ctx;
                if (key < ctx) {
                    float w = 0.f;
#pragma unroll
                    for (int e = 0; e < 2 * NT; ++e) {
                        const float y[4] = {x[u][e].x, x[u][e].y, x[u][e].z, x[u][e].w};
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int hl = 4 * e + z;
                            if (hl < G)
                                w += ptx::ex2(y[z] - all_m[hl]) * all_l[hl];
                        }
                    }
                    p.scores_out[srow + key] = keep ? fmaf(p.decay, old[u], w) : w;
                }
            }
        }
    }
    if (ctas > 1)
        cluster.sync(); // the others may still read this CTA's results
}

template <int D, int NT, bool kInt8, bool kWeights>
int count_ctas(const WindowArgs &a, int *ctas)
{
    using L = WinLayout<D, NT, kInt8>;
    const int64_t room = (int64_t)a.max_blocks_per_seq * a.dims.block_size, most = (int64_t)a.window + a.sinks;
    return count_cluster_ctas((int64_t)a.num_seqs * a.dims.num_kv_heads, std::min(room, most), room <= most,
                              [](int c, int *clusters) {
                                  return active_clusters<decode_window_kernel<D, NT, kInt8, kWeights>>(
                                      "window decode", c, kThreads, L::kSmemBytes, clusters);
                              },
                              ctas);
}

template <int D, int NT, bool kInt8, bool kWeights>
int launch(const WindowArgs &a, const WinParams &p, cudaStream_t stream)
{
    using L = WinLayout<D, NT, kInt8>;
    if (int rc = ensure_smem<decode_window_kernel<D, NT, kInt8, kWeights>>(L::kSmemBytes, "window decode"))
        return rc;
    if (int rc = ensure_wide_clusters<decode_window_kernel<D, NT, kInt8, kWeights>>("window decode"))
        return rc;
    int ctas = 1;
    if (int rc = count_ctas<D, NT, kInt8, kWeights>(a, &ctas))
        return rc;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.num_seqs * a.dims.num_kv_heads * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)ctas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_window_kernel<D, NT, kInt8, kWeights>, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(PA_ERR_CUDA, "window decode launch: %s", cudaGetErrorString(e));
    }
    return PA_OK;
}

template <int D, int NT>
int launch_kind(const WindowArgs &a, const WinParams &p, cudaStream_t s)
{
    if (a.raw)
        return a.k_scale ? launch<D, NT, true, true>(a, p, s) : launch<D, NT, false, true>(a, p, s);
    return a.k_scale ? launch<D, NT, true, false>(a, p, s) : launch<D, NT, false, false>(a, p, s);
}

} // namespace

int launch_decode_window(const WindowArgs &a, void *stream)
{
    WinParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.k_cache = a.k_cache, p.v_cache = a.v_cache;
    p.k_scale = static_cast<const __half *>(a.k_scale), p.v_scale = static_cast<const __half *>(a.v_scale);
    p.block_tables = a.block_tables, p.context_lens = a.context_lens, p.table_rows = a.table_rows;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.scale_log2 = a.scale * kLog2e;
    p.num_heads = a.dims.num_heads, p.num_kv_heads = a.dims.num_kv_heads;
    p.group = a.dims.num_heads / a.dims.num_kv_heads;
    p.block_size = a.dims.block_size, p.num_blocks = a.dims.num_blocks;
    p.num_rows = a.num_rows, p.max_blocks = a.max_blocks_per_seq;
    p.window = a.window, p.sinks = a.sinks;
    p.decay = a.decay, p.scores = a.scores, p.scores_out = a.scores_out, p.raw = a.raw;
    p.raw_heads = window_raw_heads(a.dims);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool two = p.group > 8;
    if (a.dims.head_dim == 128)
        return two ? launch_kind<128, 2>(a, p, s) : launch_kind<128, 1>(a, p, s);
    return two ? launch_kind<64, 2>(a, p, s) : launch_kind<64, 1>(a, p, s);
}

int read_window_error(uint32_t *code)
{
    uint32_t v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_window_error, sizeof v);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbol(g_window_error, &zero, sizeof zero);
    if (e != cudaSuccess)
        return fail(PA_ERR_CUDA, "reading window decode error word: %s", cudaGetErrorString(e));
    *code |= (v & 1u) << 6; // the shared-prefix decode's bit: a block id outside the pool
    return PA_OK;
}

} // namespace pa

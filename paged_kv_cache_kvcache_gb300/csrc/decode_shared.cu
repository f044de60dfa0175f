// Single-token decode of a batch whose sequences share long prefixes: the shared pages are
// read once for the whole group instead of once per sequence.
//
// Sources (page title, section):
//  - "vLLM / SGLang 面试源码深挖", section 4 (beam search and KV block fork): parent and
//    child sequences share block ids; section 3: requests behind one prompt hit the same
//    cached prefix blocks.
//  - "面试问答准备: nano-vLLM 推理引擎优化", the Split-K entry: segments of a context emit a
//    max, a normaliser and an fp32 accumulator, merged by log-sum-exp.
//
// Mathematics.  For a key range R let m = max_R s, l = sum_R 2^(s - m), o = sum_R 2^(s - m) v / l
// (s in log2 units).  Ranges merge exactly: with e_R = m_R + log2 l_R and M = max e_R,
//   out = sum_R 2^(e_R - M) o_R / sum_R 2^(e_R - M).
// So a sequence's context may be cut at its group's shared prefix, and the prefix part of all
// sequences of the group is ONE product: rows = (sequence, query head of the KV head's group),
// all reading the same K/V.  With R rows a K/V byte is worth R flops (bf16), so a prefix is
// bound by HBM up to about 290 rows per KV head and by the tensor cores beyond.
//
// One persistent launch runs every part.  A work item is (rows, KV head, key range, block-table
// row): a prefix part carries many sequences, a suffix part one.  A CTA holds two query tiles of
// 128 rows and runs its items in two ways:
//  * a prefix part of more than 128 rows is a PAIR: both tiles against one stream of K/V, bound by
//    what one tile's softmax and hand-offs take beyond the other's products (measured 1.62 us per 128
//    keys, of which the products are 1.0; tensor pipe 58 % busy on the SMs in use);
//  * every other part is a SINGLE: one tile, 128 keys whose products take about 1100 cycles of the
//    tensor core while their 64 KB of K/V take about 2800 cycles of this SM's share of HBM.  But
//    score product, softmax and value product of one tile follow one another (about 2700 cycles
//    with their hand-offs), so the two tiles are two LANES, each walking singles of its own, one's
//    products under the other's softmax and loads.  Most of a single's rows are padding; warps
//    without a valid row skip the softmax.  Where there are more items than lanes, the parts of
//    single sequences run apart, in the decode kernels, in a launch that may run beside this one.
// The host cuts the key ranges and deals pairs to CTAs and singles to lanes (longest first onto
// the least loaded).  Structure of a CTA as in the prefill kernel: K, V and query producers
// (TMA, one 3-D box per physical block), one MMA warp (tcgen05, S and O in tensor memory, P fed
// back through tensor memory), one softmax warpgroup per tile; the rings run on across items.
//
// INT8 cache.  A launch before turns what the shared parts read into fp16, once for all query
// tiles and heads: keys and values (code * scale, rounded by 2^-11 of it at most; fp16 holds them to
// 65504) and the queries.  The products then run as on a bf16 cache, with fp16 weights.  (Exact
// codes with the scales in the softmax took 3.4 us per 128 keys and pair instead of 1.6: 64 more
// 16-byte loads per row; converting in shared memory took 4.2.)
//
// Short contexts (the plan decides, see pack_shared.cpp) gain nothing from sharing: they go whole
// through the decode kernels, which start in less time and have nothing to merge.
//
// Every hand-off waits with a time limit; a wait that runs out sets an error bit and the
// kernel returns, once nothing that it issued can be in flight any more.  A block id outside the pool reads as zeros and sets an error bit.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace pa {

// bit 0: a bounded wait timed out; bit 1: a block id outside the pool was met
__device__ uint32_t g_shared_error;

namespace {

// warps 0-7: softmax (two warpgroups), 8: K producer, 9: MMA issuer and TMEM owner, 10: V
// producer, 11: query producer.  168 registers per thread at launch; setmaxnreg moves part of
// warps 8-11's share to the softmax warps.  (ptxas -v: 36 bytes of spill stores a thread and 172 of spill
// loads, not traced to their place.)
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168;
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
static_assert(128 * (2 * kSoftmaxRegs + kOtherRegs) == kThreads * kLaunchRegs, "register hand-over");
constexpr int kKWarp = 8, kMmaWarp = 9, kVWarp = 10, kQWarp = 11;
// Rows of a TMA box of large blocks: a range's last boxes read past its end, 16 rows on average
// (with one box of 128 per tile a batch of 200 suffixes of 350 keys read 12 % more than its keys).
constexpr int kBoxRows = 32;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f; // log2 units
template <int D>
struct ShLayout {
    static constexpr int kPanels = D / 64;        // 64-element (128-byte) panels along head_dim
    static constexpr int kPanelBytes = 128 * 128; // 128 rows x 128 bytes
    static constexpr int kTileBytes = kPanels * kPanelBytes;
    static constexpr int kKStages = D == 128 ? 3 : 4;
    static constexpr int kVStages = D == 128 ? 2 : 4;
    static constexpr int kQ = 0; // two query tiles
    static constexpr int kK = kQ + 2 * kTileBytes;
    static constexpr int kV = kK + kKStages * kTileBytes;
    static constexpr int kBar = kV + kVStages * kTileBytes;
    static constexpr int kSmemBytes = kBar + 256 + 1024; // + alignment slack
    static_assert(kKStages <= 4 && kVStages <= 4, "barrier slots");
    static_assert(kSmemBytes <= 232448, "shared memory per CTA");
};

struct ShParams {
    int32_t scratch_rows; // INT8: rows of the scratch cache
    const int4 *items;
    const int4 *cta_items;
    const int2 *seq_parts;
    const int32_t *block_tables;
    __nv_bfloat16 *out;
    float *part_o;
    float *part_lse;
    float scale_log2;
    int32_t num_heads;
    int32_t group;
    int32_t rows_per_tile; // sequences per 128-row tile
    int32_t block_size;
    int32_t box_rows;
    int32_t max_blocks;
    int32_t num_blocks;
    // bf16: `go` into the word (NULL: none), once the launches before have ended, for the launch beside
    uint64_t *go_word;
    uint64_t go;
};

struct Bars {
    uint32_t base;
    __device__ uint32_t q_full(int t) const { return base + 8 * t; }
    __device__ uint32_t q_free(int t) const { return base + 8 * (2 + t); }
    __device__ uint32_t k_full(int s) const { return base + 8 * (4 + s); }
    __device__ uint32_t k_free(int s) const { return base + 8 * (8 + s); }
    __device__ uint32_t v_full(int s) const { return base + 8 * (12 + s); }
    __device__ uint32_t v_free(int s) const { return base + 8 * (16 + s); }
    __device__ uint32_t s_full(int t) const { return base + 8 * (20 + t); }
    __device__ uint32_t p_full(int t) const { return base + 8 * (22 + t); }
    __device__ uint32_t o_full(int t) const { return base + 8 * (24 + t); }
    __device__ uint32_t v_tail(int s) const { return base + 8 * (26 + s); }
    __device__ uint32_t tmem_slot() const { return base + 8 * 30; }
};
constexpr int kTmemSlotOffset = 8 * 30;
constexpr int kAbortOffset = 8 * 31;

struct Item {
    int s0, nseq, g; // sequences s0 .. s0 + nseq - 1 (rows of q), KV head
    int row, k0, k1; // block-table row, key range (k0 a multiple of the box)
    int part;        // which of each sequence's parts this is
    int scratch;     // INT8: scratch row of key 0
    __device__ int tiles() const { return (k1 - k0 + 127) >> 7; }
    __device__ bool tail() const { return ((k1 - k0) & 127) != 0; } // the last key tile runs past k1
};

// Entries [idx, end) of the item list, the next one fetched while the current one runs.
struct ItemIter {
    const int4 *items;
    int idx, end;
    int4 a0, a1;
    __device__ ItemIter(const int4 *items_, int from, int to) : items(items_), idx(from), end(to) { fetch(); }
    __device__ bool more() const { return idx < end; }
    __device__ void fetch()
    {
        if (idx < end) {
            a0 = ptx::ld_nc_v4_now(items + 2 * idx);
            a1 = ptx::ld_nc_v4_now(items + 2 * idx + 1);
        }
    }
    __device__ Item peek() const { return {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w}; }
    __device__ Item next(bool fetch_now = true)
    {
        const Item w = peek();
        ++idx;
        if (fetch_now)
            fetch();
        return w;
    }
};

// A lane's place in its singles: key tile j of n of the current one.
struct Lane {
    ItemIter it;
    Item w;
    int j, n;
    bool active;
    // `first`: item `from`, already at hand
    __device__ Lane(const int4 *items, int from, int to, const Item &first)
        : it(items, min(from + 1, to), to), w(first), j(0), n(first.tiles()),
          active(from < to)
    {
    }
    __device__ void next_item()
    {
        j = 0;
        active = it.more();
        if (active) {
            w = it.next();
            n = w.tiles();
        }
    }
    __device__ void step() // past the current key tile
    {
        if (++j == n)
            next_item();
    }
};

struct Waiter {
    volatile uint32_t *abort;
    __device__ bool operator()(uint32_t bar, uint32_t parity) const
    {
        if (ptx::mbar_try_wait(bar, parity))
            return true;
        if (*abort)
            return false;
        if (ptx::mbar_wait(bar, parity))
            return true;
        *abort = 1u;
        atomicOr(&g_shared_error, 1u);
        return false;
    }
};

// 16 INT8 codes (one 16-byte vector) times an fp16 scale, rounded to fp16 (as two 16-byte vectors),
// clamped to fp16's range.  A code is exact in fp16 (the bits 0x6400 | (x + 128) are 1152 + x), so the
// product is rounded once, by 2^-11 of it at most.  (By way of fp32, with int-to-float conversions at a
// fraction of the other instructions' rate, the copies for 16384 keys took 1.5 us longer.)
__device__ __forceinline__ void codes_to_f16(const uint4 &c, __half2 scale, uint4 &lo, uint4 &hi)
{
    const uint32_t u[4] = {c.x, c.y, c.z, c.w};
    const __half2 most = __half2half2(__ushort_as_half(0x7bff)), least = __hneg2(most);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t bits = ptx::prmt(u[i >> 1] ^ 0x80808080u, 0x64646464u, i & 1 ? 0x4342u : 0x4140u);
        const uint32_t code = ptx::sub_f16x2(bits, 0x64806480u);
        const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&code), scale);
        const __half2 y = __hmin2_nan(__hmax2_nan(x, least), most);
        w[i] = *reinterpret_cast<const uint32_t *>(&y);
    }
    lo = make_uint4(w[0], w[1], w[2], w[3]);
    hi = make_uint4(w[4], w[5], w[6], w[7]);
}

struct CodesParams {
    const int4 *tiles; // block-table row, first key, end of the keys, scratch row of the first key
    const int32_t *block_tables;
    const uint4 *k_codes, *v_codes;    // INT8 cache, 16 codes each
    const uint16_t *k_scale, *v_scale; // fp16 bits
    uint4 *k_out, *v_out;              // fp16 scratch [scratch_rows][num_kv_heads][D]
    const uint4 *q;                    // bf16
    uint4 *q_out;                      // fp16
    int32_t block_size, max_blocks, num_blocks, num_kv_heads, key_vecs, head_vecs;
    int32_t tile_ctas; // CTAs that convert keys; the others convert queries
    int64_t q_vecs;    // of 8 values
    uint64_t *go_word; // as ShParams'
    uint64_t go;
};

// What the products of the CTAs' lists read on an INT8 cache, in fp16: the shared prefixes' (and,
// where single sequences do not run apart, the other) keys and values (code * scale; 16 keys per
// CTA, K and V) and the queries.  Rows behind the last key and those of block ids outside the pool
// become zeros.  1 byte read and 2 written (to L2) per code; bound by its chain of three dependent
// loads: 11 us cold for 16384 keys of 4 heads, 17 MB read and 34 MB written.
constexpr int kCodesKeys = 16;
__global__ void __launch_bounds__(256) shared_codes_kernel(const CodesParams p)
{
    ptx::grid_dependency_wait();
    if (p.go_word && blockIdx.x == 0 && threadIdx.x == 0)
        ptx::st_release(p.go_word, p.go);
    ptx::launch_dependents();
    if ((int)blockIdx.x >= p.tile_ctas) {
        const int64_t i = (int64_t)((int)blockIdx.x - p.tile_ctas) * 256 + threadIdx.x;
        if (i >= p.q_vecs)
            return;
        const uint4 v = p.q[i];
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float lo = __uint_as_float(u[e] << 16), hi = __uint_as_float(u[e] & 0xffff0000u);
            w[e] = ptx::pack_f16(ptx::clamp_f16_nan(lo), ptx::clamp_f16_nan(hi));
        }
        p.q_out[i] = make_uint4(w[0], w[1], w[2], w[3]);
        return;
    }
    const int4 t = p.tiles[blockIdx.x / (128 / kCodesKeys)];
    const int first = t.y + (int)(blockIdx.x % (128 / kCodesKeys)) * kCodesKeys;
    const int out0 = t.w + first - t.y;
    const int bs = p.block_size;
    const int total = kCodesKeys * p.key_vecs;
    constexpr int kU = 2;
    for (int i0 = threadIdx.x; i0 < total; i0 += 256 * kU) {
        uint4 k[kU], v[kU];
        __half2 ks[kU], vs[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + 256 * u;
            k[u] = v[u] = make_uint4(0, 0, 0, 0);
            ks[u] = vs[u] = __half2half2(__ushort_as_half(0));
            const int key = first + i / p.key_vecs;
            if (i < total && key < t.z) {
                const int phys = p.block_tables[(size_t)t.x * p.max_blocks + key / bs];
                if ((uint32_t)phys < (uint32_t)p.num_blocks) {
                    const int vec = i % p.key_vecs, off = key & (bs - 1);
                    const size_t at = ((size_t)phys * bs + off) * p.key_vecs + vec;
                    const size_t sc = ((size_t)phys * p.num_kv_heads + vec / p.head_vecs) * bs + off;
                    k[u] = p.k_codes[at];
                    v[u] = p.v_codes[at];
                    ks[u] = __half2half2(__ushort_as_half(p.k_scale[sc]));
                    vs[u] = __half2half2(__ushort_as_half(p.v_scale[sc]));
                } else {
                    atomicOr(&g_shared_error, 2u);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + 256 * u;
            if (i < total) {
                const size_t at = 2 * ((size_t)out0 * p.key_vecs + i);
                uint4 lo, hi;
                codes_to_f16(k[u], ks[u], lo, hi);
                ptx::st_global_v8(p.k_out + at, lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w);
                codes_to_f16(v[u], vs[u], lo, hi);
                ptx::st_global_v8(p.v_out + at, lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w);
            }
        }
    }
}

template <int D, bool kInt8>
__global__ void __launch_bounds__(kThreads, 1)
    decode_shared_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q1,
                         const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const ShParams p)
{
    using L = ShLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *sgen = smem_raw + (sbase - raw);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const Bars bars{sbase + L::kBar};
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(sgen + L::kBar + kAbortOffset);
    const Waiter wait{abort_flag};
    const int G = p.group;
    const int P = p.rows_per_tile;

    // The launch after this one may be set up: a merge, which waits for this grid's end, or the parts of
    // single sequences, which wait for the word that this launch (INT8: the conversion) gives when the
    // launches before it have ended.
    if (kInt8)
        ptx::launch_dependents();
    if (warp >= 8 && lane == 0) {
        if (warp == kQWarp) {
            ptx::prefetch_tmap(&tm_q);
            ptx::prefetch_tmap(&tm_q1);
        } else if (warp == kKWarp) {
            ptx::prefetch_tmap(&tm_k);
        } else if (warp == kVWarp) {
            ptx::prefetch_tmap(&tm_v);
        }
    }
    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(bars.q_full(t), 1);
            ptx::mbar_init(bars.q_free(t), 1);
            ptx::mbar_init(bars.s_full(t), 1);
            ptx::mbar_init(bars.p_full(t), 4);
            ptx::mbar_init(bars.o_full(t), 1);
        }
        for (int s = 0; s < L::kKStages; ++s) {
            ptx::mbar_init(bars.k_full(s), 1);
            ptx::mbar_init(bars.k_free(s), 1);
        }
        for (int s = 0; s < L::kVStages; ++s) {
            ptx::mbar_init(bars.v_full(s), 1);
            ptx::mbar_init(bars.v_free(s), 1);
            ptx::mbar_init(bars.v_tail(s), 1);
        }
        *abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(bars.tmem_slot(), kTmemCols);
        ptx::tmem_relinquish();
    }
    // This CTA's pairs and its lanes' singles.  The K and V producers look up the rows of their first
    // key tiles while the barriers and the tensor memory are set up: three dependent loads (list,
    // item, block) would otherwise stand before the first tile, 0.6 us of a small call's 5.
    const int4 *record = p.cta_items + (size_t)blockIdx.x * (kSharedCtaInts / 4);
    const int4 span = __ldg(record);
    // cache row of sub-box `lane` of key tile j of w; one past the pool reads as zeros
    auto sub_row = [&](const Item &w, int j) -> int {
        const int key = w.k0 + j * 128 + lane * p.box_rows;
        if (lane * p.box_rows >= 128 || key >= w.k1)
            return kInt8 ? p.scratch_rows : p.num_blocks * p.block_size;
        if (kInt8)
            return w.scratch + key;
        const int phys = p.block_tables[(size_t)w.row * p.max_blocks + key / p.block_size];
        if ((uint32_t)phys >= (uint32_t)p.num_blocks) {
            atomicOr(&g_shared_error, 2u);
            return p.num_blocks * p.block_size;
        }
        return phys * p.block_size + (key & (p.block_size - 1));
    };
    // the first pair or else lane 0's first item, and lane 1's (zeros, no keys, where there is none)
    Item first{}, second{};
    int row0 = 0, row1 = 0;
    if (warp >= 8) {
        if (!kInt8) { // nothing but the plan is read before
            ptx::grid_dependency_wait();
            if (p.go_word && blockIdx.x == 0 && warp == kKWarp && lane == 0)
                ptx::st_release(p.go_word, p.go);
            ptx::launch_dependents();
        }
        const int4 a0 = __ldg(record + 2), a1 = __ldg(record + 3), b0 = __ldg(record + 4), b1 = __ldg(record + 5);
        first = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
        second = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
        if (warp == kKWarp || warp == kVWarp) {
            row0 = sub_row(first, 0);
            row1 = sub_row(second, 0);
        }
    }
    // lane 0's first item: the record has it if there are no pairs
    auto lane0_first = [&]() -> Item {
        if (span.x == span.y || span.y == span.z)
            return first;
        const int4 a0 = __ldg(p.items + 2 * span.y), a1 = __ldg(p.items + 2 * span.y + 1);
        return {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
    };
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sgen + L::kBar + kTmemSlotOffset);
    auto wwait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };

    if (warp >= 8) {
        ptx::reg_dealloc<kOtherRegs>();
        // INT8: this launch is set up while the scratch copies are written; nothing is read before they are
        if (kInt8 && warp != kMmaWarp)
            ptx::grid_dependency_wait();
        uint32_t nq0 = 0, nq1 = 0; // query loads of each tile so far
        // query rows of `w` (from sequence w.s0 + skip) into tile t, once the last score product that
        // read the buffer is complete
        auto load_q = [&](const Item &w, int t, int skip) -> bool {
            uint32_t &n = t == 0 ? nq0 : nq1;
            if (n > 0 && !wwait(bars.q_free(t), (n - 1) & 1))
                return false;
            ++n;
            if (lane == 0) {
                const bool one = w.nseq == 1;
                ptx::mbar_arrive_expect_tx(bars.q_full(t), (uint32_t)(L::kPanels * 128 * G * (one ? 1 : P)));
                for (int pp = 0; pp < L::kPanels; ++pp)
                    ptx::tma_load_3d(sbase + L::kQ + t * L::kTileBytes + pp * L::kPanelBytes, one ? &tm_q1 : &tm_q,
                                     bars.q_full(t), pp * 64, w.g * G, w.s0 + skip);
            }
            __syncwarp();
            return true;
        };
        if (warp == kQWarp) {
            // ------------------------------------------------------------ query producer
            bool ok = true;
            for (ItemIter it(p.items, span.x, span.y); ok && it.more();) {
                const Item w = it.next();
                ok = load_q(w, 0, 0) && load_q(w, 1, P);
            }
            // the lanes advance tile by tile together: loads in the order in which they are needed
            Lane l0(p.items, span.y, span.z, lane0_first()), l1(p.items, span.z, span.w, second);
            int at0 = 0, at1 = 0; // key tiles before each lane's next item
            while (ok && (l0.active || l1.active)) {
                const bool is0 = l0.active && (!l1.active || at0 <= at1);
                ok = load_q(is0 ? l0.w : l1.w, is0 ? 0 : 1, 0);
                if (is0) {
                    at0 += l0.n;
                    l0.next_item();
                } else {
                    at1 += l1.n;
                    l1.next_item();
                }
            }
        } else if (warp == kKWarp || warp == kVWarp) {
            // ------------------------------------------------------------ K and V producers
            const bool is_k = warp == kKWarp;
            const int nstages = is_k ? L::kKStages : L::kVStages;
            const uint32_t ring = sbase + (is_k ? L::kK : L::kV);
            const CUtensorMap *tm = is_k ? &tm_k : &tm_v;
            const int box_rows = p.box_rows;
            const int nsub = 128 / box_rows;
            int st = 0;
            uint32_t ph = 0; // times the ring has wrapped
            int X = 0;       // key tiles of pairs so far
            const uint64_t once = ptx::policy_evict_first(), keep = ptx::policy_evict_last();
            bool ok = true;
            // key tile j of w, whose sub-boxes lie at cache row `cur`, into the next slot
            auto load = [&](const Item &w, int j, int cur, uint64_t policy) {
                const uint32_t full = is_k ? bars.k_full(st) : bars.v_full(st);
                if (ph > 0 && !(ok = wwait(is_k ? bars.k_free(st) : bars.v_free(st), (ph - 1) & 1)))
                    return;
                const uint32_t dst = ring + st * L::kTileBytes;
                if (lane == 0)
                    ptx::mbar_arrive_expect_tx(full, (uint32_t)L::kTileBytes);
                __syncwarp();
                if (lane < nsub) {
                    for (int pp = 0; pp < L::kPanels; ++pp)
                        ptx::tma_load_3d_hint(dst + pp * L::kPanelBytes + lane * box_rows * 128, tm, full, pp * 64, w.g,
                                              cur, policy);
                }
                __syncwarp();
                if (!kInt8 && !is_k && (w.k1 - w.k0) - j * 128 < 128) {
                    // rows of keys past the range may hold anything (even NaN bit patterns): zeroed, so
                    // that a weight of 0 cannot turn them into NaN
                    if (!(ok = wwait(full, ph & 1)))
                        return;
                    uint8_t *tile = sgen + L::kV + st * L::kTileBytes;
                    const int first = w.k1 - w.k0 - j * 128;
                    const int chunks = (128 - first) * 8;
                    for (int pp = 0; pp < L::kPanels; ++pp)
                        for (int c = lane; c < chunks; c += 32)
                            *reinterpret_cast<uint4 *>(tile + pp * L::kPanelBytes + (first + (c >> 3)) * 128 +
                                                       (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        ptx::mbar_arrive(bars.v_tail(st));
                }
                if (++st == nstages) {
                    st = 0;
                    ++ph;
                }
            };
            for (ItemIter it(p.items, span.x, span.y); ok && it.more();) {
                const Item w = it.next();
                const int n = w.tiles();
                int next = X == 0 ? row0 : sub_row(w, 0);
                for (int j = 0; ok && j < n; ++j, ++X) {
                    const int cur = next;
                    if (j + 1 < n)
                        next = sub_row(w, j + 1);
                    load(w, j, cur, keep);
                }
            }
            Lane l0(p.items, span.y, span.z, lane0_first()), l1(p.items, span.z, span.w, second);
            int r0 = X == 0 ? row0 : l0.active ? sub_row(l0.w, 0) : 0, r1 = row1;
            auto advance = [&](Lane &l, int &r) { // this tile's load, the next one's row looked up before it
                const Item w = l.w;
                const int j = l.j, cur = r;
                l.step();
                if (l.active)
                    r = sub_row(l.w, l.j);
                load(w, j, cur, w.nseq == 1 ? once : keep);
            };
            while (ok && (l0.active || l1.active)) {
                if (l0.active)
                    advance(l0, r0);
                if (ok && l1.active)
                    advance(l1, r1);
            }
        } else if (warp == kMmaWarp) {
            // ------------------------------------------------------------ MMA issuer (converged warp)
            constexpr uint32_t idesc_s = kInt8 ? ptx::idesc_f16(128, 128, 0) : ptx::idesc_bf16(128, 128, 0);
            constexpr uint32_t idesc_o = kInt8 ? ptx::idesc_f16(128, D, 1) : ptx::idesc_bf16(128, D, 1);
            const uint32_t hi_k = (uint32_t)(ptx::smem_desc(0, 16, 1024, ptx::kSwizzle128B) >> 32);
            const uint32_t hi_v = (uint32_t)(ptx::smem_desc(0, L::kPanelBytes, 1024, ptx::kSwizzle128B) >> 32);
            auto desc = [](uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; };
            int ks = 0, kph = 0, vs = 0, vph = 0;
            uint32_t qpar = 0, ppar = 0; // bit t: parity of tile t's queries and weights consumed so far
            uint32_t tailpar = 0;        // bit s: parity of the tail tiles V slot s has held
            bool ok = true;
            auto issue_s = [&](int t) {
                uint32_t qa = (uint32_t)ptx::smem_desc(sbase + L::kQ + t * L::kTileBytes, 16, 1024, ptx::kSwizzle128B);
                uint32_t kb = (uint32_t)ptx::smem_desc(sbase + L::kK + ks * L::kTileBytes, 16, 1024, ptx::kSwizzle128B);
                asm volatile("" : "+r"(qa), "+r"(kb));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = ((kk >> 2) * L::kPanelBytes + (kk & 3) * 32) >> 4;
                    ptx::mma_bf16_ss_warp(tmem + t * 256, desc(qa + o, hi_k), desc(kb + o, hi_k), idesc_s, kk > 0);
                }
                ptx::mma_commit_warp(bars.s_full(t));
            };
            auto issue_pv = [&](int t, bool first) {
                uint32_t vb = (uint32_t)ptx::smem_desc(sbase + L::kV + vs * L::kTileBytes, L::kPanelBytes, 1024,
                                                       ptx::kSwizzle128B);
                asm volatile("" : "+r"(vb));
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    ptx::mma_bf16_ts_warp(tmem + t * 256 + 128, tmem + t * 256 + kk * 8,
                                          desc(vb + kk * (2048 >> 4), hi_v), idesc_o, (!first || kk > 0) ? 1u : 0u);
            };
            auto wait_q = [&](int t) {
                ok = ok && wwait(bars.q_full(t), (qpar >> t) & 1u);
                qpar ^= 1u << t;
            };
            auto wait_p = [&](int t) {
                ok = ok && wwait(bars.p_full(t), (ppar >> t) & 1u);
                ppar ^= 1u << t;
            };
            auto wait_k = [&]() {
                ok = ok && wwait(bars.k_full(ks), kph);
                ptx::tc_fence_after();
            };
            auto wait_v = [&](bool tail) {
                ok = ok && wwait(bars.v_full(vs), vph);
                if (!kInt8 && tail) { // (the scratch rows behind a context are zeros)
                    ok = ok && wwait(bars.v_tail(vs), (tailpar >> vs) & 1u);
                    tailpar ^= 1u << vs;
                }
                ptx::tc_fence_after();
            };
            auto pass_k = [&]() { // the K tile has been read by everything issued so far
                ptx::mma_commit_warp(bars.k_free(ks));
                if (++ks == L::kKStages) {
                    ks = 0;
                    kph ^= 1;
                }
            };
            auto pass_v = [&]() {
                ptx::mma_commit_warp(bars.v_free(vs));
                if (++vs == L::kVStages) {
                    vs = 0;
                    vph ^= 1;
                }
            };
            for (ItemIter it(p.items, span.x, span.y); ok && it.more();) {
                const Item w = it.next();
                const int n = w.tiles();
                const bool tail = w.tail();
                wait_q(0);
                wait_k();
                if (!ok)
                    break;
                issue_s(0);
                wait_q(1);
                if (!ok)
                    break;
                ptx::tc_fence_after();
                issue_s(1);
                if (n == 1) {
                    ptx::mma_commit_warp(bars.q_free(0));
                    ptx::mma_commit_warp(bars.q_free(1));
                }
                pass_k();
                for (int j = 0; j < n; ++j) {
                    const bool more = j + 1 < n;
#pragma unroll
                    for (int t = 0; t < 2; ++t) { // PV(t, j), then S(t, j + 1) into the same columns
                        wait_p(t);
                        if (t == 0)
                            wait_v(tail && !more);
                        else
                            ptx::tc_fence_after();
                        if (!ok)
                            break;
                        issue_pv(t, j == 0);
                        if (!more) {
                            ptx::mma_commit_warp(bars.o_full(t));
                        } else {
                            if (t == 0)
                                wait_k();
                            if (!ok)
                                break;
                            issue_s(t);
                            if (j + 2 == n)
                                ptx::mma_commit_warp(bars.q_free(t));
                        }
                    }
                    if (!ok)
                        break;
                    pass_v();
                    if (more)
                        pass_k();
                }
            }
            Lane l0(p.items, span.y, span.z, lane0_first()), l1(p.items, span.z, span.w, second);
            // score product of the lane's current key tile
            auto score = [&](const Lane &l, int t) {
                if (l.j == 0)
                    wait_q(t);
                wait_k();
                if (!ok)
                    return;
                issue_s(t);
                if (l.j + 1 == l.n)
                    ptx::mma_commit_warp(bars.q_free(t));
                pass_k();
            };
            // value product of the lane's current key tile, then the next one's scores
            auto step = [&](Lane &l, int t) {
                const bool last = l.j + 1 == l.n;
                wait_p(t);
                wait_v(last && l.w.tail());
                if (!ok)
                    return;
                issue_pv(t, l.j == 0);
                if (last)
                    ptx::mma_commit_warp(bars.o_full(t));
                pass_v();
                l.step();
                if (l.active)
                    score(l, t);
            };
            if (ok && l0.active)
                score(l0, 0);
            if (ok && l1.active)
                score(l1, 1);
            while (ok && (l0.active || l1.active)) {
                if (l0.active)
                    step(l0, 0);
                if (ok && l1.active)
                    step(l1, 1);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax + epilogue
        ptx::reg_alloc<kSoftmaxRegs>();
        const int t = warp >> 2;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const int rpos = r / G, rhead = r % G;
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_col = tmem + lane_addr + t * 256;
        const uint32_t o_col = s_col + 128;
        const float sl2 = p.scale_log2;
        constexpr float kBias = kInt8 ? 7.f : 0.f; // 2^(7 + kRescaleThreshold) stays in fp16
        uint32_t ns = 0, no = 0;
        bool ok = true;
        ItemIter items(p.items, span.x, span.y);
        bool single = false;
        while (ok) {
            if (!items.more()) {
                if (single)
                    break;
                single = true;
                items = t == 0 ? ItemIter(p.items, span.y, span.z) : ItemIter(p.items, span.z, span.w);
                continue;
            }
            const Item w = items.next(false);
            const int nseq = single ? w.nseq : t == 0 ? P : w.nseq - P;
            const int n = w.tiles();
            const bool row_valid = r < G * nseq;
            const bool warp_valid = quarter * 32 < G * nseq;
            const int seq = w.s0 + (single ? 0 : t * P) + rpos;
            // first slot and number of parts of this row's sequence (an item's sequences may differ: one
            // whose context ends with the prefix has no suffix part)
            const int2 sp = row_valid ? __ldg(p.seq_parts + seq) : make_int2(0, 1);
            float m_ref = -INFINITY, l_sum = 0.f;
            for (int j = 0; j < n; ++j) {
                if (!(ok = wwait(bars.s_full(t), ns & 1)))
                    break;
                ns ^= 1;
                if (warp_valid) {
                    ptx::tc_fence_after();
                    const int lim = w.k1 - w.k0 - j * 128; // keys of this tile (128 or more: all)
                    uint32_t sr[128];
                    float mx;
                    if (lim < 128) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            ptx::tmem_ld32(s_col + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * q]));
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 128; ++c)
                            sr[c] = c < lim ? sr[c] : __float_as_uint(-INFINITY);
                        float m8[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            m8[i] = ptx::max3(__uint_as_float(sr[16 * i]), __uint_as_float(sr[16 * i + 1]),
                                              __uint_as_float(sr[16 * i + 2]));
#pragma unroll
                        for (int c = 3; c < 16; c += 2)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                m8[i] = c + 1 < 16 ? ptx::max3(m8[i], __uint_as_float(sr[16 * i + c]),
                                                               __uint_as_float(sr[16 * i + c + 1]))
                                                   : fmaxf(m8[i], __uint_as_float(sr[16 * i + c]));
                        mx = fmaxf(fmaxf(ptx::max3(m8[0], m8[1], m8[2]), ptx::max3(m8[3], m8[4], m8[5])),
                                   fmaxf(m8[6], m8[7]));
                    } else {
                        float m4[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            m4[q] = ptx::tmem_ld32_max(s_col + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * q]));
                        ptx::tmem_wait_ld();
                        mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    }
                    const float mt = mx * sl2;
                    float alpha = 1.f;
                    bool rescale = false;
                    if (row_valid && (mt > m_ref + kRescaleThreshold || (m_ref == -INFINITY && mt != -INFINITY))) {
                        const float m_new = fmaxf(m_ref, mt);
                        alpha = ptx::ex2(m_ref - m_new); // 0 on the first tile
                        rescale = j > 0;
                        l_sum *= alpha;
                        m_ref = m_new;
                    }
                    // P = 2^(s * scale * log2 e - m) written over S as pairs of the values' own type: bf16 (weights
                    // in [0, 2^8], each rounded by 2^-8 of it at most), or fp16 with 2^kBias times the weight
                    // (2^-11; the weights that fp16 cannot hold, below 2^-31 of the largest, are lost: 2^-16 of
                    // the sum over 32768 keys).  The row sum stays fp32.
                    const uint64_t sl2x2 = ptx::f2(sl2, sl2);
                    const float negm = m_ref == -INFINITY ? 0.f : kBias - m_ref;
                    const uint64_t negm2 = ptx::f2(negm, negm);
                    uint64_t sum2[4] = {ptx::f2(0.f, 0.f), ptx::f2(0.f, 0.f), ptx::f2(0.f, 0.f), ptx::f2(0.f, 0.f)};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[32];
#pragma unroll
                        for (int c = 64 * h; c < 64 * h + 64; c += 2) {
                            float x0, x1;
                            ptx::f2_split(ptx::f2_fma(ptx::f2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])),
                                                      sl2x2, negm2),
                                          x0, x1);
                            const float e0 = ptx::ex2(x0), e1 = ptx::ex2(x1); // masked columns: 2^-inf = 0
                            sum2[(c >> 1) & 3] = ptx::f2_add(sum2[(c >> 1) & 3], ptx::f2(e0, e1));
                            pk[(c >> 1) & 31] = kInt8 ? ptx::pack_f16(e0, e1) : ptx::pack_bf16(e0, e1);
                        }
                        ptx::tmem_st32(s_col + 32 * h, pk);
                    }
                    float s0, s1, s2, s3, s4, s5, s6, s7;
                    ptx::f2_split(sum2[0], s0, s1);
                    ptx::f2_split(sum2[1], s2, s3);
                    ptx::f2_split(sum2[2], s4, s5);
                    ptx::f2_split(sum2[3], s6, s7);
                    l_sum += ((s0 + s1) + (s2 + s3)) + ((s4 + s5) + (s6 + s7));
                    // O is stable here: PV(j-1) completed before S(j) did (in-order products), and PV(j)
                    // waits for the arrival below
                    if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
                        for (int cc = 0; cc < D / 32; ++cc) {
                            uint32_t o[32];
                            ptx::tmem_ld32(o_col + cc * 32, o);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                            ptx::tmem_st32(o_col + cc * 32, o);
                        }
                    }
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                }
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(bars.p_full(t));
            }
            items.fetch();
            if (!ok)
                break;
            // epilogue: O / l to the output (a sequence's only part) or, in fp32 with its log2-sum-exp,
            // to the workspace
            if (!(ok = wwait(bars.o_full(t), no & 1)))
                break;
            no ^= 1;
            if (!warp_valid)
                continue;
            ptx::tc_fence_after();
            // (a sum of NaN goes on, to the output and to the merge)
            const float inv = (row_valid && l_sum != 0.f) ? 1.f / l_sum : 0.f;
            const size_t head = (size_t)w.g * G + rhead;
            const bool partial = sp.y > 1;
            const size_t slot = (size_t)sp.x + w.part;
            float *po = p.part_o + (slot * p.num_heads + head) * D;
            if (partial && !*abort_flag)
                p.part_lse[slot * p.num_heads + head] = l_sum != 0.f ? m_ref - kBias + __log2f(l_sum) : -INFINITY;
            __nv_bfloat16 *orow = p.out + ((size_t)seq * p.num_heads + head) * D;
            uint32_t o[D / 32][32];
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc)
                ptx::tmem_ld32(o_col + cc * 32, o[cc]);
            ptx::tmem_wait_ld();
            if (row_valid && !*abort_flag) {
                if (partial) {
#pragma unroll
                    for (int cc = 0; cc < D / 32; ++cc)
#pragma unroll
                        for (int c = 0; c < 32; c += 8) {
                            uint32_t x[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                x[i] = __float_as_uint(__uint_as_float(o[cc][c + i]) * inv);
                            ptx::st_global_v8(po + cc * 32 + c, x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]);
                        }
                } else {
#pragma unroll
                    for (int cc = 0; cc < D / 32; ++cc)
#pragma unroll
                        for (int c = 0; c < 32; c += 8) {
                            uint32_t x[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                x[i] = ptx::pack_bf16(__uint_as_float(o[cc][c + 2 * i]) * inv,
                                                      __uint_as_float(o[cc][c + 2 * i + 1]) * inv);
                            *reinterpret_cast<uint4 *>(orow + cc * 32 + c) = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                }
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // A wait ran out: copies and products issued since may be in flight.  They end within microseconds;
        // shared and tensor memory are kept for 20 ms.  (Counted, to wait on their barriers, they cost
        // every call 0.3 to 1 us.)
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 20000000u) {
        }
    }
    if (warp == kMmaWarp) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

// out[b][h] = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M) over the parts of sequence b: none
// (empty context) writes zeros, one was written by its work item.  A part whose sum is NaN has the
// log-sum-exp NaN, and so has the output.  D/32 values per lane, kBatch
// parts' loads in flight; a (sequence, head)'s parts are shared out in order to kSplit warps (of
// the four or eight of a block), whose sums meet in shared memory in warp order.  Bound by the
// latency of the loads: 65 parts in one warp took 18 us, in eight 3.
template <int D, int kSplit>
__global__ void __launch_bounds__(kSplit == 8 ? 256 : 128)
    shared_combine_kernel(const float *part_o, const float *part_lse, const int2 *seq_parts, __nv_bfloat16 *out,
                          int num_heads, uint64_t *go_word)
{
    constexpr int E = D / 32;
    constexpr int kBatch = 8;
    constexpr int kHeads = kSplit == 1 ? 4 : 1; // heads per block
    const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y * kHeads + (kSplit == 1 ? warp : 0);
    const int2 sp = __ldg(seq_parts + b); // the plan's, written long before this launch's predecessor
    ptx::launch_dependents();
    ptx::grid_dependency_wait();          // the parts are complete and visible
    if (go_word && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *go_word = 0; // taken back: a replayed call gives the same one again
    if (sp.y == 1 || h >= num_heads)
        return;
    const int per = kSplit == 1 ? sp.y : (sp.y + kSplit - 1) / kSplit;
    const int from = kSplit == 1 ? 0 : min(warp * per, sp.y), n = min(sp.y - from, per);
    const float *lse = part_lse + (size_t)sp.x * num_heads + h;
    const float *po = part_o + (((size_t)sp.x + from) * num_heads + h) * D + lane * E;
    const size_t o_stride = (size_t)num_heads * D;
    float M = -INFINITY;
    for (int s = lane; s < sp.y; s += 32)
        M = fmaxf(M, lse[(size_t)s * num_heads]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    lse += (size_t)from * num_heads;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] = 0.f;
    float W = 0.f;
    for (int s = 0; s < n; s += kBatch) {
        float l[kBatch];
        float o[kBatch][E];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (s + i < n) {
                l[i] = lse[(size_t)(s + i) * num_heads];
                if constexpr (E == 4)
                    *reinterpret_cast<float4 *>(o[i]) = *reinterpret_cast<const float4 *>(po + (size_t)(s + i) * o_stride);
                else
                    *reinterpret_cast<float2 *>(o[i]) = *reinterpret_cast<const float2 *>(po + (size_t)(s + i) * o_stride);
            }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (s + i < n) {
                const float w = l[i] == -INFINITY ? 0.f : ptx::ex2(l[i] - M);
                W += w;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    acc[e] += w * o[i][e];
            }
    }
    if constexpr (kSplit > 1) {
        __shared__ float sums[kSplit][D + 1]; // a warp's D sums, then its weight
#pragma unroll
        for (int e = 0; e < E; ++e)
            sums[warp][lane * E + e] = acc[e];
        if (lane == 0)
            sums[warp][D] = W;
        __syncthreads();
        if (warp != 0)
            return;
        W = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = 0.f;
#pragma unroll
        for (int s = 0; s < kSplit; ++s) {
            W += sums[s][D];
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] += sums[s][lane * E + e];
        }
    }
    const float inv = W != 0.f ? 1.f / W : 0.f; // (NaN of a part: NaN)
    uint32_t x[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e)
        x[e] = ptx::pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    uint32_t *dst = reinterpret_cast<uint32_t *>(out + ((size_t)b * num_heads + h) * D + lane * E);
    if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(x[0], x[1]);
    else
        dst[0] = x[0];
}

// One KV head's rows of a bf16 cache in 128-byte swizzled panels of 64.
template <int D>
int encode_cache(CUtensorMap *m, const void *cache, int num_kv_heads, uint64_t rows, uint32_t box_rows, const char *what)
{
    return encode_tmap_3d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cache, D, num_kv_heads, rows, (uint64_t)D * 2,
                          (uint64_t)num_kv_heads * D * 2, 64, 1, box_rows, CU_TENSOR_MAP_SWIZZLE_128B, what);
}

// INT8: the scratch copies for the CTAs' lists.
int launch_codes(const SharedArgs &a, uint64_t go, cudaStream_t stream)
{
    const pa_dims &d = a.dims;
    const size_t half = (size_t)a.num_scratch_tiles * 128 * d.num_kv_heads * d.head_dim * 2;
    CodesParams c{};
    c.tiles = reinterpret_cast<const int4 *>(a.scratch_tiles);
    c.block_tables = a.block_tables;
    c.k_codes = static_cast<const uint4 *>(a.k_cache);
    c.v_codes = static_cast<const uint4 *>(a.v_cache);
    c.k_scale = static_cast<const uint16_t *>(a.k_scale);
    c.v_scale = static_cast<const uint16_t *>(a.v_scale);
    c.k_out = static_cast<uint4 *>(a.scratch);
    c.v_out = reinterpret_cast<uint4 *>(static_cast<char *>(a.scratch) + half);
    c.q = static_cast<const uint4 *>(a.q);
    c.q_out = reinterpret_cast<uint4 *>(static_cast<char *>(a.scratch) + 2 * half);
    c.block_size = d.block_size;
    c.max_blocks = a.max_blocks_per_seq;
    c.num_blocks = d.num_blocks;
    c.num_kv_heads = d.num_kv_heads;
    c.head_vecs = d.head_dim / 16;
    c.key_vecs = d.num_kv_heads * c.head_vecs;
    c.tile_ctas = a.num_scratch_tiles * (128 / kCodesKeys);
    c.q_vecs = (int64_t)a.num_seqs * d.num_heads * d.head_dim / 8;
    c.go_word = a.go_word;
    c.go = go;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(c.tile_ctas + (c.q_vecs + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, shared_codes_kernel, c);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(PA_ERR_CUDA, "shared decode code conversion launch: %s", cudaGetErrorString(e));
    }
    return PA_OK;
}

// Items (sequence, key range, partial slot) of single sequences through the decode kernels; with a
// go_word beside the shared parts' products, on the SMs that those leave.  (INT8, beside
// the conversion instead, with the products after both: 64 x 16384 took 75 us, not 50; these parts
// are long and few, and the products waited for them.)
int launch_singles(const SharedArgs &a, const int32_t *items, int32_t num_items, uint64_t go, cudaStream_t stream)
{
    DecodeArgs s{};
    s.dims = a.dims;
    s.q = a.q;
    s.k_cache = a.k_cache;
    s.v_cache = a.v_cache;
    s.k_scale = a.k_scale;
    s.v_scale = a.v_scale;
    s.block_tables = a.block_tables;
    s.items = items;
    s.out = a.out;
    s.part_o = a.part_o;
    s.part_lse = a.part_lse;
    s.scale = a.scale;
    s.num_seqs = a.num_seqs;
    s.num_items = num_items;
    s.max_blocks_per_seq = a.max_blocks_per_seq;
    s.table_rows = a.table_rows;
    s.go_word = a.go_word;
    s.go = go;
    int sms = 0;
    if (int rc = sm_count(&sms))
        return rc;
    // then eight warps each instead of four, which shortens the chain of steps: 8 contexts of 300 tokens
    // 6.2 us instead of 6.6, of 808 9.2 instead of 11.0, INT8 10.6 instead of 13.8; with more items than
    // SMs the wider ones have no room beside one another
    s.few = (int64_t)num_items * a.dims.num_kv_heads <= sms - (a.go_word ? a.num_ctas : 0);
    return a.k_scale ? launch_decode_int8(s, stream) : launch_decode(s, stream);
}

template <int D, bool kInt8>
int launch(const SharedArgs &a, cudaStream_t stream)
{
    using L = ShLayout<D>;
    if (int rc = ensure_smem<decode_shared_kernel<D, kInt8>>(L::kSmemBytes, "shared decode"))
        return rc;
    static std::atomic<int> launch_regs{0};
    int nreg = launch_regs.load(std::memory_order_acquire);
    if (nreg == 0) {
        cudaFuncAttributes fa{};
        const cudaError_t e = cudaFuncGetAttributes(&fa, decode_shared_kernel<D, kInt8>);
        if (e != cudaSuccess)
            return fail(PA_ERR_CUDA, "shared decode kernel attributes: %s", cudaGetErrorString(e));
        launch_regs.store(nreg = fa.numRegs, std::memory_order_release);
    }
    if (nreg != kLaunchRegs)
        return fail(PA_ERR_UNSUPPORTED, "shared decode kernel built with %d registers per thread, needs %d", nreg,
                    kLaunchRegs);
    const pa_dims &d = a.dims;
    const int G = d.num_heads / d.num_kv_heads;
    // this call's word: another for each call (multiples of an odd number), none that a workspace's first
    // contents are likely to hold
    static std::atomic<uint64_t> calls{0};
    const uint64_t go = a.go_word ? (calls.fetch_add(1, std::memory_order_relaxed) + 1) * 0x9e3779b97f4a7c15ull : 0;
    if (a.num_items > 0) {
        if (kInt8)
            if (int rc = launch_codes(a, go, stream))
                return rc;
        const uint32_t box_rows = !kInt8 && d.block_size < kBoxRows ? (uint32_t)d.block_size : (uint32_t)kBoxRows;
        // INT8: the products read the scratch cache
        const size_t half = (size_t)a.num_scratch_tiles * 128 * d.num_kv_heads * D * 2;
        const void *q = kInt8 ? static_cast<const char *>(a.scratch) + 2 * half : a.q;
        const void *k_cache = kInt8 ? a.scratch : a.k_cache;
        const void *v_cache = kInt8 ? static_cast<const char *>(a.scratch) + half : a.v_cache;
        const uint64_t rows = kInt8 ? (uint64_t)a.num_scratch_tiles * 128 : (uint64_t)d.num_blocks * d.block_size;
        constexpr CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16; // (copies bits: fp16 as well)
        constexpr CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
        const uint64_t qs = (uint64_t)d.num_heads * D * 2;
        CUtensorMap tq, tq1{}, tk, tv;
        int rc;
        if ((rc = encode_tmap_3d(&tq, bf16, q, D, d.num_heads, (uint64_t)a.num_seqs, (uint64_t)D * 2, qs, 64,
                                 (uint32_t)G, (uint32_t)a.rows_per_tile, sw, "q")) != PA_OK ||
            (a.num_single_items == 0 && // (else the lists have no parts of single sequences)
             (rc = encode_tmap_3d(&tq1, bf16, q, D, d.num_heads, (uint64_t)a.num_seqs, (uint64_t)D * 2, qs, 64,
                                  (uint32_t)G, 1, sw, "q")) != PA_OK) ||
            (rc = encode_cache<D>(&tk, k_cache, d.num_kv_heads, rows, box_rows, "k_cache")) != PA_OK ||
            (rc = encode_cache<D>(&tv, v_cache, d.num_kv_heads, rows, box_rows, "v_cache")) != PA_OK)
            return rc;
        ShParams p{};
        p.scratch_rows = kInt8 ? a.num_scratch_tiles * 128 : 0;
        p.items = reinterpret_cast<const int4 *>(a.items);
        p.cta_items = reinterpret_cast<const int4 *>(a.cta_items);
        p.seq_parts = reinterpret_cast<const int2 *>(a.seq_parts);
        p.block_tables = a.block_tables;
        p.out = static_cast<__nv_bfloat16 *>(a.out);
        p.part_o = a.part_o;
        p.part_lse = a.part_lse;
        p.scale_log2 = a.scale * kLog2e;
        p.num_heads = d.num_heads;
        p.group = G;
        p.rows_per_tile = a.rows_per_tile;
        p.block_size = d.block_size;
        p.box_rows = (int32_t)box_rows;
        p.max_blocks = a.max_blocks_per_seq;
        p.num_blocks = d.num_blocks;
        p.go_word = kInt8 ? nullptr : a.go_word;
        p.go = go;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)a.num_ctas);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = L::kSmemBytes;
        cfg.stream = stream;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_shared_kernel<D, kInt8>, tq, tq1, tk, tv, p);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return fail(PA_ERR_CUDA, "shared decode launch: %s", cudaGetErrorString(e));
        }
    }
    if (a.num_single_items > 0)
        if (int rc = launch_singles(a, a.single_items, a.num_single_items, go, stream))
            return rc;
    if (!a.merge && !a.go_word)
        return PA_OK;
    // Programmatic launch: the merge's blocks are set up while the parts still run and wait
    // inside for the end of that grid.  Without a grid before it, it waits for nothing.  (One
    // cooperative launch whose CTAs met before merging took 3 us longer on a batch of 8 x 300
    // tokens and 15 us longer on 256 x 33300.)
    cudaLaunchConfig_t cfg{};
    // several warps per (sequence, head) where there are few of them: with 1792 (9 parts each) four made
    // the merge 8.8 us, not 6.1; with 224 (65 parts), eight made a call 16.7 us, not 28
    const int64_t merges = (int64_t)a.num_seqs * d.num_heads;
    const int split = a.max_parts <= 8 || merges > 1024 ? 1 : a.max_parts <= 32 ? 4 : 8;
    cfg.gridDim = dim3((unsigned)a.num_seqs, (unsigned)(split == 1 ? (d.num_heads + 3) / 4 : d.num_heads));
    cfg.blockDim = dim3(split == 8 ? 256 : 128);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    auto combine = split == 1   ? shared_combine_kernel<D, 1>
                   : split == 4 ? shared_combine_kernel<D, 4>
                                : shared_combine_kernel<D, 8>;
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, combine, (const float *)a.part_o, (const float *)a.part_lse,
                           reinterpret_cast<const int2 *>(a.seq_parts), static_cast<__nv_bfloat16 *>(a.out),
                           (int)d.num_heads, a.go_word);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(PA_ERR_CUDA, "shared decode merge launch: %s", cudaGetErrorString(e));
    }
    return PA_OK;
}

} // namespace

int launch_decode_shared(const SharedArgs &a, void *stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.direct_items)
        return launch_singles(a, a.direct_items, a.num_seqs, 0, s);
    if (a.k_scale)
        return a.dims.head_dim == 128 ? launch<128, true>(a, s) : launch<64, true>(a, s);
    return a.dims.head_dim == 128 ? launch<128, false>(a, s) : launch<64, false>(a, s);
}

int read_shared_error(uint32_t *code)
{
    uint32_t v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_shared_error, sizeof v);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbol(g_shared_error, &zero, sizeof zero);
    if (e != cudaSuccess)
        return fail(PA_ERR_CUDA, "reading shared-decode error word: %s", cudaGetErrorString(e));
    *code |= (v & 3u) << 5;
    return PA_OK;
}

} // namespace pa

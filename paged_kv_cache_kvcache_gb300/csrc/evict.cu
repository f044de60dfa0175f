// Rows of a page pool shrink to a budget of tokens: what the attention weighed least goes.
//
// Of a row of n > budget tokens stay the first `first`, the last `last` and, of the others, those of the largest
// totals: total_j = sum over the KV heads of score[g][j] (pa_decode_weights keeps the scores), of equal ones the
// lower index.  What stays moves together in order: token kept[k] goes to place k, its keys and values in all
// layers, its scores, and the pages behind place budget - 1 lose an entry.
//
// Sources (page title, section): "手搓 vLLM 推理引擎", Step 2 (BlockManager: block tables, reference counts);
// "vLLM / SGLang 面试源码深挖", section 4 (shared blocks must not be written).
//
// Two launches.  The choice: one CTA per row, totals once into shared memory as ordered integers, the smallest
// one that stays by three rounds of counting (11, 11 and 10 bits), then ballots give every kept token its place;
// bound by latency (a row of 2048 tokens of 8 heads 8 us: the look-ups of row, length and scores 3, two or three
// rounds of counting 2, the places 2).  The move: a CTA takes a slice of the token rows of one (row,
// layer, K or V) and walks the places upwards: as kept[k] >= k, a batch's places lie below the next
// batch's sources, so it moves in place, the next batch's loads in flight while this one's are stored.  Bound by
// HBM (each moved token read and written once: 16 rows of 4096 to 2048 tokens in 28 layers 600 us, 6.3 TB/s; a row's
// places and tokens are looked up 1024 at a time, which took it from 1013).  The last CTA of a row changes its table, length and counts.
// The call is all or nothing: the choice checks every row, and the move looks at all verdicts first.
#include <algorithm>
#include <type_traits>

#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace pa {

__device__ uint32_t g_evict_error; // bit 0: a malformed call or state

namespace {

constexpr int kChooseThreads = 1024;
constexpr int kChooseWarps = kChooseThreads / 32;
constexpr int kBins = 2048;
constexpr int kKeysInSmem = 49152;
constexpr int kUnsure = 1024; // totals that total_exact forms without all the others
constexpr int kMoveThreads = 256;
constexpr int kVecs = 4; // 16-byte vectors per thread and batch
constexpr int kBatchTokens = kMoveThreads * kVecs; // at most: of one vector, value or scale each

struct EvictParams {
    int32_t *tables, *context_lens, *refs;
    const int32_t *rows;
    int32_t n, num_rows, max_blocks, num_blocks, block_size, num_kv_heads;
    const float *scores;
    float *scores_out;
    int32_t budget, first, last;
    int32_t *kept;   // [n][budget]
    int32_t *state;  // [n] length of the row, -1: refused
    int32_t *moved;  // [n] first place whose token moves
    uint32_t *done;  // [n] units of the move that are through
    int32_t keys;    // places of the key buffer in shared memory
};

// Larger totals have larger keys; NaN is below every number.
__device__ __forceinline__ uint32_t order(float x)
{
    if (x != x)
        return 0u;
    const uint32_t u = __float_as_uint(x + 0.f); // (-0 is 0)
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The exact sum of a token's scores, rounded to fp32: a fixed-point sum of 320 bits in units of 2^-149 (out of line, for
// the few tokens whose sum totals_of is not sure of).
__device__ __noinline__ float total_exact(const float *at, int heads, int64_t pitch)
{
    constexpr int kWords = 5; // 2^31 scores below 2^128, and a sign
    uint64_t sum[kWords] = {};
    bool up = false, down = false; // an infinity
    for (int h = 0; h < heads; ++h) {
        const uint32_t u = __float_as_uint(at[h * pitch]), ex = u >> 23 & 255u;
        const bool minus = u >> 31;
        if (ex == 255u) {
            if (u & 0x7fffffu)
                return __uint_as_float(0x7fffffffu); // NaN
            (minus ? down : up) = true;
            continue;
        }
        const uint64_t m = (u & 0x7fffffu) | (ex ? 0x800000u : 0u);
        const int shift = ex ? (int)ex - 1 : 0, word = shift >> 6, off = shift & 63;
        const uint64_t lo = m << off, hi = off > 40 ? m >> (64 - off) : 0;
        uint64_t carry = minus; // (minus x: its complement and 1)
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const uint64_t part = w == word ? lo : w == word + 1 ? hi : 0;
            const uint64_t add = minus ? ~part : part;
            const uint64_t a = sum[w] + add, b = a + carry;
            carry = (a < add) | (b < a);
            sum[w] = b;
        }
    }
    if (up || down)
        return up && down ? __uint_as_float(0x7fffffffu) : up ? INFINITY : -INFINITY;
    const bool minus = sum[kWords - 1] >> 63;
    uint64_t carry = minus;
    int top = -1; // its highest bit
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        if (minus) {
            sum[w] = ~sum[w] + carry;
            carry = carry && sum[w] == 0;
        }
        if (sum[w])
            top = 64 * w + 63 - __clzll((long long)sum[w]);
    }
    uint32_t bits;
    if (top < 24) { // (all of it; 0 where there is none)
        bits = (uint32_t)sum[0];
    } else {
        const int cut = top - 23; // bits below the 24 that stay
        uint64_t below = 0, head = 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const int at_bit = cut - 64 * w; // of this word
            if (at_bit >= 64)
                below |= sum[w] != 0 && at_bit > 64 ? 1u : 0u;
            if (at_bit > 0 && at_bit < 64)
                head |= sum[w] >> at_bit;
            else if (at_bit <= 0 && at_bit > -64)
                head |= sum[w] << -at_bit;
        }
        bool half = false;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const int bit = cut - 1 - 64 * w; // the first that goes
            if (bit >= 0 && bit < 64) {
                half = sum[w] >> bit & 1u;
                below |= sum[w] & ((1ull << bit) - 1ull);
            }
        }
        const uint32_t m = (uint32_t)head & 0xffffffu;
        // the leading bit counts one in the exponent; rounding up carries into it
        bits = m + ((uint32_t)cut << 23) + (half && (below || (m & 1u)) ? 1u : 0u);
        bits = cut > 253 || bits > 0x7f800000u ? 0x7f800000u : bits;
    }
    return __uint_as_float(bits | (minus ? 0x80000000u : 0u));
}

// The sum over the heads, rounded to fp32, of kTokens tokens, `step` apart and before `left`, with kHeads of each one's
// scores in flight together (one: there is no other): out(o, key, sure).  s + e is carried with the errors of e's own sums
// alone (two-sum; fp64 adds run at 1/64 of fp32's rate and took longer than the reads).  Of scores that are not negative,
// as weights are, those are below heads^2 2^-48 of the sum, and none where every score is above heads 2^-24 of it (the
// errors are multiples of its last bit then, zeros aside).  So a sum is sure if both ends of twice that range round to it, or if there is
// no error; others (next to the middle of two numbers, with a negative score, past fp32's range) are total_exact's.
template <int kTokens, int kHeads, class Out>
__device__ __forceinline__ void totals_of(const float *at, int left, int step, int heads, int64_t pitch, Out out)
{
    float s[kTokens], e[kTokens];
    uint32_t signs[kTokens], least[kTokens];
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
        s[t] = e[t] = 0.f, signs[t] = 0u, least[t] = 0xffffffffu;
    for (int h0 = 0; h0 < heads; h0 += kHeads) {
        float x[kTokens][kHeads];
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
#pragma unroll
            for (int t = 0; t < kTokens; ++t)
                x[t][h] = h0 + h < heads && t * step < left ? at[(h0 + h) * pitch + t * step] : 0.f;
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
#pragma unroll
            for (int t = 0; t < kTokens; ++t) {
                if constexpr (kHeads == 1) {
                    s[t] = x[t][h];
                } else {
                    const float u = __fadd_rn(s[t], x[t][h]);
                    const float b = __fsub_rn(u, s[t]);
                    e[t] = __fadd_rn(e[t], __fadd_rn(__fsub_rn(s[t], __fsub_rn(u, b)), __fsub_rn(x[t][h], b)));
                    s[t] = u;
                    signs[t] |= __float_as_uint(x[t][h]);
                    least[t] = min(least[t], __float_as_uint(x[t][h]) - 1u); // (0 is none)
                }
            }
    }
    const float range = (float)heads * (float)heads * 0x1p-47f, above = (float)heads * 0x1p-23f;
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
        if (t * step < left) {
            if constexpr (kHeads == 1) {
                out(t * step, order(s[t]), true);
            } else {
                const float d = __fmul_rn(s[t], range);
                const float r = __fadd_rn(s[t], __fadd_rn(e[t], d)), r0 = __fadd_rn(s[t], __fsub_rn(e[t], d));
                const bool exact = __uint_as_float(least[t]) > __fmul_rn(s[t], above) && s[t] <= 0x1p+127f;
                out(t * step, order(exact ? __fadd_rn(s[t], e[t]) : r), (int)signs[t] >= 0 && (r == r0 || exact));
            }
        }
}

// The same out of line, for rows whose keys do not fit shared memory.
__device__ __noinline__ uint32_t total_far(const float *at, int heads, int64_t pitch)
{
    uint32_t key;
    totals_of<1, 8>(at, 1, 1, heads, pitch,
                    [&](int, uint32_t x, bool sure) { key = sure ? x : order(total_exact(at, heads, pitch)); });
    return key;
}

// Keys of the n places that the list names, from the exact sums; of all from begin to end if there are more than it holds.
__device__ __noinline__ void mend_keys(uint32_t *keys, const int *list, int n, const float *scores, int heads, int64_t pitch,
                                       int begin, int end)
{
    const bool all = n > kUnsure;
    for (int x = threadIdx.x; x < (all ? end - begin : n); x += kChooseThreads) {
        const int j = all ? begin + x : list[x];
        keys[j] = order(total_exact(scores + j, heads, pitch));
    }
}

// exclusive sum over the CTA's threads; *sum: all
__device__ __forceinline__ int scan_cta(int v, int *warps, int *sum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads(); // warps[] may still be read
    if (lane == 31)
        warps[warp] = x;
    __syncthreads();
    int w = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o)
            w += y;
    }
    *sum = __shfl_sync(0xffffffffu, w, 31);
    const int before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    return before + x - v;
}

__global__ void __launch_bounds__(kChooseThreads) evict_choose_kernel(const EvictParams p)
{
    extern __shared__ uint32_t keys[];
    __shared__ int hist[kBins];
    __shared__ int warps[kChooseWarps], warps2[kChooseWarps];
    __shared__ int digit, above, equals, lowest, unsure;
    __shared__ int unsure_at[kUnsure];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bs = p.block_size, room = p.max_blocks * bs, budget = p.budget;
    const int row = p.rows[i];
    const bool in = (uint32_t)row < (uint32_t)p.num_rows;
    const int n = in ? p.context_lens[row] : -1;
    bool bad = n < 0 || n > room;
    for (int x = tid; x < i; x += kChooseThreads) // a row once
        bad = bad || p.rows[x] == row;
    int32_t *kept = p.kept + (int64_t)i * budget;
    if (tid == 0)
        unsure = 0;
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            p.state[i] = -1;
            atomicOr(&g_evict_error, 1u);
        }
        return;
    }
    if (n <= budget) {
        for (int k = tid; k < budget; k += kChooseThreads)
            kept[k] = k < n ? k : -1;
        if (tid == 0) {
            p.state[i] = n;
            p.moved[i] = n;
            p.done[i] = 0u;
        }
        return;
    }

    // the row's first pages, looked up while the totals are formed
    const int32_t *table = p.tables + (int64_t)row * p.max_blocks;
    const int pages = (n + bs - 1) / bs;
    const int page0 = tid < pages ? table[tid] : 0;
    const float *scores = p.scores + (int64_t)row * p.num_kv_heads * room;
    const bool stored = n <= p.keys;
    const int begin = p.first, end = n - p.last; // of those to choose from
    if (stored) {
        // eight or more scores of a thread in flight together
        auto form = [&](auto tokens, auto heads) {
            for (int j = begin + tid; j < end; j += tokens.value * kChooseThreads)
                totals_of<tokens.value, heads.value>(scores + j, end - j, kChooseThreads, p.num_kv_heads, room,
                                                     [&](int o, uint32_t x, bool sure) {
                                                         keys[j + o] = x;
                                                         if (!sure)
                                                             if (const int to = atomicAdd(&unsure, 1); to < kUnsure)
                                                                 unsure_at[to] = j + o;
                                                     });
        };
        using std::integral_constant;
        if (p.num_kv_heads == 1)
            form(integral_constant<int, 8>{}, integral_constant<int, 1>{});
        else if (p.num_kv_heads <= 4)
            form(integral_constant<int, 4>{}, integral_constant<int, 4>{});
        else
            form(integral_constant<int, 2>{}, integral_constant<int, 8>{});
    }
    __syncthreads();
    if (unsure > 0) // (seldom)
        mend_keys(keys, unsure_at, unsure, scores, p.num_kv_heads, room, begin, end);
    const int refs0 = tid < pages && (uint32_t)page0 < (uint32_t)p.num_blocks ? p.refs[page0] : 0;
    auto key = [&](int j) { return stored ? keys[j] : total_far(scores + j, p.num_kv_heads, room); };
    if (tid == 0)
        lowest = n;

    // the m-th largest key: its bits from the top, and how many of the keys that share them stay (no more bits are
    // needed once all of those do)
    int need = budget - p.first - p.last, low = 0;
    uint32_t prefix = 0;
    const bool any = need > 0;
    for (int round = 0; any && round < 3; ++round) {
        const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, bits = round == 2 ? 10 : 11;
        for (int x = tid; x < kBins; x += kChooseThreads)
            hist[x] = 0;
        __syncthreads();
        for (int j = begin + tid; j < end; j += kChooseThreads) {
            const uint32_t x = key(j);
            if (round == 0 || x >> (shift + bits) == prefix)
                atomicAdd(&hist[(x >> shift) & ((1u << bits) - 1u)], 1);
        }
        __syncthreads();
        // two bins per thread, from the largest down
        const int hi = kBins - 1 - 2 * tid;
        const int a = hist[hi], b = hist[hi - 1];
        int sum;
        const int before = scan_cta(a + b, warps, &sum);
        if (before < need && need <= before + a) {
            digit = hi;
            above = before;
            equals = a;
        } else if (before + a < need && need <= before + a + b) {
            digit = hi - 1;
            above = before + a;
            equals = b;
        }
        __syncthreads();
        prefix = (prefix << bits) | (uint32_t)digit;
        need -= above;
        low = shift;
        if (need == equals)
            break;
        __syncthreads();
    }

    // places: a warp has a run of tokens; of what lies before it, `more` stay for sure and `equal` are of the last key
    const int run = ((n + kChooseWarps - 1) / kChooseWarps + 31) & ~31;
    const int from = min(warp * run, n), to = min(from + run, n);
    auto look = [&](int j, bool &sure, bool &same) {
        sure = same = false;
        if (j < to) {
            if (j < begin || j >= end) {
                sure = true;
            } else if (any) {
                const uint32_t x = key(j) >> low;
                sure = x > prefix;
                same = x == prefix;
            }
        }
    };
    __syncthreads(); // (keys, where nothing was counted)
    int more = 0, equal = 0;
    for (int j = from; j < to; j += 32) {
        bool sure, same;
        look(j + lane, sure, same);
        more += __popc(__ballot_sync(0xffffffffu, sure));
        equal += __popc(__ballot_sync(0xffffffffu, same));
    }
    if (lane == 0) {
        warps[warp] = more;
        warps2[warp] = equal;
    }
    __syncthreads();
    static_assert(kChooseWarps == 32, "a warp's lane looks at each warp's counts");
    more = __reduce_add_sync(0xffffffffu, lane < warp ? warps[lane] : 0);
    equal = __reduce_add_sync(0xffffffffu, lane < warp ? warps2[lane] : 0);
    const uint32_t below = (1u << lane) - 1u;
    for (int j = from; j < to; j += 32) {
        bool sure, same;
        look(j + lane, sure, same);
        const uint32_t ms = __ballot_sync(0xffffffffu, sure), me = __ballot_sync(0xffffffffu, same);
        const int eq = equal + __popc(me & below);
        const bool stays = sure || (same && eq < need);
        if (stays)
            kept[more + __popc(ms & below) + min(eq, need)] = j + lane;
        const uint32_t gone = __ballot_sync(0xffffffffu, !stays && j + lane < to);
        if (gone && lane == 0)
            atomicMin(&lowest, j + __ffs(gone) - 1);
        more += __popc(ms);
        equal += __popc(me);
    }
    __syncthreads();

    // the row's pages are in use, and those that are written are its own
    const int moved = lowest; // the tokens before the first that goes stay where they are
    const int own = moved < budget ? moved / bs : pages, own_end = (budget + bs - 1) / bs;
    for (int x = tid; x < pages; x += kChooseThreads) {
        const int page = x == tid ? page0 : table[x];
        const bool inside = (uint32_t)page < (uint32_t)p.num_blocks;
        const int refs = x == tid ? refs0 : inside ? p.refs[page] : 0;
        bad = bad || !inside || refs < 1 || (x >= own && x < own_end && refs != 1);
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
        p.state[i] = bad ? -1 : n;
        p.moved[i] = moved;
        p.done[i] = 0u;
        if (bad)
            atomicOr(&g_evict_error, 1u);
    }
}

struct MovePlanes {
    char *k, *v, *ks, *vs; // layer 0; scales NULL: bf16
    uint64_t layer, scale_layer; // bytes between layers
    int32_t layers, token_bytes; // bytes of a token's row in one layer of k (or v)
    int32_t log_slice;           // 16-byte vectors of a slice, as a power of two
    int32_t slices;              // slices of a token's row
    int32_t log_heads;           // heads whose scales move together, as a power of two
    int32_t parts;               // such groups of heads; bf16: 0
    int32_t units;               // per row: (layer, K or V, slice), then (layer, K or V, part) of the scales, then heads
                                 // of the scores
};

// Elements T of the places [from, count) from where their tokens are: `map` (of kBatchTokens places at a time) holds
// each place's and its token's slot, element e of slot x is at(x, e); a token has per <= 2^log_per of them.  Threads of a
// warp take elements of one token or, kAcross, tokens of one element: what lies side by side in a page.
template <class T, bool kAcross, class At>
__device__ __forceinline__ void move_up(const int32_t *kept, const int32_t *table, int log_bs, int from, int count, int per,
                                        int log_per, int2 *map, At at)
{
    static_assert(kMoveThreads == 256 && kVecs == 4, "shifts below");
    // log of a batch's tokens; thread t's u-th element is of token (t & mask) or t >> log_per, and so on
    const int log_tokens = 10 - log_per, tokens = 1 << log_tokens;
    const int tid = threadIdx.x;
    auto token_of = [&](int u) {
        return kAcross ? (u * kMoveThreads + tid) & (tokens - 1) : (tid >> log_per) + u * (kMoveThreads >> log_per);
    };
    auto elem_of = [&](int u) { return kAcross ? (u * kMoveThreads + tid) >> log_tokens : tid & ((1 << log_per) - 1); };
    auto slot = [&](int token) { return (table[token >> log_bs] << log_bs) + (token & ((1 << log_bs) - 1)); };
    for (int base = from; base < count; base += kBatchTokens) {
        const int n = min(count - base, kBatchTokens);
        __syncthreads(); // the map may still be read
        for (int x = threadIdx.x; x < n; x += kMoveThreads)
            map[x] = make_int2(slot(base + x), slot(kept[base + x]));
        __syncthreads();
        T a[kVecs], b[kVecs];
        auto load = [&](int first, T(&x)[kVecs]) {
#pragma unroll
            for (int u = 0; u < kVecs; ++u) {
                const int k = first + token_of(u), v = elem_of(u);
                if (k < n && v < per)
                    x[u] = *at(map[k].y, v);
            }
        };
        auto store = [&](int first, const T(&x)[kVecs]) {
#pragma unroll
            for (int u = 0; u < kVecs; ++u) {
                const int k = first + token_of(u), v = elem_of(u);
                if (k < n && v < per)
                    *at(map[k].x, v) = x[u];
            }
        };
        load(0, a);
        for (int k = 0; k < n; k += 2 * tokens) {
            load(k + tokens, b);
            __syncthreads(); // every thread has this batch's values: its places may be written
            store(k, a);
            load(k + 2 * tokens, a);
            __syncthreads();
            store(k + tokens, b);
        }
    }
}

__global__ void __launch_bounds__(kMoveThreads, 4) evict_move_kernel(const EvictParams p, const MovePlanes q)
{
    __shared__ uint32_t place;
    __shared__ int2 map[kBatchTokens];
    ptx::grid_dependency_wait();
    const int i = blockIdx.x / q.units;
    int unit = blockIdx.x - i * q.units;
    const int tid = threadIdx.x, bs = p.block_size, budget = p.budget;
    bool refused = false;
    const int row = p.rows[i], n = p.state[i], first_moved = p.moved[i]; // (used if no row is refused)
    for (int x = tid; x < p.n; x += kMoveThreads)
        refused = refused || p.state[x] < 0;
    int32_t *kept = p.kept + (int64_t)i * budget;
    if (__syncthreads_or(refused)) { // nothing moves
        if (unit == 0)
            for (int k = tid; k < budget; k += kMoveThreads)
                kept[k] = -1;
        return;
    }
    const int left = min(n, budget);
    const int64_t room = (int64_t)p.max_blocks * bs;
    int32_t *table = p.tables + (int64_t)row * p.max_blocks;
    const int planes = 2 * q.layers;
    const int moved = min(first_moved, left);
    const int log_bs = __ffs(bs) - 1;

    if (unit < planes * q.slices) {
        const int plane = unit / q.slices, slice = unit - plane * q.slices;
        const int per = min(1 << q.log_slice, q.token_bytes / 16 - (slice << q.log_slice));
        char *base = (plane & 1 ? q.v : q.k) + (plane >> 1) * q.layer + ((int64_t)slice << q.log_slice) * 16;
        move_up<uint4, false>(kept, table, log_bs, moved, left, per, q.log_slice, map, [&](int slot, int v) {
            return reinterpret_cast<uint4 *>(base + (int64_t)slot * q.token_bytes) + v;
        });
    } else if ((unit -= planes * q.slices) < planes * q.parts) {
        const int plane = unit / q.parts, head = (unit - plane * q.parts) << q.log_heads;
        const int per = min(1 << q.log_heads, p.num_kv_heads - head);
        uint16_t *base = reinterpret_cast<uint16_t *>((plane & 1 ? q.vs : q.ks) + (plane >> 1) * q.scale_layer);
        move_up<uint16_t, true>(kept, table, log_bs, moved, left, per, q.log_heads, map, [&](int slot, int v) {
            return base + ((((int64_t)(slot >> log_bs) * p.num_kv_heads + head + v) << log_bs) + (slot & (bs - 1)));
        });
    } else { // one head's scores, a batch read before it is written as above
        unit -= planes * q.parts;
        const int64_t at = ((int64_t)row * p.num_kv_heads + unit) * room;
        const float *from = p.scores + at;
        float *to = p.scores_out + at;
        const int start = from == to ? moved : 0;
        float a[kVecs];
        for (int k0 = start; k0 < left; k0 += kBatchTokens) {
#pragma unroll
            for (int u = 0; u < kVecs; ++u)
                if (const int k = k0 + u * kMoveThreads + tid; k < left)
                    a[u] = from[kept[k]];
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kVecs; ++u)
                if (const int k = k0 + u * kMoveThreads + tid; k < left)
                    to[k] = a[u];
        }
        __syncthreads();
        for (int k = left + tid; k < n; k += kMoveThreads)
            to[k] = 0.f;
    }

    ptx::launch_dependents(); // (at the start the next launch's CTAs would take this one's places)

    // the row's last unit: nothing reads its table any more
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        place = atomicAdd(p.done + i, 1u);
    }
    __syncthreads();
    if (place == (uint32_t)q.units - 1u && n > budget) {
        for (int x = (budget + bs - 1) / bs + tid; x < (n + bs - 1) / bs; x += kMoveThreads) {
            atomicSub(p.refs + table[x], 1); // (another row of the call may give back the same page)
            table[x] = -1;
        }
        if (tid == 0)
            p.context_lens[row] = budget;
    }
}

template <class... Args>
int launch_ex(const char *what, void (*kernel)(Args...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
              const Args &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(PA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    }
    return PA_OK;
}

} // namespace

int launch_pool_evict(const PoolArgs &a, const int32_t *rows, int n, const float *scores, float *scores_out, int budget,
                      int first, int last, int32_t *kept, void *stream)
{
    int sms = 0;
    if (int rc = sm_count(&sms))
        return rc;
    const pa_dims &d = a.dims;
    const pa_pool &o = a.pool;
    EvictParams p{};
    p.tables = o.block_tables, p.context_lens = o.context_lens, p.refs = o.ref_counts;
    p.rows = rows, p.n = n, p.num_rows = o.num_rows, p.max_blocks = o.max_blocks;
    p.num_blocks = d.num_blocks, p.block_size = d.block_size, p.num_kv_heads = d.num_kv_heads;
    p.scores = scores, p.scores_out = scores_out;
    p.budget = budget, p.first = first, p.last = last, p.kept = kept;
    p.state = static_cast<int32_t *>(a.workspace); // of the pool's 8 ints and more per row
    p.moved = p.state + o.num_rows;
    p.done = reinterpret_cast<uint32_t *>(p.moved + o.num_rows);
    p.keys = (int)std::min<int64_t>((int64_t)o.max_blocks * d.block_size, kKeysInSmem);
    MovePlanes q{};
    q.k = static_cast<char *>(o.k_cache), q.v = static_cast<char *>(o.v_cache);
    q.ks = static_cast<char *>(o.k_scale), q.vs = static_cast<char *>(o.v_scale);
    q.layer = o.layer_stride, q.scale_layer = o.scale_layer_stride;
    q.layers = o.num_layers;
    q.token_bytes = d.num_kv_heads * d.head_dim * (o.k_scale ? 1 : 2);
    // slices: up to 512 bytes of a token's row (of 1 KB 16 rows of 4096 to 2048 tokens in 28 layers took 616 us, of 256
    // bytes 631, of 512 600), less (down to 64 bytes) while that gives the SMs too few CTAs.  Scales: of all heads, of
    // fewer by the same rule (a CTA per head took 30 us longer where 36 short rows of 22 layers of 8 heads hardly move).
    auto cut = [&](int elems, int most, int least, int32_t *log) {
        auto parts = [&] { return (elems + (1 << *log) - 1) >> *log; };
        for (*log = 0; *log < most && 1 << *log < elems;)
            ++*log;
        while (*log > least && (int64_t)n * q.layers * 2 * parts() < 4 * sms)
            --*log;
        return parts();
    };
    q.slices = cut(q.token_bytes / 16, 5, 2, &q.log_slice);
    q.parts = q.ks ? cut(d.num_kv_heads, 6, 0, &q.log_heads) : 0;
    const int64_t units = (int64_t)2 * q.layers * (q.slices + q.parts) + d.num_kv_heads;
    if (units * n > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "pa_pool_evict: %d rows of %d layers exceed one launch", n, q.layers);
    q.units = (int32_t)units;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t smem = (size_t)p.keys * 4;
    if (int rc = ensure_smem<evict_choose_kernel>(kKeysInSmem * 4, "evict"))
        return rc;
    if (int rc = launch_ex("evict choice", evict_choose_kernel, (unsigned)n, kChooseThreads, smem, s, p))
        return rc;
    return launch_ex("evict move", evict_move_kernel, (unsigned)(units * n), kMoveThreads, 0, s, p, q);
}

int read_evict_error(uint32_t *code)
{
    uint32_t v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_evict_error, sizeof v);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbol(g_evict_error, &zero, sizeof zero);
    if (e != cudaSuccess)
        return fail(PA_ERR_CUDA, "reading evict error word: %s", cudaGetErrorString(e));
    *code |= (v & 1u) << 8;
    return PA_OK;
}

} // namespace pa

// Host-side plan of the shared-prefix decode: key ranges, work items, their CTAs.
//
// Sources: as pack.cpp (metadata is built on the CPU next to the scheduling loop and uploaded
// with one copy); "vLLM / SGLang 面试源码深挖", section 4 (forked sequences name the same
// blocks) for what is shared.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <queue>
#include <vector>

#include <cuda_runtime.h>

#include "internal.h"

namespace pa {
namespace {

constexpr int32_t kTile = kPrefillKeyTile;

// Time model in microseconds, used only to choose the key ranges and to deal the items out
// (measured on GB300, D = 128).  A pair (two query tiles on one K/V stream) occupies both lanes of
// its CTA, its step bound by the softmax and its hand-offs.  A single occupies one lane; alone in its CTA its step
// takes kSharedStep, beside another's kSingleStep.  An item adds its query load and its output.  A
// partial costs its bytes written and read again.
//
// The parts of single sequences run in the lanes' lists too where every item has a lane of its own
// (4 x 2148 tokens 9.5 us, 8 x 16500 17.0); where there are more items, or none is shared, they run apart, in the decode
// kernels on the SMs that the shared parts leave (10.3 and 17.8 us there, but 64 x 4600 20.8 us
// instead of 28.4, 200 x 16600 63.8 instead of 66.7, and 24 ragged groups 69 instead of 82): several
// of their CTAs on an SM hide one another's latency, where a CTA of ours has two lanes.
// One plan serves both caches: the length chosen makes the product of their two times least.  The
// rates are those that fit best the times of 36 batches (1 to 256 sequences behind 512 to 32768
// tokens, three head layouts, both caches, 22 lengths of the parts, every call on tensors that L2 has
// lost): the length chosen is 1.5 % (bf16) and 2 % (INT8) slower than the best one in the mean.
constexpr float kPairStep = 1.62f, kSingleStep = 2.4f, kSharedStep = 1.9f, kPairItem = 4.0f, kSingleItem = 2.0f,
                kMergeBytesPerUs = 3.0e6f;
constexpr float kBytesPerUs = 6.9e6f, kSmBytesPerUs = 0.06e6f; // the decode kernels', all SMs and one
constexpr float kInt8Rate = 0.8f, kCodesPerUs = 6.0e6f;        // part of those rates, conversion
constexpr float kApartStart = 1.f, kApartTail = 4.f, kApartBegin = 2.f, kApartKey = 0.006f, kApartKeyInt8 = 0.0085f;
// What a call takes beyond that (set-up and merge), and what the decode kernels take for the contexts
// whole, one part each: a start, a step of 16 keys per warp after the other (twice the warps where
// there are few contexts), or the bytes of all contexts from L2 and HBM.  Fitted to 120 batches of 2
// to 128 sequences of 84 to 1580 tokens.
constexpr float kSharedStart = 5.0f, kSharedStartInt8 = 6.0f;
constexpr float kDirectStart = 4.0f, kDirectKey = 0.0075f, kDirectKeyInt8 = 0.011f, kDirectKeyFew = 0.0064f,
                kDirectKeyFewInt8 = 0.0082f, kDirectBytesPerUs = 11.0e6f, kDirectBytesPerUsInt8 = 6.5e6f;

struct Run { // consecutive sequences of a group that share `shared` tokens
    int32_t s0, n, shared;
    int32_t scratch; // row of key 0 in the INT8 decode's scratch cache
};

struct Range { // one part of `seqs` contexts: units items per split
    int32_t keys, units_pair, units_single, seqs;
};

float item_cost(int32_t tiles, bool pair)
{
    return pair ? (float)tiles * kPairStep + kPairItem : (float)tiles * kSingleStep + kSingleItem;
}

struct Work {
    int32_t s0, n, g, row, k0, k1, part, scratch;
    float cost;
};

int32_t splits_of(int32_t tiles, int32_t per) { return (tiles + per - 1) / per; }

} // namespace
} // namespace pa

using namespace pa;

static int pack_decode_shared(const pa_dims *dims, int32_t num_seqs, const int32_t *context_lens,
                              int32_t num_groups, const int32_t *group_offsets, const int32_t *shared_lens,
                              const int32_t *block_offsets, const int32_t *block_ids, const int32_t *table_rows,
                              int32_t max_blocks_per_seq, int32_t split_tokens, void *host_buf, size_t host_buf_bytes,
                              pa_shared_meta *meta)
{
    int rc = check_dims(dims);
    if (rc != PA_OK)
        return rc;
    if (!meta)
        return fail(PA_ERR_INVALID_ARG, "meta is NULL");
    if (num_seqs < 0 || num_groups < 0)
        return fail(PA_ERR_INVALID_ARG, "num_seqs or num_groups < 0");
    if (num_seqs > 0 && (!context_lens || !group_offsets))
        return fail(PA_ERR_INVALID_ARG, "context_lens/group_offsets is NULL");
    if (split_tokens < 0 || split_tokens % kTile != 0)
        return fail(PA_ERR_INVALID_ARG, "split_tokens (%d) must be 0 or a positive multiple of %d", split_tokens, kTile);
    const pa_dims &d = *dims;
    const int32_t bs = d.block_size;
    if (num_seqs > 0) {
        if (group_offsets[0] != 0 || group_offsets[num_groups] != num_seqs)
            return fail(PA_ERR_INVALID_ARG, "group_offsets must start at 0 and end at num_seqs (%d)", num_seqs);
        for (int32_t i = 0; i < num_groups; ++i)
            if (group_offsets[i + 1] < group_offsets[i])
                return fail(PA_ERR_INVALID_ARG, "group_offsets not non-decreasing at group %d", i);
    }
    int32_t max_ctx = 0;
    for (int32_t b = 0; b < num_seqs; ++b) {
        if (context_lens[b] < 0)
            return fail(PA_ERR_INVALID_ARG, "context_lens[%d] < 0", b);
        if ((int64_t)context_lens[b] > (int64_t)INT32_MAX - 2 * kTile)
            return fail(PA_ERR_INVALID_ARG, "context_lens[%d] too long", b);
        max_ctx = std::max(max_ctx, context_lens[b]);
    }
    const bool packed = block_offsets != nullptr;
    int32_t mb = 1;
    if (packed) {
        if (table_rows)
            return fail(PA_ERR_INVALID_ARG, "table_rows goes with device tables: block lists give each sequence a row");
        if (num_seqs > 0 &&
            (rc = check_seq_blocks(d, num_seqs, context_lens, block_offsets, block_ids, &mb)) != PA_OK)
            return rc;
    } else if (num_seqs > 0) {
        if (!shared_lens)
            return fail(PA_ERR_INVALID_ARG, "shared_lens is NULL: without block lists it cannot be found");
        mb = max_blocks_per_seq;
        const int64_t need = ((int64_t)max_ctx + bs - 1) / bs;
        if (mb < 1 || need > mb)
            return fail(PA_ERR_INVALID_ARG, "max_blocks_per_seq (%d) must be positive and hold %lld blocks", mb,
                        (long long)need);
        if (table_rows)
            for (int32_t b = 0; b < num_seqs; ++b)
                if (table_rows[b] < 0)
                    return fail(PA_ERR_INVALID_ARG, "table_rows[%d] < 0", b);
    }
    if (max_ctx > 0 && d.num_blocks == 0)
        return fail(PA_ERR_INVALID_ARG, "empty KV pool");

    // runs: a group's sequences with a context, consecutive ones together (entries of context 0
    // take no part and end a run)
    const int group = d.num_heads / d.num_kv_heads;
    const int32_t P = std::max(1, kPrefillRows / group);
    std::vector<Run> runs;
    struct Copied { // keys [from, to) of a row, at a scratch row
        int32_t row, from, to, scratch;
    };
    std::vector<Copied> copies; // what the INT8 decode's items read
    int64_t scratch_tiles = 0;
    for (int32_t i = 0; num_seqs > 0 && i < num_groups; ++i) {
        const int32_t b0 = group_offsets[i], b1 = group_offsets[i + 1];
        int32_t live = 0, least = INT32_MAX, first = -1;
        for (int32_t b = b0; b < b1; ++b)
            if (context_lens[b] > 0) {
                ++live;
                least = std::min(least, context_lens[b]);
                first = first < 0 ? b : first;
            }
        if (live == 0)
            continue;
        const int32_t most = least / bs * bs; // whole blocks that every sequence of the group fills
        int32_t shared = shared_lens ? shared_lens[i] : most;
        if (shared_lens && (shared < 0 || shared % bs != 0 || shared > most))
            return fail(PA_ERR_INVALID_ARG,
                        "shared_lens[%d] = %d must be a multiple of the block size in [0, %d], the whole blocks of the "
                        "group's shortest context",
                        i, shared, most);
        if (packed)
            for (int32_t b = b0; b < b1; ++b) {
                if (context_lens[b] == 0)
                    continue;
                const int32_t *x = block_ids + block_offsets[first], *y = block_ids + block_offsets[b];
                int32_t n = 0;
                while (n < shared / bs && x[n] == y[n])
                    ++n;
                if (shared_lens && n < shared / bs)
                    return fail(PA_ERR_INVALID_ARG, "sequence %d does not share block %d of its group's %d", b, n,
                                shared / bs);
                shared = n * bs;
            }
        if (live == 1)
            shared = 0; // one sequence shares nothing: its context is one part
        // (several runs of a group read the same scratch rows)
        const int32_t group_scratch = (int32_t)std::min<int64_t>(scratch_tiles * kTile, INT32_MAX);
        if (shared > 0) {
            copies.push_back({table_rows ? table_rows[first] : first, 0, shared, group_scratch});
            scratch_tiles += (shared + kTile - 1) / kTile;
        }
        for (int32_t b = b0; b < b1;) {
            if (context_lens[b] == 0) {
                ++b;
                continue;
            }
            int32_t e = b;
            while (e < b1 && context_lens[e] > 0)
                ++e;
            runs.push_back({b, e - b, shared, group_scratch});
            b = e;
        }
    }

    // choose the key tiles per item: the least of a few candidates' estimated time
    int dev = 0, sms = 152;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaGetLastError();
    std::vector<Range> ranges;
    for (const Run &r : runs) {
        if (r.shared > 0) {
            const int32_t pairs = r.n / (2 * P), rest = r.n % (2 * P);
            ranges.push_back({r.shared, (pairs + (rest > P)) * d.num_kv_heads,
                              (rest > 0 && rest <= P ? 1 : 0) * d.num_kv_heads, r.n});
        }
        for (int32_t b = r.s0; b < r.s0 + r.n; ++b)
            if (context_lens[b] > r.shared)
                ranges.push_back({context_lens[b] - r.shared, 0, d.num_kv_heads, 1});
    }
    const float key_bytes = (float)d.num_kv_heads * d.head_dim * 4;
    const float slot_us = (float)d.num_heads * d.head_dim * 8.f / kMergeBytesPerUs;
    bool apart = false;
    struct Times {
        float bf16, int8;
    };
    // parts of c key tiles at most: the times, and whether the parts of single sequences run apart
    auto estimate = [&](int32_t c) -> Times {
        float pair = 0.f, shared = 0.f, one = 0.f, work = 0.f; // longest items, CTA time of the shared parts
        float bytes = 0.f, one_bytes = 0.f, codes = 0.f, slots = 0.f, longest = 0.f;
        int64_t pairs = 0, singles = 0, ones = 0;
        for (const Range &x : ranges) {
            const int32_t tiles = splits_of(x.keys, kTile), s = splits_of(tiles, c), len = splits_of(tiles, s);
            slots += (float)s * x.seqs;
            if (x.seqs == 1) {
                ones += (int64_t)s * x.units_single;
                one = std::max(one, item_cost(len, false));
                one_bytes += x.keys * key_bytes;
                longest = std::max(longest, (float)std::min(len * kTile, x.keys));
                continue;
            }
            pairs += (int64_t)s * x.units_pair;
            singles += (int64_t)s * x.units_single;
            if (x.units_pair)
                pair = std::max(pair, item_cost(len, true));
            if (x.units_single)
                shared = std::max(shared, len * kSharedStep + kSingleItem);
            work += x.units_pair * (tiles * kPairStep + s * kPairItem) + x.units_single * (tiles * kSharedStep + s * kSingleItem);
            bytes += x.units_pair > d.num_kv_heads ? 0.f : x.keys * key_bytes;
            codes += x.keys * key_bytes / 2;
        }
        // the shared parts in equal rounds over as few CTAs as that takes; on the SMs left and, after
        // them, on all, those of single sequences
        const float merge = slots * slot_us;
        const int64_t units = pairs + singles, rounds = (units + sms - 1) / sms;
        const int64_t ctas = units ? (units + rounds - 1) / rounds : 0;
        float t = std::max(pair, shared);
        if (rounds > 1)
            t = std::max(t, work / (float)ctas + 0.25f * work / (float)units);
        auto beside = [&](float n, float rate, float per_key) {
            const float left = std::max(0.f, n - t * rate * std::min(kBytesPerUs, (float)(sms - ctas) * kSmBytesPerUs));
            return std::max(t + (left > 0.f ? left / (rate * kBytesPerUs) + kApartTail : 0.f), kApartBegin + per_key * longest) +
                   kApartStart;
        };
        apart = units == 0 || 2 * pairs + singles + ones > 2 * (int64_t)sms;
        if (!apart) {
            const float in = std::max(std::max(pair, shared * (kSingleStep / kSharedStep)), one) + merge;
            return {in, in + (codes + one_bytes / 2) / kCodesPerUs};
        }
        return {std::max(beside(one_bytes, 1.f, kApartKey), (bytes + one_bytes) / kBytesPerUs) + merge,
                beside(one_bytes / 2, kInt8Rate, kApartKeyInt8) + codes / kCodesPerUs + merge};
    };
    int32_t per = split_tokens / kTile;
    if (per == 0) {
        static const int32_t kPer[] = {1,  2,  3,  4,  5,  6,  7,  8,  9,  10,  11,  12,  13,  14,
                                       16, 18, 20, 22, 26, 32, 45, 64, 90, 128, 181, 256, 512, 1 << 24};
        float best = INFINITY;
        for (int32_t c : kPer) {
            const Times t = estimate(c);
            const float both = (kSharedStart + t.bf16) * (kSharedStartInt8 + t.int8);
            if (both < best) {
                best = both;
                per = c;
            }
        }
        per = std::max(per, 1);
    }
    const Times times = estimate(per); // (and apart)

    int64_t all_keys = 0;
    for (int32_t b = 0; b < num_seqs; ++b)
        all_keys += context_lens[b];
    const float keys_bytes = (float)all_keys * d.num_kv_heads * d.head_dim * 2;
    const bool few = (int64_t)num_seqs * d.num_kv_heads <= sms;
    const float steps = max_ctx * (few ? kDirectKeyFew : kDirectKey);
    const float steps_int8 = max_ctx * (few ? kDirectKeyFewInt8 : kDirectKeyInt8);
    const bool direct = split_tokens == 0 && kDirectStart + std::max(steps, 2 * keys_bytes / kDirectBytesPerUs) <
                                                 kSharedStart + times.bf16;
    const bool direct_int8 = split_tokens == 0 && kDirectStart + std::max(steps_int8, keys_bytes / kDirectBytesPerUsInt8) <
                                                      kSharedStartInt8 + times.int8;

    // items and partial slots
    std::vector<Work> works;
    std::vector<int32_t> parts(num_seqs, 0); // parts of each sequence
    for (const Run &r : runs) {
        const int32_t ptiles = (r.shared + kTile - 1) / kTile;
        const int32_t ps = ptiles > 0 ? splits_of(ptiles, per) : 0;
        for (int32_t b = r.s0; b < r.s0 + r.n; ++b) {
            const int32_t t = (context_lens[b] - r.shared + kTile - 1) / kTile;
            parts[b] = ps + (t > 0 ? splits_of(t, per) : 0);
        }
    }
    auto cut = [&](int32_t s0, int32_t n, int32_t row, int32_t from, int32_t to, int32_t first_part, int32_t scratch) {
        const int32_t tiles = (to - from + kTile - 1) / kTile;
        const int32_t s = splits_of(tiles, per);
        for (int32_t i = 0; i < s; ++i) {
            const int32_t t0 = (int32_t)((int64_t)tiles * i / s), t1 = (int32_t)((int64_t)tiles * (i + 1) / s);
            const int32_t k0 = from + t0 * kTile, k1 = std::min(to, from + t1 * kTile);
            for (int32_t g = 0; g < d.num_kv_heads; ++g)
                for (int32_t q = 0; q < n; q += 2 * P) {
                    const int32_t m = std::min(n - q, 2 * P);
                    works.push_back({s0 + q, m, g, row, k0, k1, first_part + i, scratch,
                                     item_cost(t1 - t0, m > P)});
                }
        }
    };
    for (const Run &r : runs) {
        const int32_t ptiles = (r.shared + kTile - 1) / kTile;
        const int32_t ps = ptiles > 0 ? splits_of(ptiles, per) : 0;
        if (ps > 0)
            cut(r.s0, r.n, table_rows ? table_rows[r.s0] : r.s0, 0, r.shared, 0, r.scratch);
        for (int32_t b = r.s0; b < r.s0 + r.n; ++b)
            if (context_lens[b] > r.shared) {
                const int32_t row = table_rows ? table_rows[b] : b;
                const int32_t at = (int32_t)std::min<int64_t>(scratch_tiles * kTile, INT32_MAX);
                if (!apart) {
                    copies.push_back({row, r.shared, context_lens[b], at});
                    scratch_tiles += splits_of(context_lens[b] - r.shared, kTile);
                }
                cut(b, 1, row, r.shared, context_lens[b], ps, apart ? 0 : at - r.shared);
            }
    }
    if (works.size() > (size_t)INT32_MAX / kSharedItemInts)
        return fail(PA_ERR_INVALID_ARG, "too many work items");
    int64_t partials = 0;
    int32_t max_parts = 0;
    bool merge = false;
    for (int32_t b = 0; b < num_seqs; ++b) {
        max_parts = std::max(max_parts, parts[b]);
        partials += parts[b] > 1 ? parts[b] : 0;
        merge = merge || parts[b] != 1;
    }
    if (partials > INT32_MAX)
        return fail(PA_ERR_INVALID_ARG, "too many partial results");
    if (scratch_tiles * kTile > INT32_MAX)
        return fail(PA_ERR_INVALID_ARG, "the groups' shared tokens exceed int32");
    int32_t singles = 0, shared_items = 0;
    for (const Work &w : works) {
        singles += w.n == 1 && w.g == 0;
        shared_items += w.n > 1;
    }
    // apart: the CTAs' lists hold the parts of several sequences only, on the CTAs of their rounds
    const int32_t listed = apart ? shared_items : (int32_t)works.size();
    const int32_t rounds = apart ? (listed + sms - 1) / sms : 1;
    const int32_t ctas = rounds > 0 ? std::min(sms, (listed + rounds - 1) / rounds) : 0;

    Layout L;
    *meta = pa_shared_meta{};
    meta->num_seqs = num_seqs;
    meta->num_groups = num_groups;
    meta->num_heads = d.num_heads;
    meta->num_kv_heads = d.num_kv_heads;
    meta->head_dim = d.head_dim;
    meta->block_size = bs;
    meta->max_blocks_per_seq = mb;
    meta->num_items = listed;
    meta->apart = apart ? 1 : 0;
    meta->num_ctas = ctas;
    meta->num_partials = (int32_t)partials;
    meta->max_parts = max_parts;
    meta->rows_per_tile = P;
    meta->merge = merge ? 1 : 0;
    meta->split_tokens = (int32_t)std::min<int64_t>((int64_t)per * kTile, INT32_MAX / kTile * kTile);
    meta->tables_packed = packed ? 1 : 0;
    meta->num_single_items = singles;
    meta->num_shared_items = shared_items;
    meta->num_scratch_tiles = (int32_t)scratch_tiles;
    meta->direct = (direct ? 1 : 0) | (direct_int8 ? 2 : 0);
    for (const Run &r : runs)
        meta->tokens_saved += (uint64_t)r.shared * (uint64_t)(r.n - 1);
    meta->off_block_tables = L.take(packed ? sizeof(int32_t) * (size_t)num_seqs * mb : 0);
    meta->off_slot_mapping = L.take(packed ? sizeof(int32_t) * (size_t)num_seqs : 0);
    meta->off_items = L.take(sizeof(int32_t) * kSharedItemInts * (size_t)listed);
    meta->off_cta_items = L.take(sizeof(int32_t) * kSharedCtaInts * (size_t)ctas);
    meta->off_seq_parts = L.take(sizeof(int32_t) * 2 * (size_t)num_seqs);
    meta->off_single_items = L.take(sizeof(int32_t) * 4 * (size_t)singles);
    meta->off_table_rows = L.take(sizeof(int32_t) * (size_t)num_seqs);
    meta->off_direct_items = L.take(sizeof(int32_t) * 4 * (size_t)num_seqs);
    meta->off_scratch_tiles = L.take(sizeof(int32_t) * 4 * (size_t)scratch_tiles);
    meta->total_bytes = L.off;
    const size_t results = shared_part_bytes(d, partials) + shared_go_bytes(*meta);
    meta->workspace_bytes = direct ? 0 : results;
    meta->workspace_bytes_int8 = direct_int8 ? 0 : results + shared_scratch_bytes(d, scratch_tiles, num_seqs);
    if (!host_buf)
        return PA_OK;
    if (host_buf_bytes < meta->total_bytes)
        return fail(PA_ERR_WORKSPACE, "metadata buffer has %zu bytes, needs %llu", host_buf_bytes,
                    (unsigned long long)meta->total_bytes);

    char *base = static_cast<char *>(host_buf);
    int32_t *it = reinterpret_cast<int32_t *>(base + meta->off_items);
    int32_t *ci = reinterpret_cast<int32_t *>(base + meta->off_cta_items);
    int32_t *sp = reinterpret_cast<int32_t *>(base + meta->off_seq_parts);
    if (packed && num_seqs > 0) {
        write_block_tables(d, num_seqs, context_lens, block_offsets, block_ids, mb,
                           reinterpret_cast<int32_t *>(base + meta->off_block_tables));
        int32_t *slots = reinterpret_cast<int32_t *>(base + meta->off_slot_mapping);
        for (int32_t b = 0; b < num_seqs; ++b) {
            const int32_t pos = context_lens[b] - 1;
            slots[b] = pos < 0 ? -1 : block_ids[block_offsets[b] + pos / bs] * bs + pos % bs;
        }
    }
    int32_t *rows = reinterpret_cast<int32_t *>(base + meta->off_table_rows);
    std::vector<int32_t> longest(num_seqs);
    for (int32_t b = 0; b < num_seqs; ++b) {
        rows[b] = table_rows ? table_rows[b] : b;
        longest[b] = b;
    }
    std::stable_sort(longest.begin(), longest.end(), [&](int32_t x, int32_t y) { return context_lens[x] > context_lens[y]; });
    int32_t *whole = reinterpret_cast<int32_t *>(base + meta->off_direct_items);
    for (int32_t b : longest) {
        whole[0] = b;
        whole[1] = 0;
        whole[2] = context_lens[b];
        whole[3] = -1;
        whole += 4;
    }
    int32_t *tile = reinterpret_cast<int32_t *>(base + meta->off_scratch_tiles);
    for (const Copied &x : copies)
        for (int32_t k = x.from; k < x.to; k += kTile, tile += 4) {
            tile[0] = x.row;
            tile[1] = k;
            tile[2] = x.to;
            tile[3] = x.scratch + k - x.from;
        }
    for (int32_t b = 0, slot = 0; b < num_seqs; ++b) {
        sp[2 * b] = slot;
        sp[2 * b + 1] = parts[b];
        slot += parts[b] > 1 ? parts[b] : 0;
    }
    // Deal out, longest first, to the least loaded: pairs to CTAs (both lanes), then singles to
    // lanes, those of several sequences before those of one.  Queue 3c holds CTA c's pairs, 3c + 1 and 3c + 2 its lanes' singles.
    std::vector<int32_t> order(works.size()), queue_of(works.size()), fill(3 * (size_t)ctas, 0);
    for (size_t i = 0; i < order.size(); ++i)
        order[i] = (int32_t)i;
    std::stable_sort(order.begin(), order.end(), [&](int32_t x, int32_t y) {
        // pairs, parts of several sequences, parts of one
        auto rank = [&](int32_t i) { return works[i].n > P ? 0 : works[i].n > 1 ? 1 : 2; };
        return rank(x) != rank(y) ? rank(x) < rank(y) : works[x].cost > works[y].cost;
    });
    using Load = std::pair<float, int32_t>;
    std::vector<float> load((size_t)ctas, 0.f);
    std::priority_queue<Load, std::vector<Load>, std::greater<Load>> heap;
    for (int32_t c = 0; c < ctas; ++c)
        heap.push({0.f, c});
    size_t at = 0;
    for (; at < order.size() && works[order[at]].n > P; ++at) {
        Load l = heap.top();
        heap.pop();
        queue_of[order[at]] = 3 * l.second;
        ++fill[3 * (size_t)l.second];
        load[l.second] = l.first += works[order[at]].cost;
        heap.push(l);
    }
    heap = {};
    for (int32_t c = 0; c < 2 * ctas; ++c) // first lanes before second ones
        heap.push({load[c % ctas], c});
    for (; at < (size_t)listed; ++at) {
        Load l = heap.top();
        heap.pop();
        const int32_t q = 3 * (l.second % ctas) + 1 + l.second / ctas;
        queue_of[order[at]] = q;
        ++fill[q];
        l.first += works[order[at]].cost;
        heap.push(l);
    }
    std::vector<int32_t> next(fill.size(), 0);
    for (size_t q = 1; q < fill.size(); ++q)
        next[q] = next[q - 1] + fill[q - 1];
    for (int32_t c = 0; c < ctas; ++c) {
        int32_t *e = ci + (size_t)kSharedCtaInts * c;
        std::memset(e, 0, sizeof(int32_t) * kSharedCtaInts);
        for (int32_t i = 0; i < 3; ++i)
            e[i] = next[3 * (size_t)c + i];
        e[3] = next[3 * (size_t)c + 2] + fill[3 * (size_t)c + 2];
    }
    int32_t *one = reinterpret_cast<int32_t *>(base + meta->off_single_items);
    for (int32_t i : order) {
        const Work &w = works[i];
        if (w.n == 1 && w.g == 0) {
            one[0] = w.s0;
            one[1] = w.k0;
            one[2] = w.k1;
            one[3] = parts[w.s0] > 1 ? sp[2 * w.s0] + w.part : -1;
            one += 4;
        }
        if (apart && w.n == 1)
            continue;
        int32_t *e = it + (size_t)kSharedItemInts * next[queue_of[i]]++;
        e[0] = w.s0;
        e[1] = w.n;
        e[2] = w.g;
        e[3] = w.row;
        e[4] = w.k0;
        e[5] = w.k1;
        e[6] = w.part;
        e[7] = w.scratch;
    }
    for (int32_t c = 0; c < ctas; ++c) { // what a CTA loads first, beside its lists' bounds
        int32_t *e = ci + (size_t)kSharedCtaInts * c;
        const int32_t first = e[0] < e[1] ? e[0] : e[1], second = e[2];
        if (first < (e[0] < e[1] ? e[1] : e[2]))
            std::memcpy(e + 8, it + (size_t)kSharedItemInts * first, sizeof(int32_t) * kSharedItemInts);
        if (second < e[3])
            std::memcpy(e + 16, it + (size_t)kSharedItemInts * second, sizeof(int32_t) * kSharedItemInts);
    }
    return PA_OK;
}

extern "C" int pa_pack_decode_shared(const pa_dims *dims, int32_t num_seqs, const int32_t *context_lens,
                                     int32_t num_groups, const int32_t *group_offsets, const int32_t *shared_lens,
                                     const int32_t *block_offsets, const int32_t *block_ids, const int32_t *table_rows,
                                     int32_t max_blocks_per_seq, int32_t split_tokens, void *host_buf,
                                     size_t host_buf_bytes, pa_shared_meta *meta)
{
    try { // no exception (out of memory) leaves a C entry point
        return pack_decode_shared(dims, num_seqs, context_lens, num_groups, group_offsets, shared_lens, block_offsets,
                                  block_ids, table_rows, max_blocks_per_seq, split_tokens, host_buf, host_buf_bytes,
                                  meta);
    } catch (...) {
        return fail(PA_ERR_WORKSPACE, "pa_pack_decode_shared: out of host memory");
    }
}

// A page pool whose state lives on the device: block tables, context lengths and reference
// counts beside the pages of all layers, changed by the stream that also decodes.
//
// Sources (page title, section): "手搓 vLLM 推理引擎", Step 2 (BlockManager: blocks with a
// reference count, allocate, deallocate, may_append) and Step 5 (slot = block * block_size +
// offset); "vLLM / SGLang 面试源码深挖", section 4 (a fork shares the parent's full blocks and
// copies the partly filled one).  The page's free list is the set of blocks of count 0 here,
// taken lowest id first: the result then depends on the state alone and not on the order in
// which pages came back, and nothing but the counts has to be kept consistent.
//
// append, fork and compact need order-dependent counts (the i-th new page is the i-th free
// id), so one thread-block cluster plans the call: every CTA holds a slice of the ids or
// rows, block-wide scans give ranks, and the CTAs' totals meet through distributed shared
// memory.  The plan is all or nothing: it is checked to the end before any state changes, and a
// refused call sets an error bit and leaves the pool as it was.  Moving pages is a second,
// grid-wide launch, bound by HBM (each byte read and written once); it is launched
// programmatically, so that its start-up runs under the plan.
#include <algorithm>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace pa {

// bit 0: a call was refused for lack of free pages or of table width; bit 1: a malformed call or state
__device__ uint32_t g_pool_error;

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kIdsPerThread = 4;
constexpr int kMoveThreads = 256;
constexpr int kPieceBytes = 16 << 10; // one CTA's unit of page copying: 4 x 16 bytes per thread

// Workspace: header, marks [num_rows], starts [num_rows], copies int4 [num_rows],
// list [num_blocks], list2 [num_blocks].
struct Ws {
    int32_t *head; // [0] copies or moves of the call
    int32_t *marks, *starts;
    int4 *copies;
    int32_t *list, *list2;
};

__host__ __device__ inline Ws carve(void *p, int num_rows, int num_blocks)
{
    Ws w;
    int32_t *q = static_cast<int32_t *>(p);
    w.head = q;
    w.copies = reinterpret_cast<int4 *>(q + 16);
    w.marks = q + 16 + 4 * (size_t)num_rows;
    w.starts = w.marks + num_rows;
    w.list = w.starts + num_rows;
    w.list2 = w.list + num_blocks;
    return w;
}

struct Smem {
    int warp[kWarps];
    int total[2];      // this CTA's total of a scan, by scan parity
    int flags[2];      // this CTA's OR, by parity
};

// Scans and reductions over the cluster's threads in (CTA rank, thread) order.  Each call is
// one cluster barrier; totals alternate between two words, so the next call's writes cannot
// meet a slow reader of this call's.
struct ClusterOps {
    Smem &s;
    cg::cluster_group cl;
    int parity = 0;

    __device__ explicit ClusterOps(Smem &s_) : s(s_), cl(cg::this_cluster()) {}
    __device__ int ctas() const { return (int)cl.num_blocks(); }
    __device__ int rank() const { return (int)cl.block_rank(); }
    __device__ int threads() const { return ctas() * kThreads; }
    __device__ int thread() const { return rank() * kThreads + (int)threadIdx.x; }

    // exclusive sum of v over all threads before this one; *total = the sum over all
    __device__ int scan(int v, int *total)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        if (lane == 31)
            s.warp[warp] = x;
        __syncthreads();
        const int w = s.warp[lane];
        int wx = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, wx, o);
            if (lane >= o)
                wx += y;
        }
        const int before = __shfl_sync(0xffffffffu, wx - w, warp);
        if (threadIdx.x == kThreads - 1)
            s.total[parity] = wx;
        cl.sync(); // also orders s.warp's reads before the next call's writes
        int base = 0, sum = 0;
        for (int c = 0; c < ctas(); ++c) {
            const int t = *cl.map_shared_rank(&s.total[parity], c);
            base += c < rank() ? t : 0;
            sum += t;
        }
        parity ^= 1;
        *total = sum;
        return base + before + x - v;
    }
    // OR over all threads of the cluster
    __device__ int any(int v)
    {
        const int mine = __syncthreads_or(v & 1) | (__syncthreads_or(v & 2) ? 2 : 0);
        if (threadIdx.x == 0)
            s.flags[parity] = mine;
        cl.sync();
        int f = 0;
        for (int c = 0; c < ctas(); ++c)
            f |= *cl.map_shared_rank(&s.flags[parity], c);
        parity ^= 1;
        return f;
    }
};

struct PoolParams {
    int32_t *tables;
    int32_t *context_lens;
    int32_t *refs;
    int32_t num_rows, max_blocks, num_blocks, block_size;
};

// The lowest `want` ids of reference count 0 into list; returns how many there are (at most
// want).  Rounds of 4 ids per thread, ending when enough are found.
__device__ int lowest_free(ClusterOps &ops, const PoolParams &p, int want, int32_t *list)
{
    const int per_round = ops.threads() * kIdsPerThread;
    int found = 0;
    for (int base = 0; base < p.num_blocks && found < want; base += per_round) {
        const int id = base + ops.thread() * kIdsPerThread;
        uint32_t free = 0;
        if (id + kIdsPerThread <= p.num_blocks) {
            const int4 r = *reinterpret_cast<const int4 *>(p.refs + id); // 16-byte aligned: checked on the host
            free = (r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3;
        } else {
            for (int i = 0; i < kIdsPerThread; ++i)
                if (id + i < p.num_blocks && p.refs[id + i] == 0)
                    free |= 1u << i;
        }
        int sum;
        int at = found + ops.scan(__popc(free), &sum);
        for (int i = 0; i < kIdsPerThread; ++i)
            if (free >> i & 1u) {
                if (at < want)
                    list[at] = id + i;
                ++at;
            }
        found += sum;
    }
    return min(found, want);
}

__device__ __forceinline__ int pages(int tokens, int bs) { return (tokens + bs - 1) / bs; }

// ---------------------------------------------------------------- append

__global__ void __launch_bounds__(kThreads)
    pool_append_kernel(const PoolParams p, const int32_t *__restrict__ rows, const int32_t *__restrict__ cu, int n,
                       int32_t *__restrict__ slots, int num_tokens, void *workspace)
{
    __shared__ Smem sm;
    ClusterOps ops(sm);
    const Ws w = carve(workspace, p.num_rows, p.num_blocks);
    const int nt = ops.threads(), me = ops.thread(), bs = p.block_size;
    int bad = 0, want = 0;
    if (me == 0 && (cu[0] != 0 || cu[n] != num_tokens))
        bad = 2;
    for (int base = 0; base < n; base += nt) {
        const int i = base + me;
        int need = 0;
        if (i < n) {
            const int r = rows[i];
            const int64_t count = (int64_t)cu[i + 1] - cu[i];
            if ((uint32_t)r >= (uint32_t)p.num_rows || count < 0) {
                bad |= 2;
            } else {
                w.marks[r] = i;
                const int ctx = p.context_lens[r];
                if (ctx < 0 || (int64_t)ctx > (int64_t)p.max_blocks * bs) {
                    bad |= 2;
                } else if (ctx + count > (int64_t)p.max_blocks * bs) {
                    bad |= 1;
                } else {
                    need = pages(ctx + (int)count, bs) - pages(ctx, bs);
                    if (count > 0 && ctx % bs != 0) { // the partly filled page takes the first tokens: it must be the row's own
                        const int page = p.tables[(size_t)r * p.max_blocks + ctx / bs];
                        if ((uint32_t)page >= (uint32_t)p.num_blocks || p.refs[page] != 1)
                            bad |= 2;
                    }
                }
            }
        }
        int sum;
        const int at = want + ops.scan(need, &sum);
        if (i < n)
            w.starts[i] = at;
        want += sum;
        if (want < 0 || want > p.num_blocks) { // more than the pool holds: no need to count on
            bad |= 1;
            break;
        }
    }
    if (!(ops.any(bad))) { // all marks are written
        for (int i = me; i < n; i += nt)
            if (w.marks[rows[i]] != i)
                bad |= 2; // the same row twice
    }
    bad = ops.any(bad);
    if (!bad && lowest_free(ops, p, want, w.list) < want)
        bad = 1;
    if (bad) {
        if (me == 0)
            atomicOr(&g_pool_error, (uint32_t)bad);
        for (int t = me; t < num_tokens; t += nt)
            slots[t] = -1;
        ops.cl.sync();
        return;
    }
    ops.cl.sync(); // the list
    // tokens: a warp's 32 consecutive ones lie in one row or a few neighbouring ones
    for (int t0 = me & ~31; t0 < num_tokens; t0 += nt) {
        int lo = 0, hi = n; // cu[lo] <= t0 < cu[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t0)
                lo = mid;
            else
                hi = mid;
        }
        const int t = t0 + (me & 31);
        if (t < num_tokens) {
            int i = lo;
            while (cu[i + 1] <= t)
                ++i;
            const int r = rows[i], ctx = p.context_lens[r], pos = ctx + t - cu[i];
            const int page = pos / bs, old = pages(ctx, bs);
            const int id = page < old ? p.tables[(size_t)r * p.max_blocks + page] : w.list[w.starts[i] + page - old];
            slots[t] = id * bs + pos % bs;
        }
    }
    // new pages into the tables
    for (int j = me; j < want; j += nt) {
        int lo = 0, hi = n; // the last row whose pages start at or before j
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (w.starts[mid] <= j)
                lo = mid;
            else
                hi = mid;
        }
        const int r = rows[lo], id = w.list[j];
        p.tables[(size_t)r * p.max_blocks + pages(p.context_lens[r], bs) + j - w.starts[lo]] = id;
        p.refs[id] = 1;
    }
    ops.cl.sync(); // every reader of the old lengths is done
    for (int i = me; i < n; i += nt) {
        const int count = cu[i + 1] - cu[i];
        if (count > 0)
            p.context_lens[rows[i]] += count;
    }
}

// ---------------------------------------------------------------- fork

__global__ void __launch_bounds__(kThreads)
    pool_fork_kernel(const PoolParams p, const int32_t *__restrict__ parents, const int32_t *__restrict__ children,
                     int n, void *workspace)
{
    __shared__ Smem sm;
    ptx::launch_dependents();
    ClusterOps ops(sm);
    const Ws w = carve(workspace, p.num_rows, p.num_blocks);
    const int nt = ops.threads(), me = ops.thread(), bs = p.block_size;
    int bad = 0, want = 0;
    for (int base = 0; base < n; base += nt) {
        const int i = base + me;
        int need = 0;
        if (i < n) {
            const int r = parents[i], c = children[i];
            if ((uint32_t)r >= (uint32_t)p.num_rows || (uint32_t)c >= (uint32_t)p.num_rows) {
                bad |= 2;
            } else {
                w.marks[c] = i;
                const int ctx = p.context_lens[r];
                if (ctx < 0 || (int64_t)ctx > (int64_t)p.max_blocks * bs || p.context_lens[c] != 0) {
                    bad |= 2;
                } else if (ctx % bs != 0) {
                    need = 1;
                    const int page = p.tables[(size_t)r * p.max_blocks + ctx / bs];
                    if ((uint32_t)page >= (uint32_t)p.num_blocks)
                        bad |= 2;
                }
            }
        }
        int sum;
        const int at = want + ops.scan(need, &sum);
        if (i < n)
            w.starts[i] = need ? at : -1;
        want += sum;
    }
    if (!ops.any(bad)) {
        for (int i = me; i < n; i += nt) {
            // a child named twice, or a child that is a parent too (its mark, if it is one of this call's)
            const int r = parents[i], m = w.marks[r];
            if (w.marks[children[i]] != i || ((uint32_t)m < (uint32_t)n && children[m] == r))
                bad |= 2;
        }
    }
    bad = ops.any(bad);
    if (!bad && lowest_free(ops, p, want, w.list) < want)
        bad = 1;
    if (bad) {
        if (me == 0) {
            atomicOr(&g_pool_error, (uint32_t)bad);
            w.head[0] = 0;
        }
        ops.cl.sync();
        return;
    }
    ops.cl.sync(); // the list
    for (int i = me; i < n; i += nt) {
        const int r = parents[i], ctx = p.context_lens[r], s = w.starts[i];
        const int src = s >= 0 ? p.tables[(size_t)r * p.max_blocks + ctx / bs] : -1;
        const int dst = s >= 0 ? w.list[s] : -1;
        w.copies[i] = make_int4(src, dst, ctx % bs, ctx / bs);
        if (s >= 0)
            p.refs[dst] = 1;
        p.context_lens[children[i]] = ctx; // a child is no parent, so no reader of this call sees it
    }
    if (me == 0)
        w.head[0] = n;
    ops.cl.sync();
}

// Pages of all layers: K, V and, for an INT8 cache, the scales.
struct Planes {
    uint4 *k, *v;
    uint16_t *ks, *vs; // NULL: bf16 cache
    uint64_t layer_vecs, scale_layer; // layer strides in 16-byte vectors and in scales
    int32_t layers, page_vecs, row_vecs, pieces, block_size, num_kv_heads;
};

// Piece `u` (layer, K or V, 16 KB of the page) of copying the first `rows` rows of page src to dst.
__device__ __forceinline__ void copy_piece(const Planes &q, int u, int src, int dst, int rows)
{
    constexpr int kU = kPieceBytes / 16 / kMoveThreads;
    const int piece = u % q.pieces, plane = u / q.pieces;
    const int layer = plane >> 1;
    uint4 *base = (plane & 1 ? q.v : q.k) + (size_t)layer * q.layer_vecs;
    const int first = piece * (kPieceBytes / 16);
    const int last = min(first + kPieceBytes / 16, rows * q.row_vecs);
    const uint4 *from = base + (size_t)src * q.page_vecs;
    uint4 *to = base + (size_t)dst * q.page_vecs;
    uint4 x[kU];
#pragma unroll
    for (int e = 0; e < kU; ++e) {
        const int i = first + e * kMoveThreads + (int)threadIdx.x;
        if (i < last)
            x[e] = __ldcs(from + i);
    }
#pragma unroll
    for (int e = 0; e < kU; ++e) {
        const int i = first + e * kMoveThreads + (int)threadIdx.x;
        if (i < last)
            __stcs(to + i, x[e]);
    }
    if (q.ks && piece == 0) { // each KV head's run of `rows` scales
        uint16_t *sc = (plane & 1 ? q.vs : q.ks) + (size_t)layer * q.scale_layer;
        const size_t page = (size_t)q.num_kv_heads * q.block_size;
        for (int i = threadIdx.x; i < rows * q.num_kv_heads; i += kMoveThreads) {
            const size_t at = (size_t)(i / rows) * q.block_size + i % rows;
            sc[dst * page + at] = sc[src * page + at];
        }
    }
}

// The forked rows' tables and counts, and their partly filled pages.
__global__ void __launch_bounds__(kMoveThreads)
    pool_fork_copy_kernel(const PoolParams p, const Planes q, const int32_t *__restrict__ parents,
                          const int32_t *__restrict__ children, void *workspace)
{
    ptx::grid_dependency_wait();
    const Ws w = carve(workspace, p.num_rows, p.num_blocks);
    const int n = w.head[0]; // 0: refused
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const int4 c = w.copies[i];
        const int32_t *from = p.tables + (size_t)parents[i] * p.max_blocks;
        int32_t *to = p.tables + (size_t)children[i] * p.max_blocks;
        for (int j = threadIdx.x; j < c.w; j += kMoveThreads) {
            const int id = from[j];
            if ((uint32_t)id < (uint32_t)p.num_blocks)
                atomicAdd(p.refs + id, 1);
            else
                atomicOr(&g_pool_error, 2u);
            to[j] = id;
        }
        if (threadIdx.x == 0 && c.y >= 0)
            to[c.w] = c.y;
    }
    const int per = 2 * q.layers * q.pieces;
    const int64_t units = (int64_t)n * per;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int4 c = w.copies[u / per];
        if (c.y >= 0)
            copy_piece(q, (int)(u % per), c.x, c.y, c.z);
    }
}

// ---------------------------------------------------------------- free

// One CTA per row.  The context length is taken by exchange, so a row named twice is given back once.
__global__ void __launch_bounds__(128) pool_free_kernel(const PoolParams p, const int32_t *__restrict__ rows)
{
    __shared__ int s_ctx;
    const int r = rows[blockIdx.x];
    if ((uint32_t)r >= (uint32_t)p.num_rows) {
        if (threadIdx.x == 0)
            atomicOr(&g_pool_error, 2u);
        return;
    }
    if (threadIdx.x == 0)
        s_ctx = atomicExch(p.context_lens + r, 0);
    __syncthreads();
    const int ctx = s_ctx;
    if (ctx < 0 || (int64_t)ctx > (int64_t)p.max_blocks * p.block_size) {
        if (threadIdx.x == 0)
            atomicOr(&g_pool_error, 2u);
        return;
    }
    int32_t *row = p.tables + (size_t)r * p.max_blocks;
    const int n = pages(ctx, p.block_size);
    for (int j = threadIdx.x; j < n; j += 128) {
        const int id = row[j];
        row[j] = -1;
        if ((uint32_t)id >= (uint32_t)p.num_blocks) {
            atomicOr(&g_pool_error, 2u);
        } else if (atomicSub(p.refs + id, 1) <= 0) { // counted out already: put back what was taken
            atomicAdd(p.refs + id, 1);
            atomicOr(&g_pool_error, 2u);
        }
    }
}

// ---------------------------------------------------------------- compact

// remap, the counts under the new ids and the moves (list2[k] -> list[k]).  U used pages: the
// used ids >= U move, in order, to the free ids < U.  Sources and destinations are disjoint.
__global__ void __launch_bounds__(kThreads)
    pool_compact_kernel(const PoolParams p, int32_t *__restrict__ remap, int32_t *refs_out, void *workspace)
{
    __shared__ Smem sm;
    ptx::launch_dependents();
    ClusterOps ops(sm);
    const Ws w = carve(workspace, p.num_rows, p.num_blocks);
    const int nt = ops.threads(), me = ops.thread(), N = p.num_blocks;
    int mine = 0;
    for (int id = me; id < N; id += nt)
        mine += p.refs[id] > 0;
    int U;
    ops.scan(mine, &U);
    int holes = 0, high = 0; // free ids below U and used ids from U on, so far
    for (int base = 0; base < N; base += nt) {
        const int id = base + me;
        const bool used = id < N && p.refs[id] > 0;
        const bool hole = id < U && id < N && !used, move = used && id >= U;
        int sum; // both ranks in one scan: at most 8192 threads, so 14 bits each
        const int at = ops.scan((int)hole | (int)move << 16, &sum);
        if (hole)
            w.list[holes + (at & 0xffff)] = id;
        if (move)
            w.list2[high + (at >> 16)] = id;
        if (id < N && !move)
            remap[id] = used ? id : -1;
        holes += sum & 0xffff;
        high += sum >> 16;
    }
    ops.cl.sync(); // both lists; holes == high
    for (int k = me; k < high; k += nt) {
        const int src = w.list2[k], dst = w.list[k];
        remap[src] = dst;
        refs_out[dst] = p.refs[src];
    }
    if (me == 0)
        w.head[0] = high;
    ops.cl.sync(); // the sources' counts are read
    for (int id = me; id < N; id += nt) {
        if (id >= U)
            refs_out[id] = 0;
        else if (refs_out != p.refs && p.refs[id] > 0)
            refs_out[id] = p.refs[id];
    }
    ops.cl.sync();
}

__global__ void __launch_bounds__(kMoveThreads)
    pool_move_kernel(const PoolParams p, const Planes q, const int32_t *__restrict__ remap, int32_t *tables_out,
                     void *workspace)
{
    ptx::grid_dependency_wait();
    const Ws w = carve(workspace, p.num_rows, p.num_blocks);
    const int64_t cells = (int64_t)p.num_rows * p.max_blocks;
    for (int64_t i = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; i < cells; i += (int64_t)gridDim.x * kMoveThreads) {
        const int id = p.tables[i];
        int to = -1;
        if ((uint32_t)id < (uint32_t)p.num_blocks) {
            to = remap[id];
            if (to < 0)
                atomicOr(&g_pool_error, 2u); // a table names a page of count 0
        } else if (id != -1) {
            atomicOr(&g_pool_error, 2u);
        }
        tables_out[i] = to;
    }
    const int per = 2 * q.layers * q.pieces;
    const int64_t units = (int64_t)w.head[0] * per;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int k = (int)(u / per);
        copy_piece(q, (int)(u % per), w.list2[k], w.list[k], q.block_size);
    }
}

// ---------------------------------------------------------------- launches

PoolParams params_of(const PoolArgs &a)
{
    return {a.pool.block_tables, a.pool.context_lens,  a.pool.ref_counts, a.pool.num_rows,
            a.pool.max_blocks,   a.dims.num_blocks,    a.dims.block_size};
}

Planes planes_of(const PoolArgs &a)
{
    const pa_pool &o = a.pool;
    const int elem = o.k_scale ? 1 : 2;
    Planes q{};
    q.k = static_cast<uint4 *>(o.k_cache);
    q.v = static_cast<uint4 *>(o.v_cache);
    q.ks = static_cast<uint16_t *>(o.k_scale);
    q.vs = static_cast<uint16_t *>(o.v_scale);
    q.layer_vecs = o.layer_stride / 16;
    q.scale_layer = o.scale_layer_stride / 2;
    q.layers = o.num_layers;
    q.row_vecs = a.dims.num_kv_heads * a.dims.head_dim * elem / 16;
    q.page_vecs = q.row_vecs * a.dims.block_size;
    q.pieces = (q.page_vecs * 16 + kPieceBytes - 1) / kPieceBytes;
    q.block_size = a.dims.block_size;
    q.num_kv_heads = a.dims.num_kv_heads;
    return q;
}

template <typename... P, typename... A>
int launch_ex(const char *what, void (*kernel)(P...), unsigned grid, unsigned block, unsigned cluster, bool dependent,
              void *stream, A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    if (dependent) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
    } else {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(PA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    }
    return PA_OK;
}

// CTAs of the planning cluster.
unsigned plan_ctas(int64_t work) { return work <= 4 * kThreads ? 1u : 8u; }

} // namespace

size_t pool_workspace_bytes(int num_rows, int num_blocks)
{
    return align_up((16 + 6 * (size_t)num_rows + 2 * (size_t)num_blocks) * 4, 256);
}

int launch_pool_append(const PoolArgs &a, const int32_t *rows, const int32_t *cu, int n, int32_t *slots, int num_tokens,
                       void *stream)
{
    const unsigned c = plan_ctas(std::max<int64_t>(a.dims.num_blocks, std::max(num_tokens, n)));
    return launch_ex("pool append", pool_append_kernel, c, kThreads, c, false, stream, params_of(a), rows, cu, n, slots,
                     num_tokens, a.workspace);
}

int launch_pool_fork(const PoolArgs &a, const int32_t *parents, const int32_t *children, int n, void *stream)
{
    int sms = 0;
    if (int rc = sm_count(&sms))
        return rc;
    const unsigned c = plan_ctas(std::max(a.dims.num_blocks, n));
    if (int rc = launch_ex("pool fork", pool_fork_kernel, c, kThreads, c, false, stream, params_of(a), parents, children,
                           n, a.workspace))
        return rc;
    const Planes q = planes_of(a);
    const int64_t units = std::max<int64_t>(n, (int64_t)n * 2 * q.layers * q.pieces);
    return launch_ex("pool fork copy", pool_fork_copy_kernel, (unsigned)std::min<int64_t>(units, (int64_t)sms * 8),
                     kMoveThreads, 1, true, stream, params_of(a), q, parents, children, a.workspace);
}

int launch_pool_free(const PoolArgs &a, const int32_t *rows, int n, void *stream)
{
    pool_free_kernel<<<(unsigned)n, 128, 0, static_cast<cudaStream_t>(stream)>>>(params_of(a), rows);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(PA_ERR_CUDA, "pool free launch: %s", cudaGetErrorString(e));
    return PA_OK;
}

int launch_pool_compact(const PoolArgs &a, int32_t *remap, int32_t *tables_out, int32_t *refs_out, void *stream)
{
    int sms = 0;
    if (int rc = sm_count(&sms))
        return rc;
    const unsigned c = plan_ctas(a.dims.num_blocks);
    if (int rc = launch_ex("pool compact", pool_compact_kernel, c, kThreads, c, false, stream, params_of(a), remap,
                           refs_out, a.workspace))
        return rc;
    const Planes q = planes_of(a);
    const int64_t cells = (int64_t)a.pool.num_rows * a.pool.max_blocks;
    const int64_t units = std::max<int64_t>((cells + kMoveThreads - 1) / kMoveThreads,
                                            (int64_t)(a.dims.num_blocks / 2) * 2 * q.layers * q.pieces);
    return launch_ex("pool move", pool_move_kernel, (unsigned)std::max<int64_t>(1, std::min<int64_t>(units, sms * 8)), kMoveThreads, 1, true, stream, params_of(a), q,
                     (const int32_t *)remap, tables_out, a.workspace);
}

int read_pool_error(uint32_t *code)
{
    uint32_t v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_pool_error, sizeof v);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbol(g_pool_error, &zero, sizeof zero);
    if (e != cudaSuccess)
        return fail(PA_ERR_CUDA, "reading pool error word: %s", cudaGetErrorString(e));
    *code |= (v & 3u) << 7;
    return PA_OK;
}

} // namespace pa

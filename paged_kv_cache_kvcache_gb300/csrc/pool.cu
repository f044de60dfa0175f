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
// append, fork and compact need order-dependent counts (the i-th new page is the i-th free id), so
// a call is planned where threads can scan: by one CTA for small pools (everything in shared
// memory, bound by its four dependent look-ups: row, length, last page, its count), by a cluster of
// eight for large ones (the ids scanned by all, the CTAs' totals meeting through distributed shared
// memory).  The plan is all or nothing: it is checked to the end before any state changes, and a
// refused call sets an error bit and leaves the pool as it was.  What is many (slots of a prompt
// batch, pages to move) is a second, grid-wide launch, bound by HBM; it is launched
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
constexpr int kIds = 16;              // ids per thread and round of a search for free pages
constexpr int kClusterCtas = 8;
constexpr int kMoveThreads = 256;
constexpr int kPieceBytes = 16 << 10; // one CTA's unit of page copying: 4 x 16 bytes per thread
constexpr int kRowBits = 65536;       // rows whose use in a call is kept in a bitmap in shared memory
constexpr int kSmallList = 4096;      // free ids kept in shared memory
constexpr int kPlanCells = 4096;      // table cells that a plan looks at by itself
constexpr int kCheckCtas = 608;       // CTAs that look at more, at most (a planning CTA has a thread for each)

// Workspace: header, copies int4 [num_rows], marks, starts, lens, cums [num_rows],
// list [num_blocks], list2 [num_blocks], checks [kCheckCtas].
struct Ws {
    int32_t *head; // [0] copies or moves of the call, -1: refused; [1] pieces of the copies; [2] compact: u(U)
    int4 *copies;
    int32_t *marks, *starts, *lens, *cums;
    int32_t *list, *list2;
    int32_t *checks; // verdicts of pool_check_kernel's CTAs
};

__host__ __device__ inline Ws carve(void *p, int num_rows, int num_blocks)
{
    Ws w;
    int32_t *q = static_cast<int32_t *>(p);
    w.head = q;
    w.copies = reinterpret_cast<int4 *>(q + 16);
    w.marks = q + 16 + 4 * (size_t)num_rows;
    w.starts = w.marks + num_rows;
    w.lens = w.starts + num_rows;
    w.cums = w.lens + num_rows;
    w.list = w.cums + num_rows;
    w.list2 = w.list + num_blocks;
    w.checks = w.list2 + num_blocks;
    return w;
}
constexpr int kWsRowInts = 8, kWsBlockInts = 2;

struct Smem {
    int warp[2][kWarps];
    int total[2][kClusterCtas]; // the CTAs' totals of a scan, by scan parity
    int bad;               // first CTA: refusal bits
    int want;              // and pages the call needs
    uint32_t bits[kRowBits / 32];
    int starts[kThreads], lens[kThreads];
    int list[kSmallList];
};

// Scans over the threads of one CTA (kCluster false) or of the cluster, in (CTA rank, thread)
// order.  Buffers alternate by call, so one barrier per call is enough: the next call's writes
// cannot meet a slow reader of this one's.
template <bool kCluster>
struct Team {
    Smem &s;
    int parity = 0; // of this CTA's scans (the first CTA's counting of rows makes it differ between CTAs)
    int turn = 0;   // of the team's

    __device__ explicit Team(Smem &s_) : s(s_) {}
    __device__ int ctas() const { return kCluster ? (int)cg::this_cluster().num_blocks() : 1; }
    __device__ int rank() const { return kCluster ? (int)cg::this_cluster().block_rank() : 0; }
    __device__ int threads() const { return ctas() * kThreads; }
    __device__ int thread() const { return rank() * kThreads + (int)threadIdx.x; }
    __device__ void sync()
    {
        if constexpr (kCluster)
            cg::this_cluster().sync();
        else
            __syncthreads();
    }
    // Before the first scan or refuse() every CTA must run: its shared memory is written by the others.
    // Where no sync() stands before it, the kernel begins with arrive() and waits here after its first loads.
    __device__ void arrive()
    {
        if constexpr (kCluster)
            cg::this_cluster().barrier_arrive();
    }
    __device__ void all_run()
    {
        if constexpr (kCluster)
            cg::this_cluster().barrier_wait();
    }
    // exclusive sum of v over the CTA's threads before this one; *total = the CTA's sum
    __device__ int scan_cta(int v, int *total)
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
            s.warp[parity][warp] = x;
        __syncthreads();
        const int w = s.warp[parity][lane];
        int wx = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, wx, o);
            if (lane >= o)
                wx += y;
        }
        parity ^= 1;
        *total = __shfl_sync(0xffffffffu, wx, 31);
        return __shfl_sync(0xffffffffu, wx - w, warp) + x - v;
    }
    // the same over all threads of the team
    __device__ int scan(int v, int *total)
    {
        int mine;
        const int before = scan_cta(v, &mine);
        if constexpr (!kCluster) {
            *total = mine;
            return before;
        }
        // every CTA tells every other (all threads reading all totals from there took 2 us)
        if (threadIdx.x < kClusterCtas)
            *cg::this_cluster().map_shared_rank(&s.total[turn][rank()], threadIdx.x) = mine;
        sync();
        int base = 0, sum = 0;
#pragma unroll
        for (int c = 0; c < kClusterCtas; ++c) {
            const int t = s.total[turn][c];
            base += c < rank() ? t : 0;
            sum += t;
        }
        turn ^= 1;
        *total = sum;
        return base + before;
    }
    // notes in every CTA that the call is refused: after all_run(), seen after the next sync() or scan()
    __device__ void refuse(int bits)
    {
        if constexpr (kCluster) {
            for (int c = 0; c < kClusterCtas; ++c)
                atomicOr(cg::this_cluster().map_shared_rank(&s.bad, c), bits);
        } else {
            atomicOr(&s.bad, bits);
        }
    }
    // a word of the first CTA's shared memory, after the barrier that follows its write
    __device__ int of_first(int *word)
    {
        if constexpr (kCluster)
            return *cg::this_cluster().map_shared_rank(word, 0);
        return *word;
    }
    // the first CTA's n starts and lens into every CTA's shared memory
    __device__ void rows_of_first(int n)
    {
        if constexpr (kCluster) {
            if (rank() == 0)
                return;
            const int *starts = cg::this_cluster().map_shared_rank(s.starts, 0);
            const int *lens = cg::this_cluster().map_shared_rank(s.lens, 0);
            for (int i = threadIdx.x; i < n; i += kThreads) {
                s.starts[i] = starts[i];
                s.lens[i] = lens[i];
            }
        }
    }
};

struct PoolParams {
    int32_t *tables;
    int32_t *context_lens;
    int32_t *refs;
    int32_t num_rows, max_blocks, num_blocks, block_size;
    int32_t row_tokens; // most tokens a row can hold (an int32 with room for a page)
};

// A round looks at `words` (up to kIds) ids per thread, as few as one round of all threads needs.  A
// warp's 32 * words consecutive ids begin at first_id; its lane has the ids + 32 e + lane, so that what
// it reads and writes for them is contiguous (16 consecutive ids per thread took 9 us of a round for
// the list of 16384 free pages alone, each store of a warp touching 32 sectors).
template <bool kCluster>
__device__ __forceinline__ int round_words(const Team<kCluster> &team, const PoolParams &p)
{
    return min(kIds, (p.num_blocks + team.threads() - 1) / team.threads());
}
template <bool kCluster>
__device__ __forceinline__ int first_id(const Team<kCluster> &team, const PoolParams &p, int words, int64_t base)
{
    return (int)min(base + (int64_t)(team.thread() & ~31) * words, (int64_t)p.num_blocks);
}
// Counts of this lane's ids; those past the pool count as used.
__device__ __forceinline__ void load_refs(const PoolParams &p, int words, int first, int (&r)[kIds])
{
    const int left = p.num_blocks - first - (int)(threadIdx.x & 31u);
    const int32_t *at = p.refs + first + (threadIdx.x & 31u);
#pragma unroll
    for (int e = 0; e < kIds; ++e) {
        if (e >= words)
            break;
        r[e] = 32 * e < left ? at[32 * e] : 1;
    }
}
__device__ __forceinline__ uint32_t lanes_below() { return (1u << (threadIdx.x & 31u)) - 1u; }

// The lowest `want` ids of count 0 into list; returns how many there are (at most want).  `r`:
// the counts of this thread's ids of the first round, loaded by the caller ahead of time.
template <bool kCluster>
__device__ int lowest_free(Team<kCluster> &team, const PoolParams &p, int want, int32_t *list, int (&r)[kIds])
{
    const int words = round_words(team, p);
    const int lane = threadIdx.x & 31;
    int found = 0;
    for (int64_t base = 0; base < p.num_blocks && found < want; base += (int64_t)team.threads() * words) {
        const int first = first_id(team, p, words, base);
        if (base > 0)
            load_refs(p, words, first, r);
        uint32_t m[kIds];
        int mine = 0;
#pragma unroll
        for (int e = 0; e < kIds; ++e) {
            if (e >= words)
                break;
            m[e] = __ballot_sync(0xffffffffu, r[e] == 0);
            mine += __popc(m[e]);
        }
        int sum;
        int at = found + __shfl_sync(0xffffffffu, team.scan(lane == 0 ? mine : 0, &sum), 0);
#pragma unroll
        for (int e = 0; e < kIds; ++e) {
            if (e >= words || at >= want)
                break;
            const int k = at + __popc(m[e] & lanes_below());
            if ((m[e] >> lane & 1u) && k < want)
                list[k] = first + 32 * e + lane;
            at += __popc(m[e]);
        }
        found += sum;
    }
    return min(found, want);
}

__device__ __forceinline__ int pages(int tokens, int bs) { return (tokens + bs - 1) / bs; }

// Notes that entry i of the call names row r; true if another entry already did (bitmap), or, for
// pools of very many rows, to be asked again with marked_twice after a barrier.
__device__ __forceinline__ bool mark_row(Smem &s, const Ws &w, int num_rows, int r, int i)
{
    if (num_rows <= kRowBits)
        return atomicOr(&s.bits[r >> 5], 1u << (r & 31)) >> (r & 31) & 1u;
    w.marks[r] = i;
    return false;
}
__device__ __forceinline__ bool marked_twice(const Ws &w, int num_rows, int r, int i)
{
    return num_rows > kRowBits && w.marks[r] != i;
}

// The last index of [0, n) whose entry of the ascending `a` is at most x (a[0] <= x).
__device__ __forceinline__ int last_at_most(const int32_t *a, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The same by a warp, all lanes with the same arguments: 32 entries are compared in the time of one.
__device__ __forceinline__ int last_at_most_warp(const int32_t *a, int n, int x)
{
    int lo = 0;
    while (n > 1) {
        const int step = (n + 31) / 32, at = (int)(threadIdx.x & 31u) * step;
        const int upto = __popc(__ballot_sync(0xffffffffu, at < n && a[lo + at] <= x)) - 1;
        lo += upto * step;
        n = min(step, n - upto * step);
    }
    return lo;
}

// What the planning kernels begin with: shared memory cleared, this thread's counts on their way.
template <bool kCluster>
__device__ __forceinline__ void plan_begin(Team<kCluster> &team, const PoolParams &p, int (&refs)[kIds])
{
    const int per_thread = round_words(team, p);
    load_refs(p, per_thread, first_id(team, p, per_thread, 0), refs);
    const int words = (min(p.num_rows, kRowBits) + 31) / 32;
    if (team.rank() == 0)
        for (int i = threadIdx.x; i < words; i += kThreads)
            team.s.bits[i] = 0;
    if (threadIdx.x == 0)
        team.s.bad = 0;
    __syncthreads();
}

// ---------------------------------------------------------------- checks

// Whether one of this thread's cells (from, from + step, ...) names no page in use: kFork, of the
// parents' table rows, up to their lengths; else (a compaction) of all n rows, entries of -1 excepted.
// Four at a time: each is a chain of four (two) dependent loads.
template <bool kFork>
__device__ __forceinline__ bool bad_cells(const PoolParams &p, const int32_t *parents, int n, int from,
                                          int step)
{
    constexpr int kU = 4;
    const int64_t cells = (int64_t)n * p.max_blocks;
    bool bad = false;
    for (int64_t c0 = from; c0 < cells; c0 += (int64_t)kU * step) {
        int id[kU];
        bool look[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t c = c0 + (int64_t)u * step;
            if constexpr (!kFork) {
                id[u] = c < cells ? p.tables[c] : -1;
                look[u] = id[u] != -1;
                continue;
            }
            const int i = (int)c / p.max_blocks, j = (int)c % p.max_blocks; // (cells fit an int32)
            const int r = c < cells ? parents[i] : -1;
            look[u] = (uint32_t)r < (uint32_t)p.num_rows && j < pages(p.context_lens[r], p.block_size);
            id[u] = look[u] ? p.tables[(size_t)r * p.max_blocks + j] : 0;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
            bad |= look[u] && ((uint32_t)id[u] >= (uint32_t)p.num_blocks || p.refs[id[u]] <= 0);
    }
    return bad;
}

// Many cells, over the whole grid: a verdict per CTA, which the plan behind collects.  (A fork of 64 rows
// into 256, 5632 cells, one token each and their end took 48.2 us with the cells looked at in the plan, 48.4
// with this launch, 45.7 unchecked; more cells take the planning CTA a chain of loads per 4096, this less.)
template <bool kFork>
__global__ void __launch_bounds__(256)
    pool_check_kernel(const PoolParams p, const int32_t *parents, int n, void *workspace)
{
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int any = __syncthreads_or(bad_cells<kFork>(p, parents, n, (int)blockIdx.x * 256 + (int)threadIdx.x, (int)gridDim.x * 256));
    if (threadIdx.x == 0)
        carve(workspace, p.num_rows, p.num_blocks).checks[blockIdx.x] = any;
}

// The plan's side: the verdicts of `checked` CTAs, or this thread's share of the cells itself.
template <bool kFork, bool kCluster>
__device__ __forceinline__ bool found_bad(const Team<kCluster> &team, const PoolParams &p, const Ws &w,
                                          const int32_t *parents, int n, int checked)
{
    if (checked == 0)
        return bad_cells<kFork>(p, parents, n, team.thread(), team.threads());
    return team.thread() < checked && w.checks[team.thread()] != 0;
}

// ---------------------------------------------------------------- append

// Slots of new tokens: token t of entry i is token lens[i] + t - cu[i] of its row.
__device__ __forceinline__ int slot_of(const PoolParams &p, int row, int pos)
{
    return p.tables[(size_t)row * p.max_blocks + pos / p.block_size] * p.block_size + pos % p.block_size;
}

// The rows are checked and counted by the first CTA, the free ids found by all.  kSlots: the slots
// are written here (few tokens), else by pool_slots_kernel.
template <bool kCluster, bool kSlots>
__global__ void __launch_bounds__(kThreads)
    pool_append_kernel(const PoolParams p, const int32_t *rows, const int32_t *cu, int n,
                       int32_t *slots, int num_tokens, void *workspace)
{
    __shared__ Smem sm;
    if (!kSlots)
        ptx::launch_dependents();
    ptx::grid_dependency_wait();
    Team<kCluster> team(sm);
    const Ws w = carve(workspace, p.num_rows, p.num_blocks);
    const int nt = team.threads(), me = team.thread(), bs = p.block_size;
    int refs[kIds];
    plan_begin(team, p, refs);
    const bool small = n <= kThreads; // the rows' counts stay in shared memory
    int32_t *starts = small ? sm.starts : w.starts, *lens = small ? sm.lens : w.lens;
    if (team.rank() == 0) {
        int want = 0;
        if (threadIdx.x == 0 && (cu[0] != 0 || cu[n] != num_tokens))
            atomicOr(&sm.bad, 2);
        for (int base = 0; base < n; base += kThreads) {
            const int i = base + (int)threadIdx.x;
            int need = 0, bad = 0, ctx = 0;
            if (i < n) {
                const int r = rows[i];
                const int64_t count = (int64_t)cu[i + 1] - cu[i];
                if ((uint32_t)r >= (uint32_t)p.num_rows || count < 0) {
                    bad = 2;
                } else {
                    ctx = p.context_lens[r];
                    bad = mark_row(sm, w, p.num_rows, r, i) ? 2 : 0;
                    if (ctx < 0 || ctx > p.row_tokens) {
                        bad = 2;
                    } else if (ctx + count > p.row_tokens) {
                        bad |= 1;
                    } else {
                        need = pages(ctx + (int)count, bs) - pages(ctx, bs);
                        if (count > 0 && ctx % bs != 0) { // the partly filled page must be the row's own
                            const int page = p.tables[(size_t)r * p.max_blocks + ctx / bs];
                            if ((uint32_t)page >= (uint32_t)p.num_blocks || p.refs[page] != 1)
                                bad |= 2;
                        }
                    }
                }
                lens[i] = ctx;
            }
            if (bad)
                atomicOr(&sm.bad, bad);
            int sum;
            const int at = want + team.scan_cta(need, &sum); // at most num_rows * max_blocks: an int32
            if (i < n)
                starts[i] = at;
            want += sum;
        }
        if (p.num_rows > kRowBits) {
            __syncthreads(); // all marks
            for (int i = threadIdx.x; i < n; i += kThreads)
                if ((uint32_t)rows[i] < (uint32_t)p.num_rows && marked_twice(w, p.num_rows, rows[i], i))
                    atomicOr(&sm.bad, 2);
        }
        if (threadIdx.x == 0)
            sm.want = want;
    }
    team.sync();
    const int want = team.of_first(&sm.want);
    int bad = team.of_first(&sm.bad);
    if (small)
        team.rows_of_first(n); // (there is a barrier between here and their use)
    if (want > p.num_blocks)
        bad |= 1;
    int32_t *list = !kCluster && want <= kSmallList ? sm.list : w.list;
    if (!bad && lowest_free(team, p, want, list, refs) < want)
        bad = 1;
    if (bad) {
        if (me == 0) {
            atomicOr(&g_pool_error, (uint32_t)bad);
            w.head[0] = -1;
        }
        if (kSlots)
            for (int t = me; t < num_tokens; t += nt)
                slots[t] = -1;
        team.sync(); // nobody leaves while its shared memory may be read
        return;
    }
    if (!kSlots && me == 0)
        w.head[0] = n;
    team.sync(); // the list
    for (int j = me; j < want; j += nt) { // new pages into the tables
        const int i = last_at_most(starts, n, j), id = list[j];
        p.tables[(size_t)rows[i] * p.max_blocks + pages(lens[i], bs) + j - starts[i]] = id;
        p.refs[id] = 1;
    }
    for (int i = me; i < n; i += nt) {
        const int count = cu[i + 1] - cu[i];
        if (count > 0)
            p.context_lens[rows[i]] = lens[i] + count;
    }
    if (kSlots) {
        for (int t = me; t < num_tokens; t += nt) {
            const int i = last_at_most(cu, n, t), pos = lens[i] + t - cu[i];
            const int page = pos / bs, old = pages(lens[i], bs);
            // (the tables' new entries are other threads' writes: the list has them)
            slots[t] = page < old ? slot_of(p, rows[i], pos) : list[starts[i] + page - old] * bs + pos % bs;
        }
    }
    team.sync();
}

// The slots of many tokens, from the tables as the plan left them: four tokens per thread, the
// warp's first row found once.
__global__ void __launch_bounds__(256)
    pool_slots_kernel(const PoolParams p, const int32_t *rows, const int32_t *cu, int n,
                      int32_t *slots, int num_tokens, void *workspace)
{
    ptx::grid_dependency_wait();
    const bool refused = *static_cast<const int32_t *>(workspace) < 0;
    const int64_t t0 = ((int64_t)blockIdx.x * 256 + (threadIdx.x & ~31u)) * 4, t = t0 + 4 * (threadIdx.x & 31u);
    if (t0 >= num_tokens)
        return;
    int v[4] = {-1, -1, -1, -1};
    const int m = (int)min((int64_t)4, num_tokens - t); // at most 0: nothing for this lane
    if (!refused) {
        int i = last_at_most_warp(cu, n, (int)t0);
        int begin = cu[i], end = cu[i + 1];
        int row = -1, from = 0; // the row, and the position of its token `begin`
        for (int e = 0; e < m; ++e) {
            while (end <= t + e) {
                begin = end;
                end = cu[++i + 1];
                row = -1;
            }
            if (row < 0) {
                row = rows[i];
                from = p.context_lens[row] - (end - begin);
            }
            v[e] = slot_of(p, row, from + (int)(t + e) - begin);
        }
    }
    if (m == 4 && (reinterpret_cast<uintptr_t>(slots) & 15u) == 0) {
        *reinterpret_cast<int4 *>(slots + t) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
        for (int e = 0; e < m; ++e)
            slots[t + e] = v[e];
    }
}

// ---------------------------------------------------------------- fork

template <bool kCluster>
__global__ void __launch_bounds__(kThreads)
    pool_fork_kernel(const PoolParams p, const int32_t *parents, const int32_t *children,
                     int n, int row_bytes, int checked, void *workspace)
{
    __shared__ Smem sm;
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    Team<kCluster> team(sm);
    const Ws w = carve(workspace, p.num_rows, p.num_blocks);
    const int nt = team.threads(), me = team.thread(), bs = p.block_size;
    int refs[kIds];
    plan_begin(team, p, refs);
    team.arrive();
    const bool wrong = found_bad<true>(team, p, w, parents, n, checked);
    team.all_run();
    if (wrong)
        team.refuse(2);
    const bool small = n <= kThreads;
    int32_t *starts = small ? sm.starts : w.starts, *lens = small ? sm.lens : w.lens;
    if (team.rank() == 0) {
        int want = 0, pieces = 0;
        for (int base = 0; base < n; base += kThreads) {
            const int i = base + (int)threadIdx.x;
            int need = 0, bad = 0, ctx = 0, bits = 0;
            if (i < n) {
                const int r = parents[i], c = children[i];
                if ((uint32_t)r >= (uint32_t)p.num_rows || (uint32_t)c >= (uint32_t)p.num_rows) {
                    bad = 2;
                } else {
                    ctx = p.context_lens[r];
                    bad = mark_row(sm, w, p.num_rows, c, i) ? 2 : 0;
                    if (ctx < 0 || ctx > p.row_tokens || p.context_lens[c] != 0) {
                        bad = 2;
                    } else if (ctx % bs != 0) {
                        need = 1;
                        bits = (int)(((int64_t)(ctx % bs) * row_bytes + kPieceBytes - 1) / kPieceBytes);
                    }
                }
                lens[i] = ctx;
            }
            if (bad)
                atomicOr(&sm.bad, bad);
            int sum;
            const int at = want + team.scan_cta(need, &sum);
            if (i < n)
                starts[i] = at;
            want += sum;
            const int first = pieces + team.scan_cta(bits, &sum);
            if (i < n)
                w.cums[i] = first;
            pieces += sum;
        }
        __syncthreads(); // all marks
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int r = parents[i], c = children[i];
            if ((uint32_t)r >= (uint32_t)p.num_rows || (uint32_t)c >= (uint32_t)p.num_rows)
                continue;
            bool wrong; // a child named twice, or a parent that is a child of this call
            if (p.num_rows <= kRowBits) {
                wrong = sm.bits[r >> 5] >> (r & 31) & 1u;
            } else {
                const int m = w.marks[r];
                wrong = marked_twice(w, p.num_rows, c, i) || ((uint32_t)m < (uint32_t)n && children[m] == r);
            }
            if (wrong)
                atomicOr(&sm.bad, 2);
        }
        if (threadIdx.x == 0) {
            sm.want = want;
            w.head[1] = pieces;
        }
    }
    team.sync();
    const int want = team.of_first(&sm.want);
    int bad = team.of_first(&sm.bad);
    if (small)
        team.rows_of_first(n);
    int32_t *list = !kCluster && want <= kSmallList ? sm.list : w.list;
    if (!bad && lowest_free(team, p, want, list, refs) < want)
        bad = 1;
    if (bad) {
        if (me == 0) {
            atomicOr(&g_pool_error, (uint32_t)bad);
            w.head[0] = -1;
        }
        team.sync();
        return;
    }
    team.sync(); // the list
    for (int i = me; i < n; i += nt) {
        const int r = parents[i], ctx = lens[i];
        int src = -1, dst = -1;
        if (ctx % bs != 0) {
            src = p.tables[(size_t)r * p.max_blocks + ctx / bs];
            dst = list[starts[i]];
            p.refs[dst] = 1;
        }
        w.copies[i] = make_int4(src, dst, ctx % bs, ctx / bs);
        p.context_lens[children[i]] = ctx; // (lens has the parents': no reader of this call sees it)
    }
    if (me == 0)
        w.head[0] = n;
    team.sync();
}

// Pages of all layers: K, V and, for an INT8 cache, the scales.
struct Planes {
    uint4 *k, *v;
    uint16_t *ks, *vs; // NULL: bf16 cache
    uint64_t layer_vecs, scale_layer; // layer strides in 16-byte vectors and in scales
    int32_t layers, page_vecs, row_vecs, pieces, block_size, num_kv_heads;
};

// One piece of a copy: (plane = layer, K or V), 16 KB of the first `rows` rows of page src.
struct Piece {
    const uint4 *from;
    uint4 *to;
    int n; // 16-byte vectors
    int plane, src, dst, scale_rows; // scale_rows: the page's first piece brings that many rows' scales
};
__device__ __forceinline__ Piece piece_of(const Planes &q, int plane, int piece, int src, int dst, int rows)
{
    constexpr int kVecs = kPieceBytes / 16;
    uint4 *base = (plane & 1 ? q.v : q.k) + (size_t)(plane >> 1) * q.layer_vecs + (size_t)piece * kVecs;
    return {base + (size_t)src * q.page_vecs, base + (size_t)dst * q.page_vecs,
            min(kVecs, rows * q.row_vecs - piece * kVecs), plane, src, dst, piece == 0 ? rows : 0};
}

// Copies pieces u = blockIdx.x, + gridDim.x, ... < units, of(u) giving each; a piece is loaded
// before the one before it is stored, so that a CTA always has loads in flight.
template <typename F>
__device__ __forceinline__ void copy_pieces(const Planes &q, int64_t units, F of)
{
    constexpr int kU = kPieceBytes / 16 / kMoveThreads;
    auto load = [&](const Piece &c, uint4 (&x)[kU]) {
#pragma unroll
        for (int e = 0; e < kU; ++e) {
            const int i = e * kMoveThreads + (int)threadIdx.x;
            if (i < c.n)
                x[e] = __ldcs(c.from + i);
        }
    };
    int64_t u = blockIdx.x;
    if (u >= units)
        return;
    Piece c = of(u);
    uint4 x[kU];
    load(c, x);
    for (;;) {
        u += gridDim.x;
        const bool more = u < units;
        Piece d = c;
        uint4 y[kU];
        if (more) {
            d = of(u);
            load(d, y);
        }
#pragma unroll
        for (int e = 0; e < kU; ++e) {
            const int i = e * kMoveThreads + (int)threadIdx.x;
            if (i < c.n)
                __stcs(c.to + i, x[e]);
        }
        if (q.ks && c.scale_rows > 0) { // each KV head's run of scales
            uint16_t *sc = (c.plane & 1 ? q.vs : q.ks) + (size_t)(c.plane >> 1) * q.scale_layer;
            const size_t page = (size_t)q.num_kv_heads * q.block_size;
            for (int i = threadIdx.x; i < c.scale_rows * q.num_kv_heads; i += kMoveThreads) {
                const size_t at = (size_t)(i / c.scale_rows) * q.block_size + i % c.scale_rows;
                sc[c.dst * page + at] = sc[c.src * page + at];
            }
        }
        if (!more)
            return;
        c = d;
#pragma unroll
        for (int e = 0; e < kU; ++e)
            x[e] = y[e];
    }
}

// The forked rows' tables and counts, and their partly filled pages: all layers of the i-th of
// all pieces before those of the next.
__global__ void __launch_bounds__(kMoveThreads)
    pool_fork_copy_kernel(const PoolParams p, const Planes q, const int32_t *parents,
                          const int32_t *children, void *workspace)
{
    ptx::grid_dependency_wait();
    const Ws w = carve(workspace, p.num_rows, p.num_blocks);
    const int n = w.head[0], planes = 2 * q.layers;
    if (n < 0) // refused
        return;
    const int64_t units = (int64_t)w.head[1] * planes;
    copy_pieces(q, units, [&](int64_t u) {
        const int g = (int)(u / planes), i = last_at_most_warp(w.cums, n, g);
        const int4 c = w.copies[i];
        return piece_of(q, (int)(u % planes), g - w.cums[i], c.x, c.y, c.z);
    });
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const int4 c = w.copies[i];
        const int32_t *from = p.tables + (size_t)parents[i] * p.max_blocks;
        int32_t *to = p.tables + (size_t)children[i] * p.max_blocks;
        for (int j = threadIdx.x; j < c.w; j += kMoveThreads) {
            const int id = from[j]; // (in the pool and in use: checked before the plan)
            atomicAdd(p.refs + id, 1);
            to[j] = id;
        }
        if (threadIdx.x == 0 && c.y >= 0)
            to[c.w] = c.y;
    }
}

// ---------------------------------------------------------------- free

// One CTA per row.  The context length is taken by exchange, so a row named twice is given back once.
__global__ void __launch_bounds__(128) pool_free_kernel(const PoolParams p, const int32_t *rows)
{
    __shared__ int s_ctx;
    ptx::grid_dependency_wait();
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
    if (ctx < 0 || ctx > p.row_tokens) {
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
// used ids >= U move, in order, to the free ids < U; sources and destinations are disjoint.  With
// u(id) the used ids before id, a free id < U is hole id - u(id), and a used id >= U takes
// hole u(id) - u(U).  Refused (a table names a page not in use, a count is negative): remap and the out
// arrays tell of pages that stay where they are.
template <bool kCluster>
__global__ void __launch_bounds__(kThreads)
    pool_compact_kernel(const PoolParams p, int32_t *remap, int32_t *refs_out, int checked, void *workspace)
{
    __shared__ Smem sm;
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    Team<kCluster> team(sm);
    if (threadIdx.x == 0)
        sm.bad = 0;
    __syncthreads();
    team.arrive();
    const Ws w = carve(workspace, p.num_rows, p.num_blocks);
    const int nt = team.threads(), me = team.thread(), N = p.num_blocks;
    const int words = round_words(team, p), lane = threadIdx.x & 31;
    const int64_t per_round = (int64_t)nt * words;
    bool wrong = found_bad<false>(team, p, w, nullptr, p.num_rows, checked);
    uint32_t used[kIds]; // of this warp's ids: lane l of word e is id first + 32 e + l
    auto look = [&](int first) {
        int refs[kIds];
        load_refs(p, words, first, refs);
        int sum = 0;
#pragma unroll
        for (int e = 0; e < kIds; ++e) {
            if (e >= words)
                break;
            wrong |= refs[e] < 0;
            used[e] = __ballot_sync(0xffffffffu, refs[e] != 0 && 32 * e + lane < N - first);
            sum += __popc(used[e]);
        }
        return sum;
    };
    // sum over the warps before this one, of a value that its lanes agree on
    auto before_warp = [&](int v, int *total) { return __shfl_sync(0xffffffffu, team.scan(lane == 0 ? v : 0, total), 0); };
    // U and, where one round holds all ids, u(this warp's first id)
    int mine = 0;
    const bool one = N <= per_round;
    for (int64_t base = 0; base < N; base += per_round)
        mine += look(first_id(team, p, words, base));
    team.all_run();
    if (wrong)
        team.refuse(2);
    int U, before = before_warp(mine, &U);
    if (sm.bad) {
        if (me == 0) {
            atomicOr(&g_pool_error, 2u);
            w.head[0] = -1;
        }
        for (int id = me; id < N; id += nt) {
            const int count = p.refs[id];
            remap[id] = count != 0 ? id : -1;
            if (refs_out != p.refs)
                refs_out[id] = count;
        }
        return;
    }
    // u(U): by the warp that holds id U, in the round that holds it
    int seen = 0;
    for (int64_t base = 0; base < N; base += per_round) {
        const int first = first_id(team, p, words, base);
        int sum = U;
        if (!one)
            before = seen + before_warp(look(first), &sum);
        const int at = U - first;
        if (at >= 0 && at < 32 * words && U < N) {
            int u = before;
#pragma unroll
            for (int e = 0; e < kIds; ++e)
                if (e <= at >> 5)
                    u += __popc(e < at >> 5 ? used[e] : used[e] & ((1u << (at & 31)) - 1u));
            if (lane == 0)
                w.head[2] = u;
        }
        seen += sum;
    }
    if (me == 0 && U == N)
        w.head[2] = N; // no id U: nothing moves
    team.sync();
    const int below = w.head[2];
    seen = 0;
    for (int64_t base = 0; base < N; base += per_round) {
        const int first = first_id(team, p, words, base);
        if (!one) {
            int sum;
            before = seen + before_warp(look(first), &sum);
            seen += sum;
        }
        int u0 = before;
#pragma unroll
        for (int e = 0; e < kIds; ++e) {
            if (e >= words)
                break;
            if (32 * e + lane < N - first) {
                const int x = first + 32 * e + lane, u = u0 + __popc(used[e] & lanes_below());
                if (used[e] >> lane & 1u) {
                    if (x >= U)
                        w.list2[u - below] = x;
                    else
                        remap[x] = x;
                } else {
                    if (x < U)
                        w.list[x - u] = x;
                    remap[x] = -1;
                }
            }
            u0 += __popc(used[e]);
        }
    }
    const int moves = U - below;
    if (me == 0)
        w.head[0] = moves;
    team.sync(); // both lists
    for (int k = me; k < moves; k += nt) {
        const int src = w.list2[k], dst = w.list[k];
        remap[src] = dst;
        refs_out[dst] = p.refs[src];
    }
    team.sync(); // the sources' counts are read
    for (int id = me; id < N; id += nt) {
        if (id >= U)
            refs_out[id] = 0;
        else if (refs_out != p.refs && p.refs[id] > 0)
            refs_out[id] = p.refs[id];
    }
    team.sync();
}

__global__ void __launch_bounds__(kMoveThreads)
    pool_move_kernel(const PoolParams p, const Planes q, const int32_t *remap, int32_t *tables_out,
                     void *workspace)
{
    ptx::grid_dependency_wait();
    const Ws w = carve(workspace, p.num_rows, p.num_blocks);
    const int64_t cells = (int64_t)p.num_rows * p.max_blocks;
    const int moves = w.head[0]; // -1: refused
    for (int64_t i = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; i < cells; i += (int64_t)gridDim.x * kMoveThreads) {
        const int id = p.tables[i]; // -1 or (checked before the plan) a page in use
        tables_out[i] = moves < 0 || id < 0 ? id : remap[id];
    }
    const int per = 2 * q.layers * q.pieces;
    const int64_t units = (int64_t)moves * per;
    copy_pieces(q, units, [&](int64_t u) {
        const int k = (int)(u / per), v = (int)(u % per);
        return piece_of(q, v / q.pieces, v % q.pieces, w.list2[k], w.list[k], q.block_size);
    });
}

// ---------------------------------------------------------------- launches

PoolParams params_of(const PoolArgs &a)
{
    const int64_t tokens = (int64_t)a.pool.max_blocks * a.dims.block_size;
    return {a.pool.block_tables, a.pool.context_lens, a.pool.ref_counts,  a.pool.num_rows,
            a.pool.max_blocks,   a.dims.num_blocks,   a.dims.block_size,
            (int32_t)std::min<int64_t>(tokens, INT32_MAX - a.dims.block_size)};
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
int launch_ex(const char *what, void (*kernel)(P...), unsigned grid, unsigned block, unsigned cluster, void *stream,
              A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.stream = static_cast<cudaStream_t>(stream);
    // every kernel here waits for the launch before it (and may be set up during it)
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(PA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    }
    return PA_OK;
}

// One CTA looks through 16384 ids in a round, a cluster through 131072, but it takes 2 us more to
// start and meet.  A search for free pages ends when it has found enough.  8 tokens appended to 8
// rows, then freed, one CTA against the cluster, in a pool empty / half full / 0.95 full: 32768 pages
// 7.2 / 10.2 / 10.9 us against 9.3 / 9.8 / 9.9, 49152 pages 7.0 / 10.8 / 12.7 against 9.4 / 10.1 / 9.3.
// A compaction goes through all ids, three times if they take several rounds: 8192 pages 6.3 us
// against 7.8, 16384 pages 8.3 / 8.1, 32768 pages 19.1 / 8.7.
constexpr int kRoundIds = kThreads * kIds;
bool search_by_cluster(const PoolArgs &a) { return a.dims.num_blocks > 2 * kRoundIds; }
bool compact_by_cluster(const PoolArgs &a) { return a.dims.num_blocks > kRoundIds; }

// CTAs of the launch that looks at a call's table cells; 0: they are few, the plan does it
int check_ctas(int64_t cells)
{
    return cells <= kPlanCells ? 0 : (int)std::min<int64_t>(kCheckCtas, (cells + 1023) / 1024);
}

} // namespace

size_t pool_workspace_bytes(int num_rows, int num_blocks)
{
    return align_up((16 + kWsRowInts * (size_t)num_rows + kWsBlockInts * (size_t)num_blocks + kCheckCtas) * 4, 256);
}

int launch_pool_append(const PoolArgs &a, const int32_t *rows, const int32_t *cu, int n, int32_t *slots, int num_tokens,
                       void *stream)
{
    // a planning CTA writes a few thousand slots in the time that another launch takes
    const bool many = num_tokens > 4 * kThreads, cluster = search_by_cluster(a);
    auto kernel = many ? (cluster ? pool_append_kernel<true, false> : pool_append_kernel<false, false>)
                       : (cluster ? pool_append_kernel<true, true> : pool_append_kernel<false, true>);
    const unsigned c = cluster ? kClusterCtas : 1;
    if (int rc = launch_ex("pool append", kernel, c, kThreads, c, stream, params_of(a), rows, cu, n, slots,
                           num_tokens, a.workspace))
        return rc;
    if (!many)
        return PA_OK;
    return launch_ex("pool slots", pool_slots_kernel, (unsigned)(((int64_t)num_tokens + 1023) / 1024), 256, 1, stream,
                     params_of(a), rows, cu, n, slots, num_tokens, a.workspace);
}

int launch_pool_fork(const PoolArgs &a, const int32_t *parents, const int32_t *children, int n, void *stream)
{
    int sms = 0;
    if (int rc = sm_count(&sms))
        return rc;
    const Planes q = planes_of(a);
    const bool cluster = search_by_cluster(a);
    const unsigned c = cluster ? kClusterCtas : 1;
    const int checked = check_ctas((int64_t)n * a.pool.max_blocks);
    if (checked > 0)
        if (int rc = launch_ex("pool check", pool_check_kernel<true>, (unsigned)checked, 256, 1, stream, params_of(a),
                               parents, n, a.workspace))
            return rc;
    if (int rc = launch_ex("pool fork", cluster ? pool_fork_kernel<true> : pool_fork_kernel<false>, c, kThreads, c,
                           stream, params_of(a), parents, children, n, (int)(q.row_vecs * 16), checked, a.workspace))
        return rc;
    const int64_t units = std::max<int64_t>(n, (int64_t)n * 2 * q.layers * q.pieces);
    return launch_ex("pool fork copy", pool_fork_copy_kernel, (unsigned)std::min<int64_t>(units, (int64_t)sms * 8),
                     kMoveThreads, 1, stream, params_of(a), q, parents, children, a.workspace);
}

int launch_pool_free(const PoolArgs &a, const int32_t *rows, int n, void *stream)
{
    return launch_ex("pool free", pool_free_kernel, (unsigned)n, 128, 1, stream, params_of(a), rows);
}

int launch_pool_compact(const PoolArgs &a, int32_t *remap, int32_t *tables_out, int32_t *refs_out, void *stream)
{
    int sms = 0;
    if (int rc = sm_count(&sms))
        return rc;
    const bool cluster = compact_by_cluster(a);
    const unsigned c = cluster ? kClusterCtas : 1;
    const int64_t cells = (int64_t)a.pool.num_rows * a.pool.max_blocks;
    const int checked = check_ctas(cells);
    if (checked > 0)
        if (int rc = launch_ex("pool check", pool_check_kernel<false>, (unsigned)checked, 256, 1, stream, params_of(a),
                               (const int32_t *)nullptr, a.pool.num_rows, a.workspace))
            return rc;
    if (int rc = launch_ex("pool compact", cluster ? pool_compact_kernel<true> : pool_compact_kernel<false>, c, kThreads,
                           c, stream, params_of(a), remap, refs_out, checked, a.workspace))
        return rc;
    const Planes q = planes_of(a);
    const int64_t units = std::max<int64_t>((cells + kMoveThreads - 1) / kMoveThreads,
                                            (int64_t)(a.dims.num_blocks / 2) * 2 * q.layers * q.pieces);
    return launch_ex("pool move", pool_move_kernel, (unsigned)std::max<int64_t>(1, std::min<int64_t>(units, sms * 8)),
                     kMoveThreads, 1, stream, params_of(a), q, (const int32_t *)remap, tables_out, a.workspace);
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

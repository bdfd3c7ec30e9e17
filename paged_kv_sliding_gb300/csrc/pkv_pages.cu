// The pages of a cache, kept on the device: rows of a page table grow, fork, are freed and
// packed together, and the pages themselves are copied, without a host round trip.
//
// State: table [num_rows, row_stride] page ids, lens [num_rows] tokens of a row (its first
// ceil(len / P) entries are in use) and refs [num_pages], how many entries in use name a
// page. A page is free iff its refs are 0, so nothing else has to be kept, and "the lowest
// free ids, in the order of the call" makes every result a function of the inputs alone.
//   extend: ceil((len + add) / P) - ceil(len / P) new pages for each row, slots of the tokens
//   fork:   the child's row names the parent's full pages (refs + 1); a last page that is
//           not full is one the child will write, so it gets a free one and (src, dst)
//   free:   refs - 1 for the row's pages, len = 0
//   compact: with n live pages, the live ids >= n move to the free ids < n, both ascending
// extend and fork take their entries together: if one does not fit (a row out of range or
// named twice, no page left) the call changes nothing and records why.
//
// Free pages have to be ranked, a scan over refs. rank_kernel does it, with the entries'
// own prefix sums and checks, as one cluster of 8 CTAs, whose barriers and shared memories
// spare the second and third launch of a scan over the grid, or CTAs that spin on one
// another: every warp counts a segment of its own, the 256 counts are exchanged, and a
// second pass over the segment (now in L2) writes the ids of the ranks that are wanted.
// What it found is applied by a CTA to each entry over the whole GPU: on the cluster's 8
// SMs alone, extending 256 rows by 512 thousand tokens took 33 us, now a tenth of it.
// Bound by latency: chains of dependent loads, over 4 bytes a page and entry.
#include <cooperative_groups.h>

#include <string>
#include <utility>

#include "pkv_internal.h"
#include "pkv_nvtx.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kCtas = 8;  // portable cluster size
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kAllWarps = kCtas * kWarps;
constexpr int kDeep = 4;  // 16-byte loads that a lane keeps in flight over refs
constexpr int kApplyThreads = 256;
constexpr int32_t kBad = 1, kTooMany = 2;  // of the verdict word

struct PoolParams {
    int32_t *table, *lens, *refs;
    int64_t row_stride;
    int32_t num_rows, num_pages, page_size;
    int32_t *status;
    // workspace
    int32_t *claim;      // [num_rows] entry of the call that named a row
    int32_t *first;      // [num_rows] rank of an entry's first new page
    int64_t *first_slot; // [num_rows] its first slot in the call's slots (fork: the parent's length,
                         // which a child's may replace when a row is both)
    int32_t *free_ids;   // [num_pages] the free pages by rank (compact: a page's rank)
    int32_t *word;       // extend, fork: what does not fit; compact: the live pages
    int64_t *tokens;     // extend: the call's new tokens
};

// ceil(x / p) for 0 <= x < 2^31.
__device__ __forceinline__ int ceil_div(int64_t x, int p) { return (int)(((unsigned)x + (unsigned)p - 1u) / (unsigned)p); }

// What every warp of the cluster counted, in each CTA's shared memory: new pages, free
// pages and new tokens of its segment.
struct Board {
    uint32_t pages[kAllWarps];
    uint32_t frees[kAllWarps];
    long long tokens[kAllWarps];
};

// Neighbouring segments go to different CTAs: the lowest free pages, which a call wants, lie
// in the first few (all in one CTA, ranking 32 thousand of them took 8 us longer).
__device__ __forceinline__ int warp_of_cluster(const cg::cluster_group &cluster, int warp)
{
    return warp * kCtas + (int)cluster.block_rank();
}

__device__ __forceinline__ uint32_t warp_sum(uint32_t x) { return __reduce_add_sync(0xffffffffu, x); }

__device__ __forceinline__ long long warp_sum64(long long x)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Exclusive prefix over the lanes of a warp.
__device__ __forceinline__ int warp_before(int x, int lane)
{
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o)
            s += y;
    }
    return s - x;
}

__device__ __forceinline__ long long warp_before64(long long x, int lane)
{
    long long s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o)
            s += y;
    }
    return s - x;
}

// Segment of `n` items that warp gw of the cluster handles: [lo, hi), multiples of `unit`.
__device__ __forceinline__ void segment(int n, int unit, int gw, int &lo, int &hi)
{
    const int per = ((n + kAllWarps - 1) / kAllWarps + unit - 1) / unit * unit;
    lo = (int)min((long long)n, (long long)gw * per);
    hi = (int)min((long long)n, (long long)lo + per);
}

// refs of the four pages from p on (a page past the end reads as in use).
__device__ __forceinline__ int4 refs4(const int32_t *refs, int p, int end)
{
    if (p + 4 <= end)
        return __ldcg(reinterpret_cast<const int4 *>(refs + p));
    int4 r = make_int4(1, 1, 1, 1);
    if (p < end)
        r.x = __ldcg(refs + p);
    if (p + 1 < end)
        r.y = __ldcg(refs + p + 1);
    if (p + 2 < end)
        r.z = __ldcg(refs + p + 2);
    return r;
}

__device__ __forceinline__ int count_free(const int4 &r) { return (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0); }

// Free pages of [lo, hi), which starts at a multiple of 4.
__device__ int segment_free(const int32_t *refs, int lo, int hi, int lane)
{
    int n = 0, base = lo;
    for (; base + 128 * kDeep <= hi; base += 128 * kDeep) {
        int4 r[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u)
            r[u] = __ldcg(reinterpret_cast<const int4 *>(refs + base + 128 * u) + lane);
#pragma unroll
        for (int u = 0; u < kDeep; ++u)
            n += count_free(r[u]);
    }
    for (int p = base + 4 * lane; p < hi; p += 128)
        n += count_free(refs4(refs, p, hi));
    return (int)warp_sum((uint32_t)n);
}

// The ids of the free pages of [lo, hi), the first of which has rank `rank`, into
// free_ids[rank], as far as ranks below `want` go.
__device__ void write_free(const PoolParams &p, int lo, int hi, int rank, int want, int lane)
{
    for (int base = lo; base < hi && rank < want; base += 128 * kDeep) {
        int4 r[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u)
            r[u] = refs4(p.refs, base + 128 * u + 4 * lane, hi);
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            const int at = base + 128 * u + 4 * lane;
            const uint32_t m0 = __ballot_sync(0xffffffffu, r[u].x == 0), m1 = __ballot_sync(0xffffffffu, r[u].y == 0);
            const uint32_t m2 = __ballot_sync(0xffffffffu, r[u].z == 0), m3 = __ballot_sync(0xffffffffu, r[u].w == 0);
            const uint32_t lower = (1u << lane) - 1u;
            int k = rank + __popc(m0 & lower) + __popc(m1 & lower) + __popc(m2 & lower) + __popc(m3 & lower);
            if (r[u].x == 0 && k < want)
                p.free_ids[k] = at;
            k += r[u].x == 0;
            if (r[u].y == 0 && k < want)
                p.free_ids[k] = at + 1;
            k += r[u].y == 0;
            if (r[u].z == 0 && k < want)
                p.free_ids[k] = at + 2;
            k += r[u].z == 0;
            if (r[u].w == 0 && k < want)
                p.free_ids[k] = at + 3;
            rank += __popc(m0) + __popc(m1) + __popc(m2) + __popc(m3);
        }
    }
}

// Tell every CTA of the cluster what this warp counted (8 lanes, a CTA each; the CTAs have
// all started: the caller waited for it), and wait for the others. Afterwards the board is
// only read where it lies, so that a CTA may leave when it likes.
__device__ void exchange(cg::cluster_group &cluster, Board &b, int gw, int lane, uint32_t pages, uint32_t frees,
                         long long tokens)
{
    if (lane < kCtas) {
        Board *to = cluster.map_shared_rank(&b, lane);
        to->pages[gw] = pages;
        to->frees[gw] = frees;
        to->tokens[gw] = tokens;
    }
    cluster.sync();
}

// Sum over the warps before gw, and over all, of one of the board's arrays (32-bit counts:
// as halves, whose sums stay below 2^32).
__device__ __forceinline__ void before_and_total(const uint32_t *all, int gw, int lane, long long &before, long long &total)
{
    uint32_t s_lo = 0, s_hi = 0, t_lo = 0, t_hi = 0;
#pragma unroll
    for (int k = 0; k < kAllWarps / 32; ++k) {
        const uint32_t v = all[32 * k + lane], lo = v & 0xffffu, hi = v >> 16;
        const bool mine = 32 * k + lane < gw;
        t_lo += lo;
        t_hi += hi;
        s_lo += mine ? lo : 0;
        s_hi += mine ? hi : 0;
    }
    before = warp_sum(s_lo) + ((long long)warp_sum(s_hi) << 16);
    total = warp_sum(t_lo) + ((long long)warp_sum(t_hi) << 16);
}

__device__ __forceinline__ void before_and_total(const long long *all, int gw, int lane, long long &before,
                                                 long long &total)
{
    long long s = 0, t = 0;
#pragma unroll
    for (int k = 0; k < kAllWarps / 32; ++k) {
        const long long v = all[32 * k + lane];
        t += v;
        s += 32 * k + lane < gw ? v : 0;
    }
    before = warp_sum64(s);
    total = warp_sum64(t);
}

__device__ __forceinline__ bool len_fine(const PoolParams &p, int64_t len)
{
    return len >= 0 && ceil_div(len, p.page_size) <= p.row_stride;
}

enum Op { kExtend, kFork };

// Rank the pages and slots of a call's entries, and the free pages; the verdict word says
// whether the call can be done. kExtend: rows, add. kFork: rows = children, add = parents.
template <Op OP>
__global__ void __launch_bounds__(kThreads) rank_kernel(const PoolParams p, const int32_t *rows, const int32_t *add, int n,
                                                        bool slots, int64_t slots_capacity)
{
    __shared__ Board b;
    cg::cluster_group cluster = cg::this_cluster();
    auto started = cluster.barrier_arrive();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, gw = warp_of_cluster(cluster, warp);
    const int P = p.page_size;
    grid_dependency_wait();
    grid_launch_dependents();
    if (gw == 0 && lane == 0)
        *p.word = 0;

    // What each entry of the warp's segment needs, and the free pages of its segment. The
    // first 32 entries (nearly always all) stay in registers for the second pass.
    int e_lo, e_hi, p_lo, p_hi;
    segment(n, 1, gw, e_lo, e_hi);
    segment(p.num_pages, 4, gw, p_lo, p_hi);
    struct Entry {
        int row, more;  // more: add, or the parent
        int need;       // new pages; -1: does not fit
        long long tokens;
    };
    auto index = [&](int i) -> Entry { return {i < e_hi ? rows[i] : -1, i < e_hi ? add[i] : 0, 0, 0}; };
    auto measure = [&](int i, Entry &e) {
        if (i >= e_hi)
            return;
        e.need = -1;
        if ((unsigned)e.row >= (unsigned)p.num_rows)
            return;
        const int64_t len = p.lens[e.row];
        if (OP == kExtend) {
            if (e.more < 0 || !len_fine(p, len) || len + e.more > INT32_MAX || !len_fine(p, len + e.more))
                return;
            e.tokens = e.more;
            e.need = ceil_div(len + e.more, P) - ceil_div(len, P);
        } else {
            if ((unsigned)e.more >= (unsigned)p.num_rows || len != 0)
                return;
            e.tokens = p.lens[e.more];
            e.need = !len_fine(p, e.tokens) ? -1 : (int)((unsigned)e.tokens % (unsigned)P != 0);
        }
    };
    Entry first = index(e_lo + lane);
    const int frees = segment_free(p.refs, p_lo, p_hi, lane);
    long long pages = 0, tokens = 0;
    bool bad = false;
    for (int i0 = e_lo; i0 < e_hi; i0 += 32) {
        const int i = i0 + lane;
        Entry e = i0 == e_lo ? first : index(i);
        measure(i, e);
        if (e.need < 0)
            bad = true;
        else if (i < e_hi)
            p.claim[e.row] = i;
        pages += max(e.need, 0);
        tokens += e.tokens;
        if (i0 == e_lo)
            first = e;
    }
    pages = warp_sum64(pages);
    tokens = warp_sum64(tokens);
    cluster.barrier_wait(std::move(started));
    // (more pages than there are: too many in any case)
    exchange(cluster, b, gw, lane, (uint32_t)min(pages, p.num_pages + 1LL), (uint32_t)frees, tokens);

    // Ranks: an entry's first new page and slot, the ids of the free pages that are wanted.
    int claimed = e_lo + lane < e_hi && (unsigned)first.row < (unsigned)p.num_rows ? __ldcg(p.claim + first.row) : 0;
    long long page_at, want, rank, there, token_at = 0, all_tokens = 0;
    before_and_total(b.pages, gw, lane, page_at, want);
    before_and_total(b.frees, gw, lane, rank, there);
    if (OP == kExtend)
        before_and_total(b.tokens, gw, lane, token_at, all_tokens);
    if (want <= there)
        write_free(p, p_lo, p_hi, (int)rank, (int)want, lane);
    for (int i0 = e_lo; i0 < e_hi; i0 += 32) {
        const int i = i0 + lane;
        Entry e = first;
        if (i0 != e_lo) {
            e = index(i);
            measure(i, e);
            claimed = i < e_hi && (unsigned)e.row < (unsigned)p.num_rows ? __ldcg(p.claim + e.row) : 0;
        }
        const int need = max(e.need, 0), before = warp_before(need, lane);
        const long long t_before = OP == kExtend ? warp_before64(e.tokens, lane) : 0;
        if (i < e_hi) {
            p.first[i] = (int32_t)(page_at + before);
            p.first_slot[i] = OP == kExtend ? token_at + t_before : e.tokens;
            if ((unsigned)e.row < (unsigned)p.num_rows && claimed != i)
                bad = true;  // another entry names the row too
        }
        page_at += __shfl_sync(0xffffffffu, before + need, 31);
        token_at += __shfl_sync(0xffffffffu, t_before + e.tokens, 31);
    }
    if (gw == 0 && lane == 0) {
        *p.tokens = all_tokens;
        if (want > there)
            atomicOr(p.word, kTooMany);
    }
    if (bad || (OP == kExtend && slots && all_tokens > slots_capacity))
        atomicOr(p.word, kBad);
}

// Whether the ranked call can be done; if not, block 0 records why.
__device__ bool granted(const PoolParams &p)
{
    const int verdict = *p.word;
    if (verdict && blockIdx.x == 0 && threadIdx.x == 0)
        record_status(p.status, verdict & kBad ? PKV_ERR_DEVICE_BOUNDS : PKV_ERR_OOM);
    return verdict == 0;
}

// One CTA an entry.
__global__ void __launch_bounds__(kApplyThreads) extend_kernel(const PoolParams p, const int32_t *rows, const int32_t *add,
                                                               int64_t *slots, int64_t slots_capacity)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int i = blockIdx.x, P = p.page_size;
    const bool done = granted(p);
    if (slots)  // behind the call's tokens no slot: the calls that take them skip it
        for (int64_t k = (done ? *p.tokens : 0) + (int64_t)i * kApplyThreads + threadIdx.x; k < slots_capacity;
             k += (int64_t)gridDim.x * kApplyThreads)
            slots[k] = -1;
    if (!done)
        return;
    const int row = rows[i], len = p.lens[row], more = add[i];
    const int have = ceil_div(len, P), upto = ceil_div((int64_t)len + more, P);
    int32_t *entries = p.table + row * p.row_stride;
    const int32_t *fresh = p.free_ids + p.first[i];
    if (slots) {
        int64_t *out = slots + p.first_slot[i];
        int last = 0;      // the page that is filled up first
        int64_t skip = 0;  // its tokens, if the entry is no page id: they have no slot
        if (more > 0 && (unsigned)len % (unsigned)P != 0) {
            last = entries[have - 1];
            if ((unsigned)last >= (unsigned)p.num_pages) {
                skip = min((int64_t)more, (int64_t)have * P - len);
                for (int64_t t = threadIdx.x; t < skip; t += kApplyThreads)
                    out[t] = -1;
                if (threadIdx.x == 0)
                    record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
            }
        }
        constexpr int U = 4;  // tokens of a thread in flight
        for (int64_t t0 = skip + threadIdx.x; t0 < more; t0 += U * kApplyThreads) {
            int page[U], in[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t t = t0 + u * kApplyThreads;
                const unsigned at = (unsigned)(len + t);
                const int k = at / (unsigned)P;
                in[u] = at - (unsigned)k * P;
                page[u] = k < have ? last : t < more ? fresh[k - have] : 0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t0 + u * kApplyThreads < more)
                    out[t0 + u * kApplyThreads] = (int64_t)page[u] * P + in[u];
        }
    }
    for (int64_t k = (int64_t)have + threadIdx.x; k < upto; k += kApplyThreads) {
        const int page = fresh[k - have];
        entries[k] = page;
        p.refs[page] = 1;
    }
    __syncthreads();  // every thread has the row's old length
    if (threadIdx.x == 0)
        p.lens[row] = len + more;
}

__global__ void __launch_bounds__(kApplyThreads) fork_kernel(const PoolParams p, const int32_t *children,
                                                             const int32_t *parents, int32_t *src, int32_t *dst)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int i = blockIdx.x;
    if (!granted(p)) {
        if (threadIdx.x == 0)
            src[i] = dst[i] = -1;
        return;
    }
    const int child = children[i], len = (int)p.first_slot[i], full = len / p.page_size;
    const int32_t *from = p.table + parents[i] * p.row_stride;
    int32_t *to = p.table + child * p.row_stride;
    for (int k = threadIdx.x; k < full; k += kApplyThreads) {
        const int page = from[k];
        to[k] = page;
        if ((unsigned)page < (unsigned)p.num_pages)
            atomicAdd(p.refs + page, 1);
        else
            record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
    }
    if (threadIdx.x == 0) {
        int a = -1, z = -1;
        if (len % p.page_size != 0) {
            a = from[full];
            z = p.free_ids[p.first[i]];
            to[full] = z;
            p.refs[z] = 1;
            if ((unsigned)a >= (unsigned)p.num_pages) {
                a = z = -1;
                record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
            }
        }
        src[i] = a;
        dst[i] = z;
        p.lens[child] = len;
    }
}

// One CTA an entry, each taken by itself: whoever finds a row's length gives its pages
// back, so that a row named twice is freed once.
__global__ void __launch_bounds__(kApplyThreads) free_kernel(const PoolParams p, const int32_t *rows)
{
    __shared__ int shared_len;
    grid_dependency_wait();
    grid_launch_dependents();
    const int row = rows[blockIdx.x];
    if (threadIdx.x == 0) {
        int len = 0;
        if ((unsigned)row < (unsigned)p.num_rows && len_fine(p, p.lens[row]))
            len = atomicExch(p.lens + row, 0);
        else
            record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
        shared_len = len;
    }
    __syncthreads();
    const int pages = ceil_div(shared_len, p.page_size);
    const int32_t *entries = p.table + row * p.row_stride;
    for (int k = threadIdx.x; k < pages; k += kApplyThreads) {
        const int page = entries[k];
        if ((unsigned)page >= (unsigned)p.num_pages) {
            record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
        } else if (atomicSub(p.refs + page, 1) <= 0) {  // more entries named the page than were counted
            atomicAdd(p.refs + page, 1);
            record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
        }
    }
}

// The moves of a compaction: src, dst, their number, refs_out, and in the workspace each
// moved page's rank and the number of live pages.
__global__ void __launch_bounds__(kThreads) moves_kernel(const PoolParams p, int32_t *refs_out, int32_t *src,
                                                         int32_t *dst, int max_moves, int32_t *count)
{
    __shared__ Board b;
    __shared__ int edge_live;  // live pages below n_live in the segment that n_live falls into
    cg::cluster_group cluster = cg::this_cluster();
    auto started = cluster.barrier_arrive();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, gw = warp_of_cluster(cluster, warp);
    grid_dependency_wait();
    grid_launch_dependents();
    int lo, hi;
    segment(p.num_pages, 4, gw, lo, hi);
    const int frees = segment_free(p.refs, lo, hi, lane);
    cluster.barrier_wait(std::move(started));
    exchange(cluster, b, gw, lane, (uint32_t)(hi - lo - frees), (uint32_t)frees, 0);  // pages: the live ones
    long long live_before, n_live, free_before, n_free;
    before_and_total(b.pages, gw, lane, live_before, n_live);
    before_and_total(b.frees, gw, lane, free_before, n_free);
    // The holes are the free pages below n_live: a warp's first has rank free_before. The
    // movers are the live pages from n_live on: rank = live pages before it minus those
    // below n_live, n_live - holes.
    const int N = (int)n_live;
    const int per = ((p.num_pages + kAllWarps - 1) / kAllWarps + 3) / 4 * 4;
    const int edge = min(N / max(per, 1), kAllWarps - 1);
    if (warp == 0) {
        int e_lo, e_hi;
        segment(p.num_pages, 4, edge, e_lo, e_hi);
        const int n = max(min(e_hi, N) - e_lo, 0) - segment_free(p.refs, e_lo, min(e_hi, N), lane);
        if (lane == 0)
            edge_live = n;
    }
    __syncthreads();
    long long edge_before, unused;
    before_and_total(b.pages, edge, lane, edge_before, unused);
    const int live_below = (int)edge_before + edge_live;
    const int moves = N - live_below;  // as many movers as holes
    const bool fits = moves <= max_moves;
    if (fits) {
        int live_rank = (int)live_before - live_below, free_rank = (int)free_before;
        for (int base = lo; base < hi; base += 128) {
            const int at = base + 4 * lane;
            const int4 r4 = refs4(p.refs, at, hi);
            const int r[4] = {r4.x, r4.y, r4.z, r4.w};
            int f = 0, l = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f += at + k < hi && r[k] == 0;
                l += at + k < hi && r[k] != 0;
            }
            const int f_before = warp_before(f, lane), l_before = warp_before(l, lane);
            int fr = free_rank + f_before, lr = live_rank + l_before;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int q = at + k;
                if (q >= hi)
                    break;
                if (refs_out != p.refs && (q >= N || r[k] != 0))  // what stays, and the ids given up
                    refs_out[q] = q < N ? r[k] : 0;
                if (r[k] == 0) {
                    if (q < N)
                        dst[fr] = q;
                    else
                        p.free_ids[q] = -1;
                    ++fr;
                } else {
                    if (q >= N) {
                        src[lr] = q;
                        p.free_ids[q] = lr;
                    }
                    ++lr;
                }
            }
            free_rank += __shfl_sync(0xffffffffu, f_before + f, 31);
            live_rank += __shfl_sync(0xffffffffu, l_before + l, 31);
        }
    }
    cluster.sync();
    const int at = gw * 32 + lane;
    if (fits) {
        for (int k = at; k < moves; k += kAllWarps * 32) {
            const int from = __ldcg(src + k);
            refs_out[__ldcg(dst + k)] = __ldcg(p.refs + from);
            if (refs_out == p.refs)
                refs_out[from] = 0;
        }
    } else if (refs_out != p.refs) {
        for (int q = at; q < p.num_pages; q += kAllWarps * 32)
            refs_out[q] = __ldcg(p.refs + q);
    }
    if (at == 0) {
        *count = fits ? moves : 0;
        *p.word = fits ? N : INT32_MAX;  // ids below it stay what they are
        if (!fits)
            record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
    }
}

// Table entries by the moves: one CTA a row.
constexpr int kRewriteThreads = 128;

__global__ void __launch_bounds__(kRewriteThreads) rewrite_kernel(const PoolParams p, int32_t *table_out, int64_t out_stride,
                                                      int32_t *lens_out, const int32_t *dst)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int row = blockIdx.x;
    const int n_live = *p.word;
    const int64_t len = p.lens[row];
    if (threadIdx.x == 0 && lens_out != p.lens)  // a length that is none too: out is as broken as the pool
        lens_out[row] = (int32_t)len;
    if (!len_fine(p, len)) {
        if (threadIdx.x == 0)
            record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
        return;
    }
    const int n = ceil_div(len, p.page_size);
    const int32_t *from = p.table + row * p.row_stride;
    int32_t *to = table_out + row * out_stride;
    for (int k = threadIdx.x; k < n; k += kRewriteThreads) {
        int page = from[k];
        if ((unsigned)page >= (unsigned)p.num_pages) {
            record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
        } else if (page >= n_live) {
            const int rank = p.free_ids[page];
            if (rank >= 0)
                page = dst[rank];
            else
                record_status(p.status, PKV_ERR_DEVICE_BOUNDS);  // an entry that refs did not count
        }
        to[k] = page;
    }
}

// Whole pages of K and V, of every layer, in 16-byte granules: a CTA takes tiles of
// kTile granules of one cache, each thread kUnroll of them, all loaded before the first
// is stored. Bound by HBM.
constexpr int kCopyThreads = 256, kUnroll = 8, kTile = kCopyThreads * kUnroll;

struct CopyParams {
    uint8_t *k, *v;
    int64_t layer_bytes;  // from one layer's cache to the next
    int32_t num_layers, num_pages;
    int32_t granules;     // of a page
    int32_t n;
    const int32_t *src, *dst, *count;
    int32_t *status;
};

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int n = p.count ? max(0, min(p.n, *p.count)) : p.n;
    const long long per_cache = ((long long)n * p.granules + kTile - 1) / kTile;
    for (long long tile = blockIdx.x; tile < per_cache * 2 * p.num_layers; tile += gridDim.x) {
        const long long which = tile / per_cache;
        uint8_t *cache = (which & 1 ? p.v : p.k) + (which >> 1) * p.layer_bytes;
        const long long g0 = (tile - which * per_cache) * kTile;
        const int pair0 = (int)(g0 / p.granules), rest = (int)(g0 - (long long)pair0 * p.granules);
        uint4 x[kUnroll];
        int64_t to[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const unsigned g = (unsigned)rest + u * kCopyThreads + threadIdx.x;
            const int step = g / (unsigned)p.granules;
            const int pair = pair0 + step;
            to[u] = -1;
            if (pair < n) {
                const int a = p.src[pair], z = p.dst[pair];
                if (a >= p.num_pages || z >= p.num_pages) {
                    if (p.status)
                        record_status(p.status, PKV_ERR_DEVICE_BOUNDS);
                } else if (a >= 0 && z >= 0) {
                    const int64_t in = (int64_t)(g - (unsigned)step * (unsigned)p.granules) * 16;
                    const int64_t page = (int64_t)p.granules * 16;
                    x[u] = *reinterpret_cast<const uint4 *>(cache + a * page + in);
                    to[u] = z * page + in;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (to[u] >= 0)
                *reinterpret_cast<uint4 *>(cache + to[u]) = x[u];
    }
}

int refuse(int status, const char *call, const char *what)
{
    set_last_error((std::string(call) + ": " + what).c_str());
    return status;
}

bool misaligned(const void *p, uintptr_t a) { return (uintptr_t)p % a != 0; }

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

struct Carve {
    int64_t claim, first, first_slot, free_ids, word, tokens, bytes;
};

Carve carve(int32_t num_rows, int32_t num_pages)
{
    Carve c{};
    c.claim = 0;
    c.first = align256(c.claim + 4LL * num_rows);
    c.first_slot = align256(c.first + 4LL * num_rows);
    c.free_ids = align256(c.first_slot + 8LL * num_rows);
    c.word = align256(c.free_ids + 4LL * num_pages);
    c.tokens = c.word + 8;
    c.bytes = c.word + 256;
    return c;
}

// The pool's checks, and its parameters.
int take_pool(const char *call, const pkv_page_pool *pool, PoolParams &p)
{
    if (!pool)
        return refuse(PKV_ERR_INVALID_ARG, call, "pool is NULL");
    if (pool->num_rows < 0 || pool->num_pages < 0 || pool->row_stride < 0 || pool->page_size <= 0)
        return refuse(PKV_ERR_INVALID_ARG, call, "negative size, or page_size <= 0");
    // (segments and loop steps of the scans are rounded up in 32 bits)
    if (pool->row_stride > INT32_MAX || pool->num_pages > INT32_MAX - 4096 || pool->num_rows > INT32_MAX - 4096)
        return refuse(PKV_ERR_UNSUPPORTED, call, "a row or a pool of about 2^31 pages, or as many rows");
    if ((pool->num_rows > 0 && (!pool->lens || (pool->row_stride > 0 && !pool->table))) ||
        (pool->num_pages > 0 && !pool->refs) || !pool->status)
        return refuse(PKV_ERR_INVALID_ARG, call, "table, lens, refs and status are required");
    if (misaligned(pool->table, 4) || misaligned(pool->lens, 4) || misaligned(pool->refs, 16) ||
        misaligned(pool->status, 4) || misaligned(pool->workspace, 16))
        return refuse(PKV_ERR_INVALID_ARG, call, "refs and workspace must be 16-byte aligned, the others 4-byte");
    const Carve c = carve(pool->num_rows, pool->num_pages);
    if (!pool->workspace || pool->workspace_bytes < c.bytes)
        return refuse(PKV_ERR_INVALID_ARG, call, "workspace is NULL or below pkv_pages_workspace's size");
    uint8_t *w = (uint8_t *)pool->workspace;
    p = PoolParams{};
    p.table = pool->table;
    p.lens = pool->lens;
    p.refs = pool->refs;
    p.row_stride = pool->row_stride;
    p.num_rows = pool->num_rows;
    p.num_pages = pool->num_pages;
    p.page_size = pool->page_size;
    p.status = pool->status;
    p.claim = (int32_t *)(w + c.claim);
    p.first = (int32_t *)(w + c.first);
    p.first_slot = (int64_t *)(w + c.first_slot);
    p.free_ids = (int32_t *)(w + c.free_ids);
    p.word = (int32_t *)(w + c.word);
    p.tokens = (int64_t *)(w + c.tokens);
    return PKV_OK;
}

int take_entries(const char *call, const PoolParams &p, int32_t n, const void *a, const void *b)
{
    if (n < 0)
        return refuse(PKV_ERR_INVALID_ARG, call, "n is negative");
    if (n > p.num_rows)
        return refuse(PKV_ERR_INVALID_ARG, call, "more entries than the pool has rows");
    if (n > 0 && (!a || !b || misaligned(a, 4) || misaligned(b, 4)))
        return refuse(PKV_ERR_INVALID_ARG, call, "an index array is NULL or misaligned");
    return PKV_OK;
}

// One launch behind the work of the stream, its start allowed to overlap the end of the
// kernel before it (which every kernel here waits for first thing).
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int grid, int threads, int cluster, void *stream, Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int launched(const char *call, cudaError_t ce)
{
    return ce == cudaSuccess ? PKV_OK : refuse(PKV_ERR_CUDA, call, cudaGetErrorString(ce));
}

}  // namespace
}  // namespace pkv

extern "C" {

PKV_API int pkv_pages_workspace(int32_t num_rows, int32_t num_pages, int64_t *bytes)
{
    using namespace pkv;
    if (!bytes || num_rows < 0 || num_pages < 0)
        return refuse(PKV_ERR_INVALID_ARG, "pkv_pages_workspace", "bytes is NULL or a size negative");
    *bytes = carve(num_rows, num_pages).bytes;
    return PKV_OK;
}

PKV_API int pkv_pages_extend(const pkv_page_pool *pool, const int32_t *rows, const int32_t *add, int32_t n,
                             int64_t *slots, int64_t slots_capacity, void *stream)
{
    using namespace pkv;
    NvtxRange range("pkv_pages_extend");
    set_last_error("");
    PoolParams p;
    int st = take_pool("pkv_pages_extend", pool, p);
    if (st == PKV_OK)
        st = take_entries("pkv_pages_extend", p, n, rows, add);
    if (st != PKV_OK)
        return st;
    if (slots_capacity < 0 || misaligned(slots, 8))
        return refuse(PKV_ERR_INVALID_ARG, "pkv_pages_extend", "slots are misaligned or their capacity negative");
    if (n == 0)  // -1 in every slot
        return slots && slots_capacity > 0
                   ? launched("pkv_pages_extend",
                              cudaMemsetAsync(slots, 0xff, slots_capacity * sizeof(int64_t), (cudaStream_t)stream))
                   : PKV_OK;
    cudaError_t ce = launch(rank_kernel<kExtend>, kCtas, kThreads, kCtas, stream, p, rows, add, (int)n, slots != nullptr,
                            slots_capacity);
    if (ce == cudaSuccess)
        ce = launch(extend_kernel, n, kApplyThreads, 1, stream, p, rows, add, slots, slots_capacity);
    return launched("pkv_pages_extend", ce);
}

PKV_API int pkv_pages_fork(const pkv_page_pool *pool, const int32_t *parents, const int32_t *children, int32_t n,
                           int32_t *src, int32_t *dst, void *stream)
{
    using namespace pkv;
    NvtxRange range("pkv_pages_fork");
    set_last_error("");
    PoolParams p;
    int st = take_pool("pkv_pages_fork", pool, p);
    if (st == PKV_OK)
        st = take_entries("pkv_pages_fork", p, n, parents, children);
    if (st == PKV_OK)
        st = take_entries("pkv_pages_fork", p, n, src, dst);
    if (st != PKV_OK || n == 0)
        return st;
    cudaError_t ce = launch(rank_kernel<kFork>, kCtas, kThreads, kCtas, stream, p, children, parents, (int)n, false,
                            (int64_t)0);
    if (ce == cudaSuccess)
        ce = launch(fork_kernel, n, kApplyThreads, 1, stream, p, children, parents, src, dst);
    return launched("pkv_pages_fork", ce);
}

PKV_API int pkv_pages_free(const pkv_page_pool *pool, const int32_t *rows, int32_t n, void *stream)
{
    using namespace pkv;
    NvtxRange range("pkv_pages_free");
    set_last_error("");
    PoolParams p;
    int st = take_pool("pkv_pages_free", pool, p);
    if (st == PKV_OK)
        st = take_entries("pkv_pages_free", p, n, rows, rows);
    if (st != PKV_OK || n == 0)
        return st;
    return launched("pkv_pages_free", launch(free_kernel, n, kApplyThreads, 1, stream, p, rows));
}

PKV_API int pkv_pages_compact(const pkv_page_pool *pool, const pkv_page_pool *out, int32_t *src, int32_t *dst,
                              int32_t max_moves, int32_t *count, void *stream)
{
    using namespace pkv;
    NvtxRange range("pkv_pages_compact");
    set_last_error("");
    PoolParams p, o;
    int st = take_pool("pkv_pages_compact", pool, p);
    if (st == PKV_OK)
        st = take_pool("pkv_pages_compact", out, o);
    if (st != PKV_OK)
        return st;
    if (o.num_rows != p.num_rows || o.num_pages != p.num_pages || o.page_size != p.page_size ||
        o.row_stride < p.row_stride)
        return refuse(PKV_ERR_INVALID_ARG, "pkv_pages_compact", "the two pools differ in their sizes");
    if (o.table == p.table && o.row_stride != p.row_stride)
        return refuse(PKV_ERR_INVALID_ARG, "pkv_pages_compact", "one table with two row strides");
    if (max_moves < 0 || (max_moves > 0 && (!src || !dst)) || !count || misaligned(src, 4) || misaligned(dst, 4) ||
        misaligned(count, 4))
        return refuse(PKV_ERR_INVALID_ARG, "pkv_pages_compact", "src, dst and count are required");
    cudaError_t ce = launch(moves_kernel, kCtas, kThreads, kCtas, stream, p, o.refs, src, dst, (int)max_moves, count);
    if (ce == cudaSuccess && p.num_rows > 0)
        ce = launch(rewrite_kernel, p.num_rows, kRewriteThreads, 1, stream, p, o.table, o.row_stride, o.lens,
                    (const int32_t *)dst);
    return launched("pkv_pages_compact", ce);
}

PKV_API int pkv_copy_pages(void *k_cache, void *v_cache, int32_t num_layers, int64_t layer_bytes, int32_t num_pages,
                           int64_t page_bytes, const int32_t *src, const int32_t *dst, int32_t n, const int32_t *count,
                           int32_t *status, void *stream)
{
    using namespace pkv;
    NvtxRange range("pkv_copy_pages");
    set_last_error("");
    if (n < 0 || num_layers < 0 || num_pages < 0 || page_bytes < 0 || layer_bytes < 0)
        return refuse(PKV_ERR_INVALID_ARG, "pkv_copy_pages", "negative size");
    if (page_bytes % 16 || layer_bytes % 16 || page_bytes > (1LL << 30))
        return refuse(PKV_ERR_UNSUPPORTED, "pkv_copy_pages",
                      "page_bytes and layer_bytes must be multiples of 16, a page at most 2^30 bytes");
    if (n == 0 || num_layers == 0 || page_bytes == 0)
        return PKV_OK;
    if (!k_cache || !v_cache || !src || !dst)
        return refuse(PKV_ERR_INVALID_ARG, "pkv_copy_pages", "a required pointer is NULL");
    if (misaligned(k_cache, 16) || misaligned(v_cache, 16) || misaligned(src, 4) || misaligned(dst, 4) ||
        misaligned(count, 4) || misaligned(status, 4))
        return refuse(PKV_ERR_INVALID_ARG, "pkv_copy_pages", "caches must be 16-byte aligned, the others 4-byte");
    CopyParams p{};
    p.k = (uint8_t *)k_cache;
    p.v = (uint8_t *)v_cache;
    p.layer_bytes = layer_bytes;
    p.num_layers = num_layers;
    p.num_pages = num_pages;
    p.granules = (int32_t)(page_bytes / 16);
    p.n = n;
    p.src = src;
    p.dst = dst;
    p.count = count;
    p.status = status;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t tiles = ((int64_t)n * p.granules + kTile - 1) / kTile * 2 * num_layers;
    const int grid = (int)(tiles < sms * 8LL ? tiles : sms * 8LL);
    return launched("pkv_copy_pages", launch(copy_kernel, grid, kCopyThreads, 1, stream, p));
}

}  // extern "C"

// Pages of the paged key/value cache: reserving, freeing, forking, compacting,
// and writing new tokens into them.
//
// The tables live on the device and every decision is taken there, so a step
// can be captured into a graph and none waits for the host.  A page is free
// when its reference count is 0; whoever needs pages gets the free ones with
// the lowest numbers, in list order, so results do not depend on timing.
//
// Which pages are free is an ordered scan over the reference counts.  It runs
// in one CTA (1024 threads, 16 counts a thread and step), which stops once
// enough are found; the moving of data that follows runs on all SMs and is
// bound by HBM (each page read once and written once).
#include <algorithm>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace eta {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kScan = 16;          // reference counts per thread and step

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_done() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Exclusive prefix of v over the block's threads, and the total.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *wsum, T &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    T w = wsum[lane];   // 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T t = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += t;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const T before = warp == 0 ? T(0) : __shfl_sync(0xffffffffu, w, warp - 1);
    return before + inc - v;
}

// Whether an earlier entry of the list names the same row (the first wins), of
// those that `counts` lets count.  Whole warp; every lane gets the answer.
template <typename Counts>
__device__ __forceinline__ bool named_before(const int *list, int i, int row, const Counts &counts) {
    const int lane = threadIdx.x & 31;
    for (int j0 = 0; j0 < i; j0 += 32) {
        const int j = j0 + lane;
        const bool same = j < i && list[j] == row && counts(j);
        if (__any_sync(0xffffffffu, same)) return true;
    }
    return false;
}

// 16 reference counts from `base`; counts past the end read as in use.
__device__ __forceinline__ void load_refs(const int *refs, int pages, long long base, int (&r)[kScan]) {
    if (base + kScan <= pages) {
#pragma unroll
        for (int q = 0; q < kScan / 4; ++q) {
            const int4 v = *reinterpret_cast<const int4 *>(refs + base + 4 * q);
            r[4 * q] = v.x;
            r[4 * q + 1] = v.y;
            r[4 * q + 2] = v.z;
            r[4 * q + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int q = 0; q < kScan; ++q) r[q] = base + q < pages ? refs[base + q] : 1;
    }
}

// The first `want` free pages, lowest first, into list[]; returns how many
// were found.  Whole block.
__device__ __forceinline__ int find_free(const int *refs, int pages, int want, int *list, int *wsum) {
    int found = 0;
    for (long long c0 = 0; c0 < pages && found < want; c0 += static_cast<long long>(kPlanThreads) * kScan) {
        const long long base = c0 + static_cast<long long>(threadIdx.x) * kScan;
        int r[kScan], n = 0, total;
        load_refs(refs, pages, base, r);
#pragma unroll
        for (int q = 0; q < kScan; ++q) n += r[q] <= 0 ? 1 : 0;
        int at = found + block_scan(n, wsum, total);
#pragma unroll
        for (int q = 0; q < kScan; ++q)
            if (r[q] <= 0) {
                if (at < want) list[at] = static_cast<int>(base) + q;
                ++at;
            }
        found += total;
    }
    __syncthreads();   // the list is complete (block scope)
    return min(found, want);
}

__device__ __forceinline__ int pages_of(int tokens, int S) { return (tokens + S - 1) / S; }

// What a fork's plan leaves in the workspace for the copies.
struct Plan {
    int *totals;     // [0]: pages handed out in all
    int *need_end;   // pages handed out up to and with this entry
    int *need;       // pages it got; -1: refused
    int *info;       // the parent's length
    int *list;       // the pages handed out
};
__device__ __host__ inline Plan carve_plan(void *ws, int n) {
    int *w = static_cast<int *>(ws);
    Plan q;
    q.totals = w;
    q.need_end = w + 16;
    q.need = q.need_end + n;
    q.info = q.need + n;
    q.list = q.info + n;
    return q;
}

constexpr int kSmallList = 2048;   // free pages kept in shared memory

// Shared memory of the planning kernels, which take 1024 entries at a time, a
// thread to an entry.
struct PlanShared {
    int wsum[32];
    long long wneed[32];
    int named[kPlanThreads];    // the list's rows of these entries (-1: one that changes nothing)
    int end[kPlanThreads];      // needs up to and with an entry (of these entries), or pages + 1 if that is less
    int list[kSmallList];
    int handed;
};

// Whether an earlier entry of the list names the same row (the first wins), of
// those that `counts` lets count.  Entries from c0 on are in sh.named.
template <typename Counts>
__device__ __forceinline__ bool named_before(const PlanShared &sh, const int *list, int c0, int row, const Counts &counts) {
    bool same = false;
    for (int j = 0; j < c0; ++j) same |= list[j] == row && counts(j);
    for (int j = 0; j < static_cast<int>(threadIdx.x); ++j) same |= sh.named[j] == row;
    return same;
}

// Grants the needs of up to 1024 entries (need: this thread's; -1 refused) in
// order while free pages last, and marks the pages handed out.  After one
// entry did not get its pages none that needs pages does (`full` carries that
// on).  Returns whether this entry was granted; `list` is where the pages lie,
// `handed` how many, and sh.end says whose they are.
__device__ __forceinline__ bool grant(const CacheView &c, PlanShared &sh, int need, int *big_list, bool &full, int *&list,
                                      int &handed) {
    // (together the needs may pass 32 bits; more than there are pages is never met)
    const long long most = static_cast<long long>(c.pages) + 1;
    long long sum;
    const long long before = block_scan(static_cast<long long>(max(need, 0)), sh.wneed, sum);
    const int end = static_cast<int>(min(before + max(need, 0), most)), total = static_cast<int>(min(sum, most));
    sh.end[threadIdx.x] = end;
    if (threadIdx.x == 0) sh.handed = 0;
    list = total <= kSmallList ? sh.list : big_list;
    const int found = full ? 0 : find_free(c.ref_counts, c.pages, total, list, sh.wsum);
    if (full) __syncthreads();
    const bool ok = need == 0 || (need > 0 && end <= found);
    if (ok && need > 0) atomicMax(&sh.handed, end);
    full = full || found < total;
    __syncthreads();
    handed = sh.handed;
    for (int k = threadIdx.x; k < handed; k += kPlanThreads) c.ref_counts[list[k]] = 1;
    return ok;
}
// The entry (of these up to 1024) that page k was handed to: the first whose needs reach past k.
__device__ __forceinline__ int owner_of(const PlanShared &sh, int k) {
    int lo = 0, hi = kPlanThreads - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (sh.end[mid] > k) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const CacheView c, const int *seqs, const int *n_new, int n,
                                                               int *granted, void *ws, int *err) {
    __shared__ PlanShared sh;
    __shared__ int have[kPlanThreads];
    pdl_wait();
    const int S = c.page_size, tid = threadIdx.x;
    bool full = false;
    for (int c0 = 0; c0 < n; c0 += kPlanThreads) {
        const int i = c0 + tid;
        __syncthreads();   // the entries before are done with
        const int s = i < n ? seqs[i] : -1, add = i < n ? n_new[i] : 0;
        sh.named[tid] = add > 0 ? s : -1;
        __syncthreads();
        int need = -1, len = 0;
        bool bad = false;
        if (i < n) {
            bad = s < 0 || s >= c.rows || add < 0;
            if (!bad) {
                len = c.seq_lens[s];
                bad = len < 0 || (add > 0 && named_before(sh, seqs, c0, s, [&](int j) { return n_new[j] > 0; }));
            }
            if (!bad && static_cast<long long>(len) + add <= static_cast<long long>(c.max_pages) * S) {
                need = pages_of(len + add, S) - pages_of(len, S);
                if (add > 0 && (len & (S - 1)) != 0) {
                    // the new tokens begin inside the last page: it must be this sequence's own
                    const int id = c.page_table[static_cast<long long>(s) * c.max_pages + len / S];
                    bad = id < 0 || id >= c.pages || c.ref_counts[id] > 1;
                    if (bad) need = -1;
                }
            }
            if (bad) atomicOr(err, kErrWordBadRow);
        }
        have[tid] = pages_of(len, S);
        int *list, handed;
        const bool ok = grant(c, sh, need, carve_plan(ws, n).list, full, list, handed);
        for (int k = tid; k < handed; k += kPlanThreads) {
            const int e = owner_of(sh, k), first = e > 0 ? sh.end[e - 1] : 0;
            c.page_table[static_cast<long long>(sh.named[e]) * c.max_pages + have[e] + k - first] = list[k];
        }
        if (i < n) {
            granted[i] = ok ? 1 : 0;
            if (ok && add > 0) c.seq_lens[s] = len + add;
        }
    }
    pdl_done();
}

constexpr int kFreeThreads = 256;

__global__ void __launch_bounds__(kFreeThreads) free_kernel(const CacheView c, const int *seqs, const int *keep, int n,
                                                            int *err) {
    pdl_wait();
    const int i = blockIdx.x;
    const int s = seqs[i];
    __shared__ int bad;
    if (threadIdx.x < 32) {
        const bool no = s < 0 || s >= c.rows || named_before(seqs, i, s, [](int) { return true; });
        if (threadIdx.x == 0) bad = no;
    }
    __syncthreads();
    if (bad) {
        if (threadIdx.x == 0) atomicOr(err, kErrWordBadRow);
    } else {
        const int len = min(c.seq_lens[s], c.max_pages * c.page_size);
        const int left = max(0, min(keep ? keep[i] : 0, len));
        int *row = c.page_table + static_cast<long long>(s) * c.max_pages;
        for (int k = pages_of(left, c.page_size) + threadIdx.x; k < c.max_pages; k += kFreeThreads) {
            const int id = row[k];
            if (id < 0) continue;
            row[k] = -1;
            if (id < c.pages) atomicSub(c.ref_counts + id, 1);
            else atomicOr(err, kErrWordBadRow);
        }
        __syncthreads();   // everyone has read the length
        if (threadIdx.x == 0) c.seq_lens[s] = left;
    }
    pdl_done();
}

// Fork, first part: who gets which pages.  need[i] = -1: refused.  Lengths and
// rows are written by the second part, so that all entries see the sequences
// as they were.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const CacheView c, const int *parents, const int *children,
                                                                 int n, int copy, int *granted, void *ws, int *err) {
    __shared__ PlanShared sh;
    pdl_wait();
    const Plan q = carve_plan(ws, n);
    const int S = c.page_size, cap = c.max_pages * S, tid = threadIdx.x;
    bool full = false;
    int base = 0;
    for (int c0 = 0; c0 < n; c0 += kPlanThreads) {
        const int i = c0 + tid;
        __syncthreads();   // the entries before are done with
        const int a = i < n ? parents[i] : -1, b = i < n ? children[i] : -1;
        sh.named[tid] = b;
        __syncthreads();
        int need = -1, len = 0;
        if (i < n) {
            if (a >= 0 && a < c.rows && b >= 0 && b < c.rows) {
                len = c.seq_lens[a];
                if (c.seq_lens[b] == 0 && len >= 0 && len <= cap && !named_before(sh, children, c0, b, [](int) { return true; }))
                    need = copy ? pages_of(len, S) : (len % S ? 1 : 0);
            }
            if (need < 0) atomicOr(err, kErrWordBadRow);
        }
        int *list, handed;
        const bool ok = grant(c, sh, need, q.list + base, full, list, handed);
        if (list == sh.list)
            for (int k = tid; k < handed; k += kPlanThreads) q.list[base + k] = list[k];
        if (i < n) {
            granted[i] = ok ? 1 : 0;
            q.need[i] = ok ? need : -1;
            q.need_end[i] = base + sh.end[tid];
            q.info[i] = len;
        }
        base += handed;
    }
    if (tid == 0) q.totals[0] = base;
    pdl_done();
}

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;                               // 16-byte pieces per thread in flight
constexpr int kCopyPiece = kCopyThreads * kCopyVecs;       // 16-byte pieces per work item

// One piece of a page of one layer of K or V.  `held`: slots to copy (the
// whole page: page_size).
__device__ __forceinline__ void copy_piece(const CacheView &c, uint4 *pool, int layer, int src, int dst, int part, int held) {
    const long long lay = layer * c.layer_vecs;
    const uint4 *s = pool + lay + src * c.page_vecs;
    uint4 *d = pool + lay + dst * c.page_vecs;
    const int v0 = part * kCopyPiece + threadIdx.x;
    uint4 buf[kCopyVecs];
    bool in[kCopyVecs];
#pragma unroll
    for (int q = 0; q < kCopyVecs; ++q) {
        const int v = v0 + q * kCopyThreads;
        in[q] = v < c.block_vecs;
        if (held < c.page_size && in[q]) in[q] = (v / c.slot_vecs) % c.page_size < held;
        if (in[q]) buf[q] = __ldcs(s + v);
    }
#pragma unroll
    for (int q = 0; q < kCopyVecs; ++q)
        if (in[q]) __stcs(d + v0 + q * kCopyThreads, buf[q]);
}

struct Move {
    int src, dst, held;   // src < 0: nothing to copy
};
// Pages whose block of one layer is small: a group of threads (a power of two, so
// that a page gives each about kCopyVecs pieces, 32 .. 256) takes a page, or a part
// of it, across layers, K and V.  Compacting 32768 pages of 4 layers x 1 KB 179 us
// (528 an item to a block, as below), 16384 of 2 x 4 KB 134 (171), 8192 of 2 x 9 KB
// 118 (123), 8192 of 2 x 12 KB 154 (147).
constexpr int kSmallBlock = 640;   // 10 KB
template <typename Where>
__device__ __forceinline__ void copy_small_pages(const CacheView &c, int pages, const Where &where) {
    const int per_page = 2 * c.layers * c.block_vecs;
    int group = 32;
    while (group < kCopyThreads && group * kCopyVecs < per_page) group *= 2;
    const int parts = (per_page + group * kCopyVecs - 1) / (group * kCopyVecs), side = kCopyThreads / group;
    const int mine = static_cast<int>(threadIdx.x) & (group - 1);
    const long long items = static_cast<long long>(pages) * parts, step = static_cast<long long>(gridDim.x) * side;
    long long it = static_cast<long long>(blockIdx.x) * side + threadIdx.x / group;
    if (it >= items) return;
    Move next = where(static_cast<int>(it / parts));
    for (; it < items; it += step) {
        const Move m = next;
        const int v0 = static_cast<int>(it % parts) * group * kCopyVecs + mine;
        if (it + step < items) next = where(static_cast<int>((it + step) / parts));
        if (m.src < 0) continue;
        uint4 buf[kCopyVecs], *to[kCopyVecs];
        bool in[kCopyVecs];
#pragma unroll
        for (int q = 0; q < kCopyVecs; ++q) {
            const int v = v0 + q * group, block = v / c.block_vecs, off = v - block * c.block_vecs;
            in[q] = v < per_page && (m.held >= c.page_size || (off / c.slot_vecs) % c.page_size < m.held);
            uint4 *at = (block & 1 ? c.v : c.k) + (block >> 1) * c.layer_vecs + off;
            to[q] = at + m.dst * c.page_vecs;
            if (in[q]) buf[q] = __ldcs(at + m.src * c.page_vecs);
        }
#pragma unroll
        for (int q = 0; q < kCopyVecs; ++q)
            if (in[q]) __stcs(to[q], buf[q]);
    }
}

// Copies `pages` pages in every layer: work items (page, layer, K or V, piece),
// the pieces of a page together, dealt to all blocks.  The next item's place is
// looked up before this item's data is waited for.
template <bool SMALL, typename Where>
__device__ __forceinline__ void copy_pages(const CacheView &c, int pages, const Where &where) {
    if constexpr (SMALL) {
        copy_small_pages(c, pages, where);
        return;
    }
    const int pieces = (c.block_vecs + kCopyPiece - 1) / kCopyPiece;
    const long long per_page = 2LL * c.layers * pieces, items = pages * per_page;
    long long it = blockIdx.x;
    if (it >= items) return;
    Move next = where(static_cast<int>(it / per_page));
    for (; it < items; it += gridDim.x) {
        const Move m = next;
        int rest = static_cast<int>(it % per_page);
        if (it + gridDim.x < items) next = where(static_cast<int>((it + gridDim.x) / per_page));
        if (m.src < 0) continue;
        const int part = rest % pieces;
        rest /= pieces;
        copy_piece(c, rest & 1 ? c.v : c.k, rest >> 1, m.src, m.dst, part, m.held);
    }
}

// Whether a pool's pages are copied as small ones.  (Kernels of their own: with both ways in one the copy of large pages
// had 64 registers instead of 46 and a CTA less on an SM: 8192 pages of 131 KB 168.4 us instead of 166.5.)
bool small_pages(const CacheView &c) { return c.block_vecs < kSmallBlock && c.layers < (1 << 16); }

// Fork, second part: the children's rows, the reference counts, the copies.
template <bool SMALL>
__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(const CacheView c, const int *parents, const int *children,
                                                                  int n, int copy, const void *ws, int *err) {
    pdl_wait();
    const Plan q = carve_plan(const_cast<void *>(ws), n);
    const int S = c.page_size;
    // rows: one block per entry at a time
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const int need = q.need[i];
        if (need < 0) continue;
        const int len = q.info[i], shared = copy ? 0 : len / S;
        const int *from = c.page_table + static_cast<long long>(parents[i]) * c.max_pages;
        int *to = c.page_table + static_cast<long long>(children[i]) * c.max_pages;
        for (int k = threadIdx.x; k < c.max_pages; k += kCopyThreads) {
            int id = -1;
            if (k < shared + need) {
                const int src = from[k];
                const bool there = src >= 0 && src < c.pages;
                if (k < shared) {
                    id = there ? src : -1;
                    if (there) atomicAdd(c.ref_counts + id, 1);
                } else {
                    id = q.list[q.need_end[i] - need + k - shared];
                    if (!there) {   // nothing to copy: the page goes back
                        c.ref_counts[id] = 0;
                        id = -1;
                    }
                }
                if (!there) atomicOr(err, kErrWordBadRow);   // what the parent lacks the child lacks too
            }
            to[k] = id;
        }
        if (threadIdx.x == 0) c.seq_lens[children[i]] = len;
    }
    copy_pages<SMALL>(c, q.totals[0], [&](int k) -> Move {
        // the entry that page k was handed to: the first with need_end > k
        int lo = 0, hi = n - 1;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (q.need_end[mid] > k) hi = mid;
            else lo = mid + 1;
        }
        const int len = q.info[lo], need = q.need[lo];
        const int col = (copy ? 0 : len / S) + k - (q.need_end[lo] - need);
        int src = c.page_table[static_cast<long long>(parents[lo]) * c.max_pages + col];
        if (src < 0 || src >= c.pages) {
            atomicOr(err, kErrWordBadRow);
            src = -1;
        }
        // (a block of 4-bit values is copied whole: its scales lie behind the codes)
        return Move{src, q.list[k], c.bits == 4 ? S : min(S, len - col * S)};
    });
    pdl_done();
}

constexpr int kCompactList = 4096;   // moves whose lists fit shared memory

// Compact, first part: how many pages are live, where the live pages above
// that many go, and the new reference counts.  One block: two ordered scans
// over the counts, which a thread keeps in registers between them (up to
// 16384 pages), and lists that stay in shared memory while the moves are
// written out.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CacheView c, int *refs_out, int *n_live, void *ws) {
    __shared__ int wsum[32];
    __shared__ int small_holes[kCompactList], small_strays[kCompactList];
    pdl_wait();
    int *totals = static_cast<int *>(ws), *holes = totals + 16, *strays = holes + c.pages, *map = strays + c.pages;
    constexpr long long step = static_cast<long long>(kPlanThreads) * kScan;
    const bool once = c.pages <= step;
    int r[kScan], live = 0;
    for (long long c0 = 0; c0 < c.pages; c0 += step) {
        int n = 0, total;
        const long long base = c0 + static_cast<long long>(threadIdx.x) * kScan;
        load_refs(c.ref_counts, c.pages, base, r);
#pragma unroll
        for (int q = 0; q < kScan; ++q) n += r[q] > 0 && base + q < c.pages ? 1 : 0;
        block_scan(n, wsum, total);
        live += total;
    }
    // as many holes below as live pages above, and no more than either side has
    const bool small = min(live, c.pages - live) <= kCompactList;
    int *hl = small ? small_holes : holes, *sl = small ? small_strays : strays;
    int nh = 0, ns = 0;
    for (long long c0 = 0; c0 < c.pages; c0 += step) {
        const long long base = c0 + static_cast<long long>(threadIdx.x) * kScan;
        if (!once) load_refs(c.ref_counts, c.pages, base, r);
        int both = 0, total;   // holes in the upper half, strays in the lower
#pragma unroll
        for (int q = 0; q < kScan; ++q) {
            const bool in = base + q < c.pages, used = r[q] > 0, low = base + q < live;
            both += (in && !used && low ? 1 << 16 : 0) + (in && used && !low ? 1 : 0);
        }
        const int before = block_scan(both, wsum, total);
        int ah = nh + (before >> 16), as = ns + (before & 0xffff);
        nh += total >> 16;
        ns += total & 0xffff;
#pragma unroll
        for (int q = 0; q < kScan; ++q) {
            const int id = static_cast<int>(base) + q;
            if (base + q >= c.pages) continue;
            const bool used = r[q] > 0, low = base + q < live;
            if (!used && low) hl[ah++] = id;
            if (!used && !low) map[id] = -1;
            if (used && !low) sl[as++] = id;
            if (refs_out != c.ref_counts) refs_out[id] = used && low ? r[q] : 0;
        }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < ns; k += kPlanThreads) {
        const int from = sl[k], to = hl[k], n = c.ref_counts[from];
        map[from] = to;
        refs_out[to] = n;
        if (refs_out == c.ref_counts) refs_out[from] = 0;
        if (small) {
            strays[k] = from;
            holes[k] = to;
        }
    }
    if (threadIdx.x == 0) {
        totals[0] = ns;
        totals[1] = live;
        *n_live = live;
    }
    pdl_done();
}
static_assert(kPlanThreads * kScan < (1 << 16), "two counts to a scan");

// Compact, second part: the table and the pages.
template <bool SMALL>
__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const CacheView c, int *table_out, const void *ws,
                                                                     int *err) {
    pdl_wait();
    const int *totals = static_cast<const int *>(ws), *holes = totals + 16, *strays = holes + c.pages,
              *map = strays + c.pages;
    const int live = totals[1];
    const long long entries = static_cast<long long>(c.rows) * c.max_pages;
    for (long long e = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; e < entries;
         e += static_cast<long long>(gridDim.x) * kCopyThreads) {
        int id = c.page_table[e];
        if (id >= live) {
            id = id < c.pages ? map[id] : -1;
            if (id < 0) atomicOr(err, kErrWordBadRow);   // no page of the pool, or a free one
        }
        table_out[e] = id < 0 ? -1 : id;
    }
    copy_pages<SMALL>(c, totals[0], [&](int k) -> Move { return Move{strays[k], holes[k], c.page_size}; });
    pdl_done();
}

constexpr int kAppendThreads = 256;

// One CTA takes TOK consecutive tokens.  Warp w finds the place of token w: its
// entry (32 borders of q_start to a round trip), that sequence's length, and
// the page.  A thread owns a 16-byte piece of the row of a token (K's pieces,
// then V's) and takes it for every token, so where a piece lies is worked out
// once for all of them; rows do not depend on where they go, so the first
// pieces are read before the places are known.
template <int TOK>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const CacheView c, int layer, const uint4 *Kn, const uint4 *Vn,
                                                                long long token_vecs, long long head_vecs, int T,
                                                                const int *seqs, const int *q_start, const int *granted, int n,
                                                                int *err) {
    static_assert(TOK <= kAppendThreads / 32, "one warp finds one token's place");
    __shared__ long long dst[TOK];   // first 16-byte piece of the slot's head 0, or -1
    pdl_wait();
    const int t0 = blockIdx.x * TOK, ntok = min(TOK, T - t0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = c.row_vecs, per = c.heads * row;   // pieces of one head's row; of K (or V) of a token
    // short rows: several tokens side by side
    const int side = 2 * per < kAppendThreads ? kAppendThreads / (2 * per) : 1;
    const int first = side > 1 ? threadIdx.x / (2 * per) : 0;
    int x = side > 1 ? static_cast<int>(threadIdx.x) - first * 2 * per : static_cast<int>(threadIdx.x);
    if (first >= side) x = 2 * per;   // (threads left over)
    const uint4 *src;
    uint4 *pool;
    long long off;
    auto place = [&]() {
        const bool v = x >= per;
        const int y = v ? x - per : x, h = y / row, e = y - h * row;
        src = (v ? Vn : Kn) + t0 * token_vecs + h * head_vecs + e;
        pool = v ? c.v : c.k;
        off = h * c.head_stride_vecs + e;
    };
    uint4 buf[TOK];
    auto read = [&]() {
        place();
#pragma unroll
        for (int k = 0; k < TOK; ++k)
            if (first + k * side < ntok) buf[k] = __ldcs(src + (first + k * side) * token_vecs);
    };
    if (x < 2 * per) read();
    // warp w: token t0 + w
    const int t = t0 + warp, S = c.page_size;
    long long at = -1;
    bool bad = false;
    if (warp < TOK && t < T) {
        // the last entry that begins at or before t (what it says comes along: each read that waits for another costs 0.3 us)
        int i = -1, q0 = 0, q1 = 0, s = 0;
        for (int j0 = 0; j0 < n; j0 += 32) {
            const int j = j0 + lane;
            int b = 0x7fffffff, e = 0, row_of = j;
            if (j < n) {
                b = q_start[j];
                e = q_start[j + 1];
                if (seqs) row_of = seqs[j];
            }
            const uint32_t le = __ballot_sync(0xffffffffu, b <= t);
            if (le) {
                const int last = 31 - __clz(le);
                i = j0 + last;
                q0 = __shfl_sync(0xffffffffu, b, last);
                q1 = __shfl_sync(0xffffffffu, e, last);
                s = __shfl_sync(0xffffffffu, row_of, last);
            }
            if (le != 0xffffffffu) break;
        }
        if (i >= 0 && t < q1) {
            const bool here = !granted || granted[i] != 0;
            bad = here && !(q0 >= 0 && q1 <= T && s >= 0 && s < c.rows);
            if (here && !bad) {
                const int len = c.seq_lens[s];   // (on its way while the list is looked through)
                const bool again = seqs && named_before(seqs, i, s, [&](int j) {
                    return q_start[j + 1] > q_start[j] && (!granted || granted[j] != 0);
                });
                const int pos = len - (q1 - q0) + (t - q0);
                bad = again || pos < 0 || pos / S >= c.max_pages;
                if (!bad) {
                    const int id = c.page_table[static_cast<long long>(s) * c.max_pages + pos / S];
                    // (a page that other table entries name too is read by those sequences: it is never written)
                    bad = id < 0 || id >= c.pages || c.ref_counts[id] > 1;
                    if (!bad) at = layer * c.layer_vecs + id * c.page_vecs + (pos % S) * c.slot_stride_vecs;
                }
            }
        }
    }
    // entries whose range is none, or reaches past the tokens: reported once, since none of their tokens need be met above
    if (blockIdx.x == 0 && warp == kAppendThreads / 32 - 1) {
        bool none = false;
        for (int j = lane; j < n; j += 32) {
            const int a = q_start[j], b = q_start[j + 1];
            none |= (a < 0 || b < a || b > T) && (!granted || granted[j] != 0);
        }
        if (none) atomicOr(err, kErrWordBadRow);
    }
    if (warp < TOK && lane == 0) {
        dst[warp] = at;
        if (bad) atomicOr(err, kErrWordBadRow);
    }
    __syncthreads();
    while (x < 2 * per) {
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            const int tok = first + k * side;
            if (tok >= ntok) break;
            const long long base = dst[tok];
            if (base >= 0) pool[base + off] = buf[k];
        }
        if (side > 1) break;
        x += kAppendThreads;
        if (x < 2 * per) read();
    }
    pdl_done();
}

template <typename K, typename... A>
int launch(K kern, unsigned grid, int threads, cudaStream_t stream, const A &...args) {
    return launch_dependent(kern, dim3(grid), static_cast<unsigned>(threads), 0, stream, args...);
}

int copy_grid() {
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return nsm * 8;   // 2048 threads an SM
}

}  // namespace

size_t cache_workspace_bytes(int pages, int n) {
    // the larger of a plan's (3 n + pages) and compaction's (3 pages) integers
    return (16 + std::max<size_t>(3 * static_cast<size_t>(n) + pages, 3 * static_cast<size_t>(pages))) * sizeof(int);
}

int launch_cache_reserve(const CacheView &c, const int *seqs, const int *n_new, int n, int *granted, void *ws,
                         cudaStream_t stream) {
    int *err = device_error_word();
    if (!err) return kErrCuda;
    return launch(reserve_kernel, 1, kPlanThreads, stream, c, seqs, n_new, n, granted, ws, err);
}

int launch_cache_free(const CacheView &c, const int *seqs, const int *keep, int n, cudaStream_t stream) {
    int *err = device_error_word();
    if (!err) return kErrCuda;
    return launch(free_kernel, static_cast<unsigned>(n), kFreeThreads, stream, c, seqs, keep, n, err);
}

int launch_cache_fork(const CacheView &c, const int *parents, const int *children, int n, int copy, int *granted, void *ws,
                      cudaStream_t stream) {
    int *err = device_error_word();
    const int grid = copy_grid();
    if (!err || grid <= 0) return kErrCuda;
    const int rc = launch(fork_plan_kernel, 1, kPlanThreads, stream, c, parents, children, n, copy, granted, ws, err);
    if (rc != kOk) return rc;
    return launch(small_pages(c) ? fork_apply_kernel<true> : fork_apply_kernel<false>, static_cast<unsigned>(grid), kCopyThreads,
                  stream, c, parents, children, n, copy, static_cast<const void *>(ws), err);
}

int launch_cache_compact(const CacheView &c, int *table_out, int *refs_out, int *n_live, void *ws, cudaStream_t stream) {
    int *err = device_error_word();
    const int grid = copy_grid();
    if (!err || grid <= 0) return kErrCuda;
    const int rc = launch(compact_plan_kernel, 1, kPlanThreads, stream, c, refs_out, n_live, ws);
    if (rc != kOk) return rc;
    return launch(small_pages(c) ? compact_apply_kernel<true> : compact_apply_kernel<false>, static_cast<unsigned>(grid),
                  kCopyThreads, stream, c, table_out, static_cast<const void *>(ws), err);
}

int launch_cache_append(const CacheView &c, int layer, const void *Kn, const void *Vn, long long token_vecs,
                        long long head_vecs, int T, const int *seqs, const int *q_start, const int *granted, int n,
                        cudaStream_t stream) {
    int *err = device_error_word();
    if (!err) return kErrCuda;
    const uint4 *k = static_cast<const uint4 *>(Kn), *v = static_cast<const uint4 *>(Vn);
    // up to 4096 tokens two to a CTA (131 tokens x 8 heads x 128: 2.7 us, 3.9 with
    // eight), more eight (8000: 10.2 us, 10.4 with two; 7000 tokens of 58 MB, two layers in turn: 10.4 us, 0.84 of the copy rate)
    if (T <= 4096)
        return launch(append_kernel<2>, static_cast<unsigned>((T + 1) / 2), kAppendThreads, stream, c, layer, k, v,
                      token_vecs, head_vecs, T, seqs, q_start, granted, n, err);
    return launch(append_kernel<8>, static_cast<unsigned>((T + 7) / 8), kAppendThreads, stream, c, layer, k, v,
                  token_vecs, head_vecs, T, seqs, q_start, granted, n, err);
}

}  // namespace eta

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
#include "ptx.cuh"

namespace eta {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kScan = 16;          // reference counts per thread and step

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_done() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Exclusive prefix of v over the block's threads, and the total.
__device__ __forceinline__ int block_scan(int v, int *wsum, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int w = wsum[lane];   // 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += t;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = warp == 0 ? 0 : __shfl_sync(0xffffffffu, w, warp - 1);
    return before + inc - v;
}

// Whether an earlier entry of the list names the same row (the first wins).
// Whole warp; every lane gets the answer.
__device__ __forceinline__ bool named_before(const int *list, int i, int row) {
    const int lane = threadIdx.x & 31;
    for (int j0 = 0; j0 < i; j0 += 32) {
        const bool same = j0 + lane < i && list[j0 + lane] == row;
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
__device__ int find_free(const int *refs, int pages, int want, int *list, int *wsum) {
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

// Per entry of a plan, in the workspace.
struct Plan {
    int *need_end;   // running total of the needs up to and with this entry
    int *need;       // pages it needs; -1: refused for another reason
    int *info;       // fork: the parent's length
    int *list;       // free pages found
    int *totals;     // [0]: pages granted in all
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

// Running totals of need[] (refused entries count 0); returns the grand total.
__device__ int total_needs(const Plan &q, int n, int *wsum) {
    long long sum = 0;
    for (int c0 = 0; c0 < n; c0 += kPlanThreads) {
        const int i = c0 + threadIdx.x;
        const int v = i < n ? max(q.need[i], 0) : 0;
        int total;
        const int before = block_scan(v, wsum, total);
        if (i < n) q.need_end[i] = static_cast<int>(min(sum + before + v, 0x7fffffffLL));
        sum += total;
    }
    __syncthreads();
    return static_cast<int>(min(sum, 0x7fffffffLL));
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const CacheView c, const int *seqs, const int *n_new, int n,
                                                               int *granted, void *ws, int *err) {
    __shared__ int wsum[32];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Plan q = carve_plan(ws, n);
    const int S = c.page_size;
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int s = seqs[i], add = n_new[i];
        bool ok = s >= 0 && s < c.rows && add >= 0 && !named_before(seqs, i, s);
        int need = -1;
        if (ok) {
            const int len = c.seq_lens[s];
            ok = len >= 0 && static_cast<long long>(len) + add <= static_cast<long long>(c.max_pages) * S;
            if (ok) need = pages_of(len + add, S) - pages_of(len, S);
            else if (len < 0 && lane == 0) atomicOr(err, kErrWordBadRow);
        } else if (lane == 0) {
            atomicOr(err, kErrWordBadRow);
        }
        if (lane == 0) q.need[i] = need;
    }
    __syncthreads();
    const int want = total_needs(q, n, wsum);
    const int found = find_free(c.ref_counts, c.pages, want, q.list, wsum);
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int need = q.need[i], off = q.need_end[i] - need;
        const bool ok = need == 0 || (need > 0 && q.need_end[i] <= found);
        if (ok) {
            const int s = seqs[i], len = c.seq_lens[s], have = pages_of(len, S);
            int *row = c.page_table + static_cast<long long>(s) * c.max_pages + have;
            for (int k = lane; k < need; k += 32) {
                const int id = q.list[off + k];
                row[k] = id;
                c.ref_counts[id] = 1;
            }
            __syncwarp();
            if (lane == 0) c.seq_lens[s] = len + n_new[i];
        }
        if (lane == 0) granted[i] = ok ? 1 : 0;
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
        const bool no = s < 0 || s >= c.rows || named_before(seqs, i, s);
        if (threadIdx.x == 0) bad = no;
    }
    __syncthreads();
    if (bad) {
        if (threadIdx.x == 0) atomicOr(err, kErrWordBadRow);
    } else {
        const int len = c.seq_lens[s];
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

// Fork, first part: who gets which pages.  need[i] = -1: refused.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const CacheView c, const int *parents, const int *children,
                                                                 int n, int copy, int *granted, void *ws, int *err) {
    __shared__ int wsum[32];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Plan q = carve_plan(ws, n);
    if (threadIdx.x == 0) q.totals[0] = 0;
    const int S = c.page_size, cap = c.max_pages * S;
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int a = parents[i], b = children[i];
        int need = -1, len = 0;
        if (a >= 0 && a < c.rows && b >= 0 && b < c.rows && !named_before(children, i, b)) {
            len = c.seq_lens[a];
            if (c.seq_lens[b] == 0 && len >= 0 && len <= cap) need = copy ? pages_of(len, S) : (len % S ? 1 : 0);
        }
        if (lane == 0) {
            q.need[i] = need;
            q.info[i] = len;
            if (need < 0) atomicOr(err, kErrWordBadRow);
        }
    }
    __syncthreads();
    const int want = total_needs(q, n, wsum);
    const int found = find_free(c.ref_counts, c.pages, want, q.list, wsum);
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const bool ok = q.need[i] == 0 || (q.need[i] > 0 && q.need_end[i] <= found);
        granted[i] = ok ? 1 : 0;
        if (ok) {
            c.seq_lens[children[i]] = q.info[i];
            // (of the entries that need pages the granted ones are the first, so
            // the largest running total is the number of pages handed out)
            if (q.need[i] > 0) atomicMax(q.totals, q.need_end[i]);
        } else {
            q.need[i] = -1;
        }
    }
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

// Fork, second part: the children's rows, the reference counts, the copies.
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
            if (k < shared) {
                id = from[k];
                if (id >= 0 && id < c.pages) atomicAdd(c.ref_counts + id, 1);
                else atomicOr(err, kErrWordBadRow);
            } else if (k < shared + need) {
                id = q.list[q.need_end[i] - need + k - shared];
                c.ref_counts[id] = 1;
            }
            to[k] = id;
        }
    }
    // copies: items (page, layer, K or V, piece), pieces of a page together
    const int pieces = (c.block_vecs + kCopyPiece - 1) / kCopyPiece;
    const long long per_page = 2LL * c.layers * pieces;
    const long long items = q.totals[0] * per_page;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int k = static_cast<int>(it / per_page);
        int rest = static_cast<int>(it - k * per_page);
        // the entry that page k was handed to: the first with need_end > k
        int lo = 0, hi = n - 1;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (q.need_end[mid] > k) hi = mid;
            else lo = mid + 1;
        }
        const int len = q.info[lo], need = q.need[lo];
        const int col = (copy ? 0 : len / S) + k - (q.need_end[lo] - need);
        const int src = c.page_table[static_cast<long long>(parents[lo]) * c.max_pages + col];
        if (src < 0 || src >= c.pages) {
            if (threadIdx.x == 0) atomicOr(err, kErrWordBadRow);
            continue;
        }
        const int part = rest % pieces;
        rest /= pieces;
        copy_piece(c, rest & 1 ? c.v : c.k, rest >> 1, src, q.list[k], part, min(S, len - col * S));
    }
    pdl_done();
}

// Compact, first part: how many pages are live, where the live pages above
// that many go, and the new reference counts.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CacheView c, int *refs_out, int *n_live, void *ws) {
    __shared__ int wsum[32];
    pdl_wait();
    int *totals = static_cast<int *>(ws), *holes = totals + 16, *strays = holes + c.pages, *map = strays + c.pages;
    constexpr long long step = static_cast<long long>(kPlanThreads) * kScan;
    int live = 0;
    for (long long c0 = 0; c0 < c.pages; c0 += step) {
        int r[kScan], nf = 0, total;
        const long long base = c0 + static_cast<long long>(threadIdx.x) * kScan;
        load_refs(c.ref_counts, c.pages, base, r);
#pragma unroll
        for (int q = 0; q < kScan; ++q) nf += r[q] > 0 && base + q < c.pages ? 1 : 0;
        block_scan(nf, wsum, total);
        live += total;
    }
    int nh = 0, ns = 0;
    for (long long c0 = 0; c0 < c.pages; c0 += step) {
        int r[kScan], h = 0, s = 0, total;
        const long long base = c0 + static_cast<long long>(threadIdx.x) * kScan;
        load_refs(c.ref_counts, c.pages, base, r);
#pragma unroll
        for (int q = 0; q < kScan; ++q) {
            const bool in = base + q < c.pages, used = r[q] > 0;
            h += in && !used && base + q < live ? 1 : 0;
            s += in && used && base + q >= live ? 1 : 0;
        }
        int ah = nh + block_scan(h, wsum, total);
        nh += total;
        int as = ns + block_scan(s, wsum, total);
        ns += total;
#pragma unroll
        for (int q = 0; q < kScan; ++q) {
            const long long id = base + q;
            if (id >= c.pages) continue;
            if (r[q] <= 0 && id < live) holes[ah++] = static_cast<int>(id);
            if (r[q] <= 0 && id >= live) map[id] = -1;
            if (r[q] > 0 && id >= live) {
                map[id] = as;   // its rank for now
                strays[as++] = static_cast<int>(id);
            }
        }
    }
    __syncthreads();
    // as many holes below as live pages above
    for (int k = threadIdx.x; k < ns; k += kPlanThreads) map[strays[k]] = holes[k];
    // counts: what stays, then what moves (its old place is read before it is cleared)
    if (refs_out != c.ref_counts)
        for (int id = threadIdx.x; id < c.pages; id += kPlanThreads) refs_out[id] = id < live ? max(c.ref_counts[id], 0) : 0;
    __syncthreads();
    for (int k = threadIdx.x; k < ns; k += kPlanThreads) {
        const int r = c.ref_counts[strays[k]];
        refs_out[holes[k]] = r;
        if (refs_out == c.ref_counts) refs_out[strays[k]] = 0;
    }
    if (threadIdx.x == 0) {
        totals[0] = ns;
        totals[1] = live;
        *n_live = live;
    }
    pdl_done();
}

// Compact, second part: the table and the pages.
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
    const int pieces = (c.block_vecs + kCopyPiece - 1) / kCopyPiece;
    const long long per_page = 2LL * c.layers * pieces;
    const long long items = totals[0] * per_page;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int k = static_cast<int>(it / per_page);
        int rest = static_cast<int>(it - k * per_page);
        const int part = rest % pieces;
        rest /= pieces;
        copy_piece(c, rest & 1 ? c.v : c.k, rest >> 1, strays[k], holes[k], part, c.page_size);
    }
    pdl_done();
}

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;

// One CTA takes kAppendTokens consecutive tokens.  Its first threads find each
// token's entry (binary search in q_start), page and slot; then the block
// copies the tokens' rows of K and V, 16 bytes a thread.
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const CacheView c, int layer, const uint4 *Kn, const uint4 *Vn,
                                                                long long token_vecs, long long head_vecs, int T,
                                                                const int *seqs, const int *q_start, int n, int *err) {
    __shared__ long long dst[kAppendTokens];   // first 16-byte piece of the slot's head 0, or -1
    pdl_wait();
    const int t0 = blockIdx.x * kAppendTokens;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int S = c.page_size;
    // warp w: token t0 + w
    const int t = t0 + warp;
    long long at = -1;
    if (t < T && t >= q_start[0] && t < q_start[n]) {
        int lo = 0, hi = n - 1;   // the last entry that begins at or before t
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (q_start[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        const int i = lo;
        const int q0 = q_start[i], q1 = q_start[i + 1];
        const int s = seqs ? seqs[i] : i;
        bool ok = q0 <= t && t < q1 && s >= 0 && s < c.rows && !(seqs && named_before(seqs, i, s));
        if (ok) {
            const int pos = c.seq_lens[s] - (q1 - q0) + (t - q0);
            const int col = pos / S;
            ok = pos >= 0 && col < c.max_pages;
            if (ok) {
                const int id = c.page_table[static_cast<long long>(s) * c.max_pages + col];
                ok = id >= 0 && id < c.pages;
                if (ok) at = layer * c.layer_vecs + id * c.page_vecs + (pos % S) * c.slot_stride_vecs;
            }
        }
        if (!ok && lane == 0) atomicOr(err, kErrWordBadRow);
    }
    if (lane == 0) dst[warp] = at;
    __syncthreads();
    const int row = c.row_vecs, per = c.heads * row;   // pieces of one head's row; of a token
    const int total = kAppendTokens * per;
    for (int v = threadIdx.x; v < 2 * total; v += kAppendThreads) {
        const bool isv = v >= total;
        const int x = isv ? v - total : v;
        const int tok = x / per, y = x - tok * per, h = y / row, e = y - h * row;
        const long long to = dst[tok];
        if (to < 0) continue;
        const uint4 *src = (isv ? Vn : Kn) + (t0 + tok) * token_vecs + h * head_vecs + e;
        (isv ? c.v : c.k)[to + h * c.head_stride_vecs + e] = __ldg(src);
    }
    pdl_done();
}
static_assert(kAppendTokens == kAppendThreads / 32, "one warp finds one token's place");

template <typename K, typename... A>
int launch(K kern, unsigned grid, int threads, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? kOk : kErrCuda;
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
    return launch(fork_apply_kernel, static_cast<unsigned>(grid), kCopyThreads, stream, c, parents, children, n, copy,
                  static_cast<const void *>(ws), err);
}

int launch_cache_compact(const CacheView &c, int *table_out, int *refs_out, int *n_live, void *ws, cudaStream_t stream) {
    int *err = device_error_word();
    const int grid = copy_grid();
    if (!err || grid <= 0) return kErrCuda;
    const int rc = launch(compact_plan_kernel, 1, kPlanThreads, stream, c, refs_out, n_live, ws);
    if (rc != kOk) return rc;
    return launch(compact_apply_kernel, static_cast<unsigned>(grid), kCopyThreads, stream, c, table_out,
                  static_cast<const void *>(ws), err);
}

int launch_cache_append(const CacheView &c, int layer, const void *Kn, const void *Vn, long long token_vecs,
                        long long head_vecs, int T, const int *seqs, const int *q_start, int n, cudaStream_t stream) {
    int *err = device_error_word();
    if (!err) return kErrCuda;
    const unsigned grid = static_cast<unsigned>((T + kAppendTokens - 1) / kAppendTokens);
    return launch(append_kernel, grid, kAppendThreads, stream, c, layer, static_cast<const uint4 *>(Kn),
                  static_cast<const uint4 *>(Vn), token_vecs, head_vecs, T, seqs, q_start, n, err);
}

}  // namespace eta

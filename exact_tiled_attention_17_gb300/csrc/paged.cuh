// What the attn_paged_fwd kernels share: parameters, the device side of the
// work partition (paged_index.h), and the layout of partial results.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "paged_index.h"
#include "ptx.cuh"

namespace eta {

constexpr float kPagedLog2e = 1.4426950408889634f;
constexpr float kPagedLn2 = 0.6931471805599453f;

struct PagedParams {
    PagedGeom gm;
    const void *Q, *K, *V;
    void *O;
    float *LSE;                                    // [T][Hq] or null
    long long q_token, q_head, o_token, o_head;    // strides of Q and O, in elements
    long long page_stride, head_stride, slot_stride;   // strides of one layer's K and V, in elements
    int d, Hq;
    float scale_log2;                              // scale * log2(e)
    // Partial results of units that a share's border cuts: CTA c has slot 2c
    // for a part that does not begin its unit, slot 2c + 1 for one that
    // begins it but does not end it (each at most once).
    int *part_hdr;      // [2 G][4]: valid, entry, h * 2^16... see PagedHdr
    float *part_m, *part_l;   // [2 G][rows]: running maximum (log2 units) and sum
    float *part_o;      // [2 G][rows][d]: unnormalised output
    int part_rows;
    int *err;
};

// Header of a partial slot: rows of the unit it belongs to, and whether it
// holds the unit's last tiles.  rows = 0: the slot is not in use.
struct PagedHdr {
    int rows;    // valid query rows of the unit
    int tok0;    // its first row of Q
    int head;    // its kv head
    int last;    // ends the unit
};

struct PagedPlan {
    PagedPos begin, end;
    long long wsum[32];
    long long carry;
};

// Finds this CTA's share.  All NT threads of the block take part; `plan` is
// shared memory, valid for everyone after the call.  Entries that are out of
// range are recorded in the error word by CTA 0.
template <int NT>
__device__ __forceinline__ void paged_plan(const PagedParams &p, PagedPlan *plan, int cta, int ctas) {
    const PagedGeom &gm = p.gm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int NW = NT / 32;
    // inclusive scan of v over the block; returns the exclusive prefix and the total
    auto scan = [&](long long v, long long &total) -> long long {
        long long inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        __syncthreads();   // the previous scan's sums have been read
        if (lane == 31) plan->wsum[warp] = inc;
        __syncthreads();
        long long before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += plan->wsum[w];
            total += plan->wsum[w];
        }
        return before + inc - v;
    };
    PagedEntry e;
    long long work = 0, W = 0, first = 0;
    bool bad = false;
    for (int c0 = 0; c0 < gm.n; c0 += NT) {
        const int i = c0 + tid;
        work = 0;
        if (i < gm.n) {
            bad |= !paged_entry(gm, i, e);
            work = paged_entry_work(gm, e);
        }
        long long total;
        first = scan(work, total);
        W += total;
    }
    if (bad && cta == 0) atomicOr(p.err, kErrWordBadRow);
    const int shares = paged_shares(gm, W, ctas);
    const long long x0 = paged_share_begin(W, cta, shares), x1 = paged_share_begin(W, cta + 1, shares);
    if (tid == 0) {
        plan->begin = PagedPos{gm.n, 0, 0, 0};
        plan->end = PagedPos{gm.n, 0, 0, 0};
    }
    __syncthreads();
    auto place = [&](int i, long long at) {
        if (x0 >= at && x0 < at + work) plan->begin = paged_locate(gm, e, i, x0 - at);
        if (x1 >= at && x1 < at + work) plan->end = paged_locate(gm, e, i, x1 - at);
    };
    if (gm.n <= NT) {
        place(tid, first);
    } else {
        long long base = 0;
        for (int c0 = 0; c0 < gm.n; c0 += NT) {
            const int i = c0 + tid;
            work = 0;
            if (i < gm.n) {
                paged_entry(gm, i, e);
                work = paged_entry_work(gm, e);
            }
            long long total;
            const long long at = base + scan(work, total);
            place(i, at);
            base += total;
        }
    }
    __syncthreads();
}

// Walks the units (or parts of units) of a share, in order.
struct PagedWalk {
    PagedPos pos, end;
    PagedEntry e;
    int have;   // entry e was read for
    // the current part
    int i, h, u, tile0, tile1, tiles;
    __device__ __forceinline__ void start(const PagedPlan *plan) {
        pos = plan->begin;
        end = plan->end;
        have = -1;
    }
    __device__ __forceinline__ bool next(const PagedGeom &gm) {
        while (paged_less(pos, end)) {
            if (have != pos.i) {
                paged_entry(gm, pos.i, e);
                have = pos.i;
            }
            if (e.nq == 0) {
                pos = PagedPos{pos.i + 1, 0, 0, 0};
                continue;
            }
            i = pos.i;
            h = pos.h;
            u = pos.u;
            tiles = paged_tiles(gm, e, u);
            tile0 = pos.tile;
            const bool same = i == end.i && h == end.h && u == end.u;
            tile1 = same ? min(end.tile, tiles) : tiles;
            paged_next_unit(gm, e, pos);
            if (same) pos = end;
            if (tile1 > tile0) return true;
        }
        return false;
    }
    __device__ __forceinline__ int tok0(const PagedGeom &gm) const { return u * gm.tpu; }   // within the entry
    __device__ __forceinline__ int ntok(const PagedGeom &gm) const { return min(gm.tpu, e.nq - u * gm.tpu); }
    __device__ __forceinline__ bool whole() const { return tile0 == 0 && tile1 == tiles; }
    // slot of a part that is not whole
    __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (tile0 == 0 ? 1 : 0); }
    __device__ __forceinline__ PagedHdr header(const PagedGeom &gm) const {
        return PagedHdr{ntok(gm) * gm.g, e.q0 + tok0(gm), h, tile1 == tiles ? 1 : 0};
    }
};

// The same for a whole warp, with the state in shared memory (registers are
// what the matrix kernel lacks): one lane moves on, everyone reads.
__device__ __forceinline__ bool paged_walk_warp(PagedWalk *w, const PagedGeom &gm) {
    int more = 0;
    __syncwarp();   // everyone has read the part before
    if ((threadIdx.x & 31) == 0) more = w->next(gm) ? 1 : 0;
    __syncwarp();
    return __shfl_sync(0xffffffffu, more, 0) != 0;
}

__device__ __forceinline__ void paged_write_header(const PagedParams &p, int slot, const PagedHdr &h) {
    *reinterpret_cast<int4 *>(p.part_hdr + 4 * slot) = make_int4(h.rows, h.tok0, h.head, h.last);
}
__device__ __forceinline__ PagedHdr paged_read_header(const PagedParams &p, int slot) {
    const int4 v = __ldcg(reinterpret_cast<const int4 *>(p.part_hdr + 4 * slot));
    return PagedHdr{v.x, v.y, v.z, v.w};
}

// Joins the parts of every cut unit (paged_merge.cu): ctas CTAs wrote slots.
int launch_paged_merge(const PagedParams &p, int bf16, int ctas, cudaStream_t stream);

// The variants (each sets its own unit size, partial layout and grid).
int launch_paged_simt(PagedParams p, void *workspace, cudaStream_t stream);
int launch_paged_tc(PagedParams p, void *workspace, cudaStream_t stream);
int launch_paged_decode(PagedParams p, void *workspace, cudaStream_t stream);

// Tensor maps of the bf16 kernels: Q in boxes of `tokens` tokens x g heads x 64
// columns (rows token by token), K and V in boxes of `box` slots x 64 columns of
// one page and head.
bool paged_maps(const PagedParams &p, int tokens, int box, CUtensorMap *tq, CUtensorMap *tk, CUtensorMap *tv);

// Workspace: headers, m, l, o for `ctas` CTAs and units of `rows` rows.
inline size_t paged_partial_bytes(int ctas, int rows, int d) {
    const size_t slots = 2 * static_cast<size_t>(ctas);
    return slots * 16 + slots * rows * (2 + static_cast<size_t>(d)) * sizeof(float);
}
inline void paged_carve(PagedParams &p, void *workspace, int ctas, int rows) {
    const size_t slots = 2 * static_cast<size_t>(ctas);
    char *ws = static_cast<char *>(workspace);
    p.part_hdr = reinterpret_cast<int *>(ws);
    p.part_o = reinterpret_cast<float *>(ws + slots * 16);
    p.part_m = p.part_o + slots * rows * p.d;
    p.part_l = p.part_m + slots * rows;
    p.part_rows = rows;
}

}  // namespace eta

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
    int *part_hdr;      // [2 G][4]: PagedHdr
    int *part_sum;      // [G]: what a CTA's two slots hold (paged_sum)
    float *part_m, *part_l;   // [2 G][rows]: running maximum (log2 units) and sum
    float *part_o;      // [2 G][rows][d]: unnormalised output
    int part_rows;
    int *err;
};

// Header of a slot that begins a unit (2c + 1): where its rows go.
struct PagedHdr {
    int rows;    // valid query rows of the unit
    int tok0;    // its first row of Q
    int head;    // its kv head
    int spare;
};
// A CTA's word for the merge kernel: rows of the unit that it began but did
// not end (0: none), and whether it holds a part of an earlier CTA's unit, and
// the last one.
__device__ __forceinline__ int paged_sum(int tail_rows, bool part, bool last) {
    return tail_rows << 2 | (last ? 2 : 0) | (part ? 1 : 0);
}

// The maximum that goes with a part's sum: -inf for a part without keys, and
// something finite where the sum is NaN, so that the merge passes the NaN on.
__device__ __forceinline__ float paged_part_max(float m, float l) {
    return l == 0.f ? -INFINITY : m == -INFINITY ? 0.f : m;
}

// Reads the parameters once, while the kernel waits for the one before it: a
// first touch of a line of the parameter bank takes about half a microsecond,
// and a short call touches all of them one after the other.
__device__ __forceinline__ void paged_touch(const PagedParams &p) {
    asm volatile("" ::"l"(p.gm.page_table), "l"(p.gm.q_start), "r"(p.gm.rows), "r"(p.gm.heads), "r"(p.gm.unit_cost),
                 "r"(p.gm.g_mul), "l"(p.Q), "l"(p.O), "l"(p.LSE));
    asm volatile("" ::"l"(p.q_token), "l"(p.o_token), "l"(p.o_head), "l"(p.page_stride), "l"(p.slot_stride), "r"(p.Hq),
                 "f"(p.scale_log2), "l"(p.part_sum), "l"(p.part_l), "r"(p.part_rows), "l"(p.err));
}

// One part of a unit as the warps that work on it see it (32-bit words in
// shared memory, read by everyone).
struct PagedUnit {
    int tok0, ntok;      // first row of Q, tokens
    int head;            // kv head
    int tile0, tiles;    // key tiles of this part; tiles = 0: no more work
    int vis0, len;       // keys that token 0 sees (before clamping); keys of the sequence
    int slot;            // partial slot, or -1: the whole unit
    int seq;             // table row
    // the matrix kernel, per query tile: key tiles of this part that it takes
    // part in (the first ones), and how many of them every row sees whole
    int own[2], inner[2];
    int spare[3];
};
static_assert(sizeof(PagedUnit) == 64, "units are copied 16 bytes at a time");

__device__ __forceinline__ int paged_unit_visible(const PagedGeom &gm, const PagedUnit &u, int t) {
    return gm.causal ? max(0, min(u.vis0 + t, u.len)) : u.len;
}

// A CTA's share of the work: found and walked by one warp, all lanes of which
// hold the same state.  Nothing of it is needed by the other warps but the
// units that come out.
struct PagedFeed {
    PagedPos pos, end;
    PagedEntry e;
    int have;   // entry e was read for
    int sum;    // paged_sum of the parts so far

    __device__ __forceinline__ static PagedEntry pick(const PagedEntry &v, int lane) {
        PagedEntry r;
        r.seq = __shfl_sync(0xffffffffu, v.seq, lane);
        r.q0 = __shfl_sync(0xffffffffu, v.q0, lane);
        r.nq = __shfl_sync(0xffffffffu, v.nq, lane);
        r.len = __shfl_sync(0xffffffffu, v.len, lane);
        return r;
    }

    // Entries are dealt to the lanes in runs; lane sums give the line's
    // length, and the lanes that hold the share's two borders find their
    // entries.  Out-of-range entries are recorded by CTA 0.
    __device__ __forceinline__ void start(const PagedParams &p, int cta, int ctas) {
        const PagedGeom &gm = p.gm;
        const int lane = threadIdx.x & 31;
        const int per = (gm.n + 31) >> 5, i0 = lane * per, i1 = min(i0 + per, gm.n);
        PagedEntry le{0, 0, 0, 0};
        long long work = 0;
        bool bad = false;
#pragma unroll 4
        for (int i = i0; i < i1; ++i) {
            bad |= !paged_entry(gm, i, le);
            work += paged_entry_work(gm, le);
        }
        long long inc = work;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        const long long W = __shfl_sync(0xffffffffu, inc, 31), first = inc - work;
        if (bad && cta == 0) atomicOr(p.err, kErrWordBadRow);
        const int shares = paged_shares(gm, W, ctas);
        // (a lane to a border: lane 0 the beginning, lane 1 the end)
        const long long mine = paged_share_begin(W, cta + (lane == 1 ? 1 : 0), shares);
        const long long x0 = __shfl_sync(0xffffffffu, mine, 0), x1 = __shfl_sync(0xffffffffu, mine, 1);
        const int l0 = __ffs(__ballot_sync(0xffffffffu, x0 >= first && x0 < inc)) - 1;
        const int l1 = __ffs(__ballot_sync(0xffffffffu, x1 >= first && x1 < inc)) - 1;
        // the entry of lanes l0 and l1, and what of the line lies before it
        PagedEntry be = le, ee = le;
        int bi = i0, ei = i0;
        long long bx = x0 - first, ex = x1 - first;
        if (per > 1) {
            auto seek = [&](int &i, PagedEntry &v, long long &x) {
                for (i = i0; i < i1; ++i) {
                    paged_entry(gm, i, v);
                    const long long w = paged_entry_work(gm, v);
                    if (x < w) break;
                    x -= w;
                }
            };
            if (lane == l0) seek(bi, be, bx);
            if (lane == l1) seek(ei, ee, ex);
            __syncwarp();
        }
        const int s0 = max(l0, 0), s1 = max(l1, 0);
        be = pick(be, s0);
        ee = pick(ee, s1);
        bi = __shfl_sync(0xffffffffu, bi, s0);
        ei = __shfl_sync(0xffffffffu, ei, s1);
        bx = __shfl_sync(0xffffffffu, bx, s0);
        ex = __shfl_sync(0xffffffffu, ex, s1);
        PagedPos at{gm.n, 0, 0, 0};
        if (lane == 0 && l0 >= 0) at = paged_locate(gm, be, bi, bx);
        if (lane == 1 && l1 >= 0) at = paged_locate(gm, ee, ei, ex);
        __syncwarp();
        pos.i = __shfl_sync(0xffffffffu, at.i, 0);
        pos.h = __shfl_sync(0xffffffffu, at.h, 0);
        pos.u = __shfl_sync(0xffffffffu, at.u, 0);
        pos.tile = __shfl_sync(0xffffffffu, at.tile, 0);
        end.i = __shfl_sync(0xffffffffu, at.i, 1);
        end.h = __shfl_sync(0xffffffffu, at.h, 1);
        end.u = __shfl_sync(0xffffffffu, at.u, 1);
        end.tile = __shfl_sync(0xffffffffu, at.tile, 1);
        e = be;
        have = l0 >= 0 && pos.i == bi ? bi : -1;
        sum = 0;
    }

    // The next part of the share; tiles = 0 when there is none.
    __device__ __forceinline__ void next(const PagedParams &p, int cta, PagedUnit &out) {
        const PagedGeom &gm = p.gm;
        out.tiles = 0;
        while (paged_less(pos, end)) {
            if (have != pos.i) {
                paged_entry(gm, pos.i, e);
                have = pos.i;
            }
            if (e.nq == 0) {
                pos = PagedPos{pos.i + 1, 0, 0, 0};
                continue;
            }
            const int tiles = paged_tiles(gm, e, pos.u), tile0 = pos.tile;
            const bool same = pos.i == end.i && pos.h == end.h && pos.u == end.u;
            const int tile1 = same ? min(end.tile, tiles) : tiles;
            const int t0 = pos.u * gm.tpu;
            out.tok0 = e.q0 + t0;
            out.ntok = min(gm.tpu, e.nq - t0);
            out.head = pos.h;
            out.tile0 = tile0;
            out.vis0 = e.len - e.nq + t0 + 1;
            out.len = e.len;
            out.seq = e.seq;
            paged_next_unit(gm, e, pos);
            if (same) pos = end;
            if (tile1 <= tile0) continue;
            out.tiles = tile1 - tile0;
            out.slot = tile0 == 0 && tile1 == tiles ? -1 : 2 * cta + (tile0 == 0 ? 1 : 0);
            if (tile0 > 0) sum |= paged_sum(0, true, tile1 == tiles);
            else if (tile1 < tiles) sum |= paged_sum(out.ntok * gm.g, false, false);
            break;
        }
    }
    // Leaves what the merge kernel wants to know about a part / about the CTA.
    __device__ __forceinline__ void report(const PagedParams &p, const PagedUnit &u) const;
    __device__ __forceinline__ void finish(const PagedParams &p, int cta) const {
        if ((threadIdx.x & 31) == 0) p.part_sum[cta] = sum;
    }
};

__device__ __forceinline__ void paged_write_header(const PagedParams &p, int slot, const PagedHdr &h) {
    *reinterpret_cast<int4 *>(p.part_hdr + 4 * slot) = make_int4(h.rows, h.tok0, h.head, 0);
}
__device__ __forceinline__ void PagedFeed::report(const PagedParams &p, const PagedUnit &u) const {
    if (u.slot >= 0 && u.tile0 == 0 && (threadIdx.x & 31) == 0)
        paged_write_header(p, u.slot, PagedHdr{u.ntok * p.gm.g, u.tok0, u.head, 0});
}
__device__ __forceinline__ PagedHdr paged_read_header(const PagedParams &p, int slot) {
    const int4 v = __ldcg(reinterpret_cast<const int4 *>(p.part_hdr + 4 * slot));
    return PagedHdr{v.x, v.y, v.z, v.w};
}

// Joins the parts of every cut unit (paged_merge.cu): ctas CTAs wrote slots,
// on a device of `sms` SMs.
int launch_paged_merge(const PagedParams &p, int bf16, int ctas, int sms, cudaStream_t stream);

// Rows of a unit (sizes the workspace too).  The stream kernel: 16 or 32,
// whichever holds an entry.  The CUDA-core kernels: 4, 8, 16, 32 or 64 (from 16 on
// the one that tiles).
inline int paged_decode_rows(int g, int max_q) { return static_cast<long long>(g) * max_q <= 16 ? 16 : 32; }
inline int paged_simt_rows(int g, int max_q) {
    const long long rows = static_cast<long long>(g) * max_q;
    return rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// The variants (each sets its own unit size, partial layout and grid).
int launch_paged_few(PagedParams p, void *workspace, cudaStream_t stream);
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
    return slots * 16 + (ctas * sizeof(int) + 15) / 16 * 16 + slots * rows * (2 + static_cast<size_t>(d)) * sizeof(float);
}
inline void paged_carve(PagedParams &p, void *workspace, int ctas, int rows) {
    const size_t slots = 2 * static_cast<size_t>(ctas);
    char *ws = static_cast<char *>(workspace);
    p.part_hdr = reinterpret_cast<int *>(ws);
    p.part_sum = reinterpret_cast<int *>(ws + slots * 16);
    p.part_o = reinterpret_cast<float *>(ws + slots * 16 + (ctas * sizeof(int) + 15) / 16 * 16);
    p.part_m = p.part_o + slots * rows * p.d;
    p.part_l = p.part_m + slots * rows;
    p.part_rows = rows;
}

}  // namespace eta

// Rows in and out of a paged cache where a value changes on its way: appending
// with the position rotation (queries too), appending to a cache of 4-bit
// values, and reading tokens back as contiguous rows.
//
// Rotation: the pair (a, b) of a row's columns becomes (a c - b s, b c + a s),
// with c and s from the table's row of the token's position; products and the
// sum are rounded to float32 one by one (no fused multiply-add), so that the
// result is the same wherever it is computed.
//
// 4-bit rows (e2m1.cuh): 16 columns share a scale.
//
// A lane owns 16 columns of a row: two runs of 8, contiguous, or (halves rotated)
// 8 columns of the lower half and their partners in the upper one, so a pair is
// in one lane and a group of 16 columns in two neighbouring ones.  All lanes of a
// row are in one warp.
#include <algorithm>

#include <cuda_bf16.h>

#include "e2m1.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace eta {
namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_done() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Where a token of the list lies.
struct Place {
    long long block;   // first byte of its page's block in this layer; -1: nowhere
    int slot, pos;     // slot of the page, index in its sequence
};

// One warp finds the place of row t.  WRITE: the rows are the sequences' last
// tokens, go into pages of their own, and no sequence is named twice; else they
// are tokens first[i] .. (null: the last ones).
template <bool WRITE>
__device__ __forceinline__ Place find_place(const CacheView &c, const RowList &li, int layer, int t, int *err) {
    const int lane = threadIdx.x & 31;
    Place out{-1, 0, 0};
    // the last entry that begins at or before t (what it says comes along: each read that waits for another costs 0.3 us)
    int i = -1, q0 = 0, q1 = 0, s = 0;
    for (int j0 = 0; j0 < li.n; j0 += 32) {
        const int j = j0 + lane;
        int b = 0x7fffffff, e = 0, row_of = j;
        if (j < li.n) {
            b = li.q_start[j];
            e = li.q_start[j + 1];
            if (li.seqs) row_of = li.seqs[j];
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
    if (i < 0 || t >= q1) return out;
    if (li.granted && li.granted[i] == 0) return out;
    bool bad = !(q0 >= 0 && q1 <= li.T && s >= 0 && s < c.rows);
    if (!bad) {
        const int len = c.seq_lens[s];   // (on its way while the list is looked through)
        if constexpr (WRITE) {
            if (li.seqs)
                for (int j0 = 0; j0 < i && !bad; j0 += 32) {
                    const int j = j0 + lane;
                    const bool same = j < i && li.seqs[j] == s && li.q_start[j + 1] > li.q_start[j] &&
                                      (!li.granted || li.granted[j] != 0);
                    bad = __any_sync(0xffffffffu, same);
                }
        }
        const long long from = !WRITE && li.first ? li.first[i] : static_cast<long long>(len) - (q1 - q0);
        const long long pos = from + (t - q0);
        bad = bad || pos < 0 || (li.first && from < 0) || pos >= len || pos / c.page_size >= c.max_pages;
        if (!bad) {
            const int id = c.page_table[static_cast<long long>(s) * c.max_pages + pos / c.page_size];
            // (a page that other table entries name too is read by those sequences: it is never written)
            bad = id < 0 || id >= c.pages || (WRITE && c.ref_counts[id] > 1);
            if (!bad) {
                out.block = (layer * c.layer_vecs + id * c.page_vecs) * 16;
                out.pos = static_cast<int>(pos);
                out.slot = out.pos % c.page_size;
            }
        }
    }
    if (bad && lane == 0) atomicOr(err, kErrWordBadRow);
    return out;
}

// Entries whose range is none, or reaches past the rows: reported once (one warp of the grid), since none of their rows need be met.
__device__ __forceinline__ void check_ranges(const RowList &li, int *err) {
    bool none = false;
    for (int j = threadIdx.x & 31; j < li.n; j += 32) {
        const int a = li.q_start[j], b = li.q_start[j + 1];
        none |= (a < 0 || b < a || b > li.T) && (!li.granted || li.granted[j] != 0);
    }
    if (none) atomicOr(err, kErrWordBadRow);
}

// 8 values of a row.
template <typename T>
struct Run8;
template <>
struct Run8<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const char *p) { w = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = bf16lo_to_f32(u[e]);
            x[2 * e + 1] = bf16hi_to_f32(u[e]);
        }
    }
    static __device__ __forceinline__ void put(char *p, const float (&x)[8]) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                                   pack_bf16x2(x[6], x[7]));
    }
    static __device__ __forceinline__ float one(const char *p) { return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(p)); }
};
template <>
struct Run8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const char *p) {
        a = __ldcs(reinterpret_cast<const float4 *>(p));
        b = __ldcs(reinterpret_cast<const float4 *>(p + 16));
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    static __device__ __forceinline__ void put(char *p, const float (&x)[8]) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 16) = make_float4(x[4], x[5], x[6], x[7]);
    }
    static __device__ __forceinline__ float one(const char *p) { return *reinterpret_cast<const float *>(p); }
};

__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// T: the type of the rows that come in.  Q4: the cache holds 4-bit values.
template <typename T, bool Q4, int TOK>
__global__ void __launch_bounds__(kRowThreads) append_rows_kernel(const CacheView c, int layer, const RowIn in, const RowList li,
                                                                  const Rotation r, int *err) {
    static_assert(TOK <= kRowThreads / 32, "one warp finds one token's place");
    constexpr int ES = sizeof(T);
    __shared__ Place places[TOK];
    pdl_wait();
    const int t0 = blockIdx.x * TOK, ntok = min(TOK, li.T - t0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lpr = 1 << in.lane_shift;              // lanes of a row (d / 16, up to a power of two)
    const int rows = 2 * c.heads + in.Hq;            // of a token: K, V, Q
    const int items = ntok * rows * lpr;
    const int l = threadIdx.x & (lpr - 1);
    const bool halves = r.dims > 0 && !r.neighbours, fast = halves && r.dims % 32 == 0;
    const int half = r.dims / 2;

    // what a lane works on: the row's address, its first columns, whether it turns
    struct Item {
        const char *src;
        int tok, row, c0, c1;
        bool rot;
        Run8<T> x0, x1;
    };
    auto fetch = [&](int at, Item &w) {
        w.tok = -1;
        w.x0.zero();
        w.x1.zero();
        w.c0 = 16 * l;
        w.c1 = 16 * l + 8;
        w.rot = false;
        w.row = 0;
        w.src = nullptr;
        if (at >= items || 16 * l >= in.d) return;
        const int y = at >> in.lane_shift;
        w.tok = y / rows;
        w.row = y - w.tok * rows;
        const long long t = t0 + w.tok;
        if (w.row < c.heads) w.src = in.K + t * in.token_bytes + w.row * in.head_bytes;
        else if (w.row < 2 * c.heads) w.src = in.V + t * in.token_bytes + (w.row - c.heads) * in.head_bytes;
        else w.src = in.Q + t * in.q_token_bytes + (w.row - 2 * c.heads) * in.q_head_bytes;
        w.rot = w.c0 < r.dims && (w.row < c.heads || w.row >= 2 * c.heads);
        if (w.rot && fast) {
            w.c0 = 8 * l;
            w.c1 = half + 8 * l;
        }
        w.x0.load(w.src + w.c0 * ES);
        w.x1.load(w.src + w.c1 * ES);
    };
    Item cur;
    fetch(threadIdx.x, cur);
    if (warp < TOK) {
        Place p{-1, 0, 0};
        if (t0 + warp < li.T) {
            p = find_place<true>(c, li, layer, t0 + warp, err);
            if (r.dims > 0 && p.block >= 0) {
                if (r.positions) p.pos = r.positions[t0 + warp];
                if (p.pos < 0 || p.pos >= r.rows) {   // no such row of the table
                    p.block = -1;
                    if (lane == 0) atomicOr(err, kErrWordBadRow);
                }
            }
        }
        if (lane == 0) places[warp] = p;
    }
    if (blockIdx.x == 0 && warp == kRowThreads / 32 - 1) check_ranges(li, err);
    __syncthreads();

    for (int at = threadIdx.x; at - static_cast<int>(threadIdx.x) < items; at += kRowThreads) {
        Item w = cur;
        fetch(at + kRowThreads, cur);
        const Place p = w.tok >= 0 ? places[w.tok] : Place{-1, 0, 0};
        const bool live = p.block >= 0;
        float x0[8], x1[8];
        w.x0.get(x0);
        w.x1.get(x1);
        if (w.rot && live) {
            const float *cs = r.table + static_cast<long long>(p.pos) * r.dims;
            if (fast) {
                float co[8], si[8];
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float4 a = __ldg(reinterpret_cast<const float4 *>(cs + w.c0 + e));
                    const float4 b = __ldg(reinterpret_cast<const float4 *>(cs + half + w.c0 + e));
                    co[e] = a.x, co[e + 1] = a.y, co[e + 2] = a.z, co[e + 3] = a.w;
                    si[e] = b.x, si[e + 1] = b.y, si[e + 2] = b.z, si[e + 3] = b.w;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) turn(x0[e], x1[e], co[e], si[e]);
            } else if (!halves) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    if (w.c0 + e < r.dims) turn(x0[e], x0[e + 1], __ldg(cs + (w.c0 + e) / 2), __ldg(cs + half + (w.c0 + e) / 2));
                    if (w.c1 + e < r.dims) turn(x1[e], x1[e + 1], __ldg(cs + (w.c1 + e) / 2), __ldg(cs + half + (w.c1 + e) / 2));
                }
            } else {
                // halves that do not fall on runs of 16: the partners are read one by one
                auto other = [&](float &x, int col) {
                    if (col >= r.dims) return;
                    const bool lower = col < half;
                    const int j = lower ? col : col - half;
                    float y = Run8<T>::one(w.src + (lower ? col + half : j) * ES);
                    const float co = __ldg(cs + j), si = __ldg(cs + half + j);
                    if (lower) turn(x, y, co, si);
                    else turn(y, x, co, si);
                };
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    other(x0[e], w.c0 + e);
                    other(x1[e], w.c1 + e);
                }
            }
        }
        __syncwarp();   // (Q may be turned in place: every lane of the row has read what it needs)
        if constexpr (Q4) {
            // the groups of columns c0 and c1: one lane's own 16 columns, or 8 of this lane and 8 of its neighbour
            uint32_t a0 = e2m1_amax(x0), a1 = e2m1_amax(x1);
            const uint32_t n0 = __shfl_xor_sync(0xffffffffu, a0, 1), n1 = __shfl_xor_sync(0xffffffffu, a1, 1);
            const bool split = w.rot && fast;
            a0 = max(a0, split ? n0 : a1);
            a1 = split ? max(a1, n1) : a0;
            if (live && w.row < 2 * c.heads) {
                const bool v = w.row >= c.heads;
                const int h = v ? w.row - c.heads : w.row;
                char *blk = reinterpret_cast<char *>(v ? c.v : c.k) + p.block + h * c.head_stride_vecs * 16;
                char *codes = blk + p.slot * (in.d / 2);
                char *scales = blk + c.page_size * (in.d / 2) + p.slot * (in.d / 16);
                const int s0 = e2m1_scale(a0), s1 = e2m1_scale(a1);
                *reinterpret_cast<uint32_t *>(codes + w.c0 / 2) = e2m1_pack(x0, s0);
                *reinterpret_cast<uint32_t *>(codes + w.c1 / 2) = e2m1_pack(x1, s1);
                if (!split) scales[l] = static_cast<char>(s0);
                else if (l & 1) scales[w.c1 / 16] = static_cast<char>(s1);
                else scales[w.c0 / 16] = static_cast<char>(s0);
            }
        } else if (live && w.row < 2 * c.heads) {
            const bool v = w.row >= c.heads;
            const int h = v ? w.row - c.heads : w.row;
            char *dst = reinterpret_cast<char *>(v ? c.v : c.k) + p.block + (h * c.head_stride_vecs + p.slot * c.slot_stride_vecs) * 16;
            Run8<T>::put(dst + w.c0 * ES, x0);
            Run8<T>::put(dst + w.c1 * ES, x1);
        }
        if (live && w.row >= 2 * c.heads) {
            char *dst = in.Qout + (t0 + w.tok) * in.o_token_bytes + (w.row - 2 * c.heads) * in.o_head_bytes;
            Run8<T>::put(dst + w.c0 * ES, x0);
            Run8<T>::put(dst + w.c1 * ES, x1);
        }
    }
    pdl_done();
}

// Reading: a lane takes 16 columns of a 4-bit row, or a 16-byte piece of another.
template <bool Q4, int TOK>
__global__ void __launch_bounds__(kRowThreads) read_rows_kernel(const CacheView c, int layer, const RowOut out, const RowList li,
                                                                int *err) {
    static_assert(TOK <= kRowThreads / 32, "one warp finds one token's place");
    __shared__ Place places[TOK];
    pdl_wait();
    const int t0 = blockIdx.x * TOK, ntok = min(TOK, li.T - t0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp < TOK) {
        Place p{-1, 0, 0};
        if (t0 + warp < li.T) p = find_place<false>(c, li, layer, t0 + warp, err);
        if (lane == 0) places[warp] = p;
    }
    if (blockIdx.x == 0 && warp == kRowThreads / 32 - 1) check_ranges(li, err);
    __syncthreads();
    const int per = Q4 ? out.d / 16 : c.row_vecs, rows = 2 * c.heads, items = ntok * rows * per;
    for (int at = threadIdx.x; at < items; at += kRowThreads) {
        const int y = at / per, l = at - y * per, tok = y / rows, row = y - tok * rows;
        const Place p = places[tok];
        if (p.block < 0) continue;
        const bool v = row >= c.heads;
        const int h = v ? row - c.heads : row;
        const char *blk = reinterpret_cast<const char *>(v ? c.v : c.k) + p.block + h * c.head_stride_vecs * 16;
        char *dst = (v ? out.V : out.K) + (t0 + tok) * out.token_bytes + h * out.head_bytes;
        if constexpr (Q4) {
            const uint2 codes = *reinterpret_cast<const uint2 *>(blk + p.slot * (out.d / 2) + 8 * l);
            const uint32_t s2 = e2m1_scale_h2(*reinterpret_cast<const uint8_t *>(blk + c.page_size * (out.d / 2) + p.slot * (out.d / 16) + l));
            uint32_t h2[8], w[8];
            e2m1_values(codes.x, s2, h2);
            e2m1_values(codes.y, s2, h2 + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) {   // (at most 6 significant bits: exact in bf16)
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(h2 + e));
                w[e] = pack_bf16x2(f.x, f.y);
            }
            uint4 *to = reinterpret_cast<uint4 *>(dst + 32 * l);
            to[0] = make_uint4(w[0], w[1], w[2], w[3]);
            to[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
            reinterpret_cast<uint4 *>(dst)[l] = *reinterpret_cast<const uint4 *>(blk + p.slot * c.slot_stride_vecs * 16 + 16 * l);
        }
    }
    pdl_done();
}

unsigned blocks(int T, int tok) { return static_cast<unsigned>((static_cast<long long>(T) + tok - 1) / tok); }

template <typename T, bool Q4>
int launch_append(const CacheView &c, int layer, const RowIn &in, const RowList &li, const Rotation &r, int *err, cudaStream_t stream) {
    if (li.T <= 4096)
        return launch_dependent(append_rows_kernel<T, Q4, 2>, dim3(blocks(li.T, 2)), kRowThreads, 0, stream, c, layer, in, li, r, err);
    return launch_dependent(append_rows_kernel<T, Q4, 8>, dim3(blocks(li.T, 8)), kRowThreads, 0, stream, c, layer, in, li, r, err);
}

}  // namespace

int launch_cache_rows_in(const CacheView &c, int layer, RowIn in, const RowList &li, const Rotation &r, cudaStream_t stream) {
    int *err = device_error_word();
    if (!err) return kErrCuda;
    in.lane_shift = in.d <= 32 ? 1 : in.d <= 64 ? 2 : 3;
    if (c.bits == 4) return launch_append<__nv_bfloat16, true>(c, layer, in, li, r, err, stream);
    if (c.bits == 16) return launch_append<__nv_bfloat16, false>(c, layer, in, li, r, err, stream);
    return launch_append<float, false>(c, layer, in, li, r, err, stream);
}

int launch_cache_rows_out(const CacheView &c, int layer, const RowOut &out, const RowList &li, cudaStream_t stream) {
    int *err = device_error_word();
    if (!err) return kErrCuda;
    auto go = [&](auto kern, int tok) {
        return launch_dependent(kern, dim3(blocks(li.T, tok)), kRowThreads, 0, stream, c, layer, out, li, err);
    };
    if (c.bits == 4) return go(read_rows_kernel<true, 4>, 4);
    return go(read_rows_kernel<false, 4>, 4);
}

}  // namespace eta

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
// A CTA takes TOK consecutive tokens; warp w finds where token w lies.  A lane owns 16
// columns of a row: two runs of 8, contiguous, or (halves rotated) 8 columns of the
// lower half and their partners in the upper one, so a pair is in one lane and a group
// of 16 columns in two.  All lanes of a row are in one warp.  The
// CTA's threads go through the rows of all its tokens in one line, each with the next
// two on their way.  (Four CTAs an SM, 64 registers: the appends of bf16 rows spill 4 to
// 36 bytes a thread, 92 where halves end inside a group of 16.)
#include <algorithm>

#include <cuda_bf16.h>

#include "e2m1.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace eta {
namespace {

constexpr int kRowThreads = 256;
// Tokens to a CTA, where there are more than kFewTokens (else one).  8 kv heads of 128,
// appending 4 x 1500 .. 2048 tokens (32 query heads): 2, 4 and 8 take 43, 38 and 41 us;
// reading 16 x 1000 .. 4096 of 4 bits: 74, 52 and 44.  (One warp that finds the next
// group's places while the others copy gains nothing.)
// One against many, bf16, 512 / 1024 / 2048 tokens: 8 kv and 32 query heads 8.4 and 10.3 /
// 12.3 and 11.3 / 17.9 and 14.7 us, 1 and 4 heads 8.7 and 8.9 / 10.7 and 8.9 / 15.0 and
// 9.0; reading takes the same up to 1024 (8.5), then 10.1 and 8.5.
constexpr int kAppendTokens = 4, kReadTokens = 8, kFewTokens = 1024;

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
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
    static __device__ __forceinline__ void put(char *p, const float (&x)[8]) { *reinterpret_cast<uint4 *>(p) = pack(x); }
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
    static __device__ __forceinline__ uint4 pack(const float (&)[8]) { return make_uint4(0, 0, 0, 0); }   // (16-bit rows only)
    static __device__ __forceinline__ float one(const char *p) { return *reinterpret_cast<const float *>(p); }
};

__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// 32 bytes to 32-byte aligned memory in one piece (whole sectors), or in two to what is aligned to 16.
__device__ __forceinline__ void put32(char *dst, const uint4 &a, const uint4 &b) {
    if ((reinterpret_cast<uintptr_t>(dst) & 31u) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                     "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        *reinterpret_cast<uint4 *>(dst) = a;
        *reinterpret_cast<uint4 *>(dst + 16) = b;
    }
}

// How columns are paired.  Halves of a multiple of 8 columns each, so that a lane
// holds whole pairs; others, whose partners a lane reads one by one (4 x 1500 .. 2048
// tokens of bf16, 48 and 52 of 128 columns: 39 and 74 us).  kHalvesApart: into 4 bits,
// halves that end inside a group of 16 (a branch instead costs the others 52 -> 55 us).
enum class Turn { kNone, kHalves, kHalvesApart, kNeighbours, kOddHalves };
__host__ __device__ constexpr bool in_lane_halves(Turn t) { return t == Turn::kHalves || t == Turn::kHalvesApart; }

// A row of a CTA's tokens; the CTA's threads step through them together.
struct RowAt {
    int tok, row;
    __device__ __forceinline__ void next(int step, int rows) {
        row += step;
        while (row >= rows) {
            row -= rows;
            ++tok;
        }
    }
};

// T: the type of the rows that come in.  Q4: the cache holds 4-bit values.
template <typename T, bool Q4, Turn TURN, int TOK>
__global__ void __launch_bounds__(kRowThreads, sizeof(T) == 2 ? 4 : 3) append_rows_kernel(const CacheView c, int layer, const RowIn in,
                                                                                          const RowList li, const Rotation r, int *err) {
    static_assert(TOK <= kRowThreads / 32, "one warp finds one token's place");
    constexpr int ES = sizeof(T);
    __shared__ Place places[TOK];
    pdl_wait();
    const int t0 = blockIdx.x * TOK, ntok = min(TOK, li.T - t0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int turning = c.heads + in.Hq, rows = turning + c.heads;    // of a token: K, Q, V
    const int lpr = 1 << in.lane_shift, l = threadIdx.x & (lpr - 1);   // lanes of a row (d / 16, up to a power of two)
    const int step = kRowThreads >> in.lane_shift;                     // rows that the CTA takes at once
    const int half = r.dims / 2;
    const bool mine = 16 * l < in.d;
    const bool mixed = in_lane_halves(TURN) && 16 * l < r.dims;       // this lane's runs of a turning row are a half apart

    auto address = [&](const RowAt &a) -> const char * {
        const long long t = t0 + a.tok;
        return a.row < c.heads ? in.K + t * in.token_bytes + a.row * in.head_bytes
               : a.row < turning ? in.Q + t * in.q_token_bytes + (a.row - c.heads) * in.q_head_bytes
                                 : in.V + t * in.token_bytes + (a.row - turning) * in.head_bytes;
    };
    struct Item {
        Run8<T> x0, x1;
    };
    RowAt ahead{0, 0};
    ahead.next(static_cast<int>(threadIdx.x) >> in.lane_shift, rows);
    RowAt now = ahead;
    auto fetch = [&](Item &w) {
        w.x0.zero();
        w.x1.zero();
        if (ahead.tok < ntok && mine) {
            const char *src = address(ahead);
            const bool m = mixed && ahead.row < turning;
            w.x0.load(src + (m ? 8 * l : 16 * l) * ES);
            w.x1.load(src + (m ? half + 8 * l : 16 * l + 8) * ES);
        }
        ahead.next(step, rows);
    };
    // (rows do not depend on where they go: the first are read before the places are known)
    Item buf[2];
    fetch(buf[0]);
    fetch(buf[1]);
    if (warp < TOK) {
        Place p{-1, 0, 0};
        if (t0 + warp < li.T) {
            p = find_place<true>(c, li, layer, t0 + warp, err);
            if (TURN != Turn::kNone && p.block >= 0) {
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

    auto finish = [&](const Item &w) {
        const Place p = now.tok < ntok ? places[now.tok] : Place{-1, 0, 0};
        const bool live = mine && p.block >= 0, turns = now.row < turning, m = mixed && turns;
        const int c0 = m ? 8 * l : 16 * l, c1 = m ? half + 8 * l : 16 * l + 8;
        float x0[8], x1[8];
        w.x0.get(x0);
        w.x1.get(x1);
        if (TURN != Turn::kNone && live && turns) {
            const float *cs = r.table + static_cast<long long>(p.pos) * r.dims;
            if constexpr (in_lane_halves(TURN)) {
                if (m) {
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 a = __ldg(reinterpret_cast<const float4 *>(cs + c0 + e));
                        const float4 b = __ldg(reinterpret_cast<const float4 *>(cs + half + c0 + e));
                        turn(x0[e], x1[e], a.x, b.x);
                        turn(x0[e + 1], x1[e + 1], a.y, b.y);
                        turn(x0[e + 2], x1[e + 2], a.z, b.z);
                        turn(x0[e + 3], x1[e + 3], a.w, b.w);
                    }
                }
            } else if constexpr (TURN == Turn::kNeighbours) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = c0 / 2 + e, k = c1 / 2 + e;
                    if (i < half) turn(x0[2 * e], x0[2 * e + 1], __ldg(cs + i), __ldg(cs + half + i));
                    if (k < half) turn(x1[2 * e], x1[2 * e + 1], __ldg(cs + k), __ldg(cs + half + k));
                }
            } else {
                const char *src = address(now);
                auto other = [&](float &x, int col) {
                    if (col >= r.dims) return;
                    const bool lower = col < half;
                    const int j = lower ? col : col - half;
                    float y = Run8<T>::one(src + (lower ? col + half : j) * ES);
                    const float co = __ldg(cs + j), si = __ldg(cs + half + j);
                    if (lower) turn(x, y, co, si);
                    else turn(y, x, co, si);
                };
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    other(x0[e], c0 + e);
                    other(x1[e], c1 + e);
                }
            }
        }
        __syncwarp();   // (Q may be turned in place: every lane of the row has read what it needs)
        const bool v = !turns, query = turns && now.row >= c.heads;
        const int h = v ? now.row - turning : now.row;
        if constexpr (Q4) {
            // the groups of columns c0 and c1: one lane's own 16 columns, or 8 of this lane and 8 of its neighbour
            uint32_t a0 = e2m1_amax(x0), a1 = e2m1_amax(x1);
            uint32_t n0 = __shfl_xor_sync(0xffffffffu, a0, 1), n1 = __shfl_xor_sync(0xffffffffu, a1, 1);
            if constexpr (TURN == Turn::kHalvesApart) {
                // the halves meet inside a group: the upper half's groups are lanes (1, 2), (3, 4) ..., and the last
                // run of the lower half goes with the first of the upper one, lane 0's
                const int lanes = half / 8, first = lane - l;
                n1 = __shfl_sync(0xffffffffu, a1, first + ((l & 1 ? l + 1 : l - 1) & (lpr - 1)));
                const uint32_t x = __shfl_sync(0xffffffffu, l == 0 ? a1 : a0, first + (l == 0 ? lanes - 1 : 0));
                if (l == 0) n1 = lanes == 1 ? a0 : x;
                if (l == lanes - 1) n0 = x;
            }
            a0 = max(a0, m ? n0 : a1);
            a1 = m ? max(a1, n1) : a0;
            if (live && !query) {
                char *blk = reinterpret_cast<char *>(v ? c.v : c.k) + p.block + h * c.head_stride_vecs * 16;
                char *codes = blk + p.slot * (in.d / 2);
                char *scales = blk + c.page_size * (in.d / 2) + p.slot * (in.d / 16);
                const int s0 = e2m1_scale(a0), s1 = e2m1_scale(a1);
                const uint32_t w0 = e2m1_pack(x0, s0), w1 = e2m1_pack(x1, s1);
                if (m) {
                    *reinterpret_cast<uint32_t *>(codes + c0 / 2) = w0;
                    *reinterpret_cast<uint32_t *>(codes + c1 / 2) = w1;
                    scales[l & 1 ? c1 / 16 : c0 / 16] = static_cast<char>(l & 1 ? s1 : s0);
                } else {
                    *reinterpret_cast<uint2 *>(codes + c0 / 2) = make_uint2(w0, w1);
                    scales[l] = static_cast<char>(s0);
                }
            }
        }
        if (live && (query || !Q4)) {
            char *dst = query ? in.Qout + (t0 + now.tok) * in.o_token_bytes + (h - c.heads) * in.o_head_bytes
                              : reinterpret_cast<char *>(v ? c.v : c.k) + p.block + (h * c.head_stride_vecs + p.slot * c.slot_stride_vecs) * 16;
            if (ES == 2 && !m) {
                put32(dst + c0 * ES, Run8<T>::pack(x0), Run8<T>::pack(x1));
            } else {
                Run8<T>::put(dst + c0 * ES, x0);
                Run8<T>::put(dst + c1 * ES, x1);
            }
        }
        now.next(step, rows);
    };
    // (whole warps: a row's lanes are in one, and the first row of the CTA's is the first to reach an end)
    const int rounds = (ntok * rows + step - 1) / step;
    for (int k = 0; k < rounds; k += 2) {
        const Item a = buf[0];
        fetch(buf[0]);
        finish(a);
        if (k + 1 < rounds) {
            const Item b = buf[1];
            fetch(buf[1]);
            finish(b);
        }
    }
    pdl_done();
}

// Reading: a lane takes 16 columns of a 4-bit row, or a 16-byte piece of another, four of them at once.
template <bool Q4, int TOK>
__global__ void __launch_bounds__(kRowThreads) read_rows_kernel(const CacheView c, int layer, const RowOut out, const RowList li,
                                                                int *err) {
    static_assert(TOK <= kRowThreads / 32, "one warp finds one token's place");
    constexpr int U = 4;
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
    const int rows = 2 * c.heads, step = kRowThreads >> out.lane_shift;
    const int l = threadIdx.x & ((1 << out.lane_shift) - 1);
    const bool mine = l < (Q4 ? out.d / 16 : c.row_vecs);
    RowAt at{0, 0};
    at.next(static_cast<int>(threadIdx.x) >> out.lane_shift, rows);
    while (at.tok < ntok) {
        uint4 x[U];
        uint32_t sc[U];
        char *to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            to[u] = nullptr;
            if (at.tok < ntok && mine) {
                const Place p = places[at.tok];
                const bool v = at.row >= c.heads;
                const int h = v ? at.row - c.heads : at.row;
                const char *blk = reinterpret_cast<const char *>(v ? c.v : c.k) + p.block + h * c.head_stride_vecs * 16;
                if (p.block >= 0) {
                    to[u] = (v ? out.V : out.K) + (t0 + at.tok) * out.token_bytes + h * out.head_bytes + l * (Q4 ? 32 : 16);
                    if constexpr (Q4) {
                        const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(blk + p.slot * (out.d / 2) + 8 * l));
                        x[u].x = w.x;
                        x[u].y = w.y;
                        sc[u] = *reinterpret_cast<const uint8_t *>(blk + c.page_size * (out.d / 2) + p.slot * (out.d / 16) + l);
                    } else {
                        x[u] = __ldcs(reinterpret_cast<const uint4 *>(blk + p.slot * c.slot_stride_vecs * 16 + 16 * l));
                    }
                }
            }
            at.next(step, rows);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!to[u]) continue;
            if constexpr (Q4) {
                uint32_t h2[8], w[8];
                e2m1_values(x[u].x, e2m1_scale_h2(sc[u]), h2);
                e2m1_values(x[u].y, e2m1_scale_h2(sc[u]), h2 + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) {   // (at most 6 significant bits: exact in bf16)
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(h2 + e));
                    w[e] = pack_bf16x2(f.x, f.y);
                }
                put32(to[u], make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
            } else {
                *reinterpret_cast<uint4 *>(to[u]) = x[u];
            }
        }
    }
    pdl_done();
}

unsigned blocks(int T, int tok) { return static_cast<unsigned>((static_cast<long long>(T) + tok - 1) / tok); }

template <typename T, bool Q4, Turn TURN>
int launch_turn(const CacheView &c, int layer, const RowIn &in, const RowList &li, const Rotation &r, int *err, cudaStream_t stream) {
    if (li.T <= kFewTokens)
        return launch_dependent(append_rows_kernel<T, Q4, TURN, 1>, dim3(blocks(li.T, 1)), kRowThreads, 0, stream, c, layer, in, li, r, err);
    return launch_dependent(append_rows_kernel<T, Q4, TURN, kAppendTokens>, dim3(blocks(li.T, kAppendTokens)), kRowThreads, 0, stream, c, layer,
                            in, li, r, err);
}
template <typename T, bool Q4>
int launch_append(const CacheView &c, int layer, const RowIn &in, const RowList &li, const Rotation &r, int *err, cudaStream_t stream) {
    if constexpr (Q4) {
        if (r.dims == 0) return launch_turn<T, Q4, Turn::kNone>(c, layer, in, li, r, err, stream);
    }
    if (r.neighbours) return launch_turn<T, Q4, Turn::kNeighbours>(c, layer, in, li, r, err, stream);
    if constexpr (Q4) {
        if (r.dims % 32 == 16) return launch_turn<T, Q4, Turn::kHalvesApart>(c, layer, in, li, r, err, stream);
    }
    if (r.dims % 16 == 0) return launch_turn<T, Q4, Turn::kHalves>(c, layer, in, li, r, err, stream);
    return launch_turn<T, Q4, Turn::kOddHalves>(c, layer, in, li, r, err, stream);
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

int launch_cache_rows_out(const CacheView &c, int layer, RowOut out, const RowList &li, cudaStream_t stream) {
    int *err = device_error_word();
    if (!err) return kErrCuda;
    out.lane_shift = 0;
    while ((1 << out.lane_shift) < (c.bits == 4 ? out.d / 16 : c.row_vecs)) ++out.lane_shift;
    auto go = [&](auto one, auto many) {
        if (li.T <= kFewTokens) return launch_dependent(one, dim3(blocks(li.T, 1)), kRowThreads, 0, stream, c, layer, out, li, err);
        return launch_dependent(many, dim3(blocks(li.T, kReadTokens)), kRowThreads, 0, stream, c, layer, out, li, err);
    };
    return c.bits == 4 ? go(read_rows_kernel<true, 1>, read_rows_kernel<true, kReadTokens>)
                       : go(read_rows_kernel<false, 1>, read_rows_kernel<false, kReadTokens>);
}

}  // namespace eta

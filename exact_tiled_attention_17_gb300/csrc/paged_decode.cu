// Attention of a few new tokens over a paged cache, bf16 in / f32 accumulate:
// decoding, and the checking of a few drafted tokens.
//
// A unit (paged_index.h) is one kv head with up to 16 or 32 query rows:
// a few tokens times the g query heads that share the head.  The work is a
// stream over K and V, a few FLOPs to a byte, so it is bound by HBM and the
// kernel's job is to keep enough bytes in flight.  With g heads to a stream
// the CUDA cores would not keep up (g * 2 FMAs to each element read), so both
// products run on mma.sync with the rows padded to 16: at 16 rows that is
// 16 * 4 FLOPs to a key's column, a small part of what the instruction can do.
// tcgen05 would need 128-row tiles, of which these rows fill a quarter at most.
//
//   warp 4         finds the CTA's work; TMA producer: gathers tiles of 64 keys
//                  (128 at d <= 64: the same bytes), page by page, into a ring
//                  of three stages (K and V of a tile on one barrier), and the
//                  next unit's Q rows.
//   warps 0 .. 3   consumers.  S = Q K^T: warp w takes a quarter of the keys.
//                  One vote a tile whether some row's maximum exceeds its
//                  reference by 2^8; only then do the warps exchange maxima and
//                  rescale.  P goes through shared memory as bf16 (units of
//                  16 rows: as two bf16 parts, p and what rounding left over,
//                  so that O is as exact as its own rounding; under the stream
//                  the second product costs 0.3 us at most; with 32 rows the
//                  second part's buffer, 4 KB, does not fit beside another CTA's,
//                  and P is rounded once), and warp w forms O += P V for its
//                  quarter of the columns.
// Two barriers a tile among the four warps; with two CTAs on an SM one's
// arithmetic covers the other's.
//
// Missing pages and pages past the end read as zeros (an out-of-range page
// coordinate); masked scores are replaced by -inf, and V fragments of slots
// past the end, which may hold NaN, are cleared in registers.
//
// Measured: 64 sequences of 2048 .. 8191 tokens, 8 kv heads of 128, 4 query heads
// to each: 1.41 GB in 217 us, 0.97 of the measured copy rate.  4 sequences of 300
// .. 1000: 13 us, of which 3 are launches and the rest a chain of dependent reads.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "launch.cuh"
#include "paged.cuh"

namespace eta {
namespace {

constexpr float kThreshD = 8.0f;

template <int DP, int MT>   // padded head dimension, 16-row blocks of a unit
struct PdShape {
    static constexpr int CB = DP / 64;
    static constexpr int ROWS = 16 * MT;
    static constexpr int KEYS = DP == 64 ? 128 : 64;                // of a tile
    static constexpr int KV_BYTES = KEYS * DP * 2;
    static constexpr int STAGE = 2 * KV_BYTES;
    static constexpr int CTAS = 2;                                  // per SM
    static constexpr int QB = MT == 1 ? 2 : 1;                      // Q buffers
    static constexpr int NS = 3;                                    // stages: 96 KB in flight to a CTA
    static constexpr int Q_BYTES = ROWS * DP * 2;
    static constexpr int P_BYTES = ROWS * KEYS * 2;                 // [KEYS / 64][ROWS][128 bytes]
    static constexpr int PS = MT == 1 ? 2 : 1;                      // bf16 parts of a p
    static constexpr int OFF_Q = NS * STAGE;
    static constexpr int OFF_P = OFF_Q + QB * Q_BYTES;
    static constexpr int OFF_MX = OFF_P + PS * P_BYTES;                  // [4][ROWS] maxima
    static constexpr int OFF_L = OFF_MX + 4 * ROWS * 4;             // [4][ROWS] sums
    static constexpr int OFF_BAR = OFF_L + 4 * ROWS * 4;
    // a unit's words and its Q arrive on one barrier; QEMPTY: both have been read
    static constexpr int BAR_FULL = 0, BAR_EMPTY = NS, BAR_QFULL = 2 * NS, BAR_QEMPTY = BAR_QFULL + QB;
    static constexpr int OFF_MISC = OFF_BAR + ((BAR_QEMPTY + QB) * 8 + 15) / 16 * 16;
    static constexpr int OFF_BADP = OFF_MISC + 16;                  // per stage: missing pages, bit per 16 keys
    static constexpr int OFF_UNIT = OFF_BADP + ((NS * 4 + 15) / 16) * 16;   // [QB]
    static constexpr int SMEM_BYTES = OFF_UNIT + QB * static_cast<int>(sizeof(PagedUnit)) + 1024;
    static_assert(SMEM_BYTES <= 113 * 1024, "shared memory");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int DP, int MT>
__global__ void __launch_bounds__(160, PdShape<DP, MT>::CTAS)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
    using S = PdShape<DP, MT>;
    constexpr int NS = S::NS, CB = S::CB, ROWS = S::ROWS;
    constexpr int KS = DP / 16;        // K steps of Q K^T
    constexpr int NT = DP / 32;        // 8-column blocks of O to a warp
    constexpr int KEYS = S::KEYS, KW = KEYS / 4, NK = KW / 8;   // keys of a tile, of a warp, 8-key blocks of a warp
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    const PagedGeom &gm = p.gm;
    auto bar = [&](int i) -> uint32_t { return sbase + S::OFF_BAR + 8 * i; };
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + S::OFF_MISC);
    volatile uint32_t *bad_pages = reinterpret_cast<volatile uint32_t *>(smem + S::OFF_BADP);
    PagedUnit *units = reinterpret_cast<PagedUnit *>(smem + S::OFF_UNIT);
    float *mx_sh = reinterpret_cast<float *>(smem + S::OFF_MX);
    float *l_sh = reinterpret_cast<float *>(smem + S::OFF_L);
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar(S::BAR_FULL + s), 1);
            mbar_init(bar(S::BAR_EMPTY + s), 4);
        }
        for (int b = 0; b < S::QB; ++b) {
            mbar_init(bar(S::BAR_QFULL + b), 1);
            mbar_init(bar(S::BAR_QEMPTY + b), 4);
        }
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 4 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    __syncthreads();
    paged_touch(p);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == 4) {
        // ------------------------------------------------------------------
        // Producer.  Lane (kv, box, column block) issues that copy of a tile.
        // ------------------------------------------------------------------
        auto wwait = [&](uint32_t b, uint32_t parity, int site) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.err, site));
        };
        const int box_rows = min(gm.page_size, KEYS);
        const int boxes = KEYS / box_rows;
        const int my_kv = lane / (boxes * CB), my_box = lane / CB % boxes, my_cb = lane % CB;
        const bool mine = lane < 2 * boxes * CB;
        const uint32_t dst = my_kv * S::KV_BYTES + my_cb * (KEYS * 128) + my_box * box_rows * 128;
        int t = 0, u = 0;
        bool ok = true;
        PagedFeed feed;
        feed.start(p, cta, gridDim.x);
        for (;; ++u) {
            PagedUnit w;
            feed.next(p, cta, w);
            const int qb = u % S::QB;
            if (u >= S::QB && !wwait(bar(S::BAR_QEMPTY + qb), (u / S::QB - 1) & 1, 50)) ok = false;
            if (!ok) break;   // (the others' waits run out too)
            if (lane == 0) {
                units[qb] = w;
                if (w.tiles == 0) {
                    mbar_arrive(bar(S::BAR_QFULL + qb));
                } else {
                    mbar_arrive_expect_tx(bar(S::BAR_QFULL + qb), CB * 128 * gm.g * gm.tpu);
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb)
                        tma_load_3d(sbase + S::OFF_Q + qb * S::Q_BYTES + cb * (ROWS * 128), &tm_q, bar(S::BAR_QFULL + qb),
                                    cb * 64, w.head * gm.g, w.tok0);
                }
            }
            if (w.tiles == 0) break;
            feed.report(p, w);
            const int j1 = w.tile0 + w.tiles;
            auto lookup = [&](int j) -> int {   // page of this lane's box: -1 past the end, -2 missing
                const int key = j * KEYS + my_box * box_rows;
                if (!mine || key >= w.len) return -1;
                const int id = paged_page(gm, w.seq, key >> gm.page_shift);
                return id < 0 ? -2 : id;
            };
            // table entries two tiles ahead
            int next0 = lookup(w.tile0), next1 = w.tiles > 1 ? lookup(w.tile0 + 1) : -1;
            for (int j = w.tile0; j < j1; ++j, ++t) {
                const int id = next0;
                next0 = next1;
                if (j + 2 < j1) next1 = lookup(j + 2);
                const int st = t % NS;
                if (t >= NS && !wwait(bar(S::BAR_EMPTY + st), (t / NS - 1) & 1, 51)) {
                    ok = false;
                    break;
                }
                const uint32_t missing = __ballot_sync(0xffffffffu, id == -2 && my_kv == 0 && my_cb == 0);
                if (lane == 0) {
                    uint32_t bits = 0;
                    if (missing) {
                        atomicOr(p.err, kErrWordBadRow);
                        for (int b = 0; b < boxes; ++b)
                            if ((missing >> (b * CB)) & 1u) bits |= ((1u << (box_rows / 16)) - 1u) << (b * (box_rows / 16));
                    }
                    bad_pages[st] = bits;
                    mbar_arrive_expect_tx(bar(S::BAR_FULL + st), S::STAGE);
                }
                __syncwarp();
                if (mine)
                    tma_load_4d(sbase + st * S::STAGE + dst, my_kv ? &tm_v : &tm_k, bar(S::BAR_FULL + st), my_cb * 64,
                                (j * KEYS + my_box * box_rows) & (gm.page_size - 1), w.head, id < 0 ? gm.pages : id);
            }
        }
        feed.finish(p, cta);
        // every copy has landed before this warp leaves
        for (int tt = max(0, t - NS); tt < t; ++tt) wwait(bar(S::BAR_FULL + tt % NS), (tt / NS) & 1, 52);
        // (the buffer that the last words went to was free: its Q had been read)
        for (int uu = max(0, u - S::QB + 1); uu < u; ++uu) wwait(bar(S::BAR_QFULL + uu % S::QB), (uu / S::QB) & 1, 53);
        __syncwarp();
    } else {
        // ------------------------------------------------------------------
        // Consumers
        // ------------------------------------------------------------------
        const float sl2 = p.scale_log2;
        const int quad = lane >> 2, col2 = (lane & 3) * 2, mat = lane >> 3;
        const int a_row = lane & 15, a_chunk = lane >> 4;             // ldmatrix lanes of an A fragment
        const int k_row = warp * KW + (mat >> 1) * 8 + (lane & 7), k_chunk = mat & 1;
        const int v_row = (mat & 1) * 8 + (lane & 7), v_chunk = warp * (DP / 32) + (mat >> 1);
        int t = 0;
        for (int u = 0;; ++u) {
            const int qb = u % S::QB;
            // (all four warps leave together: what one reads of a unit that never
            // came, the others read too)
            const bool came = mbar_wait(bar(S::BAR_QFULL + qb), (u / S::QB) & 1, abort_flag, p.err, 54);
            if (named_bar_red_or(1, 128, !came)) break;
            const PagedUnit w = units[qb];
            if (w.tiles == 0) break;
            const uint32_t sQ = sbase + S::OFF_Q + qb * S::Q_BYTES;
            const uint32_t sP = sbase + S::OFF_P;
            auto q_frag = [&](int mt, int kk, uint32_t (&a)[4]) {
                const int r = mt * 16 + a_row;
                ldsm4(sQ + (kk >> 2) * (ROWS * 128) + r * 128 + ((((kk & 3) * 2 + a_chunk) ^ (r & 7)) << 4), a);
            };
            uint32_t qf[MT == 1 ? KS : 1][4];
            if constexpr (MT == 1) {
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) q_frag(0, kk, qf[kk]);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(S::BAR_QEMPTY + qb));   // the next Q may overwrite it
            }
            const int rows = w.ntok * gm.g, j1 = w.tile0 + w.tiles;
            int vis[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = mt * 16 + quad + 8 * i;
                    vis[mt][i] = r < rows ? paged_unit_visible(gm, w, paged_token(gm, r)) : 0;
                }
            const int vis_all = paged_unit_visible(gm, w, 0);   // what every row sees
            float m[MT][2], l[MT][2], o[MT][NT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    m[mt][i] = -INFINITY;
                    l[mt][i] = 0.f;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
            }
            for (int j = w.tile0; j < j1; ++j, ++t) {
                const int st = t % NS;
                mbar_wait(bar(S::BAR_FULL + st), (t / NS) & 1, abort_flag, p.err, 55);
                const uint32_t sK = sbase + st * S::STAGE, sV = sK + S::KV_BYTES;
                const int key0 = j * KEYS;
                float s[MT][NK][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int n = 0; n < NK; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[mt][n][e] = 0.f;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    uint32_t b[NK / 2][4];
#pragma unroll
                    for (int n2 = 0; n2 < NK / 2; ++n2)
                        ldsm4(sK + (kk >> 2) * (KEYS * 128) + (k_row + 16 * n2) * 128 +
                                  ((((kk & 3) * 2 + k_chunk) ^ (k_row & 7)) << 4), b[n2]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t a[4];
                        if constexpr (MT > 1) q_frag(mt, kk, a);
#pragma unroll
                        for (int n2 = 0; n2 < NK / 2; ++n2) {
                            if constexpr (MT == 1) {
                                mma16816(s[mt][2 * n2], qf[kk], b[n2][0], b[n2][1]);
                                mma16816(s[mt][2 * n2 + 1], qf[kk], b[n2][2], b[n2][3]);
                            } else {
                                mma16816(s[mt][2 * n2], a, b[n2][0], b[n2][1]);
                                mma16816(s[mt][2 * n2 + 1], a, b[n2][2], b[n2][3]);
                            }
                        }
                    }
                }
                // scaled and masked scores, and whether a maximum moves
                const uint32_t bad = bad_pages[st];
                const bool edge = key0 + KEYS > vis_all || bad != 0u;
                float mx[MT][2];
                bool move = false;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float v = -INFINITY;
#pragma unroll
                        for (int n = 0; n < NK; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float x = s[mt][n][2 * i + e] * sl2;
                                if (edge) {
                                    const int key = warp * KW + n * 8 + col2 + e;
                                    x = (!((bad >> (key >> 4)) & 1u) && key0 + key < vis[mt][i]) ? x : -INFINITY;
                                }
                                s[mt][n][2 * i + e] = x;
                                v = fmaxf(v, x);
                            }
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                        mx[mt][i] = v;
                        move = move || (vis[mt][i] > 0 && v > m[mt][i] + kThreshD);
                    }
                if (named_bar_red_or(1, 128, move)) {
                    if ((lane & 3) == 0) {
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int i = 0; i < 2; ++i) mx_sh[warp * ROWS + mt * 16 + quad + 8 * i] = mx[mt][i];
                    }
                    named_bar_sync(1, 128);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float *at = mx_sh + mt * 16 + quad + 8 * i;
                            const float v = fmaxf(fmaxf(at[0], at[ROWS]), fmaxf(at[2 * ROWS], at[3 * ROWS]));
                            if (vis[mt][i] > 0 && v > m[mt][i] + kThreshD) {
                                const float a = m[mt][i] == -INFINITY ? 0.f : ex2(m[mt][i] - v);
                                m[mt][i] = v;
                                l[mt][i] *= a;
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    o[mt][n][2 * i] *= a;
                                    o[mt][n][2 * i + 1] *= a;
                                }
                            }
                        }
                }
                // P
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float mu = m[mt][i] == -INFINITY ? 0.f : m[mt][i];
                        const int r = mt * 16 + quad + 8 * i;
#pragma unroll
                        for (int n = 0; n < NK; ++n) {
                            const float p0 = ex2(s[mt][n][2 * i] - mu), p1 = ex2(s[mt][n][2 * i + 1] - mu);
                            l[mt][i] += p0 + p1;
                            const int chunk = warp * NK + n;
                            const uint32_t at = sP + (chunk >> 3) * (ROWS * 128) + r * 128 + (((chunk & 7) ^ (r & 7)) << 4) + col2 * 2;
                            const uint32_t hi = pack_bf16x2(p0, p1);
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(hi) : "memory");
                            if constexpr (S::PS == 2) {
                                const uint32_t lo = pack_bf16x2(p0 - bf16lo_to_f32(hi), p1 - bf16hi_to_f32(hi));
                                asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + S::P_BYTES), "r"(lo) : "memory");
                            }
                        }
                    }
                named_bar_sync(1, 128);
                // O += P V, this warp's columns
                const int live = w.len - key0;   // slots of the tile that hold tokens
#pragma unroll
                for (int ks = 0; ks < KEYS / 16; ++ks) {
                    uint32_t vf[NT / 2][4];
#pragma unroll
                    for (int n2 = 0; n2 < NT / 2; ++n2) {
                        const int key = ks * 16 + v_row, chunk = v_chunk + 2 * n2;
                        ldsm4t(sV + (chunk >> 3) * (KEYS * 128) + key * 128 + (((chunk & 7) ^ (key & 7)) << 4), vf[n2]);
                        if (live < KEYS) {
                            // clear what lies past the end
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int k0 = ks * 16 + (e & 1) * 8 + col2;
                                if (k0 >= live) vf[n2][e] = 0u;
                                else if (k0 + 1 >= live) vf[n2][e] &= 0xFFFFu;
                            }
                        }
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t a[4];
                        const int r = mt * 16 + a_row;
                        const uint32_t at = sP + (ks >> 2) * (ROWS * 128) + r * 128 + ((((ks & 3) * 2 + a_chunk) ^ (r & 7)) << 4);
                        ldsm4(at, a);
#pragma unroll
                        for (int n2 = 0; n2 < NT / 2; ++n2) {
                            mma16816(o[mt][2 * n2], a, vf[n2][0], vf[n2][1]);
                            mma16816(o[mt][2 * n2 + 1], a, vf[n2][2], vf[n2][3]);
                        }
                        if constexpr (S::PS == 2) {
                            ldsm4(at + S::P_BYTES, a);
#pragma unroll
                            for (int n2 = 0; n2 < NT / 2; ++n2) {
                                mma16816(o[mt][2 * n2], a, vf[n2][0], vf[n2][1]);
                                mma16816(o[mt][2 * n2 + 1], a, vf[n2][2], vf[n2][3]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(S::BAR_EMPTY + st));
            }
            if constexpr (MT > 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(S::BAR_QEMPTY + qb));
            }
            // ---------------- the unit's end ----------------
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    l[mt][i] += __shfl_xor_sync(0xffffffffu, l[mt][i], 1);
                    l[mt][i] += __shfl_xor_sync(0xffffffffu, l[mt][i], 2);
                    if ((lane & 3) == 0) l_sh[warp * ROWS + mt * 16 + quad + 8 * i] = l[mt][i];
                }
            named_bar_sync(1, 128);
            const bool whole = w.slot < 0;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = mt * 16 + quad + 8 * i;
                    if (r >= rows || *abort_flag) continue;
                    const float *at = l_sh + r;
                    const float L = (at[0] + at[ROWS]) + (at[2 * ROWS] + at[3 * ROWS]);
                    const int tr = paged_token(gm, r);
                    const long long tok = w.tok0 + tr;
                    const int head = w.head * gm.g + r - tr * gm.g;
                    const float inv = L != 0.f ? 1.f / L : 0.f;   // (a NaN goes on)
                    const size_t prow = static_cast<size_t>(whole ? 0 : w.slot) * p.part_rows + r;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int c = warp * (DP / 4) + n * 8 + col2;
                        if (c >= p.d) continue;
                        if (whole) {
                            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.O) + tok * p.o_token +
                                                 static_cast<long long>(head) * p.o_head + c;
                            *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(o[mt][n][2 * i] * inv, o[mt][n][2 * i + 1] * inv);
                        } else {
                            *reinterpret_cast<float2 *>(p.part_o + prow * p.d + c) = make_float2(o[mt][n][2 * i], o[mt][n][2 * i + 1]);
                        }
                    }
                    if (warp == 0 && (lane & 3) == 0) {
                        if (!whole) {
                            p.part_m[prow] = paged_part_max(m[mt][i], L);
                            p.part_l[prow] = L;
                        } else if (p.LSE) {
                            p.LSE[tok * p.Hq + head] = L != 0.f ? (m[mt][i] + log2f(L)) * kPagedLn2 : -INFINITY;
                        }
                    }
                }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

constexpr int kMaxDev = 64;
std::mutex g_mu;

template <int DP, int MT>
int launch_one(PagedParams &p, void *workspace, cudaStream_t stream) {
    using S = PdShape<DP, MT>;
    auto kern = paged_decode_kernel<DP, MT>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return kErrCuda;
    static std::atomic<int> grids[kMaxDev];   // CTAs that are resident at once; 0: not set up yet
    int grid = grids[dev].load(std::memory_order_acquire);
    if (grid == 0) {
        std::lock_guard<std::mutex> lk(g_mu);
        int nsm = 0, per = 0;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM_BYTES) != cudaSuccess ||
            cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, 160, S::SMEM_BYTES) != cudaSuccess)
            return kErrCuda;
        grid = std::min(nsm * std::max(per, 1), kPagedMaxDecodeCtas);
        grids[dev].store(grid, std::memory_order_release);
    }
    const PagedGeom &gm = p.gm;
    p.gm.tpu = S::ROWS / gm.g;
    p.gm.tk = S::KEYS;
    p.gm.unit_cost = S::KEYS;
    p.gm.min_share = 128;
    paged_derive(p.gm);
    CUtensorMap tq, tk, tv;
    if (!paged_maps(p, S::ROWS / gm.g, std::min(gm.page_size, S::KEYS), &tq, &tk, &tv)) return kErrCuda;
    paged_carve(p, workspace, grid, S::ROWS);
    const int rc = launch_dependent(kern, dim3(static_cast<unsigned>(grid)), 160, S::SMEM_BYTES, stream, tq, tk, tv, p);
    if (rc != kOk) return rc;
    return launch_paged_merge(p, 1, grid, grid / S::CTAS, stream);
}

}  // namespace

int launch_paged_decode(PagedParams p, void *workspace, cudaStream_t stream) {
    if (paged_decode_rows(p.gm.g, p.gm.max_q) == 16)
        return p.d <= 64 ? launch_one<64, 1>(p, workspace, stream) : launch_one<128, 1>(p, workspace, stream);
    return p.d <= 64 ? launch_one<64, 2>(p, workspace, stream) : launch_one<128, 2>(p, workspace, stream);
}

}  // namespace eta

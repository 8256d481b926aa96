// Attention of a chunk of new tokens over a paged cache, bf16 in / f32
// accumulate, on the tcgen05 tensor cores of sm_103a.
//
// What it computes: O = softmax(scale Q K^T) V and the row's LSE for the units
// of paged_index.h: one kv head, a block of new tokens, all g query heads that
// share the head.  A unit's rows are packed (token, head of the group) into
// two 128-row query tiles of 128 / g tokens each, so K and V are streamed once
// for the whole group and short chunks still fill the matrix instructions.
//
// Mapping, as in the contiguous forward: one persistent CTA per SM,
//   warps 0 .. 15  softmax: two warpgroups per query tile, each with half of
//                  the tile's 64-key halves of S and of O's columns, one
//                  thread per row; running maximum m (moved only when a tile
//                  exceeds it by 2^8, so O is rescaled rarely) and float32
//                  sum l of the unrounded p; P as bf16 over S in tensor memory
//                  (the instruction takes 16-bit operands next to a bf16 V; a
//                  second part, what the rounding left over, would add half to
//                  the products of a kernel whose tensor pipe is 60 % busy; a
//                  weight is off by 2^-8 of itself at most, the sum l is not).
//   warp 16        finds the CTA's work and announces it unit by unit; TMA
//                  producer of the Q tiles and of K_j.
//   warp 17        MMA issuer: S_q = Q_q K_j^T, O_q += P_q V_j.
//   warp 18        TMA producer of V_j.  (K_j and V_j share a ring of slots.  A
//                  tile is gathered page by page, one box of min(page, 128) rows
//                  by 64 columns per copy; at 16 tokens a page that is 32 copies
//                  a tile, which one warp issues too slowly.)
// The work of all units is cut into equal shares, one to a CTA, which may
// begin and end inside a unit; cut units are joined by the merge kernel.
//
// Pages that do not exist, and whole pages past the end, are copied from an
// out-of-range page coordinate, which fills zeros.  Slots past the end inside
// the last page may hold anything: the producer waits for that V tile itself
// and zeroes them before it hands the tile on (a masked p = 0 times NaN would
// be NaN); masked scores are replaced, never added to.
//
// Bound by the softmax and the products together (tensor pipe 60 % active): a
// step of 128 keys for both query tiles takes 1.5 us at d = 128, a unit about 5
// us more.  Measured: four chunks of 511 .. 1024 tokens over 4000 .. 8192 cached
// ones, 32 query heads of 128 on 8 kv heads: 346 GFLOP in 255 us, 1.36 PFLOP/s; 128
// tokens over 130907, 16 query heads of 64 on 4: 92 us.
#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "launch.cuh"
#include "paged.cuh"

namespace eta {
namespace {

constexpr float kThresh = 8.0f;   // the reference maximum moves by at least this (log2 units)
constexpr float kNegInfP = -__builtin_huge_valf();

template <int DP>   // padded head dimension: 64 or 128
struct PtcShape {
    static constexpr int NQ = 2, BR = 128, BC = 128;
    static constexpr int CB = DP / 64;
    static constexpr int Q_BYTES = BR * DP * 2;
    static constexpr int SLOT_BYTES = BC * DP * 2;
    static constexpr int XCH_BYTES = NQ * 2 * 128 * 8;
    static constexpr int NS_RAW = (222 * 1024 - NQ * Q_BYTES - XCH_BYTES) / SLOT_BYTES;
    static constexpr int NS = NS_RAW > 8 ? 8 : NS_RAW;
    static constexpr int SOFTMAX_WARPS = 16, WARP_MMA = 17, WARP_TMV = 18;   // (warp 16: Q, K and the work)
    static constexpr int THREADS = 19 * 32;
    static constexpr int OFF_RING = NQ * Q_BYTES;
    static constexpr int OFF_XCH = OFF_RING + NS * SLOT_BYTES;
    static constexpr int OFF_BAR = OFF_XCH + XCH_BYTES;
    static constexpr int BAR_QFULL = 0;
    static constexpr int BAR_FULL = BAR_QFULL + NQ;
    static constexpr int BAR_EMPTY = BAR_FULL + NS;
    static constexpr int BAR_SFULL = BAR_EMPTY + NS;
    static constexpr int BAR_PFULL = BAR_SFULL + NQ;
    static constexpr int BAR_OFULL = BAR_PFULL + NQ;
    static constexpr int BAR_QFREE = BAR_OFULL + NQ;
    static constexpr int BAR_OFREE = BAR_QFREE + NQ;
    static constexpr int BAR_DONE = BAR_OFREE + NQ;
    static constexpr int BAR_TAIL = BAR_DONE + 1;
    static constexpr int UB = 4;                                  // units announced ahead
    static constexpr int BAR_UFULL = BAR_TAIL + 1;
    static constexpr int BAR_UEMPTY = BAR_UFULL + UB;
    static constexpr int NBARS = (BAR_UEMPTY + UB + 1) / 2 * 2;
    static constexpr int OFF_MISC = OFF_BAR + NBARS * 8;          // tensor-memory address, abort flag
    static constexpr int OFF_BADP = OFF_MISC + 16;                // per K tile (mod 8): missing pages, bit per 16 keys
    static constexpr int OFF_UNIT = OFF_BADP + 32;                // [UB]
    static constexpr int SMEM_MIN = OFF_UNIT + UB * static_cast<int>(sizeof(PagedUnit)) + 1024;
    // (all of tensor memory is allocated: a second resident CTA would wait for it)
    static constexpr int SMEM_BYTES = SMEM_MIN <= 116 * 1024 ? 117 * 1024 : SMEM_MIN;
    __host__ __device__ static constexpr int s_col(int q) { return q * BC; }
    __host__ __device__ static constexpr int o_col(int q) { return NQ * BC + q * DP; }
    static_assert(NS >= 4 && SMEM_BYTES <= 227 * 1024, "shared memory");
    static_assert(NQ * (BC + DP) <= 512, "tensor memory");
    static_assert(OFF_UNIT % 16 == 0, "alignment");
};

// N words to 16-byte aligned memory, 32 bytes at a time where that is aligned.
template <int N>
__device__ __forceinline__ void store_words(void *dst, const uint32_t *r) {
    if ((reinterpret_cast<uintptr_t>(dst) & 31u) == 0) {
#pragma unroll
        for (int k = 0; k < N; k += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<uint32_t *>(dst) + k),
                         "r"(r[k]), "r"(r[k + 1]), "r"(r[k + 2]), "r"(r[k + 3]), "r"(r[k + 4]), "r"(r[k + 5]), "r"(r[k + 6]),
                         "r"(r[k + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int k = 0; k < N; k += 4)
            asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(static_cast<uint32_t *>(dst) + k), "r"(r[k]),
                         "r"(r[k + 1]), "r"(r[k + 2]), "r"(r[k + 3])
                         : "memory");
    }
}

template <int DP>
__global__ void __launch_bounds__(PtcShape<DP>::THREADS, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
    using S = PtcShape<DP>;
    constexpr int NQ = S::NQ, BC = S::BC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    const PagedGeom &gm = p.gm;
    auto bar = [&](int i) -> uint32_t { return sbase + S::OFF_BAR + 8 * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::OFF_MISC);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + S::OFF_MISC + 4);
    volatile uint32_t *bad_pages = reinterpret_cast<volatile uint32_t *>(smem + S::OFF_BADP);
    PagedUnit *units = reinterpret_cast<PagedUnit *>(smem + S::OFF_UNIT);
    const uint32_t sQ = sbase, sRing = sbase + S::OFF_RING;

    if (threadIdx.x == 0) {
        for (int q = 0; q < NQ; ++q) {
            mbar_init(bar(S::BAR_QFULL + q), 1);
            mbar_init(bar(S::BAR_SFULL + q), 1);
            mbar_init(bar(S::BAR_PFULL + q), 256);
            mbar_init(bar(S::BAR_OFULL + q), 1);
            mbar_init(bar(S::BAR_QFREE + q), 1);
            mbar_init(bar(S::BAR_OFREE + q), 256);
        }
        for (int s = 0; s < S::NS; ++s) {
            mbar_init(bar(S::BAR_FULL + s), 1);
            mbar_init(bar(S::BAR_EMPTY + s), 1);
        }
        mbar_init(bar(S::BAR_DONE), 1);
        mbar_init(bar(S::BAR_TAIL), 1);
        for (int u = 0; u < S::UB; ++u) {
            mbar_init(bar(S::BAR_UFULL + u), 1);
            mbar_init(bar(S::BAR_UEMPTY + u), S::SOFTMAX_WARPS + 2);
        }
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == S::WARP_MMA) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    paged_touch(p);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int tpt = 128 / gm.g;   // tokens to a query tile
    // Unit u has been announced by the producer.
    auto unit_wait = [&](int u, int site) -> bool {
        return mbar_wait(bar(S::BAR_UFULL + u % S::UB), (u / S::UB) & 1, abort_flag, p.err, site);
    };
    auto unit_done = [&](int u) {   // one lane of each warp, when the warp has read the last of it
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::BAR_UEMPTY + u % S::UB));
    };

    if (warp >= S::SOFTMAX_WARPS) {
        auto wwait = [&](uint32_t b, uint32_t parity, int site) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.err, site));
        };
        const bool leader = elect_one();
        if (warp != S::WARP_MMA) {
            // --------------------------------------------------------------
            // TMA producers.  Lane b * CB + c copies box b (box_rows keys),
            // column block c, of a tile; tile i of K is the ring's tile 2 i, of V
            // 2 i + 1.
            // --------------------------------------------------------------
            const bool is_v = warp == S::WARP_TMV;
            const CUtensorMap *tm = is_v ? &tm_v : &tm_k;
            if (leader) {
                if (!is_v) tma_prefetch_desc(&tm_q);
                tma_prefetch_desc(tm);
            }
            const int box_rows = min(gm.page_size, BC);
            const int boxes = BC / box_rows;
            const int my_box = lane / S::CB, my_cb = lane % S::CB;
            const bool mine = my_box < boxes;
            const uint32_t dst = my_cb * (BC * 128) + my_box * box_rows * 128;
            const uint64_t pol_q = l2_policy_evict_first();
            int kt = 0, tails = 0;       // K (or V) tiles issued so far
            int uo[NQ] = {0, 0};
            bool ok = true;
            PagedFeed feed;
            if (!is_v) feed.start(p, cta, gridDim.x);
            for (int u = 0; ok; ++u) {
                PagedUnit w;
                if (is_v) {
                    if (!__all_sync(0xffffffffu, unit_wait(u, 18))) break;
                    w = units[u % S::UB];
                    unit_done(u);
                    if (w.tiles == 0) break;
                } else {
                    feed.next(p, cta, w);
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        const int t1 = min(w.ntok, (q + 1) * tpt);
                        const int keys = paged_unit_visible(gm, w, t1 - 1);
                        const int tiles = keys <= BC ? 1 : (keys - 1) / BC + 1;
                        w.own[q] = t1 > q * tpt ? max(0, min(tiles - w.tile0, w.tiles)) : 0;
                        w.inner[q] = paged_unit_visible(gm, w, q * tpt) / BC - w.tile0;
                    }
                    if (u >= S::UB && !wwait(bar(S::BAR_UEMPTY + u % S::UB), (u / S::UB - 1) & 1, 7)) break;
                    if (lane == 0) {
                        units[u % S::UB] = w;
                        mbar_arrive(bar(S::BAR_UFULL + u % S::UB));
                    }
                    if (w.tiles == 0) break;
                    feed.report(p, w);
                }
                // page of box my_box of tile j: -1 past the end (no keys), -2 missing;
                // looked up four tiles ahead, since a read takes about as long as a
                // tile's matrix products
                const int j0 = w.tile0, j1 = w.tile0 + w.tiles;
                auto lookup = [&](int j) -> int {
                    const int key = j * BC + my_box * box_rows;
                    if (j >= j1 || !mine || key >= w.len) return -1;
                    const int id = paged_page(gm, w.seq, key >> gm.page_shift);
                    return id < 0 ? -2 : id;
                };
                int n0 = lookup(j0), n1 = lookup(j0 + 1), n2 = lookup(j0 + 2), n3 = lookup(j0 + 3);
                if (!is_v) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        if (w.own[q] == 0) continue;
                        if (uo[q] > 0 && !wwait(bar(S::BAR_QFREE + q), (uo[q] - 1) & 1, 4)) ok = false;
                        if (ok && leader) {
                            mbar_arrive_expect_tx(bar(S::BAR_QFULL + q), S::CB * 128 * gm.g * tpt);
#pragma unroll
                            for (int cb = 0; cb < S::CB; ++cb)
                                tma_load_3d_hint(sQ + q * S::Q_BYTES + cb * (S::BR * 128), &tm_q, bar(S::BAR_QFULL + q),
                                                 cb * 64, w.head * gm.g, w.tok0 + q * tpt, pol_q);
                        }
                        ++uo[q];
                    }
                }
                for (int j = j0; ok && j < j1; ++j, ++kt) {
                    const int id = n0;
                    n0 = n1;
                    n1 = n2;
                    n2 = n3;
                    n3 = lookup(j + 4);
                    const int t = 2 * kt + (is_v ? 1 : 0), slot = t % S::NS, round = t / S::NS;
                    if (round > 0 && !wwait(bar(S::BAR_EMPTY + slot), (round - 1) & 1, is_v ? 19 : 1)) {
                        ok = false;
                        break;
                    }
                    // rows of V to clear: past the end, in a page that was copied
                    const int clear0 = w.len - j * BC;
                    const int clear1 = min(BC, (clear0 + box_rows - 1) / box_rows * box_rows);
                    const bool tail = is_v && clear0 > 0 && clear0 < BC && clear1 > clear0;
                    const uint32_t full = bar(tail ? S::BAR_TAIL : S::BAR_FULL + slot);
                    const uint32_t missing = __ballot_sync(0xffffffffu, id == -2 && my_cb == 0);
                    if (leader) {
                        if (!is_v) {
                            // one bit for each 16 keys
                            uint32_t bits = 0;
                            if (missing) {
                                atomicOr(p.err, kErrWordBadRow);
                                for (int b = 0; b < boxes; ++b)
                                    if ((missing >> (b * S::CB)) & 1u)
                                        bits |= ((1u << (box_rows / 16)) - 1u) << (b * (box_rows / 16));
                            }
                            bad_pages[kt & 7] = bits;
                        }
                        mbar_arrive_expect_tx(full, S::SLOT_BYTES);
                    }
                    __syncwarp();
                    if (mine)   // (an out-of-range page: zeros)
                        tma_load_4d(sRing + slot * S::SLOT_BYTES + dst, tm, full, my_cb * 64,
                                    (j * BC + my_box * box_rows) & (gm.page_size - 1), w.head, id < 0 ? gm.pages : id);
                    if (tail) {
                        if (!wwait(bar(S::BAR_TAIL), tails & 1, 6)) ok = false;
                        ++tails;
                        // 128-byte rows (the swizzle stays inside a row)
                        for (int i = lane; i < (clear1 - clear0) * 8 * S::CB; i += 32) {
                            const int c = i / ((clear1 - clear0) * 8), r = i % ((clear1 - clear0) * 8);
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             sRing + slot * S::SLOT_BYTES + c * (BC * 128) + clear0 * 128 + r * 16),
                                         "r"(0u)
                                         : "memory");
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (leader) mbar_arrive(bar(S::BAR_FULL + slot));
                    }
                }
            }
            if (!is_v) feed.finish(p, cta);
            // every copy this warp started has landed before the CTA may exit
            for (int i = max(0, kt - (S::NS + 1) / 2); i < kt; ++i) {
                const int t = 2 * i + (is_v ? 1 : 0);
                if (t + S::NS >= 2 * kt) wwait(bar(S::BAR_FULL + t % S::NS), (t / S::NS) & 1, 2);
            }
            if (!is_v) {
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                    if (uo[q] > 0) wwait(bar(S::BAR_QFULL + q), (uo[q] - 1) & 1, 3);
            }
            __syncwarp();
        } else {
            // --------------------------------------------------------------
            // MMA issuer (one elected lane); the order of the contiguous
            // forward: P_0 V_j, S_0(j+1), P_1 V_j, S_1(j+1).
            // --------------------------------------------------------------
            constexpr uint32_t idesc_s = idesc_bf16_f32(128, BC, false, false);
            constexpr uint32_t idesc_o = idesc_bf16_f32(128, DP, false, true);
            const uint64_t qdesc0 = sdesc_sw128(sQ, 16, 1024);
            const uint64_t kdesc0 = sdesc_sw128(sRing, 16, 1024);
            const uint64_t vdesc0 = sdesc_sw128(sRing, BC * 128, 1024);
            const int ksteps = p.d / 16;
            int t_base = 0;
            int sq[NQ] = {0, 0}, uo[NQ] = {0, 0};
            auto commit = [&](int b) {
                if (leader) tc_commit(bar(b));
            };
            bool ok = true;
            for (int u = 0; ok; ++u) {
                if (!__all_sync(0xffffffffu, unit_wait(u, 8))) break;
                const PagedUnit *w = units + u % S::UB;
                if (w->tiles == 0) break;
                int nkv[NQ];
#pragma unroll
                for (int q = 0; q < NQ; ++q) nkv[q] = w->own[q];
                const int nkv_max = w->tiles;
                unit_done(u);
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                    if (ok && nkv[q] > 0) ok = wwait(bar(S::BAR_QFULL + q), uo[q] & 1, 10);
                if (!ok) break;
                auto full_wait = [&](int tt, int site) -> bool {
                    const int tg = t_base + tt;
                    if (!wwait(bar(S::BAR_FULL + tg % S::NS), (tg / S::NS) & 1, site)) return false;
                    tc_fence_after();
                    return true;
                };
                auto slot_of = [&](int tt) { return S::BAR_EMPTY + (t_base + tt) % S::NS; };
                auto issue_s = [&](int q, int j, int nkvq) {
                    const uint64_t a0 = qdesc0 + static_cast<uint64_t>((q * S::Q_BYTES) >> 4);
                    const uint64_t b0 = kdesc0 + static_cast<uint64_t>((((t_base + 2 * j) % S::NS) * S::SLOT_BYTES) >> 4);
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < DP / 16; ++kk) {
                            if (kk >= ksteps) break;
                            const int cb = kk >> 2, off = (kk & 3) * 32;
                            mma_bf16_ss(tmem + S::s_col(q), a0 + static_cast<uint64_t>((cb * (S::BR * 128) + off) >> 4),
                                        b0 + static_cast<uint64_t>((cb * (BC * 128) + off) >> 4), idesc_s, kk > 0 ? 1u : 0u);
                        }
                        tc_commit(bar(S::BAR_SFULL + q));
                    }
                    if (j == nkvq - 1) commit(S::BAR_QFREE + q);
                };
                auto issue_pv = [&](int q, int j) {
                    const uint64_t b0 = vdesc0 + static_cast<uint64_t>((((t_base + 2 * j + 1) % S::NS) * S::SLOT_BYTES) >> 4);
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < BC / 16; ++kk)
                            mma_bf16_ts(tmem + S::o_col(q), tmem + S::s_col(q) + (kk / 4) * 64 + (kk % 4) * 8,
                                        b0 + static_cast<uint64_t>((kk * 2048) >> 4), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
                    }
                };
                auto wait_p = [&](int q, int j) -> bool {
                    if (j == 0 && u > 0 && !wwait(bar(S::BAR_OFREE + q), (u - 1) & 1, 16)) return false;
                    if (!wwait(bar(S::BAR_PFULL + q), (sq[q] + j) & 1, 13)) return false;
                    tc_fence_after();
                    return true;
                };
                ok = full_wait(0, 11);
                if (ok) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
                        if (nkv[q] > 0) issue_s(q, 0, nkv[q]);
                    commit(slot_of(0));
                }
                for (int j = 0; ok && j < nkv_max; ++j) {
                    if (!full_wait(2 * j + 1, 12)) {
                        ok = false;
                        break;
                    }
                    bool k_ready = false;
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        if (!ok || j >= nkv[q]) continue;
                        if (wait_p(q, j)) issue_pv(q, j);
                        else ok = false;
                        if (!ok) continue;
                        if (j == nkv[q] - 1) commit(S::BAR_OFULL + q);
                        if (j + 1 < nkv[q]) {
                            if (!k_ready) {
                                if (!full_wait(2 * j + 2, 14)) {
                                    ok = false;
                                    continue;
                                }
                                k_ready = true;
                            }
                            issue_s(q, j + 1, nkv[q]);
                        }
                    }
                    commit(slot_of(2 * j + 1));
                    if (k_ready) commit(slot_of(2 * j + 2));
                }
                t_base += 2 * nkv_max;
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    if (ok && nkv[q] == 0) {
                        // nothing for this tile: O is free and "full" at once
                        if (u > 0) ok = wwait(bar(S::BAR_OFREE + q), (u - 1) & 1, 17);
                        if (ok) commit(S::BAR_OFULL + q);
                    }
                    sq[q] += nkv[q];
                    uo[q] += nkv[q] > 0 ? 1 : 0;
                }
            }
            commit(S::BAR_DONE);
            wwait(bar(S::BAR_DONE), 0, 15);
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------------
        // Softmax warpgroup h of query tile q.
        // ------------------------------------------------------------------
        const int q = warp >> 3, h = (warp >> 2) & 1, wq = warp & 3;
        const int row_in = wq * 32 + lane;
        const uint32_t t_lane = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tS = tmem + t_lane + S::s_col(q);
        const uint32_t tO = tmem + t_lane + S::o_col(q);
        const float sl2 = p.scale_log2;
        constexpr int OC = DP / 64;   // 32-column chunks of O of this warpgroup
        // this row's token within the unit, or one that no unit has (g need not divide 128)
        auto token_in = [&]() { return row_in < tpt * gm.g ? q * tpt + paged_token(gm, row_in) : 256; };
        auto xch = [&](int hh) -> uint32_t { return sbase + S::OFF_XCH + ((q * 2 + hh) * 128 + row_in) * 8; };
        auto pair_sync = [&]() { named_bar_sync(7 + q, 256); };
        auto exchange = [&](float a, float &ao) {
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(xch(h)), "f"(a) : "memory");
            pair_sync();
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ao) : "r"(xch(1 - h)) : "memory");
        };
        int sq = 0, kt = 0;
        bool ok = true;
        for (int u = 0;; ++u) {
            // (the tile's two warpgroups leave together, whichever wait gave up)
            if (named_bar_red_or(7 + q, 256, !unit_wait(u, 9))) break;
            const PagedUnit *w = units + u % S::UB;
            if (w->tiles == 0) break;
            const int nkvq = w->own[q], inner = w->inner[q];
            // (a row that is none has a reference that no maximum exceeds)
            float m = token_in() < w->ntok ? kNegInfP : -kNegInfP, l = 0.f;
            // (a wait that gives up is recorded and does not end the loop: every
            // warp still takes part in every named barrier)
            for (int j = 0; j < nkvq; ++j) {
                if (!mbar_wait(bar(S::BAR_SFULL + q), (sq + j) & 1, abort_flag, p.err, 20)) ok = false;
                tc_fence_after();
                const bool edge = j >= inner || bad_pages[(kt + j) & 7] != 0u;
                uint32_t sr[2][32];
                float mxc[2], mx = kNegInfP;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (edge) tmem_ld32(tS + h * 64 + 32 * c, sr[c]);
                    else tmem_ld32_max(tS + h * 64 + 32 * c, sr[c], mxc[c]);
                }
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    reg_fence32(sr[c]);
                    if (!edge) {
                        reg_fence_f32(mxc[c]);
                        mx = fmaxf(mx, mxc[c]);
                    } else {
                        // (read again rather than kept: edge tiles are few, registers fewer)
                        const PagedUnit *w = units + u % S::UB;
                        const int vis = paged_unit_visible(gm, *w, token_in()) - (w->tile0 + j) * BC - h * 64 - 32 * c;
                        // bits of this chunk's two 16-key groups
                        const uint32_t b2 = (bad_pages[(kt + j) & 7] >> (4 * h + 2 * c)) & 3u;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float x = __uint_as_float(sr[c][e]) * sl2;
                            x = (e < vis && !((b2 >> (e >> 4)) & 1u)) ? x : kNegInfP;
                            sr[c][e] = __float_as_uint(x);
                            mx = fmaxf(mx, x);
                        }
                    }
                }
                if (!edge) mx *= sl2;
                if (named_bar_red_or(7 + q, 256, mx > m + kThresh)) {
                    float mo;
                    exchange(mx, mo);
                    mx = fmaxf(mx, mo);
                } else {
                    mx = m;
                }
                const float m_new = mx > m + kThresh ? mx : m;
                const bool moved = m_new != m;
                const float a = moved ? ex2(m - m_new) : 1.f;
                m = m_new;
                const float m_use = (m == kNegInfP) ? 0.f : m;
                const uint64_t negm2 = f2_pack(-m_use, -m_use);
                uint64_t ls2 = f2_pack(0.f, 0.f);
                auto exps = [&](auto edge_c) {
                    constexpr bool EDGE = decltype(edge_c)::value;
                    const uint64_t sl2x2 = f2_pack(sl2, sl2);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const uint64_t xx = f2_pack(__uint_as_float(sr[c][2 * e]), __uint_as_float(sr[c][2 * e + 1]));
                            uint64_t y;
                            if constexpr (EDGE) y = f2_add(xx, negm2);
                            else y = f2_fma(xx, sl2x2, negm2);
                            float y0, y1;
                            f2_unpack(y, y0, y1);
                            const float p0 = ex2(y0), p1 = ex2(y1);
                            pk[e] = pack_bf16x2(p0, p1);
                            ls2 = f2_add(ls2, f2_pack(p0, p1));
                        }
                        tmem_st16(tS + h * 64 + 16 * c, pk);
                    }
                };
                if (edge) exps(std::true_type{});
                else exps(std::false_type{});
                if (j > 0 && __any_sync(0xffffffffu, moved)) {
                    const uint64_t a2 = f2_pack(a, a);
#pragma unroll
                    for (int c = h * OC; c < (h + 1) * OC; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32 * c, o);
                        tmem_ld_wait();
                        reg_fence32(o);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float v0, v1;
                            f2_unpack(f2_mul(f2_pack(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), a2), v0, v1);
                            o[e] = __float_as_uint(v0);
                            o[e + 1] = __float_as_uint(v1);
                        }
                        tmem_st32(tO + 32 * c, o);
                    }
                }
                float l0, l1;
                f2_unpack(ls2, l0, l1);
                l = l * a + (l0 + l1);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bar(S::BAR_PFULL + q));
            }
            // ---------------- epilogue ----------------
            float lo;
            pair_sync();
            exchange(l, lo);
            l += lo;
            pair_sync();
            if (ok) ok = mbar_wait(bar(S::BAR_OFULL + q), u & 1, abort_flag, p.err, 21);
            tc_fence_after();
            const int tok_in = token_in(), head_in = row_in - paged_token(gm, row_in) * gm.g;
            const bool whole = w->slot < 0, valid = tok_in < w->ntok;
            const bool store = valid && !*abort_flag;
            const bool any = l != 0.f;   // (a NaN goes on)
            const float scale_o = whole ? (any ? 1.f / l : 0.f) : 1.f;
            const uint64_t inv2 = f2_pack(scale_o, scale_o);
            const int unit_row = q * tpt * gm.g + row_in;
            const size_t prow = static_cast<size_t>(whole ? 0 : w->slot) * p.part_rows + unit_row;
            const long long tok = w->tok0 + tok_in;
            const int head = w->head * gm.g + head_in;
            kt += w->tiles;
            unit_done(u);
            if (nkvq > 0) {
                const long long at = valid ? tok * p.o_token + static_cast<long long>(head) * p.o_head : 0;
#pragma unroll
                for (int c = h * OC; c < (h + 1) * OC; ++c) {
                    uint32_t o[32];
                    tmem_ld32(tO + 32 * c, o);
                    tmem_ld_wait();
                    reg_fence32(o);
                    if (!store || 32 * c >= p.d) continue;
                    // whole 32-byte sectors where alignment allows
                    if (whole) {
                        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.O) + at + 32 * c;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float v0, v1;
                            f2_unpack(f2_mul(f2_pack(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), inv2), v0, v1);
                            o[e] = any ? pack_bf16x2(v0, v1) : 0u;
                        }
                        store_words<16>(dst, o);
                    } else {
                        store_words<32>(p.part_o + prow * p.d + 32 * c, o);
                    }
                }
            }
            if (h == 0 && store) {
                if (whole) {
                    if (p.LSE) p.LSE[tok * p.Hq + head] = any ? (m + log2f(l)) * kPagedLn2 : kNegInfP;
                } else {
                    p.part_m[prow] = nkvq > 0 ? paged_part_max(m, l) : kNegInfP;
                    p.part_l[prow] = l;
                }
            }
            tc_fence_before();
            mbar_arrive(bar(S::BAR_OFREE + q));
            sq += nkvq;
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    if (warp == S::WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

constexpr int kMaxDev = 64;
std::mutex g_mu;

template <int DP>
int launch_dp(PagedParams &p, void *workspace, cudaStream_t stream) {
    using S = PtcShape<DP>;
    auto kern = paged_tc_kernel<DP>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return kErrCuda;
    static std::atomic<int> sms[kMaxDev];   // 0: not set up yet
    int nsm = sms[dev].load(std::memory_order_acquire);
    if (nsm == 0) {
        std::lock_guard<std::mutex> lk(g_mu);
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM_BYTES) != cudaSuccess ||
            cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return kErrCuda;
        sms[dev].store(nsm, std::memory_order_release);
    }
    const PagedGeom &gm = p.gm;
    const int tpt = 128 / gm.g;
    CUtensorMap tq, tk, tv;
    if (!paged_maps(p, tpt, std::min(gm.page_size, S::BC), &tq, &tk, &tv)) return kErrCuda;
    const int ctas = std::min(nsm, kPagedMaxTcCtas);
    p.gm.tpu = S::NQ * tpt;
    p.gm.tk = S::BC;
    p.gm.unit_cost = 5 * S::BC;   // (1, 3 and 8 tiles: 161, 133 and 135 us for a 4096-token prompt, 5: 131)
    p.gm.min_share = 4 * S::BC;
    paged_derive(p.gm);
    paged_carve(p, workspace, ctas, S::NQ * 128);
    const int rc = launch_dependent(kern, dim3(static_cast<unsigned>(ctas)), S::THREADS, S::SMEM_BYTES, stream, tq, tk, tv, p);
    if (rc != kOk) return rc;
    return launch_paged_merge(p, 1, ctas, nsm, stream);
}

}  // namespace

int launch_paged_tc(PagedParams p, void *workspace, cudaStream_t stream) {
    return p.d <= 64 ? launch_dp<64>(p, workspace, stream) : launch_dp<128>(p, workspace, stream);
}

}  // namespace eta

// Attention of a few new tokens over a paged cache of 4-bit values (e2m1.cuh):
// decoding, and the checking of a few drafted tokens.
//
// A unit (paged_index.h) is one kv head with up to 8 or 16 query rows.  It
// streams 9 bytes for 16 values, so the bytes are few and what has to be kept
// short is the arithmetic from code to product: for each two values a conversion
// (e2m1 to float16), a multiplication by the scale, and a share of a matrix
// instruction.
//
//   producer warp  finds the CTA's work; bulk copies of tiles of 128 keys, page by page,
//                  K and V on one barrier, and (TMA) of the next unit's Q rows.
//   other warps    consumers, 16 keys of a tile at a time, each with a running
//                  maximum, sum and output of its own for all rows and columns; no
//                  exchange between warps before the unit's end.
//
// Keys are the rows of the matrix instruction (m16n8k16, float16 operands, float32
// sums), so its 8 columns hold the query rows and little is padded:
//   S^T = K Q^T    a lane has two keys and a run of d / 4 columns of each; which
//                  column stands where in the sum is free, so a lane's bytes go to
//                  the instruction as they lie, and Q is laid out to match;
//   O^T = V^T P^T  a lane has four keys and a run of d / 8 columns.  The instruction
//                  wants two keys of a column in a register: the halves of two keys'
//                  bytes are exchanged before the conversion (4 instructions to 16
//                  values).  P^T comes from S^T by transposing 8 x 8 blocks in registers.
// Which key stands in which row of the instruction is free too, as long as S and P V
// agree; an order is taken that keeps the reads of K free of bank conflicts (of V,
// two-way at d = 128, where four keys' rows of 64 bytes cannot avoid one another).
//
// Numbers.  Values are exact in float16.  A row of Q is multiplied by a power of two
// that brings its largest column to 2^14 .. 2^15 (bf16 has more exponents than
// float16): a column keeps its 8 bits down to 2^-29 of the row's largest and is off
// by 2^-39 of it at most below (half of 2^-24, beside 2^14 at least).  Weights are
// p = 2^(s - m + 7) against a reference m that moves when a score exceeds it by 8, so
// they reach 2^15 and are rounded once to float16 (2^-11 of a weight, 2^-32 of the row's
// largest at least); sums stay float32.
//
// Pages that do not exist are not copied and their keys skipped; masked scores are
// replaced by -inf; scales of slots past the end, which may hold anything, by 0.
// (A NaN in V before the end also reaches the unit's rows that do not see it, by their
// weight of 0: the caller is told.)
//
// Measured, 64 sequences of 2048 .. 8191 tokens, 8 kv heads of 128, 4 query heads to
// each: 397 MB in 80 us, 0.74 of the measured copy rate (a bf16 cache: 219 us).  The
// copies alone take 75 and the arithmetic alone 81 (graph replays of 85): 272
// instructions to 16 keys, of which 64 conversions (a half of the ALU's time), 64
// multiplications and 16 matrix instructions (of the FMA pipe's).  Three CTAs an SM and
// blocks in pairs: two CTAs 92 us, four with single blocks 101.  12 and 16 rows: 133 us
// (132 bytes of spills at d 128, 32 at 96).
// 4 sequences of 300 .. 1000: 11 us, a chain of dependent reads over two launches.
#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "e2m1.cuh"
#include "launch.cuh"
#include "paged.cuh"

namespace eta {
namespace {

template <int D_, int NT_>   // head dimension, blocks of 8 query rows
struct P4Shape {
    static constexpr int D = D_, NT = NT_, ROWS = 8 * NT;
    static constexpr int NW = 4, SPW = 2;                     // consumer warps, blocks of 16 keys of a tile to each
    static constexpr int THREADS = 32 * (NW + 1);
    static constexpr int KEYS = 16 * NW * SPW, CTAS = NT == 1 ? 3 : 2;
    static constexpr int CB = D / 2, SB = D / 16;             // bytes of a row: codes, scales
    static constexpr int OFF_V = KEYS * (CB + SB);            // of a stage: K, V
    static constexpr int STAGE = 2 * OFF_V;
    static constexpr int Q_BYTES = ROWS * D * 2;
    static constexpr int OS = D + 4;                          // floats from row to row of an output in shared memory
    // (16 rows, d 128: with 4 stages 146 us for 64 x 2048 .. 8191 tokens, with 3 and the L1 that leaves for spilled registers 133)
    static constexpr int MOST = 228 * 1024 / CTAS - 1024;     // bytes a CTA
    static constexpr int REST = 2 * Q_BYTES + NW * ROWS * (OS / 2 + 2) * 4 + 1024 + 512;
    static constexpr int NS_RAW = (MOST - REST) / STAGE, NS_MAX = NT == 2 ? 3 : 6, NS = NS_RAW < NS_MAX ? NS_RAW : NS_MAX;
    static constexpr int OFF_Q = NS * STAGE;                  // [2]
    static constexpr int OFF_O = OFF_Q + 2 * Q_BYTES;         // [NW][ROWS / 2][OS]: every other row
    static constexpr int OFF_ML = OFF_O + NW * ROWS / 2 * OS * 4;   // [2][NW][ROWS]
    static constexpr int OFF_BAR = OFF_ML + 2 * NW * ROWS * 4;
    static constexpr int BAR_FULL = 0, BAR_EMPTY = NS, BAR_QFULL = 2 * NS, BAR_QEMPTY = BAR_QFULL + 2;
    static constexpr int OFF_MISC = OFF_BAR + (BAR_QEMPTY + 2) * 8;
    static constexpr int OFF_BADP = OFF_MISC + 16;            // per stage: missing pages, bit per 16 keys
    static constexpr int OFF_UNIT = OFF_BADP + (NS * 4 + 15) / 16 * 16;   // [2]
    static constexpr int SMEM_BYTES = OFF_UNIT + 2 * static_cast<int>(sizeof(PagedUnit)) + 1024;
    static_assert(SMEM_BYTES <= MOST && NS >= 3, "shared memory");
    static_assert(OFF_Q % 128 == 0 && Q_BYTES % 128 == 0 && OFF_MISC % 16 == 0, "alignment");
    // a lane's run of K: words (8 columns each), and of V: bytes (2 columns each)
    static constexpr int KW = D / 32, KS = 2 * KW;
    static constexpr int VB = D == 96 ? 8 : D / 16;           // (d 96: 6 lanes of 8 bytes; 2 repeat the last run)
    // the key (of 8) in row i of the matrix instruction: nibble i
    static constexpr uint32_t ORDER = 0x67453210u;
};

__device__ __forceinline__ void mma16816h(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
template <int D, int NT>
__global__ void __launch_bounds__(P4Shape<D, NT>::THREADS, P4Shape<D, NT>::CTAS)
    paged4_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const PagedParams p) {
    using S = P4Shape<D, NT>;
    constexpr int NS = S::NS, ROWS = S::ROWS, NW = S::NW, KEYS = S::KEYS, KW = S::KW, KS = S::KS, VB = S::VB;
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
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar(S::BAR_FULL + s), 1);
            mbar_init(bar(S::BAR_EMPTY + s), NW);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(S::BAR_QFULL + b), 1);
            mbar_init(bar(S::BAR_QEMPTY + b), NW);
        }
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == NW && lane == 0) tma_prefetch_desc(&tm_q);
    const Paged4Box box = paged4_box(gm.page_shift, 7, D);
    __syncthreads();
    paged_touch(p);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == NW) {
        // ------------------------------------------------------------------
        // Producer.  Lane (K or V, box) issues that copy of a tile.
        // ------------------------------------------------------------------
        auto wwait = [&](uint32_t b, uint32_t parity, int site) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.err, site));
        };
        const int boxes = KEYS >> box.shift;   // 1 .. 8
        const int my_kv = lane / boxes, my_box = lane % boxes;
        const bool mine = lane < 2 * boxes;
        const char *pool = static_cast<const char *>(my_kv ? p.V : p.K);
        const uint32_t dst = my_kv * S::OFF_V + my_box * box.bytes;
        int t = 0, u = 0;
        bool ok = true;
        PagedFeed feed;
        feed.start(p, cta, gridDim.x);
        for (;; ++u) {
            PagedUnit w;
            feed.next(p, cta, w);
            const int qb = u & 1;
            if (u >= 2 && !wwait(bar(S::BAR_QEMPTY + qb), (u / 2 - 1) & 1, 60)) ok = false;
            if (!ok) break;   // (the others' waits run out too)
            if (lane == 0) {
                units[qb] = w;
                if (w.tiles == 0) {
                    mbar_arrive(bar(S::BAR_QFULL + qb));
                } else {
                    mbar_arrive_expect_tx(bar(S::BAR_QFULL + qb), D * 2 * gm.g * gm.tpu);
                    tma_load_3d(sbase + S::OFF_Q + qb * S::Q_BYTES, &tm_q, bar(S::BAR_QFULL + qb), 0, w.head * gm.g, w.tok0);
                }
            }
            if (w.tiles == 0) break;
            feed.report(p, w);
            const int j1 = w.tile0 + w.tiles;
            PagedColumns pages;
            pages.start(gm, w.seq, w.len, w.tile0 * KEYS >> gm.page_shift);
            for (int j = w.tile0; j < j1; ++j, ++t) {
                const int key = j * KEYS + (my_box << box.shift);
                const bool held = mine && key < w.len;
                const int page = pages.get(gm, w.seq, j * KEYS >> gm.page_shift, key >> gm.page_shift);
                const int id = !held ? -1 : page < 0 ? -2 : page;   // of this lane's box: -1 past the end, -2 missing
                const int st = t % NS;
                if (t >= NS && !wwait(bar(S::BAR_EMPTY + st), (t / NS - 1) & 1, 61)) {
                    ok = false;
                    break;
                }
                // (boxes without a page are not copied: nothing of them is used)
                const uint32_t missing = __ballot_sync(0xffffffffu, id == -2 && my_kv == 0);
                const uint32_t there = __ballot_sync(0xffffffffu, id >= 0);
                if (lane == 0) {
                    uint32_t bits = 0;
                    if (missing) {
                        atomicOr(p.err, kErrWordBadRow);
                        const int groups = 1 << (box.shift - 4);
                        for (int b = 0; b < boxes; ++b)
                            if ((missing >> b) & 1u) bits |= ((1u << groups) - 1u) << (b * groups);
                    }
                    bad_pages[st] = bits;
                    mbar_arrive_expect_tx(bar(S::BAR_FULL + st), __popc(there) * box.bytes);
                }
                __syncwarp();
                if (id >= 0)
                    paged4_copy(box, sbase + st * S::STAGE + dst, pool + id * p.page_stride + w.head * p.head_stride,
                                key & (gm.page_size - 1), gm.page_size, D, bar(S::BAR_FULL + st));
            }
        }
        feed.finish(p, cta);
        // every copy has landed before this warp leaves
        for (int tt = max(0, t - NS); tt < t; ++tt) wwait(bar(S::BAR_FULL + tt % NS), (tt / NS) & 1, 62);
        // (the buffer that the last words went to was free: its Q had been read)
        for (int uu = max(0, u - 1); uu < u; ++uu) wwait(bar(S::BAR_QFULL + (uu & 1)), (uu / 2) & 1, 63);
        __syncwarp();
    } else {
        // ------------------------------------------------------------------
        // Consumers.  r, c: the lane's row and column group in the matrix
        // instruction's fragments.
        // ------------------------------------------------------------------
        const int r = lane >> 2, c = lane & 3;
        auto order = [](int i) -> int { return (S::ORDER >> (4 * i)) & 7; };
        const int key_r = order(r), key_a = order(2 * c), key_b = order(2 * c + 1);
        const int vr = D == 96 ? min(r, 5) : r;   // the lane's run of V
        // where this lane's bytes of the warp's blocks lie in a tile
        int k_at[S::SPW], ks_at[S::SPW], va_at[S::SPW], vb_at[S::SPW], vsa_at[S::SPW], vsb_at[S::SPW];
#pragma unroll
        for (int b = 0; b < S::SPW; ++b) {
            const int key = (warp + b * NW) * 16, in = key & ((1 << box.shift) - 1), at = (key >> box.shift) * box.bytes;
            const int codes = at + in * S::CB, scales = at + box.codes + in * S::SB;
            k_at[b] = codes + key_r * S::CB + c * (D / 8);
            ks_at[b] = scales + key_r * S::SB + c * (D / 8) / 8;
            va_at[b] = S::OFF_V + codes + key_a * S::CB + vr * VB;
            vb_at[b] = S::OFF_V + codes + key_b * S::CB + vr * VB;
            vsa_at[b] = S::OFF_V + scales + key_a * S::SB + vr * VB / 8;
            vsb_at[b] = S::OFF_V + scales + key_b * S::SB + vr * VB / 8;
        }
        int st = 0, phase = 0;   // stage of the next tile
        for (int u = 0;; ++u) {
            const int qb = u & 1;
            // (all consumers leave together: what one reads of a unit that never came, the others read too)
            const bool came = mbar_wait(bar(S::BAR_QFULL + qb), (u / 2) & 1, abort_flag, p.err, 64);
            if (named_bar_red_or(1, 32 * NW, !came)) break;
            const PagedUnit w = units[qb];
            if (w.tiles == 0) break;
            const int rows = w.ntok * gm.g, j1 = w.tile0 + w.tiles;
            // Q: row r of each block, this lane's columns, scaled
            uint32_t qf[NT][KS][2];
            float mult[NT][2];   // what turns a sum of rows 2c, 2c + 1 into a score in log2 units
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = nt * 8 + r;
                uint32_t x[KS][2], top = 0;
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(smem + S::OFF_Q + qb * S::Q_BYTES + row * (D * 2) + c * (D / 2) + k * 8);
                    x[k][0] = v.x, x[k][1] = v.y, x[k + 1][0] = v.z, x[k + 1][1] = v.w;
                }
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (row >= rows) x[k][e] = 0u;
                        top = max(top, max((x[k][e] << 16) & 0x7fff0000u, x[k][e] & 0x7fff0000u));
                    }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int up = f16_shift(top);
                const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                const float back = f16_back(p.scale_log2, up);
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) qf[nt][k][e] = pack_f16x2(bf16lo_to_f32(x[k][e]) * f, bf16hi_to_f32(x[k][e]) * f);
#pragma unroll
                for (int i = 0; i < 2; ++i) mult[nt][i] = __shfl_sync(0xffffffffu, back, (2 * c + i) * 4);
            }
            fence_proxy_async_smem();   // (the reads are done before the next copy may write there)
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(S::BAR_QEMPTY + qb));   // (with the unit's words, which are in registers)
            int vis[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = nt * 8 + 2 * c + i;
                    vis[nt][i] = row < rows ? paged_unit_visible(gm, w, paged_token(gm, row)) : 0;
                }
            const int vis_all = paged_unit_visible(gm, w, 0);              // what every row sees
            const int vis_any = paged_unit_visible(gm, w, w.ntok - 1);     // what some row sees
            // mu: the reference less 7 (-inf: no key yet)
            float mu[NT][2], l[NT][2], o[NT][VB][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mu[nt][i] = -INFINITY;
                    l[nt][i] = 0.f;
                }
#pragma unroll
                for (int m = 0; m < VB; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][m][e] = 0.f;
            }
            // One block of 16 keys from key0 on.  EDGE: some row does not see all of them.
            auto block = [&](auto edge_c, const uint8_t *tile, int b, int key0) {
                constexpr bool EDGE = decltype(edge_c)::value;
                // ---------------- S^T = K Q^T ----------------
                uint32_t kw[2][KW], ksc[2][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t *at = tile + k_at[b] + h * (8 * S::CB), *as = tile + ks_at[b] + h * (8 * S::SB);
                    if constexpr (D == 128) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(at);
                        kw[h][0] = v.x, kw[h][1] = v.y, kw[h][2] = v.z, kw[h][3] = v.w;
                        const uint32_t x = *reinterpret_cast<const uint16_t *>(as);
                        ksc[h][0] = e2m1_scale_h2(x & 0xffu);
                        ksc[h][1] = e2m1_scale_h2(x >> 8);
                    } else if constexpr (D == 96) {
#pragma unroll
                        for (int x = 0; x < 3; ++x) kw[h][x] = *reinterpret_cast<const uint32_t *>(at + 4 * x);
                        ksc[h][0] = e2m1_scale_h2(as[0]);
                        ksc[h][1] = e2m1_scale_h2(as[1]);
                    } else if constexpr (D == 64) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(at);
                        kw[h][0] = v.x, kw[h][1] = v.y;
                        ksc[h][0] = ksc[h][1] = e2m1_scale_h2(as[0]);
                    } else {
                        kw[h][0] = *reinterpret_cast<const uint32_t *>(at);
                        ksc[h][0] = ksc[h][1] = e2m1_scale_h2(as[0]);
                    }
                }
                float s[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
                for (int x = 0; x < KW; ++x) {
                    uint32_t h[2][4];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        // (d 96: the middle word belongs to the first group in even c, to the second in odd c)
                        const uint32_t sc = D == 128 ? ksc[y][x >> 1] : D == 96 ? (x == 0 ? ksc[y][0] : x == 2 ? ksc[y][1] : c & 1 ? ksc[y][1] : ksc[y][0]) : ksc[y][0];
                        e2m1_values(kw[y][x], sc, h[y]);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t a[4] = {h[0][2 * k], h[1][2 * k], h[0][2 * k + 1], h[1][2 * k + 1]};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816h(s[nt], a, qf[nt][2 * x + k][0], qf[nt][2 * x + k][1]);
                    }
                }
                // ---------------- weights ----------------
                // element e = 2 h + i: key key_r + 8 h, row 2c + i.  y: the weight's exponent
                float y[NT][4];
                bool move = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = e & 1;
                        y[nt][e] = fmaf(s[nt][e], mult[nt][i], -mu[nt][i]);
                        if (EDGE && key0 + key_r + (e >> 1) * 8 >= vis[nt][i]) y[nt][e] = -INFINITY;
                        move = move || y[nt][e] > 15.f;
                    }
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float x[2];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                x[h] = s[nt][2 * h + i] * mult[nt][i];
                                if (EDGE && key0 + key_r + h * 8 >= vis[nt][i]) x[h] = -INFINITY;
                            }
                            float v = fmaxf(x[0], x[1]);
#pragma unroll
                            for (int z = 4; z < 32; z <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, z));
                            if (v - mu[nt][i] > 15.f) {
                                const float a = ex2(mu[nt][i] - (v - 7.f));   // (the first time: 0)
                                mu[nt][i] = v - 7.f;
                                l[nt][i] *= a;
#pragma unroll
                                for (int m = 0; m < VB; ++m) {
                                    o[nt][m][i] *= a;
                                    o[nt][m][2 + i] *= a;
                                }
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) y[nt][2 * h + i] = x[h] == -INFINITY ? -INFINITY : x[h] - mu[nt][i];
                        }
                }
                uint32_t pf[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float p0 = ex2(y[nt][2 * h]), p1 = ex2(y[nt][2 * h + 1]);
                        l[nt][0] += p0;
                        l[nt][1] += p1;
                        pf[nt][h] = transpose8(pack_f16x2(p0, p1));
                    }
                // ---------------- O^T += V^T P^T ----------------
                uint32_t sc[2];   // of keys (a, b) and (a + 8, b + 8)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t b0 = tile[vsa_at[b] + h * (8 * S::SB)], b1 = tile[vsb_at[b] + h * (8 * S::SB)];
                    if (EDGE) {
                        if (key0 + h * 8 + key_a >= w.len) b0 = 0u;
                        if (key0 + h * 8 + key_b >= w.len) b1 = 0u;
                    }
                    sc[h] = b1 * 0x800000u + b0 * 0x80u;
                }
                constexpr int VW = VB >= 4 ? VB / 4 : 1;
                uint32_t vw[2][2][VW];   // [h][a or b]
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint8_t *at = tile + (x ? vb_at[b] : va_at[b]) + h * (8 * S::CB);
                        if constexpr (VB == 8) {
                            const uint2 v = *reinterpret_cast<const uint2 *>(at);
                            vw[h][x][0] = v.x;
                            vw[h][x][VW - 1] = v.y;
                        } else if constexpr (VB == 4) {
                            vw[h][x][0] = *reinterpret_cast<const uint32_t *>(at);
                        } else {
                            vw[h][x][0] = *reinterpret_cast<const uint16_t *>(at);
                        }
                    }
#pragma unroll
                for (int x = 0; x < VW; ++x) {
                    uint32_t h[4][4];   // a0 .. a3 of four blocks
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint32_t va = vw[z][0][x], vb = vw[z][1][x];
                        e2m1_values((va & 0x0f0f0f0fu) | ((vb << 4) & 0xf0f0f0f0u), sc[z], h[2 * z]);
                        e2m1_values(((va >> 4) & 0x0f0f0f0fu) | (vb & 0xf0f0f0f0u), sc[z], h[2 * z + 1]);
                    }
#pragma unroll
                    for (int m = 0; m < 4 && 4 * x + m < VB; ++m) {
                        const uint32_t a[4] = {h[0][m], h[1][m], h[2][m], h[3][m]};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816h(o[nt][4 * x + m], a, pf[nt][0], pf[nt][1]);
                    }
                }
            };
            for (int j = w.tile0; j < j1; ++j) {
                mbar_wait(bar(S::BAR_FULL + st), phase, abort_flag, p.err, 65);
                const uint8_t *tile = smem + st * S::STAGE;
                const uint32_t bad = bad_pages[st];
                if ((j + 1) * KEYS <= vis_all && bad == 0u) {
#pragma unroll
                    for (int b = 0; b < S::SPW; ++b) block(std::false_type{}, tile, b, 0);
                } else {
#pragma unroll 1
                    for (int b = 0; b < S::SPW; ++b) {
                        const int key0 = j * KEYS + (warp + b * NW) * 16;
                        if (key0 >= vis_any || ((bad >> (warp + b * NW)) & 1u)) continue;
                        if (b == 0) block(std::true_type{}, tile, 0, key0);
                        else block(std::true_type{}, tile, S::SPW - 1, key0);
                    }
                }
                fence_proxy_async_smem();   // (the reads are done before the next copy may write there)
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(S::BAR_EMPTY + st));
                if (++st == NS) {
                    st = 0;
                    phase ^= 1;
                }
            }
            // ---------------- the unit's end: the warps' parts are joined ----------------
            // (even rows, then odd ones, through the same memory)
            float *o_sh = reinterpret_cast<float *>(smem + S::OFF_O);
            float *m_sh = reinterpret_cast<float *>(smem + S::OFF_ML), *l_sh = m_sh + NW * ROWS;
            const bool whole = w.slot < 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (i > 0) named_bar_sync(1, 32 * NW);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int row = nt * 8 + 2 * c + i;
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], x);
                    if (r == 0) {
                        m_sh[warp * ROWS + row] = paged_part_max(mu[nt][i], l[nt][i]);
                        l_sh[warp * ROWS + row] = l[nt][i];
                    }
                    if (D != 96 || r < 6) {
                        float *at = o_sh + (warp * (ROWS / 2) + nt * 4 + c) * S::OS + r * (2 * VB);
#pragma unroll
                        for (int m = 0; m < VB; m += 2)
                            *reinterpret_cast<float4 *>(at + 2 * m) =
                                make_float4(o[nt][m][i], o[nt][m][2 + i], o[nt][m + 1][i], o[nt][m + 1][2 + i]);
                    }
                }
                named_bar_sync(1, 32 * NW);
                for (int x = threadIdx.x; x < ROWS / 2 * (D / 4); x += 32 * NW) {
                    const int half = x / (D / 4), row = 2 * half + i, col = x % (D / 4) * 4;
                    if (row >= rows || *abort_flag) continue;
                    float M = -INFINITY;
#pragma unroll
                    for (int k = 0; k < NW; ++k) M = fmaxf(M, m_sh[k * ROWS + row]);
                    float L = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < NW; ++k) {
                        const float mk = m_sh[k * ROWS + row];
                        const float wt = ex2(mk - M);
                        const float4 v = *reinterpret_cast<const float4 *>(o_sh + (k * (ROWS / 2) + half) * S::OS + col);
                        if (mk != -INFINITY) {   // (a weight of 0 still passes a NaN on)
                            L = fmaf(wt, l_sh[k * ROWS + row], L);
                            acc.x = fmaf(wt, v.x, acc.x);
                            acc.y = fmaf(wt, v.y, acc.y);
                            acc.z = fmaf(wt, v.z, acc.z);
                            acc.w = fmaf(wt, v.w, acc.w);
                        }
                    }
                    const int tr = paged_token(gm, row);
                    const long long tok = w.tok0 + tr;
                    const int head = w.head * gm.g + row - tr * gm.g;
                    if (whole) {
                        const float inv = L != 0.f ? 1.f / L : 0.f;   // (a NaN goes on)
                        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.O) + tok * p.o_token + static_cast<long long>(head) * p.o_head + col;
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                        if (col == 0 && p.LSE) p.LSE[tok * p.Hq + head] = L != 0.f ? (M + log2f(L)) * kPagedLn2 : -INFINITY;
                    } else {
                        const size_t prow = static_cast<size_t>(w.slot) * p.part_rows + row;
                        *reinterpret_cast<float4 *>(p.part_o + prow * D + col) = acc;
                        if (col == 0) {
                            p.part_m[prow] = paged_part_max(M, L);
                            p.part_l[prow] = L;
                        }
                    }
                }
            }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

constexpr int kMaxDev = 64;
std::mutex g_mu;

template <int D, int NT>
int launch_one(PagedParams &p, void *workspace, cudaStream_t stream) {
    using S = P4Shape<D, NT>;
    auto kern = paged4_decode_kernel<D, NT>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return kErrCuda;
    static std::atomic<int> grids[kMaxDev];   // CTAs that are resident at once; 0: not set up yet
    int grid = grids[dev].load(std::memory_order_acquire);
    if (grid == 0) {
        std::lock_guard<std::mutex> lk(g_mu);
        int nsm = 0, per = 0;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM_BYTES) != cudaSuccess ||
            cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, S::THREADS, S::SMEM_BYTES) != cudaSuccess)
            return kErrCuda;
        grid = std::min(nsm * std::max(per, 1), kPagedMaxDecode4Ctas);
        grids[dev].store(grid, std::memory_order_release);
    }
    p.gm.tpu = S::ROWS / p.gm.g;
    p.gm.tk = S::KEYS;
    p.gm.unit_cost = S::KEYS;
    p.gm.min_share = S::KEYS;
    paged_derive(p.gm);
    CUtensorMap tq;
    if (!paged4_q_map(p, p.gm.tpu, &tq)) return kErrCuda;
    paged_carve(p, workspace, grid, S::ROWS);
    const int rc = launch_dependent(kern, dim3(static_cast<unsigned>(grid)), S::THREADS, S::SMEM_BYTES, stream, tq, p);
    if (rc != kOk) return rc;
    return launch_paged_merge(p, 1, grid, grid / S::CTAS, stream);
}

template <int NT>
int launch_nt(PagedParams &p, void *workspace, cudaStream_t stream) {
    switch (p.d) {
        case 32: return launch_one<32, NT>(p, workspace, stream);
        case 64: return launch_one<64, NT>(p, workspace, stream);
        case 96: return launch_one<96, NT>(p, workspace, stream);
        default: return launch_one<128, NT>(p, workspace, stream);
    }
}

}  // namespace

int launch_paged4_decode(PagedParams p, void *workspace, cudaStream_t stream) {
    return paged4_decode_rows(p.gm.g, p.gm.max_q) == 8 ? launch_nt<1>(p, workspace, stream) : launch_nt<2>(p, workspace, stream);
}

}  // namespace eta

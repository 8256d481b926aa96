// Joins the partial results of attn_paged_fwd: a unit whose key tiles were
// shared by several CTAs has one part (m, l, o) from each, and
//     M = max m_s,  O = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,
// the rule by which the tiled forward joins two blocks of keys.
//
// The unit that CTA c began but did not end has its first part in slot 2c + 1
// and the others in the slots 2k of the CTAs after c, up to the one that ends
// it; each CTA left one word that says which of its slots are in use.  A warp
// takes a row: a lane to a part reads m and l, then up to 8 parts' rows are
// read before the first is used.  What bounds it is this chain of dependent
// reads.  Parts are added in order: the result does not depend on timing.
//
// Units of few rows (decoding): block c looks at CTA c's unit, and all lanes
// read words, m and l at once before it is known how many parts there are.
// Units of many rows: every block reads all words and finds the cut units in
// them, so rows are dealt out evenly however few units were cut (8 units of
// 256 rows and 19 parts each: 20 us when their blocks stayed on 64 SMs); with
// two parts, as nearly always in a large batch, a warp takes four rows at once.
#include <algorithm>

#include "launch.cuh"
#include "paged.cuh"

namespace eta {
namespace {

constexpr int kMergeWarps = 8;
constexpr int kMergeThreads = 32 * kMergeWarps;
constexpr int kMergeFlight = 8;

template <int E>
__device__ __forceinline__ void load_row(const float *src, float (&v)[E]) {
    if constexpr (E == 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4 *>(src));
        v[0] = f.x;
        v[1] = f.y;
        v[2] = f.z;
        v[3] = f.w;
    } else if constexpr (E == 2) {
        const float2 f = __ldcg(reinterpret_cast<const float2 *>(src));
        v[0] = f.x;
        v[1] = f.y;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = __ldcg(src + e);
    }
}

template <int E, bool BF16>
__device__ __forceinline__ void store_row(void *base, long long at, const float (&v)[E], float inv) {
    if constexpr (BF16) {
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(base) + at;
        if constexpr (E == 4) {
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv));
        } else if constexpr (E == 2) {
            *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(v[0] * inv, v[1] * inv);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) dst[e] = __float2bfloat16_rn(v[e] * inv);
        }
    } else {
        float *dst = static_cast<float *>(base) + at;
        if constexpr (E == 4) {
            *reinterpret_cast<float4 *>(dst) = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) dst[e] = v[e] * inv;
        }
    }
}

// One row of the unit that CTA c began.  word(k): CTA k's word.  FEW: words and
// statistics are read together, whatever the words then say.
template <int E, bool BF16, bool FEW, typename Word>
__device__ __forceinline__ void merge_row(const PagedParams &p, int ctas, int c, int row, const Word &word) {
    const int lane = threadIdx.x & 31;
    float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    PagedHdr own{0, 0, 0, 0};
    if constexpr (!FEW) own = paged_read_header(p, 2 * c + 1);
    for (int base = 0; base < ctas - c; base += 32) {
        // part s is CTA c + s's (part 0: the one that begins the unit)
        const int s = base + lane;
        const int slot = s == 0 ? 2 * c + 1 : 2 * (c + s);
        const size_t x = static_cast<size_t>(slot) * p.part_rows + row;
        float m = -INFINITY, l = 0.f;
        int wd = 0;
        if constexpr (FEW) {
            if (c + s < ctas) {
                wd = word(c + s);
                m = __ldcg(p.part_m + x);
                l = __ldcg(p.part_l + x);
                if (base == 0 && lane == 0) own = paged_read_header(p, 2 * c + 1);
            }
            if (base == 0 && row >= __shfl_sync(0xffffffffu, wd, 0) >> 2) return;   // nothing begins here, or no such row
        } else {
            if (c + s < ctas) wd = word(c + s);
        }
        const uint32_t ends = __ballot_sync(0xffffffffu, s > 0 && (wd & 3) == 3);
        const int cnt = ends ? __ffs(ends) : min(32, ctas - c - base);
        const bool in = lane < cnt && (s == 0 || (wd & 1));   // (a CTA without a share has no part)
        if constexpr (FEW) {
            if (!in) m = -INFINITY;
        } else if (in) {
            m = __ldcg(p.part_m + x);
            l = __ldcg(p.part_l + x);
        }
        float Mc = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) Mc = fmaxf(Mc, __shfl_xor_sync(0xffffffffu, Mc, o));
        const float Mn = fmaxf(M, Mc);
        if (Mn != -INFINITY) {
            const float a = M == -INFINITY ? 0.f : ex2(M - Mn);
            // (a weight of 0 also stands for an o that was not written)
            const float w = m == -INFINITY ? 0.f : ex2(m - Mn);
            float wl = w == 0.f ? 0.f : w * l;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) wl += __shfl_xor_sync(0xffffffffu, wl, o);
            L = L * a + wl;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= a;
            auto add = [&](int q0) {
                constexpr int F = kMergeFlight;
                float v[F][E], ws[F];
#pragma unroll
                for (int q = 0; q < F; ++q) {
                    ws[q] = __shfl_sync(0xffffffffu, w, (q0 + q) & 31);
                    if (q0 + q >= cnt) ws[q] = 0.f;
                    const int part = base + q0 + q;
                    const size_t sl = static_cast<size_t>(part == 0 ? 2 * c + 1 : 2 * (c + part));
#pragma unroll
                    for (int e = 0; e < E; ++e) v[q][e] = 0.f;
                    if (ws[q] != 0.f) load_row<E>(p.part_o + (sl * p.part_rows + row) * p.d + E * lane, v[q]);
                }
#pragma unroll
                for (int q = 0; q < F; ++q)
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = fmaf(ws[q], v[q][e], acc[e]);
            };
            for (int q0 = 0; q0 < cnt; q0 += kMergeFlight) add(q0);
            M = Mn;
        }
        if (ends) break;
    }
    if constexpr (FEW) {
        own.tok0 = __shfl_sync(0xffffffffu, own.tok0, 0);
        own.head = __shfl_sync(0xffffffffu, own.head, 0);
    }
    const int t = paged_token(p.gm, row);
    const long long tok = own.tok0 + t;
    const int hq = own.head * p.gm.g + row - t * p.gm.g;
    store_row<E, BF16>(p.O, tok * p.o_token + static_cast<long long>(hq) * p.o_head + E * lane, acc, L != 0.f ? 1.f / L : 0.f);
    if (lane == 0 && p.LSE) p.LSE[tok * p.Hq + hq] = L != 0.f ? (M + log2f(L)) * kPagedLn2 : -INFINITY;
}

// Four rows (row, row + kMergeWarps, ...) of a unit of two parts: lane 2 q + s reads m and l of row q's part s.
template <int E, bool BF16>
__device__ __forceinline__ void merge_rows4(const PagedParams &p, int c, int row, int rows) {
    const int lane = threadIdx.x & 31;
    const PagedHdr own = paged_read_header(p, 2 * c + 1);
    const int s = lane & 1, mine = row + (lane >> 1) * kMergeWarps;
    float m = -INFINITY, l = 0.f;
    if (lane < 8 && mine < rows) {
        const size_t x = static_cast<size_t>(s == 0 ? 2 * c + 1 : 2 * (c + 1)) * p.part_rows + mine;
        m = __ldcg(p.part_m + x);
        l = __ldcg(p.part_l + x);
    }
    const float M = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    // (a weight of 0 also stands for an o that was not written)
    const float w = m == -INFINITY ? 0.f : ex2(m - M);
    float L = w == 0.f ? 0.f : w * l;
    L += __shfl_xor_sync(0xffffffffu, L, 1);
    float v[2][4][E], ws[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const size_t at = static_cast<size_t>(t == 0 ? 2 * c + 1 : 2 * (c + 1)) * p.part_rows + row;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            ws[t][q] = __shfl_sync(0xffffffffu, w, 2 * q + t);
#pragma unroll
            for (int e = 0; e < E; ++e) v[t][q][e] = 0.f;
            if (ws[t][q] != 0.f) load_row<E>(p.part_o + (at + q * kMergeWarps) * p.d + E * lane, v[t][q]);
        }
    }
    float acc[4][E];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[q][e] = fmaf(ws[1][q], v[1][q][e], ws[0][q] * v[0][q][e]);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int r = row + q * kMergeWarps;
        const float Lq = __shfl_sync(0xffffffffu, L, 2 * q), Mq = __shfl_sync(0xffffffffu, M, 2 * q);
        if (r >= rows) continue;
        const int t = paged_token(p.gm, r);
        const long long tok = own.tok0 + t;
        const int hq = own.head * p.gm.g + r - t * p.gm.g;
        store_row<E, BF16>(p.O, tok * p.o_token + static_cast<long long>(hq) * p.o_head + E * lane, acc[q],
                           Lq != 0.f ? 1.f / Lq : 0.f);
        if (lane == 0 && p.LSE) p.LSE[tok * p.Hq + hq] = Lq != 0.f ? (Mq + log2f(Lq)) * kPagedLn2 : -INFINITY;
    }
}

template <int E, bool BF16, bool FEW>   // E = d / 32 columns per lane
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedParams p, int ctas) {
    paged_touch(p);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if constexpr (FEW) {
        const int row = blockIdx.y * kMergeWarps + warp;
        if (row < p.part_rows)
            merge_row<E, BF16, true>(p, ctas, blockIdx.x, row, [&](int k) { return __ldcg(p.part_sum + k); });
    } else {
        // before: row blocks of earlier CTAs' units
        __shared__ int words[kPagedMaxTcCtas + 1], before[kPagedMaxTcCtas];
        __shared__ int wsum[kMergeWarps];
        static_assert(kPagedMaxTcCtas < kMergeThreads, "a thread to a CTA's word");
        const int wd = threadIdx.x < ctas ? __ldcg(p.part_sum + threadIdx.x) : 0;
        if (threadIdx.x <= kPagedMaxTcCtas) words[threadIdx.x] = wd;
        __syncthreads();
        // a unit whose next part is its last has two (in a large batch nearly all)
        auto two = [&](int k) { return (words[k + 1] & 3) == 3; };
        int blocks = 0;
        if (wd >> 2) {
            const int per = two(threadIdx.x) ? 4 * kMergeWarps : kMergeWarps;   // rows of a block
            blocks = ((wd >> 2) + per - 1) / per;
        }
        int inc = blocks;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        int at = inc - blocks, total = 0;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
            if (w < warp) at += wsum[w];
            total += wsum[w];
        }
        if (threadIdx.x < ctas) before[threadIdx.x] = at;
        __syncthreads();
        for (int item = blockIdx.x; item < total; item += gridDim.x) {
            int lo = 0, hi = ctas - 1;   // the last CTA with before <= item (the last of equal ones has the rows)
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (before[mid] <= item) lo = mid;
                else hi = mid - 1;
            }
            const int rows = words[lo] >> 2, block = item - before[lo];
            if (two(lo)) {
                const int row = block * 4 * kMergeWarps + warp;
                if (row < rows) merge_rows4<E, BF16>(p, lo, row, rows);
            } else {
                const int row = block * kMergeWarps + warp;
                if (row < rows) merge_row<E, BF16, false>(p, ctas, lo, row, [&](int k) { return words[k]; });
            }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int E, bool BF16, bool FEW>
int launch_one(const PagedParams &p, int ctas, int sms, cudaStream_t stream) {
    // at most ctas units are cut, of at most as many rows as an entry has
    const long long rows = std::min<long long>(p.part_rows, static_cast<long long>(p.gm.max_q) * p.gm.g);
    const unsigned per = static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps);
    const dim3 grid = FEW ? dim3(static_cast<unsigned>(ctas), per)
                          : dim3(std::min(static_cast<unsigned>(ctas) * per, 4u * static_cast<unsigned>(sms)));
    return launch_dependent(paged_merge_kernel<E, BF16, FEW>, grid, kMergeThreads, 0, stream, p, ctas);
}

template <int E>
int launch_e(const PagedParams &p, int bf16, int ctas, int sms, cudaStream_t stream) {
    if (!bf16) return launch_one<E, false, true>(p, ctas, sms, stream);
    return p.part_rows <= 64 ? launch_one<E, true, true>(p, ctas, sms, stream) : launch_one<E, true, false>(p, ctas, sms, stream);
}

}  // namespace

int launch_paged_merge(const PagedParams &p, int bf16, int ctas, int sms, cudaStream_t stream) {
    switch (p.d) {
        case 32: return launch_e<1>(p, bf16, ctas, sms, stream);
        case 64: return launch_e<2>(p, bf16, ctas, sms, stream);
        case 96: return launch_e<3>(p, bf16, ctas, sms, stream);
        case 128: return launch_e<4>(p, bf16, ctas, sms, stream);
        default: return kErrUnsupported;
    }
}

bool paged_maps(const PagedParams &p, int tokens, int box, CUtensorMap *tq, CUtensorMap *tk, CUtensorMap *tv) {
    const PagedGeom &gm = p.gm;
    const cuuint64_t qd[3] = {static_cast<cuuint64_t>(p.d), static_cast<cuuint64_t>(p.Hq), static_cast<cuuint64_t>(gm.T)};
    const cuuint64_t qs[2] = {static_cast<cuuint64_t>(p.q_head) * 2, static_cast<cuuint64_t>(p.q_token) * 2};
    const cuuint32_t qb[3] = {64u, static_cast<cuuint32_t>(gm.g), static_cast<cuuint32_t>(tokens)};
    const cuuint64_t kd[4] = {static_cast<cuuint64_t>(p.d), static_cast<cuuint64_t>(gm.page_size),
                              static_cast<cuuint64_t>(gm.heads), static_cast<cuuint64_t>(gm.pages)};
    const cuuint64_t ks[3] = {static_cast<cuuint64_t>(p.slot_stride) * 2, static_cast<cuuint64_t>(p.head_stride) * 2,
                              static_cast<cuuint64_t>(p.page_stride) * 2};
    const cuuint32_t kb[4] = {64u, static_cast<cuuint32_t>(box), 1u, 1u};
    return make_bf16_map(tq, p.Q, 3, qd, qs, qb) && make_bf16_map(tk, p.K, 4, kd, ks, kb) &&
           make_bf16_map(tv, p.V, 4, kd, ks, kb);
}

namespace {
// The kernel of a call.  bf16: the stream kernel takes units of up to 32 rows
// (tokens of an entry x query heads of a group), the matrix kernel more.  At 32 rows
// (16 x 4096 tokens, d 128, 2 kv heads: 24.6 us, matrix 24.4; 64 x 8000, 8 heads: 339,
// 338; 8 x 600: 18.2, 18.9; d 64, 64 x 8000: 217, 272); at 40, four row blocks in the
// stream kernel took 38 us where the matrix kernel took 27 (16 x 1000 .. 4096).
// float32: units of up to 8 rows are streamed through registers (32 x 8000 tokens,
// d 128, 4 rows: 160 us, tiled 365; 16 rows, 16 x 4000: 161, tiled 106).
enum class Path { kFew, kSimt, kDecode, kTc };
Path path_of(int g, int max_q, int bf16) {
    if (!bf16) return paged_simt_rows(g, max_q) <= 8 ? Path::kFew : Path::kSimt;
    return static_cast<long long>(g) * max_q <= 32 ? Path::kDecode : Path::kTc;
}
}  // namespace

size_t paged_workspace_bytes(int g, int max_q, int d, int bf16) {
    switch (path_of(g, max_q, bf16)) {
        case Path::kTc: return paged_partial_bytes(kPagedMaxTcCtas, 256, d);
        case Path::kDecode: return paged_partial_bytes(kPagedMaxDecodeCtas, paged_decode_rows(g, max_q), d);
        default: return paged_partial_bytes(kPagedMaxSimtCtas, paged_simt_rows(g, max_q), d);
    }
}

int launch_paged(const PagedParams &p, int bf16, void *workspace, cudaStream_t stream, const char **variant) {
    switch (path_of(p.gm.g, p.gm.max_q, bf16)) {
        case Path::kTc:
            if (variant) *variant = p.d <= 64 ? "paged_tc_bf16_d64" : "paged_tc_bf16_d128";
            return launch_paged_tc(p, workspace, stream);
        case Path::kDecode:
            if (variant) *variant = p.d <= 64 ? "paged_decode_bf16_d64" : "paged_decode_bf16_d128";
            return launch_paged_decode(p, workspace, stream);
        case Path::kFew:
            if (variant) *variant = "paged_few_f32";
            return launch_paged_few(p, workspace, stream);
        default:
            if (variant) *variant = "paged_simt_f32";
            return launch_paged_simt(p, workspace, stream);
    }
}

}  // namespace eta

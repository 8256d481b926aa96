// Joins the partial results of attn_paged_fwd: a unit whose key tiles were
// shared by several CTAs has one part (m, l, o) from each, and
//     M = max m_s,  O = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,
// the rule by which the tiled forward joins two blocks of keys.
//
// Grid (CTA c of the main kernel, row blocks), one warp to a row at a time.  The warps of
// block (c, y) own the unit that CTA c began but did not end (slot 2c + 1); its
// other parts lie in the slots 2k of the CTAs after c, up to the one that ends
// the unit.  What bounds this kernel is its chain of dependent reads, so a lane
// reads the header, m and l of one part at once (32 parts to a round trip,
// before it is known how many there are), and then up to 8 parts' rows are
// read before the first is used.  Parts are added in order: the result does
// not depend on timing.
#include <algorithm>

#include "paged.cuh"

namespace eta {
namespace {

constexpr int kMergeWarps = 8;
constexpr int kMergeRows = 2;      // rows of a warp
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

template <int E, bool BF16>   // E = d / 32 columns per lane
__global__ void __launch_bounds__(32 * kMergeWarps) paged_merge_kernel(const PagedParams p, int ctas) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int row = blockIdx.y * kMergeWarps + warp; row < p.part_rows; row += gridDim.y * kMergeWarps) {
        float M = -INFINITY, L = 0.f, acc[E];
    #pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        PagedHdr own{0, 0, 0, 0};
        for (int base = 0;; base += 32) {
            // part s is CTA c + s's (part 0: the one that begins the unit)
            const int s = base + lane;
            PagedHdr h{0, 0, 0, 0};
            float m = -INFINITY, l = 0.f;
            const int slot = s == 0 ? 2 * c + 1 : 2 * (c + s);
            if (c + s < ctas) {
                const size_t at = static_cast<size_t>(slot) * p.part_rows + row;
                h = paged_read_header(p, slot);
                m = __ldcg(p.part_m + at);
                l = __ldcg(p.part_l + at);
            }
            if (base == 0) {
                own.rows = __shfl_sync(0xffffffffu, h.rows, 0);
                own.tok0 = __shfl_sync(0xffffffffu, h.tok0, 0);
                own.head = __shfl_sync(0xffffffffu, h.head, 0);
                if (row >= own.rows) break;   // nothing begins here, or no more rows
            }
            const uint32_t ends = __ballot_sync(0xffffffffu, s > 0 && h.rows > 0 && h.last);
            const int cnt = ends ? __ffs(ends) : min(32, ctas - c - base);
            const bool in = lane < cnt && h.rows > 0 && m != -INFINITY;   // (a CTA without a share has no part)
            float Mc = in ? m : -INFINITY;
    #pragma unroll
            for (int o = 16; o > 0; o >>= 1) Mc = fmaxf(Mc, __shfl_xor_sync(0xffffffffu, Mc, o));
            const float Mn = fmaxf(M, Mc);
            if (Mn != -INFINITY) {
                const float a = M == -INFINITY ? 0.f : ex2(M - Mn);
                const float w = in ? ex2(m - Mn) : 0.f;
                float wl = in ? w * l : 0.f;
    #pragma unroll
                for (int o = 16; o > 0; o >>= 1) wl += __shfl_xor_sync(0xffffffffu, wl, o);
                L = L * a + wl;
    #pragma unroll
                for (int e = 0; e < E; ++e) acc[e] *= a;
                for (int q0 = 0; q0 < cnt; q0 += kMergeFlight) {
                    float v[kMergeFlight][E], ws[kMergeFlight];
    #pragma unroll
                    for (int q = 0; q < kMergeFlight; ++q) {
                        ws[q] = __shfl_sync(0xffffffffu, w, (q0 + q) & 31);
                        const int sl = __shfl_sync(0xffffffffu, slot, (q0 + q) & 31);
                        if (q0 + q >= cnt) ws[q] = 0.f;
    #pragma unroll
                        for (int e = 0; e < E; ++e) v[q][e] = 0.f;
                        if (ws[q] != 0.f) load_row<E>(p.part_o + (static_cast<size_t>(sl) * p.part_rows + row) * p.d + E * lane, v[q]);
                    }
    #pragma unroll
                    for (int q = 0; q < kMergeFlight; ++q)
    #pragma unroll
                        for (int e = 0; e < E; ++e) acc[e] = fmaf(ws[q], v[q][e], acc[e]);
                }
                M = Mn;
            }
            if (ends || base + 32 >= ctas - c) break;
        }
        if (row >= own.rows) break;
        {
            const float inv = L > 0.f ? 1.f / L : 0.f;
            const long long tok = own.tok0 + row / p.gm.g;
            const int head = own.head * p.gm.g + row % p.gm.g;
            const long long at = tok * p.o_token + static_cast<long long>(head) * p.o_head + E * lane;
            if constexpr (BF16) {
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.O) + at;
                if constexpr (E == 4) {
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                                 pack_bf16x2(acc[2] * inv, acc[3] * inv));
                } else if constexpr (E == 2) {
                    *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
                } else {
    #pragma unroll
                    for (int e = 0; e < E; ++e) dst[e] = __float2bfloat16_rn(acc[e] * inv);
                }
            } else {
                float *dst = static_cast<float *>(p.O) + at;
                if constexpr (E == 4) {
                    *reinterpret_cast<float4 *>(dst) = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
                } else {
    #pragma unroll
                    for (int e = 0; e < E; ++e) dst[e] = acc[e] * inv;
                }
            }
            if (lane == 0 && p.LSE) p.LSE[tok * p.Hq + head] = L > 0.f ? (M + log2f(L)) * kPagedLn2 : -INFINITY;
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int E, bool BF16>
int launch_one(const PagedParams &p, int ctas, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    // a unit has at most as many rows as an entry
    const int rows = static_cast<int>(std::min<long long>(p.part_rows, static_cast<long long>(p.gm.max_q) * p.gm.g));
    const int per = kMergeWarps * kMergeRows;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>((rows + per - 1) / per));
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_merge_kernel<E, BF16>, p, ctas) == cudaSuccess ? kOk : kErrCuda;
}

}  // namespace

int launch_paged_merge(const PagedParams &p, int bf16, int ctas, cudaStream_t stream) {
    switch (p.d) {
        case 32: return bf16 ? launch_one<1, true>(p, ctas, stream) : launch_one<1, false>(p, ctas, stream);
        case 64: return bf16 ? launch_one<2, true>(p, ctas, stream) : launch_one<2, false>(p, ctas, stream);
        case 96: return bf16 ? launch_one<3, true>(p, ctas, stream) : launch_one<3, false>(p, ctas, stream);
        case 128: return bf16 ? launch_one<4, true>(p, ctas, stream) : launch_one<4, false>(p, ctas, stream);
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
// The kernel of a call.  bf16: the stream kernel holds units of up to 64 rows
// (tokens of an entry x query heads of a group); more rows are matrix work.
enum class Path { kSimt, kDecode, kTc };
Path path_of(int g, int max_q, int bf16) {
    if (!bf16) return Path::kSimt;
    return static_cast<long long>(g) * max_q <= 32 ? Path::kDecode : Path::kTc;
}
}  // namespace

size_t paged_workspace_bytes(int g, int max_q, int d, int bf16) {
    if (path_of(g, max_q, bf16) == Path::kTc) return paged_partial_bytes(kPagedMaxTcCtas, 256, d);
    return paged_partial_bytes(kPagedMaxCtas, 64, d);
}

int launch_paged(const PagedParams &p, int bf16, void *workspace, cudaStream_t stream, const char **variant) {
    switch (path_of(p.gm.g, p.gm.max_q, bf16)) {
        case Path::kTc:
            if (variant) *variant = p.d <= 64 ? "paged_tc_bf16_d64" : "paged_tc_bf16_d128";
            return launch_paged_tc(p, workspace, stream);
        case Path::kDecode:
            if (variant) *variant = p.d <= 64 ? "paged_decode_bf16_d64" : "paged_decode_bf16_d128";
            return launch_paged_decode(p, workspace, stream);
        default:
            if (variant) *variant = "paged_simt_f32";
            return launch_paged_simt(p, workspace, stream);
    }
}

}  // namespace eta

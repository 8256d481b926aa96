// Joins the partial results of attn_paged_fwd: a unit whose key tiles were
// shared by several CTAs has one part (m, l, o) from each, and
//     M = max m_s,  O = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,
// the rule by which the tiled forward joins two blocks of keys.
//
// Grid (CTA c of the main kernel, row blocks).  Block (c, y) owns the unit
// that CTA c began but did not end (slot 2c + 1); its other parts lie in the
// slots 2k of the CTAs after c, up to the one that ends the unit.  One warp
// per row at a time: lanes read 32 parts' (m, l) in one round trip, then the
// lanes split d and add the parts in order, so the result does not depend on
// timing.
#include "paged.cuh"

namespace eta {
namespace {

constexpr int kMergeWarps = 4;

template <int E, bool BF16>   // E = d / 32 columns per lane
__global__ void __launch_bounds__(32 * kMergeWarps) paged_merge_kernel(const PagedParams p, int ctas) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PagedHdr hd = paged_read_header(p, 2 * c + 1);
    const int row0 = blockIdx.y * kMergeWarps + warp;
    if (hd.rows > 0) {
        // parts after the first: CTAs c + 1 .. last
        int last = c;
        for (int k0 = c + 1; k0 < ctas; k0 += 32) {
            PagedHdr hk{0, 0, 0, 0};
            if (k0 + lane < ctas) hk = paged_read_header(p, 2 * (k0 + lane));
            const uint32_t ends = __ballot_sync(0xffffffffu, hk.rows > 0 && hk.last);
            if (ends) {
                last = k0 + __ffs(ends) - 1;
                break;
            }
            last = min(k0 + 31, ctas - 1);
        }
        const int parts = last - c + 1;
        // slot of part s (0: the one that begins the unit); -1: that CTA had no share
        auto slot_of = [&](int s) { return s == 0 ? 2 * c + 1 : 2 * (c + s); };
        for (int row = row0; row < hd.rows; row += gridDim.y * kMergeWarps) {
            float M = -INFINITY;
            for (int s = lane; s < parts; s += 32) {
                const int sl = slot_of(s);
                if (s == 0 || paged_read_header(p, sl).rows > 0)
                    M = fmaxf(M, __ldcg(p.part_m + static_cast<size_t>(sl) * p.part_rows + row));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            const float mu = M == -INFINITY ? 0.f : M;
            float L = 0.f, acc[E];
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = 0.f;
            for (int s0 = 0; s0 < parts; s0 += 32) {
                float w = 0.f, l = 0.f;
                const int s = s0 + lane;
                if (s < parts) {
                    const int sl = slot_of(s);
                    if (s == 0 || paged_read_header(p, sl).rows > 0) {
                        const size_t at = static_cast<size_t>(sl) * p.part_rows + row;
                        const float m = __ldcg(p.part_m + at);
                        w = m == -INFINITY ? 0.f : ex2(m - mu);
                        l = __ldcg(p.part_l + at);
                    }
                }
                float wl = w == 0.f ? 0.f : w * l;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) wl += __shfl_xor_sync(0xffffffffu, wl, o);
                L += wl;
                const int cnt = min(32, parts - s0);
                for (int q0 = 0; q0 < cnt; q0 += 8) {
                    float v[8][E], ws[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        ws[q] = __shfl_sync(0xffffffffu, w, (q0 + q) & 31);
                        if (q0 + q >= cnt) ws[q] = 0.f;
                        const float *src = p.part_o +
                                           (static_cast<size_t>(slot_of(s0 + min(q0 + q, cnt - 1))) * p.part_rows + row) * p.d +
                                           E * lane;
#pragma unroll
                        for (int e = 0; e < E; ++e) v[q][e] = ws[q] != 0.f ? __ldcg(src + e) : 0.f;
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q)
#pragma unroll
                        for (int e = 0; e < E; ++e) acc[e] = fmaf(ws[q], v[q][e], acc[e]);
                }
            }
            const float inv = L > 0.f ? 1.f / L : 0.f;
            const long long tok = hd.tok0 + row / p.gm.g;
            const int head = hd.head * p.gm.g + row % p.gm.g;
            const long long at = tok * p.o_token + static_cast<long long>(head) * p.o_head + E * lane;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if constexpr (BF16) static_cast<__nv_bfloat16 *>(p.O)[at + e] = __float2bfloat16_rn(acc[e] * inv);
                else static_cast<float *>(p.O)[at + e] = acc[e] * inv;
            }
            if (lane == 0 && p.LSE) p.LSE[tok * p.Hq + head] = L > 0.f ? (M + log2f(L)) * kPagedLn2 : -INFINITY;
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int E, bool BF16>
int launch_one(const PagedParams &p, int ctas, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    // up to 16 rows to a block: few blocks leave at once when nothing was cut
    const int rows_y = (p.part_rows + 4 * kMergeWarps - 1) / (4 * kMergeWarps);
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(rows_y));
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
    return static_cast<long long>(g) * max_q <= 64 ? Path::kDecode : Path::kTc;
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

// Attention of a few new tokens over a paged cache, float32: IEEE products and
// sums (no TF32), exponentials from ex2.approx (relative error 2^-22 at most):
// units (paged_index.h) of at most R = 4 or 8 query rows.
//
// The work is one pass over K and V, bound by HBM, so a warp streams keys from
// global memory into registers, and a row of K lies across the lanes that hold
// the same columns of every query row: no shared memory and no barrier between
// the loads and the products.  The warps of a CTA take batches of 32 / R keys of
// a unit in turn, each with a running maximum m, sum l and output of its own,
// joined at the unit's end:
//   S      each lane multiplies its four columns: R x (32 / R) partial sums, which a
//          halving exchange over the lanes turns into one score to a lane (31
//          shuffles for 32 scores of 32 lanes);
//   P V    the lane's four columns again; p comes back to all lanes through 128
//          bytes of shared memory.
// A lane has 4 columns, so d < 128 puts several keys side by side (d 64: two, d
// 32: four; at d 96 a quarter of the lanes repeats others' work).  K of the next batch
// is on its way while P V runs, V during the next scores: 1 KB a warp (d 32, 8 rows:
// one load a lane of each) to 8 KB (d 128, 4 rows), 12 or 16 warps an SM.
// A batch lies in one page (pages begin at multiples of 16), looked up two
// batches ahead.  Keys past the end and of missing pages are not read (zeros);
// keys a row does not see have score -inf.
//
// Measured, 32 sequences of 8000 tokens, 4 rows: d 128, 4 kv heads: 1.05 GB in 160 us, 0.98 of
// the measured copy rate (units of 16 rows in the tiling kernel: 365); d 64, 8 heads:
// 166 us (366); d 96, 4 heads: 130 us, 0.91; d 32, 16 heads: 200 us, 0.79.  8 rows: d 128 206
// us, 0.76; d 96 203, 0.58; d 64 258, 0.61; d 32 372, 0.42: twice the products and
// half the bytes on their way (and at d 64 148 bytes of spills a thread; 57 % of the
// issue slots are used).
#include <algorithm>

#include "launch.cuh"
#include "paged.cuh"

namespace eta {
namespace {

constexpr int kFewWarps = 4;
constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kFewTile = 64;   // keys of a tile (the partition's step)

template <int E, int R>   // E = d / 32, R: rows of a unit
struct FewShape {
    static constexpr int D = 32 * E;
    static constexpr int NV = E >= 3 ? 32 : 8 * E;   // lanes of a key, rounded to a power of two
    static constexpr int SIDE = 32 / NV;                 // keys side by side
    static constexpr int NK = NV / R;                    // loads of a batch
    static constexpr int KEYS = NK * SIDE;               // keys of a batch: 32 / R
    // on an SM; registers decide (32 x 8000 tokens, 4 rows, d 128: three 160 us, four,
    // which spill, 191; d 64: 175 and 166)
    static constexpr int CTAS = E >= 3 ? 3 : 4;
    static_assert(KEYS == 32 / R && NK >= 1, "a score to a lane");
};

template <int E, int R>
__global__ void __launch_bounds__(kFewThreads, FewShape<E, R>::CTAS) paged_few_kernel(const PagedParams p) {
    using S = FewShape<E, R>;
    constexpr int D = S::D, NV = S::NV, SIDE = S::SIDE, NK = S::NK, KEYS = S::KEYS;
    __shared__ PagedUnit unit;
    __shared__ __align__(16) float p_sh[kFewWarps][32];
    __shared__ float m_sh[kFewWarps][R], l_sh[kFewWarps][R];
    __shared__ __align__(16) float o_sh[kFewWarps][R][D];
    const PagedGeom &gm = p.gm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    const int side = lane / NV, col = 4 * (lane % NV);   // the lane's key among SIDE, its columns
    const bool has = col < D;
    const int my_row = lane % R, my_key = (lane % NV) / R * SIDE + side;   // whose score the lane ends up with
    paged_touch(p);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float *Q = static_cast<const float *>(p.Q);
    const float *K = static_cast<const float *>(p.K);
    const float *V = static_cast<const float *>(p.V);
    PagedFeed feed;   // (warp 0)
    if (warp == 0) feed.start(p, cta, gridDim.x);
    for (;;) {
        __syncthreads();   // the unit before is done with
        if (warp == 0) {
            PagedUnit w;
            feed.next(p, cta, w);
            if (w.tiles > 0) feed.report(p, w);
            if (lane == 0) unit = w;
        }
        __syncthreads();
        const PagedUnit w = unit;
        if (w.tiles == 0) break;
        const int rows = w.ntok * gm.g;
        float q[R][4], o[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows && has) {
                const int tr = paged_token(gm, r);
                v = __ldg(reinterpret_cast<const float4 *>(
                    Q + (w.tok0 + tr) * p.q_token + static_cast<long long>(w.head * gm.g + r - tr * gm.g) * p.q_head + col));
            }
            q[r][0] = v.x * p.scale_log2;
            q[r][1] = v.y * p.scale_log2;
            q[r][2] = v.z * p.scale_log2;
            q[r][3] = v.w * p.scale_log2;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][e] = 0.f;
        }
        const int vis = my_row < rows ? paged_unit_visible(gm, w, paged_token(gm, my_row)) : 0;
        float m = -INFINITY, l = 0.f;   // of row my_row; l: of this lane's keys
        // keys of this part that some row sees; those of this warp
        const int end = min(paged_unit_visible(gm, w, w.ntok - 1), (w.tile0 + w.tiles) * kFewTile);
        constexpr int STEP = KEYS * kFewWarps;
        const int begin = w.tile0 * kFewTile + warp * KEYS;
        auto lookup = [&](int key0) -> int {   // the batch's page, -1: none
            if (key0 >= end) return -1;
            const int id = paged_page(gm, w.seq, key0 >> gm.page_shift);
            if (id < 0 && lane == 0) atomicOr(p.err, kErrWordBadRow);
            return id;
        };
        // (lanes without columns read what others do: their q is zero, their o unused)
        const long long lane_at = w.head * p.head_stride + side * p.slot_stride + (has ? col : 0);
        const long long step = SIDE * p.slot_stride;
        auto load = [&](float4 (&x)[NK], const float *pool, int key0, int id) {
            const float *at = pool + id * p.page_stride + (key0 & (gm.page_size - 1)) * p.slot_stride + lane_at;
            if (id >= 0 && key0 + KEYS <= w.len) {
#pragma unroll
                for (int k = 0; k < NK; ++k) x[k] = __ldg(reinterpret_cast<const float4 *>(at + k * step));
            } else {
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (id >= 0 && key0 + k * SIDE + side < w.len) x[k] = __ldg(reinterpret_cast<const float4 *>(at + k * step));
                }
            }
        };
        int id0 = lookup(begin), id1 = lookup(begin + STEP);
        float4 kf[NK], vf[NK];
        load(kf, K, begin, id0);
        load(vf, V, begin, id0);
        for (int key0 = begin; key0 < end; key0 += STEP) {
            const int id2 = lookup(key0 + 2 * STEP);
            // S: value i = k R + r is row r against load k (the first exchange at
            // once, so that half as many are held)
            auto dot = [&](int i) {
                const float4 &x = kf[i / R];
                const float *y = q[i % R];
                return fmaf(y[3], x.w, fmaf(y[2], x.z, fmaf(y[1], x.y, y[0] * x.x)));
            };
            auto trade = [&](float lo, float hi, int h) {
                const bool up = lane & h;
                return (up ? hi : lo) + __shfl_xor_sync(0xffffffffu, up ? lo : hi, h);
            };
            float s[NV / 2];
#pragma unroll
            for (int i = 0; i < NV / 2; ++i) s[i] = trade(dot(i), dot(i + NV / 2), NV / 2);
            load(kf, K, key0 + STEP, id1);
#pragma unroll
            for (int h = NV / 4; h > 0; h >>= 1)
#pragma unroll
                for (int i = 0; i < h; ++i) s[i] = trade(s[i], s[i + h], h);
            const float x = id0 >= 0 && key0 + my_key < vis ? s[0] : -INFINITY;
            float mx = x;
#pragma unroll
            for (int h = R; h < 32; h <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, h));
            const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
            const float al = m == -INFINITY ? 0.f : ex2(m - mu), pr = ex2(x - mu);
            l = l * al + pr;
            if (__any_sync(0xffffffffu, mn != m)) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float ar = __shfl_sync(0xffffffffu, al, r);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[r][e] *= ar;
                }
            }
            m = mn;
            p_sh[warp][lane] = pr;
            __syncwarp();
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
                for (int r4 = 0; r4 < R; r4 += 4) {
                    const float4 pp = *reinterpret_cast<const float4 *>(&p_sh[warp][side * NV + k * R + r4]);
                    const float pv[4] = {pp.x, pp.y, pp.z, pp.w};
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        o[r4 + r][0] = fmaf(pv[r], vf[k].x, o[r4 + r][0]);
                        o[r4 + r][1] = fmaf(pv[r], vf[k].y, o[r4 + r][1]);
                        o[r4 + r][2] = fmaf(pv[r], vf[k].z, o[r4 + r][2]);
                        o[r4 + r][3] = fmaf(pv[r], vf[k].w, o[r4 + r][3]);
                    }
                }
            __syncwarp();   // p has been read
            load(vf, V, key0 + STEP, id1);
            id0 = id1;
            id1 = id2;
        }
        // the warps' parts
#pragma unroll
        for (int h = R; h < 32; h <<= 1) l += __shfl_xor_sync(0xffffffffu, l, h);
        if (lane < R) {
            m_sh[warp][lane] = paged_part_max(m, l);
            l_sh[warp][lane] = l;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int h = NV; h < 32; h <<= 1) o[r][e] += __shfl_xor_sync(0xffffffffu, o[r][e], h);
            if (side == 0 && has) *reinterpret_cast<float4 *>(&o_sh[warp][r][col]) = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
        }
        __syncthreads();
        const bool whole = w.slot < 0;
        for (int i = tid; i < rows * (D / 4); i += kFewThreads) {
            const int r = i / (D / 4), c = 4 * (i % (D / 4));
            float M = -INFINITY;
#pragma unroll
            for (int x = 0; x < kFewWarps; ++x) M = fmaxf(M, m_sh[x][r]);
            float L = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
            if (M != -INFINITY) {
#pragma unroll
                for (int x = 0; x < kFewWarps; ++x) {
                    if (m_sh[x][r] == -INFINITY) continue;   // (a warp without keys)
                    const float wx = ex2(m_sh[x][r] - M);
                    const float4 v = *reinterpret_cast<const float4 *>(&o_sh[x][r][c]);
                    L = fmaf(wx, l_sh[x][r], L);
                    a[0] = fmaf(wx, v.x, a[0]);
                    a[1] = fmaf(wx, v.y, a[1]);
                    a[2] = fmaf(wx, v.z, a[2]);
                    a[3] = fmaf(wx, v.w, a[3]);
                }
            }
            const int tr = paged_token(gm, r);
            const long long tok = w.tok0 + tr;
            const int head = w.head * gm.g + r - tr * gm.g;
            const size_t prow = static_cast<size_t>(whole ? 0 : w.slot) * p.part_rows + r;
            const float inv = !whole ? 1.f : L != 0.f ? 1.f / L : 0.f;   // (a NaN goes on)
            float *dst = whole ? static_cast<float *>(p.O) + tok * p.o_token + static_cast<long long>(head) * p.o_head
                               : p.part_o + prow * D;
            *reinterpret_cast<float4 *>(dst + c) = make_float4(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
            if (c == 0) {
                if (!whole) {
                    p.part_m[prow] = paged_part_max(M, L);
                    p.part_l[prow] = L;
                } else if (p.LSE) {
                    p.LSE[tok * p.Hq + head] = L != 0.f ? (M + log2f(L)) * kPagedLn2 : -INFINITY;
                }
            }
        }
    }
    if (warp == 0) feed.finish(p, cta);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int E, int R>
int launch_one(PagedParams &p, void *workspace, cudaStream_t stream) {
    auto kern = paged_few_kernel<E, R>;
    int dev = 0, nsm = 0, per_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kFewThreads, 0) != cudaSuccess)
        return kErrCuda;
    const int ctas = std::min(std::max(per_sm, 1) * std::max(nsm, 1), kPagedMaxSimtCtas);
    p.gm.tpu = R / p.gm.g;
    p.gm.tk = kFewTile;
    p.gm.unit_cost = kFewTile;
    p.gm.min_share = 2 * kFewTile;   // (4 x 600 tokens: 12.7 us, twice that share 15.6)
    paged_derive(p.gm);
    paged_carve(p, workspace, ctas, R);
    const int rc = launch_dependent(kern, dim3(static_cast<unsigned>(ctas)), kFewThreads, 0, stream, p);
    if (rc != kOk) return rc;
    return launch_paged_merge(p, 0, ctas, nsm, stream);
}

template <int E>
int launch_rows(PagedParams &p, void *workspace, cudaStream_t stream) {
    return paged_simt_rows(p.gm.g, p.gm.max_q) == 4 ? launch_one<E, 4>(p, workspace, stream)
                                                    : launch_one<E, 8>(p, workspace, stream);
}

}  // namespace

int launch_paged_few(PagedParams p, void *workspace, cudaStream_t stream) {
    switch (p.d) {
        case 32: return launch_rows<1>(p, workspace, stream);
        case 64: return launch_rows<2>(p, workspace, stream);
        case 96: return launch_rows<3>(p, workspace, stream);
        case 128: return launch_rows<4>(p, workspace, stream);
        default: return kErrUnsupported;
    }
}

}  // namespace eta

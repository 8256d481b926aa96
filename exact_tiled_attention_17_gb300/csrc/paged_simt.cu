// Attention of new tokens over a paged cache on the CUDA cores, float32: IEEE
// products and sums (no TF32), exponentials from ex2.approx (relative error
// 2^-22 at most).
//
// O = softmax(scale Q K^T) V of each unit (paged_index.h: one kv head, a block
// of new tokens, all query heads of the group), key tile by key tile with the
// running maximum m and sum l of the online softmax.
//
// A CTA of 128 threads walks its share of the units.  Q, a tile of keys and
// its values are staged in shared memory; S and O are register tiles: 4 rows x
// 8 (d > 64: 4) keys, and 4 rows x d / 8 columns, of a thread in units of 64 rows.
// What bounds it is the multiply-add rate (1.07 GFLOP of the 200-token case below
// are 14 us), so both products run on packed pairs (fma.rn.f32x2): S pairs up
// along d, O along its rows, for which P lies key by key in shared memory.  Tiles
// are fetched with cp.async while the other product runs: K of the next tile
// during softmax and P V, V during Q K^T.
// Measured (4 x 256 tokens over 2000, 16 query heads): d 64 208 us, d 128 380, 41
// TFLOP/s; 3 x 77 .. 200 tokens over 700 .. 1500, 8 heads of 64: 47 us.  What is
// left is latency: two or three warps of a scheduler fit, and what hides it best is
// to unroll (both products by 16 steps: 208 us, by 4: 222).  16 threads along
// the keys instead of 8 (8 x 4 register tiles): 205 us at d 64, but 393 at 128 and 156
// for 125 at 32.
// Keys of pages that do not exist, and keys a row does not see, have score
// -inf; what is not a token of the sequence is fetched as zero.
#include <algorithm>

#include "launch.cuh"
#include "paged.cuh"

namespace eta {
namespace {

constexpr int kSimtThreads = 128;

template <int E, int RT>   // E = d / 32, RT: query rows of a unit
struct SimtShape {
    static constexpr int D = 32 * E;
    static constexpr int KT = RT == 64 && D > 64 ? 32 : 64;   // keys of a tile: two CTAs fit an SM (d = 128: 456 us with
                                                              // units of 32 rows and tiles of 64 keys instead, 376)
    static constexpr int TX = RT == 16 ? 16 : 8, TY = 128 / TX;   // threads along keys and columns, along rows
    static constexpr int LD = D + 4;               // padded rows: lanes reading different rows spread over the banks
    static constexpr int LP = RT + 4;              // P: [key][row]
    static constexpr int RR = RT / TY, KB = KT / TX, NC = (D + 4 * TX - 1) / (4 * TX);   // rows, keys, 4-column pieces of a thread
    static constexpr int FLOATS = RT * LD + 2 * KT * LD + KT * LP;
    static constexpr int SMEM = FLOATS * 4 + 2 * KT * 8;
    static constexpr int CTAS = (RT < 64 || KT < 64) && SMEM <= 74 * 1024 ? 3 : SMEM <= 112 * 1024 ? 2 : 1;   // at least, on an SM
};

// 16 bytes from global to shared memory; zeros if !in.
__device__ __forceinline__ void copy16(float *dst, const float *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ ulonglong2 load2(const float *p) { return *reinterpret_cast<const ulonglong2 *>(p); }

template <int E, int RT>
__global__ void __launch_bounds__(kSimtThreads, SimtShape<E, RT>::CTAS) paged_simt_kernel(const PagedParams p) {
    using S = SimtShape<E, RT>;
    constexpr int D = S::D, LD = S::LD, LP = S::LP, RR = S::RR, KT = S::KT, KB = S::KB, TX = S::TX, NC = S::NC;
    extern __shared__ __align__(16) float smem[];
    __shared__ PagedUnit unit;
    __shared__ int gaps[2][KT / 32];   // whether a tile has keys of missing pages
    float *qs = smem, *ks = qs + RT * LD, *vs = ks + KT * LD, *ps = vs + KT * LD;
    long long *key_at = reinterpret_cast<long long *>(ps + KT * LP);   // [2]: offset of each key's row, or -1
    const PagedGeom &gm = p.gm;
    const int tid = threadIdx.x, tx = tid % TX, ty = tid / TX;
    const int cta = blockIdx.x;
    paged_touch(p);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float *Q = static_cast<const float *>(p.Q);
    const float *K = static_cast<const float *>(p.K);
    const float *V = static_cast<const float *>(p.V);
    PagedFeed feed;   // (warp 0)
    if (tid < 32) feed.start(p, cta, gridDim.x);
    for (;;) {
        __syncthreads();   // the unit before is done with
        if (tid < 32) {
            PagedUnit w;
            feed.next(p, cta, w);
            if (w.tiles > 0) feed.report(p, w);
            if (tid == 0) unit = w;
        }
        __syncthreads();
        const PagedUnit w = unit;
        if (w.tiles == 0) break;
        const int rows = w.ntok * gm.g, tok0 = w.tok0, t1 = w.tile0 + w.tiles;
        const int vis_all = paged_unit_visible(gm, w, 0);   // what every row sees
        // where the keys of tile t lie
        auto places = [&](int t) {
            if (tid < KT && t < t1) {
                const int key = t * KT + tid;
                long long at = -1;
                bool gap = false;
                if (key < w.len) {
                    const int id = paged_page(gm, w.seq, key >> gm.page_shift);
                    gap = id < 0;
                    if (!gap) at = id * p.page_stride + (key & (gm.page_size - 1)) * p.slot_stride + w.head * p.head_stride;
                    else atomicOr(p.err, kErrWordBadRow);
                }
                key_at[(t & 1) * KT + tid] = at;
                const bool any = __any_sync(0xffffffffu, gap);
                if ((tid & 31) == 0) gaps[t & 1][tid >> 5] = any;
            }
        };
        auto fetch = [&](float *dst, const float *src, int t) {
            if (t < t1) {
#pragma unroll 4
                for (int i = tid; i < KT * (D / 4); i += kSimtThreads) {
                    const int r = i / (D / 4), c = 4 * (i % (D / 4));
                    const long long at = key_at[(t & 1) * KT + r];
                    copy16(dst + r * LD + c, at >= 0 ? src + at + c : src, at >= 0);
                }
            }
            copy_commit();   // (a group every time, so that the counts below hold)
        };
        places(w.tile0);
        __syncthreads();
        fetch(ks, K, w.tile0);
        fetch(vs, V, w.tile0);
        for (int i = tid; i < RT * (D / 4); i += kSimtThreads) {
            const int r = i / (D / 4), c = 4 * (i % (D / 4));
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int tr = paged_token(gm, r);
                v = __ldg(reinterpret_cast<const float4 *>(
                    Q + (tok0 + tr) * p.q_token + static_cast<long long>(w.head * gm.g + r - tr * gm.g) * p.q_head + c));
            }
            *reinterpret_cast<float4 *>(qs + r * LD + c) = v;
        }
        int vis[RR];   // keys that this thread's rows see
        float m[RR], l[RR];
        uint64_t o[RR / 2][NC][4];   // pairs of rows
#pragma unroll
        for (int a = 0; a < RR; ++a) {
            const int r = ty * RR + a;
            vis[a] = r < rows ? paged_unit_visible(gm, w, paged_token(gm, r)) : 0;
            m[a] = -INFINITY;
            l[a] = 0.f;
        }
#pragma unroll
        for (int a = 0; a < RR / 2; ++a)
#pragma unroll
            for (int b = 0; b < NC; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[a][b][e] = 0ull;
        for (int t = w.tile0; t < t1; ++t) {
            const int key0 = t * KT;
            places(t + 1);
            copy_wait<1>();    // K has landed (V may be on its way)
            __syncthreads();
            // S: rows ty * RR + a, keys tx + TX b
            float s[RR][KB];
            {
                uint64_t acc[RR][KB];
#pragma unroll
                for (int a = 0; a < RR; ++a)
#pragma unroll
                    for (int b = 0; b < KB; ++b) acc[a][b] = 0ull;
#pragma unroll 16
                for (int c = 0; c < D; c += 4) {
                    ulonglong2 kf[KB], qf[RR];
#pragma unroll
                    for (int b = 0; b < KB; ++b) kf[b] = load2(ks + (tx + TX * b) * LD + c);
#pragma unroll
                    for (int a = 0; a < RR; ++a) qf[a] = load2(qs + (ty * RR + a) * LD + c);
                    // (no product next to one that it depends on)
#pragma unroll
                    for (int a = 0; a < RR; ++a)
#pragma unroll
                        for (int b = 0; b < KB; ++b) acc[a][b] = f2_fma(qf[a].x, kf[b].x, acc[a][b]);
#pragma unroll
                    for (int a = 0; a < RR; ++a)
#pragma unroll
                        for (int b = 0; b < KB; ++b) acc[a][b] = f2_fma(qf[a].y, kf[b].y, acc[a][b]);
                }
#pragma unroll
                for (int a = 0; a < RR; ++a)
#pragma unroll
                    for (int b = 0; b < KB; ++b) {
                        float x, y;
                        f2_unpack(acc[a][b], x, y);
                        s[a][b] = (x + y) * p.scale_log2;
                    }
            }
            bool edge = key0 + KT > vis_all;
#pragma unroll
            for (int i = 0; i < KT / 32; ++i) edge = edge || gaps[t & 1][i];
            if (edge) {
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    const bool here = key_at[(t & 1) * KT + tx + TX * b] >= 0;
#pragma unroll
                    for (int a = 0; a < RR; ++a) s[a][b] = here && key0 + tx + TX * b < vis[a] ? s[a][b] : -INFINITY;
                }
            }
            __syncthreads();   // K has been read
            fetch(ks, K, t + 1);
            float alpha[RR];
#pragma unroll
            for (int a = 0; a < RR; ++a) {
                float mx = s[a][0];
#pragma unroll
                for (int b = 1; b < KB; ++b) mx = fmaxf(mx, s[a][b]);
#pragma unroll
                for (int q = 1; q < TX; q <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, q));
                const float mn = fmaxf(m[a], mx), mu = mn == -INFINITY ? 0.f : mn;
                const float al = m[a] == -INFINITY ? 0.f : ex2(m[a] - mu);
                m[a] = mn;
                float sum = 0.f;
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    s[a][b] = ex2(s[a][b] - mu);
                    sum += s[a][b];
                }
                l[a] = l[a] * al + sum;   // (this thread's keys; joined at the end)
                alpha[a] = al;
            }
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                float *at = ps + (tx + TX * b) * LP + ty * RR;
                if constexpr (RR >= 4) {
#pragma unroll
                    for (int a = 0; a < RR; a += 4)
                        *reinterpret_cast<float4 *>(at + a) = make_float4(s[a][b], s[a + 1][b], s[a + 2][b], s[a + 3][b]);
                } else {
                    *reinterpret_cast<float2 *>(at) = make_float2(s[0][b], s[1][b]);
                }
            }
#pragma unroll
            for (int a = 0; a < RR / 2; ++a) {
                if (alpha[2 * a] == 1.f && alpha[2 * a + 1] == 1.f) continue;
                const uint64_t a2 = f2_pack(alpha[2 * a], alpha[2 * a + 1]);
#pragma unroll
                for (int b = 0; b < NC; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[a][b][e] = f2_mul(o[a][b][e], a2);
            }
            copy_wait<1>();    // V has landed (the next K may be on its way)
            __syncthreads();
            // O: rows ty * RR + a, columns 4 tx + 4 TX b
#pragma unroll 16
            for (int k = 0; k < KT; ++k) {
                uint64_t pp[RR / 2];
                if constexpr (RR >= 4) {
#pragma unroll
                    for (int a = 0; a < RR / 2; a += 2) {
                        const ulonglong2 v = load2(ps + k * LP + ty * RR + 2 * a);
                        pp[a] = v.x;
                        pp[a + 1] = v.y;
                    }
                } else {
                    pp[0] = *reinterpret_cast<const uint64_t *>(ps + k * LP + ty * RR);
                }
#pragma unroll
                for (int b = 0; b < NC; ++b) {
                    const int c = 4 * tx + 4 * TX * b;
                    const float4 v = (D % (4 * TX) == 0 || c < D) ? *reinterpret_cast<const float4 *>(vs + k * LD + c)
                                                                  : make_float4(0.f, 0.f, 0.f, 0.f);
                    const uint64_t vv[4] = {f2_pack(v.x, v.x), f2_pack(v.y, v.y), f2_pack(v.z, v.z), f2_pack(v.w, v.w)};
#pragma unroll
                    for (int a = 0; a < RR / 2; ++a)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[a][b][e] = f2_fma(pp[a], vv[e], o[a][b][e]);
                }
            }
            __syncthreads();   // V has been read
            fetch(vs, V, t + 1);
        }
        copy_wait<0>();
        // the unit's rows, or this share's part of them
        const bool whole = w.slot < 0;
        const int slot = whole ? 0 : w.slot;
#pragma unroll
        for (int a = 0; a < RR; ++a) {
            float sum = l[a];
#pragma unroll
            for (int q = 1; q < TX; q <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, q);
            const int r = ty * RR + a;
            if (r >= rows) continue;
            const int tr = paged_token(gm, r);
            const long long tok = tok0 + tr;
            const int head = w.head * gm.g + r - tr * gm.g;
            const size_t prow = static_cast<size_t>(slot) * p.part_rows + r;
            const float inv = !whole ? 1.f : sum != 0.f ? 1.f / sum : 0.f;   // (a NaN goes on)
            float *dst = whole ? static_cast<float *>(p.O) + tok * p.o_token + static_cast<long long>(head) * p.o_head
                               : p.part_o + prow * D;
#pragma unroll
            for (int b = 0; b < NC; ++b) {
                const int c = 4 * tx + 4 * TX * b;
                if (D % (4 * TX) != 0 && c >= D) continue;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float lo, hi;
                    f2_unpack(o[a / 2][b][e], lo, hi);
                    v[e] = (a & 1 ? hi : lo) * inv;
                }
                *reinterpret_cast<float4 *>(dst + c) = make_float4(v[0], v[1], v[2], v[3]);
            }
            if (tx == 0) {
                if (!whole) {
                    p.part_m[prow] = paged_part_max(m[a], sum);
                    p.part_l[prow] = sum;
                } else if (p.LSE) {
                    p.LSE[tok * p.Hq + head] = sum != 0.f ? (m[a] + log2f(sum)) * kPagedLn2 : -INFINITY;
                }
            }
        }
    }
    if (tid < 32) feed.finish(p, cta);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int E, int RT>
int launch_one(PagedParams &p, void *workspace, cudaStream_t stream) {
    using S = SimtShape<E, RT>;
    auto kern = paged_simt_kernel<E, RT>;
    int dev = 0, nsm = 0, per_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kSimtThreads, S::SMEM) != cudaSuccess)
        return kErrCuda;
    const int ctas = std::min(std::max(per_sm, 1) * std::max(nsm, 1), kPagedMaxSimtCtas);
    p.gm.tpu = RT / p.gm.g;
    p.gm.tk = S::KT;
    p.gm.unit_cost = S::KT;
    p.gm.min_share = 128;
    paged_derive(p.gm);
    paged_carve(p, workspace, ctas, RT);
    const int rc = launch_dependent(kern, dim3(static_cast<unsigned>(ctas)), kSimtThreads, S::SMEM, stream, p);
    if (rc != kOk) return rc;
    return launch_paged_merge(p, 0, ctas, nsm, stream);
}

}  // namespace

template <int E>
static int launch_rows(PagedParams &p, void *workspace, cudaStream_t stream) {
    switch (paged_simt_rows(p.gm.g, p.gm.max_q)) {
        case 16: return launch_one<E, 16>(p, workspace, stream);
        case 32: return launch_one<E, 32>(p, workspace, stream);
        default: return launch_one<E, 64>(p, workspace, stream);
    }
}

int launch_paged_simt(PagedParams p, void *workspace, cudaStream_t stream) {
    switch (p.d) {
        case 32: return launch_rows<1>(p, workspace, stream);
        case 64: return launch_rows<2>(p, workspace, stream);
        case 96: return launch_rows<3>(p, workspace, stream);
        case 128: return launch_rows<4>(p, workspace, stream);
        default: return kErrUnsupported;
    }
}

}  // namespace eta

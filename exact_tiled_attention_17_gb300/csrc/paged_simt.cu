// Attention of new tokens over a paged cache on the CUDA cores: IEEE float32
// throughout (no TF32), float32 storage.
//
// O = softmax(scale Q K^T) V of each unit (paged_index.h: one kv head, a block
// of new tokens, all query heads of the group), key tile by key tile with the
// running maximum m and sum l of the online softmax.
//
// A CTA of 256 threads walks its share of the units.  Q rows, a tile of 64
// keys and its values are staged in shared memory as float32; S is a register
// tile of RT/16 rows x 4 keys per thread, P goes through shared memory and O
// is a register tile of RT/16 rows x d/16 columns.  Keys of pages that do not
// exist, and keys a row does not see, have score -inf and value 0.
#include "paged.cuh"

namespace eta {
namespace {

constexpr int kSimtThreads = 256;
constexpr int kSimtKeys = 64;

__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ void fma4(float4 a, float4 b, float &s) {
    s = fmaf(a.x, b.x, s);
    s = fmaf(a.y, b.y, s);
    s = fmaf(a.z, b.z, s);
    s = fmaf(a.w, b.w, s);
}

template <int E, int RT>   // E = d / 32, RT: query rows of a unit
struct SimtShape {
    static constexpr int D = 32 * E;
    static constexpr int LD = D + 4;          // padded rows: 16 lanes reading 16 rows meet no bank twice
    static constexpr int LP = kSimtKeys + 4;
    static constexpr int FLOATS = RT * LD + 2 * kSimtKeys * LD + RT * LP;
    static constexpr int SMEM = FLOATS * 4 + kSimtKeys * 8;
};

template <int E, int RT>
__global__ void __launch_bounds__(kSimtThreads) paged_simt_kernel(const PagedParams p) {
    using S = SimtShape<E, RT>;
    constexpr int D = S::D, LD = S::LD, LP = S::LP, RR = RT / 16;
    extern __shared__ __align__(16) float smem[];
    __shared__ PagedUnit unit;
    float *qs = smem, *ks = qs + RT * LD, *vs = ks + kSimtKeys * LD, *ps = vs + kSimtKeys * LD;
    long long *key_at = reinterpret_cast<long long *>(ps + RT * LP);   // offset of each key's row, or -1
    const PagedGeom &gm = p.gm;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
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
        const int rows = w.ntok * gm.g, tok0 = w.tok0;
        for (int i = tid; i < RT * (D / 4); i += kSimtThreads) {
            const int r = i / (D / 4), c = 4 * (i % (D / 4));
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows)
                v = load4(Q + (tok0 + paged_token(gm, r)) * p.q_token + static_cast<long long>(w.head * gm.g + (r - paged_token(gm, r) * gm.g)) * p.q_head + c);
            *reinterpret_cast<float4 *>(qs + r * LD + c) = v;
        }
        int vis[RR];   // keys that this thread's rows see
        float m[RR], l[RR];
        float4 o[RR][E == 1 ? 1 : (E + 1) / 2];
        static_assert(D / 64 <= 2, "columns per thread");
#pragma unroll
        for (int a = 0; a < RR; ++a) {
            const int r = ty * RR + a;
            vis[a] = r < rows ? paged_unit_visible(gm, w, paged_token(gm, r)) : 0;
            m[a] = -INFINITY;
            l[a] = 0.f;
#pragma unroll
            for (int b = 0; b < (E + 1) / 2; ++b) o[a][b] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int t = w.tile0; t < w.tile0 + w.tiles; ++t) {
            const int key0 = t * kSimtKeys;
            __syncthreads();   // the previous tile has been read
            if (tid < kSimtKeys) {
                const int key = key0 + tid;
                long long at = -1;
                if (key < w.len) {
                    const int id = paged_page(gm, w.seq, key >> gm.page_shift);
                    if (id >= 0) at = id * p.page_stride + (key & (gm.page_size - 1)) * p.slot_stride + w.head * p.head_stride;
                    else atomicOr(p.err, kErrWordBadRow);
                }
                key_at[tid] = at;
            }
            __syncthreads();
            for (int i = tid; i < kSimtKeys * (D / 4); i += kSimtThreads) {
                const int r = i / (D / 4), c = 4 * (i % (D / 4));
                const long long at = key_at[r];
                float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
                if (at >= 0) {
                    kv = load4(K + at + c);
                    vv = load4(V + at + c);
                }
                *reinterpret_cast<float4 *>(ks + r * LD + c) = kv;
                *reinterpret_cast<float4 *>(vs + r * LD + c) = vv;
            }
            __syncthreads();
            // S: rows ty * RR + a, keys tx + 16 b
            float s[RR][4];
#pragma unroll
            for (int a = 0; a < RR; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) s[a][b] = 0.f;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                float4 kf[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) kf[b] = *reinterpret_cast<const float4 *>(ks + (tx + 16 * b) * LD + c);
#pragma unroll
                for (int a = 0; a < RR; ++a) {
                    const float4 qf = *reinterpret_cast<const float4 *>(qs + (ty * RR + a) * LD + c);
#pragma unroll
                    for (int b = 0; b < 4; ++b) fma4(qf, kf[b], s[a][b]);
                }
            }
            bool here[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) here[b] = key_at[tx + 16 * b] >= 0;
#pragma unroll
            for (int a = 0; a < RR; ++a) {
                float mx = -INFINITY;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    s[a][b] = here[b] && key0 + tx + 16 * b < vis[a] ? s[a][b] * p.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, s[a][b]);
                }
#pragma unroll
                for (int q = 1; q < 16; q <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, q));
                const float mn = fmaxf(m[a], mx), mu = mn == -INFINITY ? 0.f : mn;
                const float al = m[a] == -INFINITY ? 0.f : exp2f(m[a] - mu);
                m[a] = mn;
                float sum = 0.f;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float e = exp2f(s[a][b] - mu);
                    sum += e;
                    ps[(ty * RR + a) * LP + tx + 16 * b] = e;
                }
#pragma unroll
                for (int q = 1; q < 16; q <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, q);
                l[a] = l[a] * al + sum;
#pragma unroll
                for (int b = 0; b < (E + 1) / 2; ++b) {
                    o[a][b].x *= al;
                    o[a][b].y *= al;
                    o[a][b].z *= al;
                    o[a][b].w *= al;
                }
            }
            __syncwarp();   // a row's P is written and read by the same half-warp
            // O: rows ty * RR + a, columns 4 tx + 64 b
#pragma unroll 4
            for (int k = 0; k < kSimtKeys; ++k) {
                float4 vf[(E + 1) / 2];
#pragma unroll
                for (int b = 0; b < (E + 1) / 2; ++b) {
                    const int c = 4 * tx + 64 * b;
                    vf[b] = c < D ? *reinterpret_cast<const float4 *>(vs + k * LD + c) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int a = 0; a < RR; ++a) {
                    const float e = ps[(ty * RR + a) * LP + k];
#pragma unroll
                    for (int b = 0; b < (E + 1) / 2; ++b) {
                        o[a][b].x = fmaf(e, vf[b].x, o[a][b].x);
                        o[a][b].y = fmaf(e, vf[b].y, o[a][b].y);
                        o[a][b].z = fmaf(e, vf[b].z, o[a][b].z);
                        o[a][b].w = fmaf(e, vf[b].w, o[a][b].w);
                    }
                }
            }
        }
        // the unit's rows, or this share's part of them
        const bool whole = w.slot < 0;
        const int slot = whole ? 0 : w.slot;
#pragma unroll
        for (int a = 0; a < RR; ++a) {
            const int r = ty * RR + a;
            if (r >= rows) continue;
            const long long tok = tok0 + paged_token(gm, r);
            const int head = w.head * gm.g + (r - paged_token(gm, r) * gm.g);
            const float inv = l[a] > 0.f ? 1.f / l[a] : 0.f;
#pragma unroll
            for (int b = 0; b < (E + 1) / 2; ++b) {
                const int c = 4 * tx + 64 * b;
                if (c >= D) continue;
                float4 v = o[a][b];
                if (!whole) {
                    *reinterpret_cast<float4 *>(p.part_o + (static_cast<size_t>(slot) * p.part_rows + r) * D + c) = v;
                    continue;
                }
                v.x *= inv;
                v.y *= inv;
                v.z *= inv;
                v.w *= inv;
                *reinterpret_cast<float4 *>(static_cast<float *>(p.O) + tok * p.o_token +
                                            static_cast<long long>(head) * p.o_head + c) = v;
            }
            if (tx == 0) {
                if (!whole) {
                    p.part_m[static_cast<size_t>(slot) * p.part_rows + r] = m[a];
                    p.part_l[static_cast<size_t>(slot) * p.part_rows + r] = l[a];
                } else if (p.LSE) {
                    p.LSE[tok * p.Hq + head] = l[a] > 0.f ? (m[a] + log2f(l[a])) * kPagedLn2 : -INFINITY;
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
    const int ctas = min(max(per_sm, 1) * max(nsm, 1), kPagedMaxCtas);
    p.gm.tpu = RT / p.gm.g;
    p.gm.tk = kSimtKeys;
    p.gm.unit_cost = kSimtKeys;
    p.gm.min_share = 2 * kSimtKeys;
    paged_derive(p.gm);
    paged_carve(p, workspace, ctas, RT);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kSimtThreads);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return kErrCuda;
    return launch_paged_merge(p, 0, ctas, nsm, stream);
}

template <int RT>
int launch_d(PagedParams &p, void *workspace, cudaStream_t stream) {
    switch (p.d) {
        case 32: return launch_one<1, RT>(p, workspace, stream);
        case 64: return launch_one<2, RT>(p, workspace, stream);
        case 96: return launch_one<3, RT>(p, workspace, stream);
        case 128: return launch_one<4, RT>(p, workspace, stream);
        default: return kErrUnsupported;
    }
}

}  // namespace

int launch_paged_simt(PagedParams p, void *workspace, cudaStream_t stream) {
    // Units of 16 rows where an entry's rows fit, else of 64.
    const bool small = static_cast<long long>(p.gm.max_q) * p.gm.g <= 16;
    return small ? launch_d<16>(p, workspace, stream) : launch_d<64>(p, workspace, stream);
}

}  // namespace eta

// Attention of new tokens over a paged cache of 4-bit values (e2m1.cuh).
//
// A warp takes a query row and looks at one key after the other; a lane has d / 32
// columns.  Everything in float32.
#include "e2m1.cuh"
#include "launch.cuh"
#include "paged.cuh"

namespace eta {
namespace {

template <int E>
__device__ __forceinline__ void row_values(const char *blk, int page_size, int slot, float (&x)[E]) {
    constexpr int D = 32 * E;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = E * lane + e;
        const uint32_t byte = *reinterpret_cast<const uint8_t *>(blk + slot * (D / 2) + c / 2);
        const uint32_t s2 = e2m1_scale_h2(*reinterpret_cast<const uint8_t *>(blk + page_size * (D / 2) + slot * (D / 16) + c / 16));
        uint32_t h[4];
        e2m1_values(byte, s2, h);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(h));
        x[e] = c & 1 ? f.y : f.x;
    }
}

template <int E>
__global__ void __launch_bounds__(128) paged_e2m1_kernel(const PagedParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PagedGeom &gm = p.gm;
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row < static_cast<long long>(gm.T) * p.Hq) {
        const int t = static_cast<int>(row / p.Hq), hq = static_cast<int>(row % p.Hq), h = hq / gm.g;
        for (int i = 0; i < gm.n; ++i) {
            PagedEntry e;
            if (!paged_entry(gm, i, e) && row == 0 && lane == 0) atomicOr(p.err, kErrWordBadRow);
            if (t < e.q0 || t >= e.q0 + e.nq) continue;
            const int vis = paged_visible(gm, e, t - e.q0);
            float q[E], o[E], k[E], m = -INFINITY, l = 0.f;
            const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(p.Q) + t * p.q_token + hq * p.q_head;
#pragma unroll
            for (int c = 0; c < E; ++c) {
                q[c] = __bfloat162float(qp[E * lane + c]);
                o[c] = 0.f;
            }
            for (int j = 0; j < vis; ++j) {
                const int id = paged_page(gm, e.seq, j >> gm.page_shift), slot = j & (gm.page_size - 1);
                if (id < 0) {
                    if (lane == 0) atomicOr(p.err, kErrWordBadRow);
                    continue;
                }
                const long long at = id * p.page_stride + h * p.head_stride;
                row_values<E>(static_cast<const char *>(p.K) + at, gm.page_size, slot, k);
                float s = 0.f;
#pragma unroll
                for (int c = 0; c < E; ++c) s = fmaf(q[c], k[c], s);
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
                s *= p.scale_log2;
                const float mn = fmaxf(m, s), a = m == -INFINITY ? 0.f : ex2(m - mn), w = ex2(s - mn);
                m = mn;
                l = l * a + w;
                row_values<E>(static_cast<const char *>(p.V) + at, gm.page_size, slot, k);
#pragma unroll
                for (int c = 0; c < E; ++c) o[c] = fmaf(w, k[c], o[c] * a);
            }
            const float inv = l != 0.f ? 1.f / l : 0.f;
            __nv_bfloat16 *op = static_cast<__nv_bfloat16 *>(p.O) + t * p.o_token + hq * p.o_head;
#pragma unroll
            for (int c = 0; c < E; ++c) op[E * lane + c] = __float2bfloat16_rn(o[c] * inv);
            if (lane == 0 && p.LSE) p.LSE[static_cast<long long>(t) * p.Hq + hq] = l != 0.f ? (m + log2f(l)) * kPagedLn2 : -INFINITY;
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace

int launch_paged_e2m1(PagedParams p, void *, cudaStream_t stream) {
    p.gm.tpu = 1;
    p.gm.tk = 64;
    paged_derive(p.gm);
    const dim3 grid(static_cast<unsigned>((static_cast<long long>(p.gm.T) * p.Hq + 3) / 4));
    switch (p.d) {
        case 32: return launch_dependent(paged_e2m1_kernel<1>, grid, 128, 0, stream, p);
        case 64: return launch_dependent(paged_e2m1_kernel<2>, grid, 128, 0, stream, p);
        case 96: return launch_dependent(paged_e2m1_kernel<3>, grid, 128, 0, stream, p);
        default: return launch_dependent(paged_e2m1_kernel<4>, grid, 128, 0, stream, p);
    }
}

}  // namespace eta

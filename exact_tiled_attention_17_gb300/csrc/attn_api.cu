// C-ABI layer: argument validation, dispatch to the kernels, the device error
// word, status and error strings.  Declared in include/attn.h.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "../../include/attn.h"
#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace eta {

// One word per device that loads the library: kernels OR a code into it when
// a bounded wait gives up.
__device__ int g_error_word;

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_mu;
int *g_err_ptr[kMaxDevices];
EncodeTiledFn g_encode = nullptr;
bool g_encode_tried = false;
thread_local const char *t_last_variant = "";

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_common(const void *Q, const void *K, const void *V, void *O, int B, int H, int N, int d, float scale,
                 const float *key_mask) {
    if (!Q || !K || !V || !O) return kErrArg;
    if (B <= 0 || H <= 0 || N <= 0 || d <= 0) return kErrArg;
    if (static_cast<long long>(B) * H * N >= (1LL << 31)) return kErrArg;
    if (static_cast<long long>(N) * d >= (1LL << 31)) return kErrArg;
    if (!(scale > 0.f) || !std::isfinite(scale)) return kErrArg;
    if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return kErrArg;
    if (key_mask && (reinterpret_cast<uintptr_t>(key_mask) & 3u)) return kErrArg;
    return kOk;
}
}  // namespace

EncodeTiledFn encode_tiled_fn() {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_encode_tried) {
        g_encode_tried = true;
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
    return g_encode;
}

namespace {
// Recently encoded tensor maps, keyed by (device, base, D, N, BH, box rows):
// repeated calls on the same buffers (a training or benchmark loop) skip the
// driver's encode.  A small table with round-robin replacement.
struct MapEntry {
    int dev, D, N, BH, box_rows;
    const void *base;
    CUtensorMap map;
};
constexpr int kMapCache = 32;
MapEntry g_maps[kMapCache];
int g_maps_n = 0, g_maps_next = 0;
std::mutex g_maps_mu;
}  // namespace

bool make_bf16_rows_map(CUtensorMap *m, const void *base, int D, int N, int BH, int box_rows) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    {
        std::lock_guard<std::mutex> lk(g_maps_mu);
        for (int i = 0; i < g_maps_n; ++i) {
            const MapEntry &e = g_maps[i];
            if (e.base == base && e.dev == dev && e.D == D && e.N == N && e.BH == BH && e.box_rows == box_rows) {
                *m = e.map;
                return true;
            }
        }
    }
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(N),
                                static_cast<cuuint64_t>(BH)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(N) * D * 2};
    const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_rows), 1u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    if (enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    std::lock_guard<std::mutex> lk(g_maps_mu);
    MapEntry &e = g_maps[g_maps_next];
    e.dev = dev;
    e.D = D;
    e.N = N;
    e.BH = BH;
    e.box_rows = box_rows;
    e.base = base;
    e.map = *m;
    g_maps_next = (g_maps_next + 1) % kMapCache;
    if (g_maps_n < kMapCache) ++g_maps_n;
    return true;
}

bool make_map(CUtensorMap *m, CUtensorMapSwizzle swizzle, const void *base, int rank, const cuuint64_t *dims,
              const cuuint64_t *strides, const cuuint32_t *box) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (rank < 1 || rank > 5 || !enc) return false;
    cuuint64_t st[4] = {};
    // a dimension of one element may come with any stride: give it a valid one
    for (int i = 1; i < rank; ++i) st[i - 1] = dims[i] > 1 ? strides[i - 1] : 16 * ((dims[0] * 2 + 15) / 16);
    const cuuint32_t estr[5] = {1u, 1u, 1u, 1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims, st, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool make_bf16_map(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                   const cuuint32_t *box) {
    return make_map(m, CU_TENSOR_MAP_SWIZZLE_128B, base, rank, dims, strides, box);
}

int *device_error_word() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_err_ptr[dev]) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_error_word) != cudaSuccess) return nullptr;
        g_err_ptr[dev] = static_cast<int *>(p);
    }
    return g_err_ptr[dev];
}

// Waits on a barrier that nothing completes, for timeout_us microseconds.
__global__ void wait_timeout_probe_kernel(unsigned long long limit_ns, int *err) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar), 1);
        abort_flag = 0u;
        fence_mbar_init();
    }
    __syncthreads();
    // Phase 0 never completes: no thread arrives.
    mbar_wait(smem_u32(&bar), 0, &abort_flag, err, 99, limit_ns);
    __syncthreads();
}

int launch_wait_timeout_probe(unsigned timeout_us, cudaStream_t stream) {
    int *err = device_error_word();
    if (!err) return kErrCuda;
    wait_timeout_probe_kernel<<<1, 32, 0, stream>>>(static_cast<unsigned long long>(timeout_us) * 1000ull, err);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}

}  // namespace eta

using namespace eta;

extern "C" {

int attn_fwd(const void *Q, const void *K, const void *V, void *O, float *LSE, int B, int H, int N, int d,
             int causal, float scale, int Br, int Bc, int dtype, const float *key_mask, void *stream) {
    int rc = check_common(Q, K, V, O, B, H, N, d, scale, key_mask);
    if (rc != kOk) return rc;
    if (causal != 0 && causal != 1) return kErrArg;
    if (LSE && (reinterpret_cast<uintptr_t>(LSE) & 3u)) return kErrArg;
    const char *variant = "";
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == ATTN_BF16) {
        if (d != 64 && d != 128) return kErrUnsupported;
        if (!((Br == 0 || Br == 64 || Br == 128) && (Bc == 0 || Bc == 64 || Bc == 128 || Bc == 256)))
            return kErrUnsupported;
        int dev = 0, major = 0, minor = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return kErrCuda;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return kErrCuda;
        if (major != 10 || minor != 3) return kErrUnsupported;  // built for sm_103a only
        // Default key tile: 128, except short causal d = 64 problems, whose few
        // tiles per CTA leave the pipeline mostly filling; 64-key tiles with two
        // S buffers ran 7% faster on 4x16x1024x64 causal.
        if (Bc == 0 && causal && d == 64 && N <= 1024) Bc = 64;
        rc = launch_fwd_tc_bf16(Q, K, V, O, LSE, B, H, N, d, causal, scale, Br, Bc, key_mask, st, &variant);
    } else if (dtype == ATTN_F32) {
        if (d > 128) return kErrUnsupported;
        if (!((Br == 0 || Br == 64) && (Bc == 0 || Bc == 64))) return kErrUnsupported;
        rc = launch_fwd_f32(static_cast<const float *>(Q), static_cast<const float *>(K),
                            static_cast<const float *>(V), static_cast<float *>(O), LSE, B, H, N, d, causal,
                            scale, key_mask, st, &variant);
    } else if (dtype == ATTN_F64) {
        return kErrUnsupported;
    } else {
        return kErrArg;
    }
    if (rc == kOk) t_last_variant = variant;
    return rc;
}

namespace {
// attn_fwd_host's device workspace: Q | K | V | O | LSE | key mask, each at a
// 256-byte boundary.
struct HostLayout {
    size_t q, k, v, o, lse, mask, total;
};
HostLayout host_layout(int B, int H, int N, int d, size_t es, bool with_mask) {
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    const size_t t = static_cast<size_t>(B) * H * N * d * es;
    const size_t r = static_cast<size_t>(B) * H * N * 4;
    HostLayout L;
    size_t off = 0;
    L.q = off; off += up(t);
    L.k = off; off += up(t);
    L.v = off; off += up(t);
    L.o = off; off += up(t);
    L.lse = off; off += up(r);
    L.mask = off; off += with_mask ? up(r) : 0;
    L.total = off;
    return L;
}
}  // namespace

size_t attn_fwd_host_workspace_size(int B, int H, int N, int d, int dtype, int with_mask) {
    if (B <= 0 || H <= 0 || N <= 0 || d <= 0) return 0;
    if (static_cast<long long>(B) * H * N >= (1LL << 31) || static_cast<long long>(N) * d >= (1LL << 31)) return 0;
    const size_t es = dtype == ATTN_F32 ? 4 : dtype == ATTN_BF16 ? 2 : 0;
    if (!es) return 0;
    return host_layout(B, H, N, d, es, with_mask != 0).total;
}

int attn_fwd_host(const void *Qh, const void *Kh, const void *Vh, void *Oh, float *LSEh, int B, int H, int N, int d,
                  int causal, float scale, int Br, int Bc, int dtype, const float *key_mask_h, void *workspace,
                  size_t ws_bytes, void *stream) {
    if (!Qh || !Kh || !Vh || !Oh) return kErrArg;
    const size_t need = attn_fwd_host_workspace_size(B, H, N, d, dtype, key_mask_h != nullptr);
    if (need == 0) return (dtype == ATTN_F32 || dtype == ATTN_BF16) ? kErrArg : kErrUnsupported;
    if (!workspace || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return kErrWorkspace;
    char *ws = static_cast<char *>(workspace);
    const HostLayout L = host_layout(B, H, N, d, dtype == ATTN_F32 ? 4 : 2, key_mask_h != nullptr);
    const size_t t = static_cast<size_t>(B) * H * N * d * (dtype == ATTN_F32 ? 4 : 2);
    const size_t r = static_cast<size_t>(B) * H * N * 4;
    // Dry run of the argument checks on the device buffers (a zero-size O
    // would be rejected by the same checks): nothing is enqueued on an
    // invalid argument.
    int rc = check_common(ws + L.q, ws + L.k, ws + L.v, ws + L.o, B, H, N, d, scale,
                          key_mask_h ? reinterpret_cast<const float *>(ws + L.mask) : nullptr);
    if (rc != kOk) return rc;
    if (causal != 0 && causal != 1) return kErrArg;
    if (dtype == ATTN_BF16) {
        if (d != 64 && d != 128) return kErrUnsupported;
        if (!((Br == 0 || Br == 64 || Br == 128) && (Bc == 0 || Bc == 64 || Bc == 128 || Bc == 256)))
            return kErrUnsupported;
    } else {
        if (d > 128) return kErrUnsupported;
        if (!((Br == 0 || Br == 64) && (Bc == 0 || Bc == 64))) return kErrUnsupported;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(ws + L.q, Qh, t, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaMemcpyAsync(ws + L.k, Kh, t, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaMemcpyAsync(ws + L.v, Vh, t, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        (key_mask_h && cudaMemcpyAsync(ws + L.mask, key_mask_h, r, cudaMemcpyHostToDevice, st) != cudaSuccess))
        return kErrCuda;
    rc = attn_fwd(ws + L.q, ws + L.k, ws + L.v, ws + L.o, LSEh ? reinterpret_cast<float *>(ws + L.lse) : nullptr, B,
                  H, N, d, causal, scale, Br, Bc, dtype,
                  key_mask_h ? reinterpret_cast<const float *>(ws + L.mask) : nullptr, stream);
    if (rc != kOk) return rc;
    if (cudaMemcpyAsync(Oh, ws + L.o, t, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        (LSEh && cudaMemcpyAsync(LSEh, ws + L.lse, r, cudaMemcpyDeviceToHost, st) != cudaSuccess))
        return kErrCuda;
    return kOk;
}

int attn_fwd_block_sparse(const void *Q, const void *K, const void *V, void *O, float *LSE, int B, int H, int N,
                          int d, int causal, float scale, int dtype, const unsigned char *block_mask,
                          const float *key_mask, void *stream) {
    int rc = check_common(Q, K, V, O, B, H, N, d, scale, key_mask);
    if (rc != kOk) return rc;
    if (!block_mask) return kErrArg;
    if (causal != 0 && causal != 1) return kErrArg;
    if (LSE && (reinterpret_cast<uintptr_t>(LSE) & 3u)) return kErrArg;
    if (dtype != ATTN_BF16) return (dtype == ATTN_F32 || dtype == ATTN_F64) ? kErrUnsupported : kErrArg;
    if (d != 64 && d != 128) return kErrUnsupported;
    if (N > ATTN_BLOCK_SPARSE_MAX_N) return kErrUnsupported;
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return kErrCuda;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return kErrCuda;
    if (major != 10 || minor != 3) return kErrUnsupported;  // built for sm_103a only
    const char *variant = "";
    rc = launch_fwd_tc_bf16_bsparse(Q, K, V, O, LSE, B, H, N, d, causal, scale, block_mask, key_mask,
                                    static_cast<cudaStream_t>(stream), &variant);
    if (rc == kOk) t_last_variant = variant;
    return rc;
}

static_assert(ATTN_BLOCK_SPARSE_BLOCK == eta::kBlockSparseBlock && ATTN_BLOCK_SPARSE_MAX_N == eta::kBlockSparseMaxN,
              "header and library agree on the block-sparse limits");

size_t attn_naive_workspace_size(int B, int H, int N, int dtype) {
    if (B <= 0 || H <= 0 || N <= 0) return 0;
    size_t es = dtype == ATTN_F32 ? 4 : dtype == ATTN_BF16 ? 2 : 0;
    if (!es) return 0;
    const unsigned long long rows = static_cast<unsigned long long>(B) * H * N;
    const unsigned long long n = static_cast<unsigned long long>(N);
    if (rows > (~0ull) / n / es) return 0;
    return static_cast<size_t>(rows * n * es);
}

int attn_naive_fwd(const void *Q, const void *K, const void *V, void *O, float *LSE, int B, int H, int N, int d,
                   int causal, float scale, int dtype, const float *key_mask, void *workspace, size_t ws_bytes,
                   void *stream) {
    int rc = check_common(Q, K, V, O, B, H, N, d, scale, key_mask);
    if (rc != kOk) return rc;
    if (causal != 0 && causal != 1) return kErrArg;
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return dtype == ATTN_F64 ? kErrUnsupported : kErrArg;
    if (d > 128) return kErrUnsupported;
    const size_t need = attn_naive_workspace_size(B, H, N, dtype);
    if (need == 0) return kErrArg;
    if (!workspace || ws_bytes < need || !aligned16(workspace)) return kErrWorkspace;
    return launch_naive(Q, K, V, O, LSE, B, H, N, d, causal, scale, dtype == ATTN_BF16 ? 1 : 0, key_mask,
                        workspace, static_cast<cudaStream_t>(stream));
}

size_t attn_deviation_workspace_size(long long n) {
    if (n <= 0) return 0;
    return deviation_workspace_bytes(n);
}

int attn_deviation(const void *a, int ta, const void *b, int tb, long long n, void *workspace, size_t ws_bytes,
                   void *stream, attn_dev_t *out) {
    if (!a || !b || !out || n <= 0) return kErrArg;
    if (ta < ATTN_F32 || ta > ATTN_F64 || tb < ATTN_F32 || tb > ATTN_F64) return kErrArg;
    const size_t need = deviation_workspace_bytes(n);
    if (!workspace || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return kErrWorkspace;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    double *res = reinterpret_cast<double *>(static_cast<char *>(workspace) + deviation_result_offset(n));
    int rc = launch_deviation(a, ta, b, tb, n, workspace, st, res);
    if (rc != kOk) return rc;
    double host[5];
    if (cudaMemcpyAsync(host, res, sizeof(host), cudaMemcpyDeviceToHost, st) != cudaSuccess) return kErrCuda;
    if (cudaStreamSynchronize(st) != cudaSuccess) return kErrCuda;
    out->max_abs = host[0];
    out->w1 = host[1];
    out->mean_abs = host[2];
    out->std_abs = host[3];
    out->mean_signed = host[4];
    out->n = n;
    return kOk;
}

static_assert(ATTN_DEVIATION_NOALLOC_MAX_N == eta::kDeviationNoAllocMaxN, "header and library agree on the limit");

int attn_deviation_noalloc(const void *a, int ta, const void *b, int tb, long long n, void *stream,
                           attn_dev_t *out) {
    if (!a || !b || !out || n <= 0) return kErrArg;
    if (ta < ATTN_F32 || ta > ATTN_F64 || tb < ATTN_F32 || tb > ATTN_F64) return kErrArg;
    if (n > ATTN_DEVIATION_NOALLOC_MAX_N) return kErrUnsupported;
    double host[5];
    const int rc = launch_deviation_noalloc(a, ta, b, tb, n, static_cast<cudaStream_t>(stream), host);
    if (rc != kOk) return rc;
    out->max_abs = host[0];
    out->w1 = host[1];
    out->mean_abs = host[2];
    out->std_abs = host[3];
    out->mean_signed = host[4];
    out->n = n;
    return kOk;
}

size_t attn_decode_workspace_size(int B, int H, int Nq, int d) {
    if (B <= 0 || H <= 0 || Nq <= 0 || d <= 0) return 0;
    if (static_cast<long long>(B) * H * Nq >= (1LL << 31)) return 0;
    return decode_workspace_bytes(B * H, Nq, d);
}

int attn_decode_fwd(const void *Q, const void *K, const void *V, void *O, float *LSE, int B, int H, int Nq, int Nk,
                    int d, int causal, float scale, int dtype, const float *key_mask, void *workspace,
                    size_t ws_bytes, void *stream) {
    if (!Q || !K || !V || !O) return kErrArg;
    if (B <= 0 || H <= 0 || Nq <= 0 || Nk <= 0 || d <= 0) return kErrArg;
    if (static_cast<long long>(B) * H * Nk >= (1LL << 31) || static_cast<long long>(Nk) * d >= (1LL << 31))
        return kErrArg;
    if (!(scale > 0.f) || !std::isfinite(scale)) return kErrArg;
    if (causal != 0 && causal != 1) return kErrArg;
    if (causal && Nq > Nk) return kErrArg;
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return dtype == ATTN_F64 ? kErrUnsupported : kErrArg;
    if (Nq > ATTN_DECODE_MAX_NQ || d > 128 || d % 32 != 0) return kErrUnsupported;
    if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return kErrArg;
    if (key_mask && (reinterpret_cast<uintptr_t>(key_mask) & 3u)) return kErrArg;
    if (!workspace || ws_bytes < attn_decode_workspace_size(B, H, Nq, d) || !aligned16(workspace))
        return kErrWorkspace;
    return launch_decode(Q, K, V, O, LSE, B, H, Nq, Nk, d, causal, scale, dtype == ATTN_BF16 ? 1 : 0, key_mask,
                         workspace, static_cast<cudaStream_t>(stream));
}

namespace {
constexpr long long kMaxTokens = 1LL << 30;   // of a sequence, and of a call
// Entries of a list.  Sequences named twice are found by looking through the
// entries before, so the longest list bounds a kernel's time (seconds), not only
// the 32-bit arithmetic on entry numbers.
constexpr int kMaxList = 1 << 20;

// Whether `outer` >= (n - 1) * inner + block, without overflow.
bool steps_over(long long outer, long long n, long long inner, long long block) {
    return outer >= block && (n <= 1 || (outer - block) / (n - 1) >= inner);
}

// Checks a cache descriptor; fills the page kernels' view of it.
int check_cache(const attn_cache_t *c, CacheView &w) {
    if (!c || !c->K || !c->V || !c->page_table || !c->seq_lens || !c->ref_counts) return kErrArg;
    if (c->dtype != ATTN_F32 && c->dtype != ATTN_BF16 && c->dtype != ATTN_E2M1)
        return c->dtype == ATTN_F64 ? kErrUnsupported : kErrArg;
    if (c->layers <= 0 || c->pages <= 0 || c->heads <= 0 || c->page_size <= 0 || c->d <= 0 || c->seqs <= 0 ||
        c->max_pages <= 0)
        return kErrArg;
    if (c->d > 128 || c->d % 32 != 0) return kErrUnsupported;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return kErrUnsupported;
    // (positions, and the ends of tiles that reach past them, stay inside 32 bits)
    if (static_cast<long long>(c->max_pages) * c->page_size > kMaxTokens) return kErrArg;
    if (!aligned16(c->K) || !aligned16(c->V) || !aligned16(c->ref_counts)) return kErrArg;
    if ((reinterpret_cast<uintptr_t>(c->page_table) & 3u) || (reinterpret_cast<uintptr_t>(c->seq_lens) & 3u)) return kErrArg;
    // elements of a 16-byte piece (4-bit values: an element is a byte), and of one head's rows of a page
    const bool q4 = c->dtype == ATTN_E2M1;
    const long long per = q4 ? 16 : c->dtype == ATTN_BF16 ? 8 : 4;
    const long long head = static_cast<long long>(c->page_size) * (q4 ? c->d / 16 * 9 : c->d);
    const long long block = c->heads * head;
    if (block / per >= (1LL << 30)) return kErrArg;
    const long long row = q4 ? c->d / 2 : c->d;
    const bool by_head = c->head_stride == head && c->slot_stride == row;
    const bool by_token = !q4 && c->slot_stride == static_cast<long long>(c->heads) * c->d && c->head_stride == c->d;
    // (with one head, or as strides of a single head may be given, both agree)
    const bool one_head = c->heads == 1 && c->slot_stride == row && c->head_stride >= 0 && c->head_stride % per == 0;
    if (!by_head && !by_token && !one_head) return kErrArg;
    if (c->page_stride < 0 || c->layer_stride < 0 || c->page_stride % per || c->layer_stride % per) return kErrArg;
    // blocks of different (layer, page) do not overlap, whichever stride is the outer one
    const bool many_l = c->layers > 1, many_p = c->pages > 1;
    if (many_p && c->page_stride < block) return kErrArg;
    if (many_l && c->layer_stride < block) return kErrArg;
    if (many_l && many_p && !steps_over(c->layer_stride, c->pages, c->page_stride, block) &&
        !steps_over(c->page_stride, c->layers, c->layer_stride, block))
        return kErrArg;
    w.k = static_cast<uint4 *>(c->K);
    w.v = static_cast<uint4 *>(c->V);
    w.page_table = c->page_table;
    w.seq_lens = c->seq_lens;
    w.ref_counts = c->ref_counts;
    w.layers = c->layers;
    w.pages = c->pages;
    w.heads = c->heads;
    w.page_size = c->page_size;
    w.rows = c->seqs;
    w.max_pages = c->max_pages;
    w.layer_vecs = c->layer_stride / per;
    w.page_vecs = c->page_stride / per;
    w.head_stride_vecs = c->head_stride / per;
    w.slot_stride_vecs = c->slot_stride / per;
    w.block_vecs = static_cast<int>(block / per);
    w.slot_vecs = static_cast<int>(c->slot_stride / per);
    w.row_vecs = static_cast<int>(c->d / per);
    w.bits = q4 ? 4 : c->dtype == ATTN_BF16 ? 16 : 32;
    return kOk;
}
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// Whether rows of d elements at (t * token, h * head) do not overlap: one of the strides steps over all of the other's range.
bool rows_apart(long long T, long long heads, long long token, long long head, long long d) {
    const bool heads_in = (heads == 1 || head >= d) && (T == 1 || steps_over(token, heads, head, d));
    const bool tokens_in = (T == 1 || token >= d) && (heads == 1 || steps_over(head, T, token, d));
    return heads_in || tokens_in;
}
// Checks what the calls that move rows of tokens share (bases, strides, the list); `none`: there is nothing to do.
int check_append(const attn_cache_t *cache, int layer, const void *K, const void *V, long long token_stride,
                 long long head_stride, const RowList &li, CacheView &w, RowIn &in, bool &none) {
    const int rc = check_cache(cache, w);
    if (rc != kOk) return rc;
    if (li.n < 0 || li.n > kMaxList || li.T < 0 || li.T > kMaxTokens || layer < 0 || layer >= w.layers) return kErrArg;
    // (the stride of a dimension of one element means nothing)
    if (li.T == 1) token_stride = 0;
    if (w.heads == 1) head_stride = 0;
    const long long es = w.bits == 32 ? 4 : 2, per = 16 / es;
    if (token_stride < 0 || head_stride < 0 || token_stride % per || head_stride % per) return kErrArg;
    in.token_bytes = token_stride * es;
    in.head_bytes = head_stride * es;
    in.d = cache->d;
    none = li.n == 0 || li.T == 0;
    if (none) return kOk;
    if (!K || !V || !li.q_start || !aligned16(K) || !aligned16(V) || !aligned4(li.q_start) || !aligned4(li.seqs) ||
        !aligned4(li.granted))
        return kErrArg;
    in.K = static_cast<const char *>(K);
    in.V = static_cast<const char *>(V);
    return kOk;
}
constexpr long long kMaxRows = 1LL << 20;   // rows of a token (K, V and Q) in the calls that count them in 32 bits
int check_workspace(const void *ws, size_t have, size_t need) {
    return !ws || have < need || !aligned16(ws) ? kErrWorkspace : kOk;
}
// sm_103a only
int check_device() {
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return kErrCuda;
    return major == 10 && minor == 3 ? kOk : kErrUnsupported;
}
}  // namespace

size_t attn_cache_workspace_size(int pages, int n) {
    if (pages <= 0 || n < 0 || n > kMaxList) return 0;
    return cache_workspace_bytes(pages, n);
}

int attn_cache_reserve(const attn_cache_t *cache, const int *seqs, const int *n_new, int n, int *granted, void *workspace,
                       size_t ws_bytes, void *stream) {
    CacheView w;
    int rc = check_cache(cache, w);
    if (rc != kOk) return rc;
    if (n < 0 || n > kMaxList) return kErrArg;
    if (n == 0) return kOk;
    if (!seqs || !n_new || !granted || !aligned4(seqs) || !aligned4(n_new) || !aligned4(granted)) return kErrArg;
    rc = check_workspace(workspace, ws_bytes, cache_workspace_bytes(w.pages, n));
    if (rc != kOk) return rc;
    return launch_cache_reserve(w, seqs, n_new, n, granted, workspace, static_cast<cudaStream_t>(stream));
}

int attn_cache_free(const attn_cache_t *cache, const int *seqs, const int *keep, int n, void *stream) {
    CacheView w;
    const int rc = check_cache(cache, w);
    if (rc != kOk) return rc;
    if (n < 0 || n > kMaxList) return kErrArg;
    if (n == 0) return kOk;
    if (!seqs || !aligned4(seqs) || !aligned4(keep)) return kErrArg;
    return launch_cache_free(w, seqs, keep, n, static_cast<cudaStream_t>(stream));
}

int attn_cache_fork(const attn_cache_t *cache, const int *parents, const int *children, int n, int copy, int *granted,
                    void *workspace, size_t ws_bytes, void *stream) {
    CacheView w;
    int rc = check_cache(cache, w);
    if (rc != kOk) return rc;
    if (n < 0 || n > kMaxList || (copy != 0 && copy != 1)) return kErrArg;
    if (n == 0) return kOk;
    if (!parents || !children || !granted || !aligned4(parents) || !aligned4(children) || !aligned4(granted)) return kErrArg;
    rc = check_workspace(workspace, ws_bytes, cache_workspace_bytes(w.pages, n));
    if (rc != kOk) return rc;
    return launch_cache_fork(w, parents, children, n, copy, granted, workspace, static_cast<cudaStream_t>(stream));
}

int attn_cache_compact(const attn_cache_t *cache, int *page_table_out, int *ref_counts_out, int *n_live, void *workspace,
                       size_t ws_bytes, void *stream) {
    CacheView w;
    int rc = check_cache(cache, w);
    if (rc != kOk) return rc;
    if (!page_table_out || !ref_counts_out || !n_live) return kErrArg;
    if (!aligned4(page_table_out) || !aligned16(ref_counts_out) || !aligned4(n_live)) return kErrArg;
    rc = check_workspace(workspace, ws_bytes, cache_workspace_bytes(w.pages, 0));
    if (rc != kOk) return rc;
    return launch_cache_compact(w, page_table_out, ref_counts_out, n_live, workspace, static_cast<cudaStream_t>(stream));
}

int attn_cache_append(const attn_cache_t *cache, int layer, const void *Knew, const void *Vnew, long long token_stride,
                      long long head_stride, int T, const int *seqs, const int *q_start, int n, void *stream) {
    return attn_cache_append_granted(cache, layer, Knew, Vnew, token_stride, head_stride, T, seqs, q_start, nullptr, n,
                                     stream);
}

int attn_cache_append_granted(const attn_cache_t *cache, int layer, const void *Knew, const void *Vnew,
                              long long token_stride, long long head_stride, int T, const int *seqs, const int *q_start,
                              const int *granted, int n, void *stream) {
    CacheView w;
    RowIn in = {};
    const RowList li{seqs, q_start, granted, nullptr, n, T};
    bool none = false;
    const int rc = check_append(cache, layer, Knew, Vnew, token_stride, head_stride, li, w, in, none);
    if (rc != kOk || none) return rc;
    if (w.bits == 4 && 2LL * w.heads > kMaxRows) return kErrUnsupported;
    if (w.bits == 4) return launch_cache_rows_in(w, layer, in, li, Rotation{}, static_cast<cudaStream_t>(stream));
    return launch_cache_append(w, layer, Knew, Vnew, in.token_bytes / 16, in.head_bytes / 16, T, seqs, q_start, granted, n,
                               static_cast<cudaStream_t>(stream));
}

int attn_cache_append_rotated(const attn_cache_t *cache, int layer, const void *Knew, const void *Vnew, long long token_stride,
                              long long head_stride, const void *Q, void *Qout, int Hq, long long q_token_stride,
                              long long q_head_stride, long long o_token_stride, long long o_head_stride, int T,
                              const int *seqs, const int *q_start, const int *granted, int n,
                              const attn_rotation_t *rotation, void *stream) {
    CacheView w;
    RowIn in = {};
    const RowList li{seqs, q_start, granted, nullptr, n, T};
    bool none = false;
    const int rc = check_append(cache, layer, Knew, Vnew, token_stride, head_stride, li, w, in, none);
    if (rc != kOk) return rc;
    if (!rotation || rotation->rows <= 0 || rotation->dims < 2 || rotation->dims % 2 || rotation->dims > cache->d ||
        (rotation->neighbours != 0 && rotation->neighbours != 1))
        return kErrArg;
    if (Hq < 0 || (Hq == 0 && (Q || Qout))) return kErrArg;
    if (2LL * w.heads + Hq > kMaxRows) return kErrUnsupported;
    if (T == 1) q_token_stride = o_token_stride = 0;
    if (Hq <= 1) q_head_stride = o_head_stride = 0;
    const long long es = w.bits == 32 ? 4 : 2, per = 16 / es;
    if (Hq > 0) {
        for (long long s : {q_token_stride, q_head_stride, o_token_stride, o_head_stride}) {
            if (s < 0 || s % per) return kErrArg;
            if (s >= (1LL << 38)) return kErrUnsupported;
        }
        if (T > 0 && !rows_apart(T, Hq, o_token_stride, o_head_stride, cache->d)) return kErrArg;
        if (Q == Qout && (q_token_stride != o_token_stride || q_head_stride != o_head_stride)) return kErrArg;
    }
    if (none) return kOk;
    if (!rotation->table || !aligned16(rotation->table) || !aligned4(rotation->positions)) return kErrArg;
    if (Hq > 0 && (!Q || !Qout || !aligned16(Q) || !aligned16(Qout))) return kErrArg;
    in.Q = static_cast<const char *>(Q);
    in.Qout = static_cast<char *>(Qout);
    in.q_token_bytes = q_token_stride * es;
    in.q_head_bytes = q_head_stride * es;
    in.o_token_bytes = o_token_stride * es;
    in.o_head_bytes = o_head_stride * es;
    in.Hq = Hq;
    const Rotation r{rotation->table, rotation->positions, rotation->rows, rotation->dims, rotation->neighbours};
    return launch_cache_rows_in(w, layer, in, li, r, static_cast<cudaStream_t>(stream));
}

int attn_cache_read(const attn_cache_t *cache, int layer, void *Kout, void *Vout, long long token_stride, long long head_stride,
                    int T, const int *seqs, const int *q_start, const int *first, int n, void *stream) {
    CacheView w;
    RowIn in = {};
    const RowList li{seqs, q_start, nullptr, first, n, T};
    bool none = false;
    const int rc = check_append(cache, layer, Kout, Vout, token_stride, head_stride, li, w, in, none);
    if (rc != kOk) return rc;
    if (2LL * w.heads > kMaxRows) return kErrUnsupported;
    const long long es = w.bits == 32 ? 4 : 2;
    if (T > 0 && !rows_apart(T, w.heads, in.token_bytes / es, in.head_bytes / es, cache->d)) return kErrArg;
    if (none) return kOk;
    if (Kout == Vout || !aligned4(first)) return kErrArg;
    const RowOut out{static_cast<char *>(Kout), static_cast<char *>(Vout), in.token_bytes, in.head_bytes, cache->d, 0};
    return launch_cache_rows_out(w, layer, out, li, static_cast<cudaStream_t>(stream));
}

size_t attn_paged_workspace_size(int Hq, int heads, int max_q, int d, int dtype) {
    if (Hq <= 0 || heads <= 0 || Hq % heads || Hq / heads > 64 || max_q <= 0 || d <= 0 || d > 128 || d % 32) return 0;
    if (dtype != ATTN_F32 && dtype != ATTN_BF16 && dtype != ATTN_E2M1) return 0;
    return paged_workspace_bytes(Hq / heads, max_q, d, dtype == ATTN_E2M1 ? 4 : dtype == ATTN_BF16 ? 16 : 32);
}

int attn_paged_fwd(const attn_cache_t *cache, int layer, const void *Q, void *O, float *LSE, long long q_token_stride,
                   long long q_head_stride, long long o_token_stride, long long o_head_stride, int T, int Hq,
                   const int *seqs, const int *q_start, int n, int max_q, int causal, float scale, void *workspace,
                   size_t ws_bytes, void *stream) {
    return attn_paged_fwd_granted(cache, layer, Q, O, LSE, q_token_stride, q_head_stride, o_token_stride, o_head_stride, T, Hq,
                                  seqs, q_start, nullptr, n, max_q, causal, scale, workspace, ws_bytes, stream);
}

int attn_paged_fwd_granted(const attn_cache_t *cache, int layer, const void *Q, void *O, float *LSE,
                           long long q_token_stride, long long q_head_stride, long long o_token_stride,
                           long long o_head_stride, int T, int Hq, const int *seqs, const int *q_start, const int *granted,
                           int n, int max_q, int causal, float scale, void *workspace, size_t ws_bytes, void *stream) {
    CacheView w;
    int rc = check_cache(cache, w);
    if (rc != kOk) return rc;
    if (layer < 0 || layer >= w.layers || T < 0 || n < 0 || n > kMaxList || Hq <= 0 || Hq % w.heads) return kErrArg;
    if (Hq / w.heads > 64) return kErrUnsupported;
    // (the kernels work in powers of two: scale * log2(e) has to be a number too, or a score of 0 would be NaN)
    if (!(scale > 0.f) || !std::isfinite(scale * kPagedLog2e)) return kErrArg;
    if (causal != 0 && causal != 1) return kErrArg;
    if (T > kMaxTokens || static_cast<long long>(T) * Hq >= (1LL << 31)) return kErrArg;
    const long long per = w.bits == 32 ? 4 : 8;
    // (the stride of a dimension of one element means nothing)
    if (T == 1) q_token_stride = o_token_stride = 0;
    if (Hq == 1) q_head_stride = o_head_stride = 0;
    for (long long s : {q_token_stride, q_head_stride, o_token_stride, o_head_stride})
        if (s < 0 || s % per) return kErrArg;
    // the tensor maps of the bf16 path take strides below 2^40 bytes, and rows of Q that differ
    for (long long s : {q_token_stride, q_head_stride, o_token_stride, o_head_stride, cache->page_stride})
        if (s >= (1LL << 38)) return kErrUnsupported;
    if ((T > 1 && q_token_stride == 0) || (Hq > 1 && q_head_stride == 0)) return kErrArg;
    if (T == 0 || n == 0) return kOk;
    if (max_q <= 0 || max_q > T) return kErrArg;
    // rows of O must not overlap: one of the strides steps over all of the other's range
    if (!rows_apart(T, Hq, o_token_stride, o_head_stride, cache->d)) return kErrArg;
    if (!Q || !O || !q_start || !aligned16(Q) || !aligned16(O) || !aligned4(q_start) || !aligned4(seqs) || !aligned4(LSE) ||
        !aligned4(granted))
        return kErrArg;
    rc = check_workspace(workspace, ws_bytes, paged_workspace_bytes(Hq / w.heads, max_q, cache->d, w.bits));
    if (rc != kOk) return rc;
    rc = check_device();
    if (rc != kOk) return rc;
    const size_t es = w.bits == 4 ? 1 : w.bits / 8;
    PagedParams p = {};
    p.gm.page_table = w.page_table;
    p.gm.seq_lens = w.seq_lens;
    p.gm.seqs = seqs;
    p.gm.q_start = q_start;
    p.gm.granted = granted;
    p.gm.n = n;
    p.gm.rows = w.rows;
    p.gm.max_pages = w.max_pages;
    p.gm.pages = w.pages;
    p.gm.page_size = w.page_size;
    p.gm.T = T;
    p.gm.max_q = max_q;
    p.gm.heads = w.heads;
    p.gm.g = Hq / w.heads;
    p.gm.causal = causal;
    p.Q = Q;
    p.K = static_cast<const char *>(cache->K) + layer * cache->layer_stride * es;
    p.V = static_cast<const char *>(cache->V) + layer * cache->layer_stride * es;
    p.O = O;
    p.LSE = LSE;
    p.q_token = q_token_stride;
    p.q_head = q_head_stride;
    p.o_token = o_token_stride;
    p.o_head = o_head_stride;
    p.page_stride = cache->page_stride;
    p.head_stride = cache->head_stride;
    p.slot_stride = cache->slot_stride;
    p.d = cache->d;
    p.Hq = Hq;
    p.scale_log2 = scale * kPagedLog2e;
    p.err = device_error_word();
    if (!p.err) return kErrCuda;
    const char *variant = "";
    rc = launch_paged(p, w.bits, workspace, static_cast<cudaStream_t>(stream), &variant);
    if (rc == kOk) t_last_variant = variant;
    return rc;
}

size_t attn_bwd_workspace_size(int B, int H, int N, int d) {
    if (B <= 0 || H <= 0 || N <= 0 || d <= 0) return 0;
    if (static_cast<long long>(B) * H * N >= (1LL << 31)) return 0;
    return bwd_workspace_bytes(B * H, N, d);
}

int attn_bwd(const void *Q, const void *K, const void *V, const void *O, const void *dO, const float *LSE, void *dQ,
             void *dK, void *dV, int B, int H, int N, int d, int causal, float scale, int dtype,
             const float *key_mask, void *workspace, size_t ws_bytes, void *stream) {
    int rc = check_common(Q, K, V, const_cast<void *>(O), B, H, N, d, scale, key_mask);
    if (rc != kOk) return rc;
    if (!dO || !LSE || !dQ || !dK || !dV) return kErrArg;
    if (!aligned16(dO) || !aligned16(dQ) || !aligned16(dK) || !aligned16(dV)) return kErrArg;
    if (reinterpret_cast<uintptr_t>(LSE) & 3u) return kErrArg;
    if (causal != 0 && causal != 1) return kErrArg;
    if (dtype == ATTN_F32) {
        if (d > 128) return kErrUnsupported;
        if (!workspace || ws_bytes < attn_bwd_workspace_size(B, H, N, d) ||
            (reinterpret_cast<uintptr_t>(workspace) & 255u))
            return kErrWorkspace;
        rc = launch_bwd_f32(static_cast<const float *>(Q), static_cast<const float *>(K), static_cast<const float *>(V),
                            static_cast<const float *>(O), static_cast<const float *>(dO), LSE, static_cast<float *>(dQ),
                            static_cast<float *>(dK), static_cast<float *>(dV), B, H, N, d, causal, scale, key_mask,
                            workspace, static_cast<cudaStream_t>(stream));
        if (rc == kOk) t_last_variant = "bwd_simt_f32";
        return rc;
    }
    if (dtype != ATTN_BF16) return dtype == ATTN_F64 ? kErrUnsupported : kErrArg;
    if (d != 64 && d != 128) return kErrUnsupported;
    if (!workspace || ws_bytes < attn_bwd_workspace_size(B, H, N, d) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return kErrWorkspace;
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return kErrCuda;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return kErrCuda;
    if (major != 10 || minor != 3) return kErrUnsupported;  // built for sm_103a only
    rc = launch_bwd_tc_bf16(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, N, d, causal, scale, key_mask, workspace,
                            static_cast<cudaStream_t>(stream));
    if (rc == kOk) t_last_variant = d == 64 ? "bwd_tc_bf16_d64_br64_bc128" : "bwd_tc_bf16_d128_br64_bc128";
    return rc;
}

int attn_emul_fwd(const void *Q, const void *K, const void *V, int dtype, double *O, int B, int H, int N, int d,
                  int causal, float scale, const float *key_mask, int algo, int Bc, int mbits, int ebits,
                  const long long *rows, long long nrows, void *stream) {
    if (!Q || !K || !V || !O) return kErrArg;
    if (B <= 0 || H <= 0 || N <= 0 || d <= 0) return kErrArg;
    if (static_cast<long long>(B) * H * N >= (1LL << 31)) return kErrArg;
    if (!(scale > 0.f) || !std::isfinite(scale)) return kErrArg;
    if (causal != 0 && causal != 1) return kErrArg;
    if (dtype < ATTN_F32 || dtype > ATTN_F64) return kErrArg;
    if (algo != ATTN_EMUL_BASELINE && algo != ATTN_EMUL_TILED) return kErrArg;
    if (mbits < 1 || mbits > 52 || ebits < 2 || ebits > 11) return kErrArg;
    if (rows && nrows < 0) return kErrArg;
    if (algo == ATTN_EMUL_TILED && (Bc < 1 || Bc > ATTN_EMUL_MAX_BC)) return kErrArg;
    if (d > 128) return kErrUnsupported;
    if (algo == ATTN_EMUL_BASELINE && N > ATTN_EMUL_MAX_N_BASELINE) return kErrUnsupported;
    if (key_mask && (reinterpret_cast<uintptr_t>(key_mask) & 3u)) return kErrArg;
    if ((reinterpret_cast<uintptr_t>(O) & 7u) || (rows && (reinterpret_cast<uintptr_t>(rows) & 7u))) return kErrArg;
    return launch_emul(Q, K, V, dtype, O, B, H, N, d, causal, scale, key_mask, algo, algo == ATTN_EMUL_TILED ? Bc : 1,
                       mbits, ebits, rows, rows ? nrows : 0, static_cast<cudaStream_t>(stream));
}

int attn_emul_round(const double *x, double *y, long long n, int mbits, int ebits, void *stream) {
    if (!x || !y || n < 0) return kErrArg;
    if (mbits < 1 || mbits > 52 || ebits < 2 || ebits > 11) return kErrArg;
    if ((reinterpret_cast<uintptr_t>(x) & 7u) || (reinterpret_cast<uintptr_t>(y) & 7u)) return kErrArg;
    if (n == 0) return kOk;
    return launch_fmt_round(x, y, n, mbits, ebits, static_cast<cudaStream_t>(stream));
}

int attn_status(void *stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(st) != cudaSuccess) return kErrCuda;
    int *err = device_error_word();
    if (!err) return kErrCuda;
    int host = 0;
    if (cudaMemcpy(&host, err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return kErrCuda;
    if (host != 0) {
        const int zero = 0;
        if (cudaMemcpy(err, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return kErrCuda;
        return (host & ~kErrWordBadRow) ? kErrDeviceTimeout : kErrArg;
    }
    return kOk;
}

const char *attn_strerror(int status) {
    switch (status) {
        case ATTN_OK: return "ok";
        case ATTN_ERR_ARG: return "invalid argument";
        case ATTN_ERR_UNSUPPORTED: return "unsupported configuration or device";
        case ATTN_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
        case ATTN_ERR_CUDA: return "CUDA runtime or driver error";
        case ATTN_ERR_DEVICE_TIMEOUT: return "a kernel's bounded wait timed out";
        default: return "unknown status";
    }
}

int attn_last_variant(char *buf, int len) {
    if (!buf || len <= 0) return kErrArg;
    const int n = static_cast<int>(strlen(t_last_variant));
    snprintf(buf, static_cast<size_t>(len), "%s", t_last_variant);
    return n;
}

int attn_debug_wait_timeout(unsigned timeout_us, void *stream) {
    if (timeout_us < 1 || timeout_us > 1000000u) return kErrArg;
    return launch_wait_timeout_probe(timeout_us, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

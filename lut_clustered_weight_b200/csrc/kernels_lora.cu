// kernels_lora.cu -- cq_lora_add: low-rank adapters of many requests beside a
// shared projection, sm_100a.  out = y + scale * B (A x) with the adapter of
// each row.
#include <algorithm>

#include "cq_common.cuh"
#include "cq_internal.h"

namespace cq {

constexpr int kLoraThreads = 256;
constexpr int kLoraMaxRank = 128;

struct LoraArgs {
    const __half *x;
    const int32_t *ids;
    const __half *a, *b;
    const float *scale;
    const int32_t *ranks;
    const float *y;
    float *out;
    int64_t ldy, ldo;
    int M, K, N, n, r;
};

// One CTA per row: a warp per entry of t = A x, then a thread per column.
__global__ void __launch_bounds__(kLoraThreads) k_lora_row(const LoraArgs p) {
    __shared__ float t[kLoraMaxRank];
    griddep_wait();
    griddep_launch();
    const int64_t m = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int id = p.ids[m];
    const float *yr = p.y + m * p.ldy;
    float *orow = p.out + m * p.ldo;
    if (id < 0 || id >= p.n) {
        if (yr != orow)
            for (int c = threadIdx.x; c < p.N; c += kLoraThreads) orow[c] = yr[c];
        return;
    }
    const int rank = p.ranks ? max(0, min(p.ranks[id], p.r)) : p.r;
    const float sc = p.scale ? p.scale[id] : 1.0f;
    const __half *xr = p.x + m * p.K;
    for (int j = warp; j < rank; j += kLoraThreads / 32) {
        const __half *ar = p.a + ((int64_t)id * p.r + j) * p.K;
        float v = 0.0f;
        for (int k = lane; k < p.K; k += 32) v += __half2float(xr[k]) * __half2float(ar[k]);
        v = warp_sum(v);
        if (lane == 0) t[j] = v;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.N; c += kLoraThreads) {
        const __half *br = p.b + ((int64_t)id * p.N + c) * p.r;
        float v = 0.0f;
        for (int j = 0; j < rank; j++) v += t[j] * __half2float(br[j]);
        orow[c] = yr[c] + sc * v;
    }
}

static bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace cq

extern "C" {

CQ_API size_t cq_lora_add_workspace_size(int64_t M, int64_t n_adapters) {
    (void)M;
    (void)n_adapters;
    return 0;
}

CQ_API cq_status cq_lora_add(const void *x, const int32_t *ids, int64_t M, int64_t K,
                             const void *a, const void *b, const float *scale,
                             const int32_t *ranks, int64_t n_adapters, int64_t r_max,
                             const float *y, int64_t ldy, float *out, int64_t ldo, int64_t N,
                             void *workspace, size_t workspace_bytes, cq_stream_t stream) {
    using namespace cq;
    if (M < 0 || K <= 0 || N <= 0 || n_adapters <= 0 || r_max <= 0)
        return CQ_ERR_INVALID_ARGUMENT;
    if (ldy < N || ldo < N || !a || !b) return CQ_ERR_INVALID_ARGUMENT;
    if (M > 0 && (!x || !ids || !y || !out)) return CQ_ERR_INVALID_ARGUMENT;
    if (y == out && ldy != ldo) return CQ_ERR_INVALID_ARGUMENT;
    const void *ps[] = {x, ids, a, b, scale, ranks, y, out, workspace};
    for (const void *p : ps)
        if (!al16(p)) return CQ_ERR_INVALID_ARGUMENT;
    if (K % 8 || N % 8 || r_max % 8 || r_max > kLoraMaxRank || ldy % 4 || ldo % 4 ||
        n_adapters > 4096 || M > (int64_t(1) << 24) || K > (int64_t(1) << 20) ||
        N > (int64_t(1) << 20))
        return CQ_ERR_UNSUPPORTED;
    if (M == 0) return CQ_OK;
    const size_t need = cq_lora_add_workspace_size(M, n_adapters);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CQ_ERR_WORKSPACE;
    LoraArgs p{};
    p.x = reinterpret_cast<const __half *>(x);
    p.ids = ids;
    p.a = reinterpret_cast<const __half *>(a);
    p.b = reinterpret_cast<const __half *>(b);
    p.scale = scale;
    p.ranks = ranks;
    p.y = y;
    p.out = out;
    p.ldy = ldy;
    p.ldo = ldo;
    p.M = (int)M;
    p.K = (int)K;
    p.N = (int)N;
    p.n = (int)n_adapters;
    p.r = (int)r_max;
    try {
        cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
        TimedScope ts(st, CQ_KERNEL_LORA_ADD);
        count_launch();
        return launch_pdl(k_lora_row, dim3((unsigned)M), dim3(kLoraThreads), 0, st, 1, p) ==
                       cudaSuccess
                   ? CQ_OK
                   : CQ_ERR_CUDA;
    } catch (...) {
        return CQ_ERR_CUDA;
    }
}

}  // extern "C"

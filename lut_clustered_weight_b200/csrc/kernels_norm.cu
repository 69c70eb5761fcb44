// kernels_norm.cu -- cq_residual_norm: norm of a block's output, gate, residual
// scale, residual add, the norm before the next block, and optionally the
// rotated codes of the result, sm_100a.
//
// r' = round(resid_scale * r + block_scale * g * post(y)), x = fp16(pre(r')).
// Everything between two roundings is fp64: a code is decided on x and x on
// r', so a value next to a rounding border has to fall on the same side
// whatever the order of a sum (an fp32 sum would move about one x in a
// thousand by an ulp, and with it now and then a code).
#include <cmath>

#include "cq_common.cuh"
#include "cq_internal.h"
#include "rotate_quantize.cuh"

namespace cq {

constexpr int kNormThreads = 256;

struct NormArgs {
    const float *y;
    const __half *gate;
    const __half *post_w, *post_b;
    const void *resid;
    void *resid_out;
    const __half *pre_w, *pre_b;
    __half *x;
    uint8_t *q;
    float *s;
    int64_t ldq;
    double eps, resid_scale, block_scale;
    int H, layer, post_norm, gate_mode, resid_bits, bits, log2b;
};

// Sum over the CTA, the same value (and order) for every thread.
template <int THREADS>
CQ_DEV double block_sum(double v, double *red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();  // red may still be read from the last sum
    if (lane == 0) red[warp] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; w++) t += red[w];
    return t;
}

// buf[0, H) = norm(buf); the caller synchronizes before and after.
CQ_DEV void norm_row(double *buf, const NormArgs &a, const __half *w, const __half *b,
                     double *red) {
    const int H = a.H;
    double mean = 0.0;
    if (a.layer) {
        double t = 0.0;
        for (int i = threadIdx.x; i < H; i += kNormThreads) t += buf[i];
        mean = block_sum<kNormThreads>(t, red) / H;
    }
    double t = 0.0;
    for (int i = threadIdx.x; i < H; i += kNormThreads) {
        const double d = buf[i] - mean;
        t += d * d;
    }
    const double inv = 1.0 / sqrt(block_sum<kNormThreads>(t, red) / H + a.eps);
    for (int i = threadIdx.x; i < H; i += kNormThreads) {
        double v = (buf[i] - mean) * inv;
        if (w) v *= (double)__half2float(w[i]);
        if (b) v += (double)__half2float(b[i]);
        buf[i] = v;
    }
}

__global__ void __launch_bounds__(kNormThreads) k_residual_norm(const NormArgs a) {
    extern __shared__ __align__(16) double buf[];
    __shared__ double red[33];
    griddep_wait();
    griddep_launch();
    const int H = a.H, tid = threadIdx.x;
    const int64_t t = blockIdx.x, row = t * H;
    const __half *r16 = reinterpret_cast<const __half *>(a.resid) + row;
    const float *r32 = reinterpret_cast<const float *>(a.resid) + row;
    if (a.y) {
        for (int i = tid; i < H; i += kNormThreads) buf[i] = (double)a.y[row + i];
        if (a.post_norm) norm_row(buf, a, a.post_w, a.post_b, red);
    }
    for (int i = tid; i < H; i += kNormThreads) {
        double r = a.resid_bits == 16 ? (double)__half2float(r16[i]) : (double)r32[i];
        if (a.y) {
            double v = buf[i];
            if (a.gate_mode) {
                const int64_t g = a.gate_mode == CQ_GATE_CHANNEL ? i
                                : a.gate_mode == CQ_GATE_TOKEN ? t : row + i;
                v *= (double)__half2float(a.gate[g]);
            }
            r = a.resid_scale * r + a.block_scale * v;
            if (a.resid_bits == 16) {
                const __half h = __double2half(r);
                reinterpret_cast<__half *>(a.resid_out)[row + i] = h;
                r = (double)__half2float(h);
            } else {
                const float f = __double2float_rn(r);
                reinterpret_cast<float *>(a.resid_out)[row + i] = f;
                r = (double)f;
            }
        }
        buf[i] = r;
    }
    norm_row(buf, a, a.pre_w, a.pre_b, red);
    for (int i = tid; i < H; i += kNormThreads) {
        const __half h = __double2half(buf[i]);
        a.x[row + i] = h;
        buf[i] = (double)__half2float(h);
    }
    if (!a.bits) return;
    __syncthreads();
    block_fwht<kNormThreads>(buf, H, a.log2b);
    const double A = block_absmax<kNormThreads>(buf, H, red);
    const RqF16 none{};
    block_quantize_range<kNormThreads>(buf, H, 0, a.bits, A, a.q + t * a.ldq, none, t, H);
    if (tid == 0)
        a.s[t] = A > 0.0 ? quant_scale(A, a.log2b, (1 << (a.bits - 1)) - 1) : 0.0f;
}

static cudaError_t launch_residual_norm(const NormArgs &a, int64_t T, cudaStream_t st) {
    TimedScope ts(st, CQ_KERNEL_RESIDUAL_NORM);
    count_launch();
    return launch_pdl(k_residual_norm, dim3((unsigned)T), dim3(kNormThreads),
                      (size_t)a.H * sizeof(double), st, 1, a);
}

static bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace cq

extern "C" CQ_API cq_status cq_residual_norm(const cq_norm_desc *d, int64_t T, const float *y,
                                             const void *gate, const void *post_weight,
                                             const void *post_bias, const void *resid,
                                             void *resid_out, const void *pre_weight,
                                             const void *pre_bias, void *x_out, void *q_out,
                                             float *s_out, cq_stream_t stream) {
    using namespace cq;
    if (!d || T < 0 || d->H <= 0) return CQ_ERR_INVALID_ARGUMENT;
    if (d->norm != CQ_NORM_RMS && d->norm != CQ_NORM_LAYER) return CQ_ERR_INVALID_ARGUMENT;
    if (d->post_norm != 0 && d->post_norm != 1) return CQ_ERR_INVALID_ARGUMENT;
    if (d->gate_mode < CQ_GATE_NONE || d->gate_mode > CQ_GATE_ELEMENT)
        return CQ_ERR_INVALID_ARGUMENT;
    if (d->resid_bits != 16 && d->resid_bits != 32) return CQ_ERR_INVALID_ARGUMENT;
    if (d->act_bits != 0 && d->act_bits != 4 && d->act_bits != 8) return CQ_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(d->eps) || !(d->eps > 0.0) || !std::isfinite(d->resid_scale) ||
        !std::isfinite(d->block_scale))
        return CQ_ERR_INVALID_ARGUMENT;
    const int b = d->had_block;
    if (d->act_bits ? (b <= 0 || (b & (b - 1)) || d->H % b) : b != 0)
        return CQ_ERR_INVALID_ARGUMENT;
    if (!y && (d->post_norm || d->gate_mode || d->resid_scale != 1.0 || d->block_scale != 1.0))
        return CQ_ERR_INVALID_ARGUMENT;
    if (!d->post_norm && (post_weight || post_bias)) return CQ_ERR_INVALID_ARGUMENT;
    if (d->norm == CQ_NORM_RMS && (post_bias || pre_bias)) return CQ_ERR_INVALID_ARGUMENT;
    if (T > 0) {
        if (!resid || !x_out || (y && !resid_out)) return CQ_ERR_INVALID_ARGUMENT;
        if ((d->gate_mode != CQ_GATE_NONE) != (gate != nullptr)) return CQ_ERR_INVALID_ARGUMENT;
        if ((d->act_bits > 0) != (q_out != nullptr) || (d->act_bits > 0) != (s_out != nullptr))
            return CQ_ERR_INVALID_ARGUMENT;
        if (x_out == resid || x_out == resid_out || static_cast<const void *>(y) == x_out ||
            (y && static_cast<const void *>(y) == resid_out))
            return CQ_ERR_INVALID_ARGUMENT;
    }
    const void *ps[] = {y,          gate,     post_weight, post_bias, resid, resid_out,
                        pre_weight, pre_bias, x_out,       q_out,     s_out};
    for (const void *p : ps)
        if (!al16(p)) return CQ_ERR_INVALID_ARGUMENT;
    if (d->H % 8 || d->H > kMaxK || T > INT32_MAX || b > 8192) return CQ_ERR_UNSUPPORTED;
    if (T == 0) return CQ_OK;
    NormArgs a{};
    a.y = y;
    a.gate = reinterpret_cast<const __half *>(gate);
    a.post_w = reinterpret_cast<const __half *>(post_weight);
    a.post_b = reinterpret_cast<const __half *>(post_bias);
    a.resid = resid;
    a.resid_out = resid_out;
    a.pre_w = reinterpret_cast<const __half *>(pre_weight);
    a.pre_b = reinterpret_cast<const __half *>(pre_bias);
    a.x = reinterpret_cast<__half *>(x_out);
    a.q = reinterpret_cast<uint8_t *>(q_out);
    a.s = s_out;
    a.H = (int)d->H;
    a.ldq = d->H * d->act_bits / 8;
    a.eps = d->eps;
    a.resid_scale = d->resid_scale;
    a.block_scale = d->block_scale;
    a.layer = d->norm == CQ_NORM_LAYER;
    a.post_norm = d->post_norm;
    a.gate_mode = d->gate_mode;
    a.resid_bits = d->resid_bits;
    a.bits = d->act_bits;
    for (a.log2b = 0; (1 << a.log2b) < b; a.log2b++) {
    }
    try {
        return launch_residual_norm(a, T, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? CQ_OK
                   : CQ_ERR_CUDA;
    } catch (...) {
        return CQ_ERR_CUDA;
    }
}

// kernels_norm.cu -- cq_residual_norm: norm of a block's output, gate, residual
// scale, residual add, the norm before the next block, and optionally the
// rotated codes of the result, sm_100a.
//
// r' = round(resid_scale * r + block_scale * g * post(y)), x = fp16(pre(r')).
// Everything between two roundings is fp64: a code is decided on x and x on
// r', so a value next to a rounding border has to fall on the same side
// whatever the order of a sum (an fp32 sum would move about one x in a
// thousand by an ulp, and with it now and then a code).
#include <algorithm>
#include <cmath>

#include "cq_common.cuh"
#include "cq_internal.h"
#include "rotate_quantize.cuh"

namespace cq {

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
    int64_t ldq, T;
    double eps, resid_scale, block_scale;
    int H, layer, post_norm, gate_mode, bits, log2b;
    int tpr, rpc;  // threads per row (a multiple of 32), rows per CTA
};

// A row's threads hold it in registers, E consecutive channels each, and share
// sums and the exchange area of the rotation through shared memory.
struct RowThreads {
    int row, j;       // row of the CTA, thread of the row
    int warps, warp0; // warps of a row, first warp of this row
    double *red;      // [2][32], the half alternates so that one barrier a sum is enough
    int flip;
};

template <bool MAX>
CQ_DEV double row_reduce(double v, RowThreads &rt) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const double u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmax(v, u) : v + u;
    }
    double *red = rt.red + 32 * rt.flip;
    rt.flip ^= 1;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[rt.warp0];
    for (int w = 1; w < rt.warps; w++) v = MAX ? fmax(v, red[rt.warp0 + w]) : v + red[rt.warp0 + w];
    return v;
}

// 8 fp16 values as fp64
CQ_DEV void halves(const uint4 &u, double *v) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = __half22float2(h[i]);
        v[2 * i] = (double)f.x;
        v[2 * i + 1] = (double)f.y;
    }
}

// v = norm(v) over the row; nv of the thread's E channels exist (0 beyond).
template <int E>
CQ_DEV void norm_regs(double (&v)[E], int nv, const NormArgs &a, const __half *w, const __half *b,
                      int c0, RowThreads &rt) {
    const double n = (double)a.H;
    if (a.layer) {
        double t = 0.0;
#pragma unroll
        for (int i = 0; i < E; i++) t += v[i];
        const double mean = row_reduce<false>(t, rt) / n;
#pragma unroll
        for (int i = 0; i < E; i++) v[i] = i < nv ? v[i] - mean : 0.0;
    }
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < E; i++) t = fma(v[i], v[i], t);
    const double inv = 1.0 / sqrt(row_reduce<false>(t, rt) / n + a.eps);
#pragma unroll
    for (int c = 0; c < E; c += 8) {
        double f[8];
        if (c < nv && w) {
            halves(*reinterpret_cast<const uint4 *>(w + c0 + c), f);
#pragma unroll
            for (int i = 0; i < 8; i++) v[c + i] *= inv * f[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) v[c + i] *= inv;
        }
        if (c < nv && b) {
            halves(*reinterpret_cast<const uint4 *>(b + c0 + c), f);
#pragma unroll
            for (int i = 0; i < 8; i++) v[c + i] += f[i];
        }
    }
}

// N butterfly levels over 2^N registers at v[0 .. 2^N)
template <int N>
CQ_DEV void butterflies(double *v) {
#pragma unroll
    for (int h = 1; h < (1 << N); h <<= 1)
#pragma unroll
        for (int i = 0; i < (1 << N); i++)
            if ((i & h) == 0) {
                const double x = v[i], y = v[i + h];
                v[i] = x + y;
                v[i + h] = x - y;
            }
}

template <int E>
struct Log2;
template <>
struct Log2<16> {
    static constexpr int v = 4;
};
template <>
struct Log2<32> {
    static constexpr int v = 5;
};

// Place of position p in the exchange area: one double of padding per E, so
// that threads writing E consecutive positions each hit different banks.
template <int E>
CQ_DEV int xplace(int p) {
    return p + (p >> Log2<E>::v);
}

// Position of register i of thread j in the stage that works on index bits
// [s, s + N): column c = j + (i >> N) * T of the row's H / 2^N columns, its
// element i & (2^N - 1).
template <int N>
CQ_DEV int xpos(int i, int j, int T, int s) {
    const int c = j + (i >> N) * T;
    return ((c >> s) << (s + N)) + ((i & ((1 << N) - 1)) << s) + (c & ((1 << s) - 1));
}

template <int E, int N>
CQ_DEV void stage(double (&v)[E], double *xch, int j, int T, int s, bool last) {
#pragma unroll
    for (int i = 0; i < E; i++) v[i] = xch[xplace<E>(xpos<N>(i, j, T, s))];
#pragma unroll
    for (int i = 0; i < E; i += 1 << N) butterflies<N>(v + i);
    if (!last) {
#pragma unroll
        for (int i = 0; i < E; i++) xch[xplace<E>(xpos<N>(i, j, T, s))] = v[i];
    }
}

template <int E, int N>
CQ_DEV void put_codes(const double (&v)[E], int8_t *cb, int j, int T, int s, double R, long long Ai,
                      int qmax) {
#pragma unroll
    for (int i = 0; i < E; i++) {
        // round(v R) to even by adding 1.5 * 2^52; within 5e-7 of a tie the exact
        // rational decides
        const double big = fma(v[i], R, 6755399441055744.0);
        const double r = fma(v[i], R, -(big - 6755399441055744.0));
        int c = __double2loint(big);
        if ((__double2hiint(r) & 0x7fffffff) >= 0x3fdffffe) c = quantize_tie(v[i], Ai, qmax);
        cb[N ? xpos<N>(i, j, T, s) : E * j + i] = (int8_t)c;
    }
}

// 16 code bytes -> 8 bytes of nibbles, low nibble first
CQ_DEV uint2 nibbles(const uint4 &u) {
    auto pack = [](uint32_t a, uint32_t b) {
        a &= 0x0f0f0f0fu;
        b &= 0x0f0f0f0fu;
        a |= a >> 4;
        b |= b >> 4;
        return prmt(a, b, 0x6420);
    };
    return make_uint2(pack(u.x, u.y), pack(u.z, u.w));
}

// Rows in registers, E channels a thread.  The rotation's index bits are taken
// log2 E at a time: the first in the layout of the loads, each further group
// after an exchange through shared memory that puts the group's 2^N values into
// one thread (2 shared accesses a value for up to log2 E levels; a lane shuffle
// of an fp64 value costs 2 instructions a level).  Codes go through shared
// memory once, as bytes, back to the layout of the loads.
template <int E, bool R16, bool CODES>
__global__ void __launch_bounds__(512) k_residual_norm(const NormArgs a) {
    extern __shared__ __align__(16) double xch_all[];
    __shared__ double red[64];
    constexpr int LE = Log2<E>::v;
    griddep_wait();
    griddep_launch();
    RowThreads rt;
    rt.row = threadIdx.x / a.tpr;
    rt.j = threadIdx.x - rt.row * a.tpr;
    rt.warps = a.tpr >> 5;
    rt.warp0 = rt.row * rt.warps;
    rt.red = red;
    rt.flip = 0;
    const int H = a.H, j = rt.j, c0 = E * j;
    const int64_t t = (int64_t)blockIdx.x * a.rpc + rt.row;
    const int nv = t < a.T ? max(0, min(E, H - c0)) : 0;  // a multiple of 8
    const int64_t at = t * H + c0;

    double v[E];
#pragma unroll
    for (int i = 0; i < E; i++) v[i] = 0.0;
    // everything the row reads once is requested before the first use
    uint4 rr[R16 ? E / 8 : E / 4];
    if (R16) {
        const uint4 *src = reinterpret_cast<const uint4 *>(reinterpret_cast<const __half *>(a.resid) + at);
#pragma unroll
        for (int c = 0; c < E / 8; c++) rr[c] = 8 * c < nv ? __ldcs(src + c) : make_uint4(0, 0, 0, 0);
    } else {
        const uint4 *src = reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(a.resid) + at);
#pragma unroll
        for (int c = 0; c < E / 4; c++) rr[c] = 4 * c < nv ? __ldcs(src + c) : make_uint4(0, 0, 0, 0);
    }
    if (a.y) {
        const float4 *src = reinterpret_cast<const float4 *>(a.y + at);
        float4 yy[E / 4];
#pragma unroll
        for (int c = 0; c < E / 4; c++)
            yy[c] = 4 * c < nv ? __ldcs(src + c) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < E / 4; c++) {
            v[4 * c] = (double)yy[c].x;
            v[4 * c + 1] = (double)yy[c].y;
            v[4 * c + 2] = (double)yy[c].z;
            v[4 * c + 3] = (double)yy[c].w;
        }
        if (a.post_norm) norm_regs<E>(v, nv, a, a.post_w, a.post_b, c0, rt);
        if (a.gate_mode == CQ_GATE_TOKEN) {
            const double g = nv > 0 ? (double)__half2float(a.gate[t]) : 0.0;
#pragma unroll
            for (int i = 0; i < E; i++) v[i] *= g;
        } else if (a.gate_mode != CQ_GATE_NONE) {
            const __half *gp = a.gate + (a.gate_mode == CQ_GATE_CHANNEL ? c0 : at);
#pragma unroll
            for (int c = 0; c < E; c += 8) {
                double f[8];
                if (c < nv) {
                    halves(*reinterpret_cast<const uint4 *>(gp + c), f);
#pragma unroll
                    for (int i = 0; i < 8; i++) v[c + i] *= f[i];
                }
            }
        }
    }
    // r' = round(resid_scale * r + block_scale * v)
    if (R16) {
#pragma unroll
        for (int c = 0; c < E / 8; c++) {
            double f[8];
            halves(rr[c], f);
            if (a.y) {
                uint4 o;
                __half *h = reinterpret_cast<__half *>(&o);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    h[i] = __double2half(fma(a.resid_scale, f[i], a.block_scale * v[8 * c + i]));
                if (8 * c < nv)
                    *reinterpret_cast<uint4 *>(reinterpret_cast<__half *>(a.resid_out) + at + 8 * c) = o;
                halves(o, f);
            }
#pragma unroll
            for (int i = 0; i < 8; i++) v[8 * c + i] = 8 * c < nv ? f[i] : 0.0;
        }
    } else {
#pragma unroll
        for (int c = 0; c < E / 4; c++) {
            const float *r = reinterpret_cast<const float *>(&rr[c]);
            float4 o;
            float *f = reinterpret_cast<float *>(&o);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                f[i] = r[i];
                if (a.y)
                    f[i] = __double2float_rn(
                        fma(a.resid_scale, (double)r[i], a.block_scale * v[4 * c + i]));
            }
            if (a.y && 4 * c < nv)
                *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.resid_out) + at + 4 * c) = o;
#pragma unroll
            for (int i = 0; i < 4; i++) v[4 * c + i] = 4 * c < nv ? (double)f[i] : 0.0;
        }
    }
    norm_regs<E>(v, nv, a, a.pre_w, a.pre_b, c0, rt);
#pragma unroll
    for (int c = 0; c < E / 8; c++) {
        uint4 o;
        __half *h = reinterpret_cast<__half *>(&o);
#pragma unroll
        for (int i = 0; i < 8; i++) h[i] = __double2half(v[8 * c + i]);
        if (8 * c < nv) *reinterpret_cast<uint4 *>(a.x + at + 8 * c) = o;
        if (CODES) halves(o, v + 8 * c);
    }
    if (!CODES) return;

    // ---- rotation (channels beyond the row are zeros of whole blocks of 8)
    switch (min(a.log2b, LE)) {
    case 0: break;
#define CQ_FIRST(N) \
    case N: \
        for (int i = 0; i < E; i += 1 << N) butterflies<N>(v + i); \
        break;
        CQ_FIRST(1) CQ_FIRST(2) CQ_FIRST(3) CQ_FIRST(4)
    default:
        if (LE == 5) butterflies<LE>(v);
#undef CQ_FIRST
    }
    const int T = H / E;  // threads of the row with channels (rotation blocks over E divide H)
    double *xch = xch_all + (size_t)rt.row * (H + T);
    int s = 0, n = 0;  // bits [s, s + n) of the last exchange (n = 0: none)
    if (a.log2b > LE) {
        const bool mine = nv > 0;
        if (mine) {
#pragma unroll
            for (int i = 0; i < E; i++) xch[xplace<E>(c0 + i)] = v[i];
        }
        for (s = LE; s < a.log2b; s += n) {
            n = min(LE, a.log2b - s);
            const bool last = s + n == a.log2b;
            __syncthreads();
            if (mine) {
                switch (n) {
                case 1: stage<E, 1>(v, xch, j, T, s, last); break;
                case 2: stage<E, 2>(v, xch, j, T, s, last); break;
                case 3: stage<E, 3>(v, xch, j, T, s, last); break;
                case 4: stage<E, 4>(v, xch, j, T, s, last); break;
                default: stage<E, LE>(v, xch, j, T, s, last); break;
                }
            }
        }
        s -= n;
    }
    // ---- codes
    double mx = 0.0;
#pragma unroll
    for (int i = 0; i < E; i++) mx = fmax(mx, fabs(v[i]));
    const double A = row_reduce<true>(mx, rt);  // its barrier also frees the exchange area
    const int qmax = (1 << (a.bits - 1)) - 1;
    const long long Ai = __double2ll_rn(A * 16777216.0);
    const double R = Ai > 0 ? __ddiv_rn((double)qmax, A) : 0.0;
    int8_t *cb = reinterpret_cast<int8_t *>(xch);
    if (nv > 0) {
        switch (n) {
        case 0: put_codes<E, 0>(v, cb, j, T, s, R, Ai, qmax); break;
        case 1: put_codes<E, 1>(v, cb, j, T, s, R, Ai, qmax); break;
        case 2: put_codes<E, 2>(v, cb, j, T, s, R, Ai, qmax); break;
        case 3: put_codes<E, 3>(v, cb, j, T, s, R, Ai, qmax); break;
        case 4: put_codes<E, 4>(v, cb, j, T, s, R, Ai, qmax); break;
        default: put_codes<E, LE>(v, cb, j, T, s, R, Ai, qmax); break;
        }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < E; c += 8) {
        if (c >= nv) break;
        const uint2 u = *reinterpret_cast<const uint2 *>(cb + c0 + c);
        if (a.bits == 8) {
            *reinterpret_cast<uint2 *>(a.q + t * a.ldq + c0 + c) = u;
        } else {
            const uint2 k = nibbles(make_uint4(u.x, u.y, 0, 0));
            *reinterpret_cast<uint32_t *>(a.q + t * a.ldq + (c0 + c) / 2) = k.x;
        }
    }
    if (j == 0 && nv > 0) a.s[t] = Ai > 0 ? quant_scale(A, a.log2b, qmax) : 0.0f;
}

template <int E>
static cudaError_t launch_rows(NormArgs a, bool r16, cudaStream_t st) {
    const int T = (a.H + E - 1) / E;
    a.tpr = (T + 31) / 32 * 32;
    // short rows share a CTA of up to 256 threads
    a.rpc = (int)std::min<int64_t>(std::max(1, 256 / a.tpr), a.T);
    const bool codes = a.bits > 0;
    const size_t smem = codes ? (size_t)a.rpc * (a.H + a.H / E) * sizeof(double) : 0;
    auto kern = r16 ? (codes ? k_residual_norm<E, true, true> : k_residual_norm<E, true, false>)
                    : (codes ? k_residual_norm<E, false, true> : k_residual_norm<E, false, false>);
    count_launch();
    return launch_pdl(kern, dim3((unsigned)((a.T + a.rpc - 1) / a.rpc)), dim3(a.tpr * a.rpc), smem,
                      st, 1, a);
}

// 16 channels a thread; 32 for rows over 8192, which would need blocks of more
// than 512 threads and with them half the registers.
static cudaError_t launch_residual_norm(const NormArgs &a, bool r16, cudaStream_t st) {
    TimedScope ts(st, CQ_KERNEL_RESIDUAL_NORM);
    return a.H <= 8192 ? launch_rows<16>(a, r16, st) : launch_rows<32>(a, r16, st);
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
    a.T = T;
    a.bits = d->act_bits;
    for (a.log2b = 0; (1 << a.log2b) < b; a.log2b++) {
    }
    try {
        return launch_residual_norm(a, d->resid_bits == 16, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? CQ_OK
                   : CQ_ERR_CUDA;
    } catch (...) {
        return CQ_ERR_CUDA;
    }
}

// kernels_rope.cu -- cq_rope_qkv: per-head norm of q and k, rotary positions,
// and the k / v rows of a cache, from the fp32 rows of a fused QKV projection,
// sm_100a.
//
// A head is head_dim / 8 units of 8 channels; a group of G lanes (a power of
// two, so that the norm's sum is a shuffle reduction) holds one head, one unit
// per lane.  A turned unit holds 4 whole pairs, so nothing crosses lanes
// but the sum: channels [4u, 4u+4) and rot/2 + [4u, 4u+4) (half layout), or
// [8u, 8u+8) (interleaved).  The angles of a token are formed once per CTA, in
// fp64: at position 10^6 an fp32 product is off by 0.06 rad.
#include <cmath>

#include "cq_common.cuh"
#include "cq_internal.h"

namespace cq {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 256;

struct RopeArgs {
    const float *qkv;
    const int32_t *positions;
    const float *inv_freq;
    const __half *qw, *kw;
    __half *q, *k, *v;
    const int64_t *slots;
    int64_t tok_stride, head_stride, n_slots;
    int n_q, n_kv, D, rot, interleaved;
    int log2g;           // lanes per head: 2^log2g >= D / 8
    int heads_per_cta;   // heads of a token per CTA (blockIdx.y: which of them)
    float attn_scale, eps;
};

CQ_DEV uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// What one lane does in a round: its unit of head h.
struct RopeUnit {
    int h, c0, c1;  // head, first channel of the unit's two halves
    bool live, turned, is_v;
    float4 a, b;
};

CQ_DEV void load_unit(RopeUnit &u, const RopeArgs &p, const float *row, int h, int h_end, int lane) {
    u.h = h;
    u.live = h < h_end && lane < (p.D >> 3);
    u.is_v = h >= p.n_q + p.n_kv;
    u.turned = !u.is_v && lane < (p.rot >> 3);
    const bool apart = u.turned && !p.interleaved;
    u.c0 = apart ? 4 * lane : 8 * lane;
    u.c1 = apart ? (p.rot >> 1) + 4 * lane : u.c0 + 4;
    u.a = u.b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (u.live) {
        const float *src = row + h * p.D;
        u.a = __ldcs(reinterpret_cast<const float4 *>(src + u.c0));
        u.b = __ldcs(reinterpret_cast<const float4 *>(src + u.c1));
    }
}

__global__ void __launch_bounds__(kRopeThreads) k_rope_qkv(const RopeArgs p) {
    __shared__ float2 cs[kRopeMaxDim / 2];
    griddep_wait();
    griddep_launch();
    const int64_t m = blockIdx.x;
    const int heads = p.n_q + 2 * p.n_kv;
    const int G = 1 << p.log2g, lane = threadIdx.x & (G - 1), groups = kRopeThreads >> p.log2g;
    const int h_end = min(heads, ((int)blockIdx.y + 1) * p.heads_per_cta);
    int h0 = blockIdx.y * p.heads_per_cta;
    const int gh = threadIdx.x >> p.log2g;
    const float *row = p.qkv + m * heads * p.D;
    // the first round's values are on their way while the angles are formed, every
    // other round's while the one before is worked on
    RopeUnit next;
    load_unit(next, p, row, h0 + gh, h_end, lane);
    const int64_t slot = p.slots ? p.slots[m] : m;
    const bool cached = !p.slots || (slot >= 0 && slot < p.n_slots);
    if (threadIdx.x < (p.rot >> 1)) {
        // in turns, so that the reduction is a subtraction of the nearest whole one
        const double turns =
            (double)p.positions[m] * (double)p.inv_freq[threadIdx.x] * 0.15915494309189535;
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        cs[threadIdx.x] = make_float2(c * p.attn_scale, s * p.attn_scale);
    }
    __syncthreads();
    // every lane of a warp runs the same rounds (the shuffles need all of them)
    for (; h0 < h_end; h0 += groups) {
        const RopeUnit u = next;
        if (h0 + groups < h_end) load_unit(next, p, row, h0 + groups + gh, h_end, lane);
        float v[8] = {u.a.x, u.a.y, u.a.z, u.a.w, u.b.x, u.b.y, u.b.z, u.b.w};
        const __half *w = u.is_v ? nullptr : u.h < p.n_q ? p.qw : p.kw;
        if (p.qw || p.kw) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i++) ss += v[i] * v[i];
            for (int o = G >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (w && u.live) {
                const float inv = 1.0f / sqrtf(ss / (float)p.D + p.eps);
                const uint2 w0 = *reinterpret_cast<const uint2 *>(w + u.c0);
                const uint2 w1 = *reinterpret_cast<const uint2 *>(w + u.c1);
                const uint32_t wh[4] = {w0.x, w0.y, w1.x, w1.y};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&wh[i]));
                    v[2 * i] *= inv * f.x;
                    v[2 * i + 1] *= inv * f.y;
                }
            }
        }
        if (!u.live) continue;
        if (u.turned) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 t = cs[4 * lane + i];
                if (p.interleaved) {
                    const float a = v[2 * i], b = v[2 * i + 1];
                    v[2 * i] = a * t.x - b * t.y;
                    v[2 * i + 1] = a * t.y + b * t.x;
                } else {
                    const float a = v[i], b = v[i + 4];
                    v[i] = a * t.x - b * t.y;
                    v[i + 4] = a * t.y + b * t.x;
                }
            }
        }
        __half *dst;
        if (u.h < p.n_q) {
            dst = p.q + (m * p.n_q + u.h) * p.D;
        } else {
            if (!cached) continue;
            const int hk = u.is_v ? u.h - p.n_q - p.n_kv : u.h - p.n_q;
            dst = (u.is_v ? p.v : p.k) + slot * p.tok_stride + hk * p.head_stride;
        }
        const uint2 lo = make_uint2(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]));
        const uint2 hi = make_uint2(pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
        if (u.c1 == u.c0 + 4 && !(u.c0 & 7)) {
            *reinterpret_cast<uint4 *>(dst + u.c0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
            *reinterpret_cast<uint2 *>(dst + u.c0) = lo;
            *reinterpret_cast<uint2 *>(dst + u.c1) = hi;
        }
    }
}

static bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace cq

extern "C" CQ_API cq_status cq_rope_qkv(const cq_rope_desc *d, int64_t M, const float *qkv,
                                        const int32_t *positions, const float *inv_freq,
                                        const void *q_weight, const void *k_weight, void *q_out,
                                        void *k_out, void *v_out, const int64_t *slots,
                                        cq_stream_t stream) {
    using namespace cq;
    if (!d || M < 0) return CQ_ERR_INVALID_ARGUMENT;
    if (d->n_q < 1 || d->n_kv < 1 || d->head_dim < 1 || d->rot_dim < 0 ||
        d->rot_dim > d->head_dim)
        return CQ_ERR_INVALID_ARGUMENT;
    if (d->interleaved != 0 && d->interleaved != 1) return CQ_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(d->attn_scale) || !std::isfinite(d->eps) || !(d->eps > 0.0f))
        return CQ_ERR_INVALID_ARGUMENT;
    if (d->kv_token_stride < 0 || d->kv_head_stride < 0 || (slots && d->n_slots < 0))
        return CQ_ERR_INVALID_ARGUMENT;
    if ((d->rot_dim > 0) != (inv_freq != nullptr)) return CQ_ERR_INVALID_ARGUMENT;
    if (M > 0 && (!qkv || !positions || !q_out || !k_out || !v_out))
        return CQ_ERR_INVALID_ARGUMENT;
    if (M > 0 && (k_out == v_out || q_out == k_out || q_out == v_out))
        return CQ_ERR_INVALID_ARGUMENT;
    const void *ps[] = {qkv, positions, inv_freq, q_weight, k_weight, q_out, k_out, v_out, slots};
    for (const void *p : ps)
        if (!al16(p)) return CQ_ERR_INVALID_ARGUMENT;
    if (d->head_dim % 8 || d->head_dim > kRopeMaxDim || d->rot_dim % 8 ||
        d->n_q > 1024 || d->n_kv > 1024 || d->n_q + 2 * d->n_kv > 1024 ||
        d->kv_token_stride % 8 || d->kv_head_stride % 8 || M > INT32_MAX)
        return CQ_ERR_UNSUPPORTED;
    if (M == 0) return CQ_OK;
    RopeArgs p{};
    p.qkv = qkv;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.qw = reinterpret_cast<const __half *>(q_weight);
    p.kw = reinterpret_cast<const __half *>(k_weight);
    p.q = reinterpret_cast<__half *>(q_out);
    p.k = reinterpret_cast<__half *>(k_out);
    p.v = reinterpret_cast<__half *>(v_out);
    p.slots = slots;
    p.tok_stride = d->kv_token_stride;
    p.head_stride = d->kv_head_stride;
    p.n_slots = d->n_slots;
    p.n_q = (int)d->n_q;
    p.n_kv = (int)d->n_kv;
    p.D = (int)d->head_dim;
    p.rot = (int)d->rot_dim;
    p.interleaved = d->interleaved;
    p.attn_scale = d->attn_scale;
    p.eps = d->eps;
    for (p.log2g = 0; (8 << p.log2g) < p.D; p.log2g++) {
    }
    // one CTA a token (the angles once); few tokens: one round of heads a CTA
    const int heads = p.n_q + 2 * p.n_kv, groups = kRopeThreads >> p.log2g;
    const int rounds = (heads + groups - 1) / groups;
    const bool split = M * rounds <= 4LL * sm_count();
    p.heads_per_cta = split ? groups : heads;
    try {
        cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
        TimedScope ts(st, CQ_KERNEL_ROPE_QKV);
        count_launch();
        return launch_pdl(k_rope_qkv, dim3((unsigned)M, split ? rounds : 1), dim3(kRopeThreads), 0, st, 1, p) ==
                       cudaSuccess
                   ? CQ_OK
                   : CQ_ERR_CUDA;
    } catch (...) {
        return CQ_ERR_CUDA;
    }
}

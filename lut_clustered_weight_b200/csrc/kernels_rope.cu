// kernels_rope.cu -- cq_rope_qkv: per-head norm of q and k, rotary positions,
// and the k / v rows of a cache, from the fp32 rows of a fused QKV projection,
// sm_100a.
//
// A head is head_dim / 8 units of 8 channels, one unit a thread and round; with a norm
// a head's units are in a group of G lanes (a power of two, so that the sum is a
// shuffle reduction), else the units of all heads follow one another.  A turned
// unit holds 4 whole pairs, so nothing crosses lanes but the sum: channels [4u, 4u+4)
// and rot/2 + [4u, 4u+4) (half layout), or [8u, 8u+8) (interleaved).  The angles of a
// token are formed once per CTA, in fp64: at position 10^6 an fp32 product is off by
// 0.06 rad.
#include <cmath>
#include <type_traits>

#include "cq_common.cuh"
#include "cq_internal.h"

namespace cq {

constexpr int kRopeThreads = 256;  // at most
constexpr int kRopeMaxDim = 256;

struct RopeArgs {
    const float *qkv;
    const int32_t *positions;
    const float *inv_freq;
    const __half *qw, *kw;
    __half *q, *k, *v;
    const int64_t *slots;
    int64_t tok_stride, head_stride, n_slots;
    int n_q, n_kv, D, rot;
    int width, log2w;    // threads per head: D / 8, or G = 2^log2w
    int step_h, step_u;  // the block's threads are step_h heads and step_u units
    int heads_per_cta;   // heads of a token per CTA (blockIdx.y: which of them)
    float attn_scale, eps;
};

CQ_DEV uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// What one thread does in a round: a unit of head h.
struct RopeUnit {
    int h, u, c0, c1;  // head, unit, first channel of the unit's two halves
    bool live, turned, is_v;
    float4 a, b;
};

template <bool INTER>
CQ_DEV void load_unit(RopeUnit &u, const RopeArgs &p, const float *row, int h, int h_end, int unit) {
    u.h = h;
    u.u = unit;
    u.live = h < h_end && unit < (p.D >> 3);
    u.is_v = h >= p.n_q + p.n_kv;
    u.turned = !u.is_v && unit < (p.rot >> 3);
    const bool apart = u.turned && !INTER;
    u.c0 = apart ? 4 * unit : 8 * unit;
    u.c1 = apart ? (p.rot >> 1) + 4 * unit : u.c0 + 4;
    u.a = u.b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (u.live) {
        const float *src = row + h * p.D;
        u.a = __ldcs(reinterpret_cast<const float4 *>(src + u.c0));
        u.b = __ldcs(reinterpret_cast<const float4 *>(src + u.c1));
    }
}

// Memory-bound where tokens are many: 4096 of 32 + 8 heads of 128 in 28.3 us, 0.82 of a
// copy's bandwidth; 33.2 with the norms, whose sum is a chain of shuffles per round, of 4 at
// this width; one token 2 us.  PACKED: the units of all heads follow one another (width
// D / 8, not a power of two; 4096 tokens of 24 + 8 heads of 80: 16.9 us, and 21.1 in groups
// of 16 lanes).  The layout and the norm are template parameters: with all of them read at
// run time it was bound by instructions (29.2 us).
template <bool NORM, bool INTER, bool PACKED>
__global__ void __launch_bounds__(kRopeThreads) k_rope_qkv(const RopeArgs p) {
    __shared__ float2 cs[kRopeMaxDim / 2];
    griddep_wait();
    griddep_launch();
    const int64_t m = blockIdx.x;
    const int heads = p.n_q + 2 * p.n_kv;
    const int h_begin = blockIdx.y * p.heads_per_cta, h_end = min(heads, h_begin + p.heads_per_cta);
    const float *row = p.qkv + m * heads * p.D;
    // the first round's values are on their way while the angles are formed, every
    // other round's while the one before is worked on
    const int h_in = PACKED ? threadIdx.x / p.width : threadIdx.x >> p.log2w;
    int nh = h_begin + h_in, nu = threadIdx.x - (PACKED ? h_in * p.width : h_in << p.log2w);
    RopeUnit next;
    load_unit<INTER>(next, p, row, nh, h_end, nu);
    const int64_t slot = p.slots ? p.slots[m] : m;
    const bool cached = !p.slots || (slot >= 0 && slot < p.n_slots);
    for (int i = threadIdx.x; i < (p.rot >> 1); i += blockDim.x) {
        // in turns, so that the reduction is a subtraction of the nearest whole one
        const double turns = (double)p.positions[m] * (double)p.inv_freq[i] * 0.15915494309189535;
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        cs[i] = make_float2(c * p.attn_scale, s * p.attn_scale);
    }
    __syncthreads();
    // every thread runs the same rounds (the shuffles need all lanes); h0: at or before the
    // head of the round's first unit (packed units move on by step_u more a round; the
    // rounds past the last head find no live unit)
    for (int h0 = h_begin; h0 < h_end; h0 += p.step_h) {
        const RopeUnit u = next;
        nh += p.step_h;
        if (PACKED) {
            nu += p.step_u;
            if (nu >= p.width) {
                nu -= p.width;
                nh++;
            }
        }
        if (h0 + p.step_h < h_end) load_unit<INTER>(next, p, row, nh, h_end, nu);
        float v[8] = {u.a.x, u.a.y, u.a.z, u.a.w, u.b.x, u.b.y, u.b.z, u.b.w};
        const __half *w = u.is_v ? nullptr : u.h < p.n_q ? p.qw : p.kw;
        if (NORM) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i++) ss += v[i] * v[i];
            for (int o = p.width >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
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
                const float2 t = cs[4 * u.u + i];
                if (INTER) {
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

// Whether k rows m tok + h head of D elements, m < M and h < n_kv (both strides at least D),
// share addresses.  Rows m and m + dm of heads h + dh and h lie |dm tok - dh head| apart,
// closest at the dm on either side of dh head / tok.
static bool rows_share(int64_t M, int64_t n_kv, int64_t tok, int64_t head, int64_t D) {
    if (static_cast<__int128>(n_kv - 1) * head + D <= tok) return false;  // a row's heads side by side
    for (int64_t dh = 1; dh < n_kv; dh++) {
        const __int128 off = static_cast<__int128>(dh) * head;
        const __int128 below = off / tok, left = off - below * tok;
        if (below >= 1 && below < M && left < D) return true;
        if (below + 1 < M && tok - left < D) return true;
    }
    return false;
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
    // heads or rows of the cache on top of one another: within a row or a head, and, where
    // the rows are known (no slots), anywhere
    if ((d->n_kv > 1 && d->kv_head_stride < d->head_dim) ||
        (M > 1 && d->kv_token_stride < d->head_dim))
        return CQ_ERR_INVALID_ARGUMENT;
    if (!slots && M > 1 &&
        rows_share(M, d->n_kv, d->kv_token_stride, d->kv_head_stride, d->head_dim))
        return CQ_ERR_INVALID_ARGUMENT;
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
    p.attn_scale = d->attn_scale;
    p.eps = d->eps;
    const bool norm = p.qw || p.kw;
    for (p.log2w = 0; (8 << p.log2w) < p.D; p.log2w++) {
    }
    p.width = norm ? 1 << p.log2w : p.D / 8;
    const bool packed = p.width != 1 << p.log2w;
    // One CTA a token (the angles once), of no more threads than its rounds need (20 heads
    // of 64 and 4096 tokens: 8.2 us with 192, 10.2 with 256); few tokens: one round of
    // whole heads a CTA.
    const int heads = p.n_q + 2 * p.n_kv, units = heads * p.width;
    const int rounds = (units + kRopeThreads - 1) / kRopeThreads;
    const int threads = ((units + rounds - 1) / rounds + 31) / 32 * 32;
    const bool split = M * rounds <= 4LL * sm_count();
    p.step_h = threads / p.width;
    p.step_u = threads % p.width;
    p.heads_per_cta = split ? p.step_h : heads;
    const unsigned parts = (heads + p.heads_per_cta - 1) / p.heads_per_cta;
    auto pick = [&](auto inter) {
        constexpr bool I = decltype(inter)::value;
        return norm ? k_rope_qkv<true, I, false> : packed ? k_rope_qkv<false, I, true> : k_rope_qkv<false, I, false>;
    };
    try {
        cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
        TimedScope ts(st, CQ_KERNEL_ROPE_QKV);
        count_launch();
        auto kern = d->interleaved ? pick(std::true_type{}) : pick(std::false_type{});
        return launch_pdl(kern, dim3((unsigned)M, parts), dim3(threads), 0, st, 1, p) == cudaSuccess
                   ? CQ_OK
                   : CQ_ERR_CUDA;
    } catch (...) {
        return CQ_ERR_CUDA;
    }
}

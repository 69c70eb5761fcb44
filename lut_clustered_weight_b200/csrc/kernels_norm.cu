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
    double eps, resid_scale, block_scale, h, inv_h, sqrt_b;
    int H, layer, post_norm, gate_mode, bits, log2b;
    int tpr, rpc;  // threads per row (a multiple of 32), rows per CTA
    int64_t ahead; // rows from a row to the one that takes its place on the SM
};

// Threads of a row.  Sums go through shared memory; the half of the
// buffer alternates, so that one barrier a sum is enough.
struct RowThreads {
    int j;            // thread of the row
    int warps, warp0; // warps of a row, first warp of this row
    double *red;      // [2][32]
    int flip;
};

CQ_DEV double row_sum(double v, RowThreads &rt) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    double *red = rt.red + 32 * rt.flip;
    rt.flip ^= 1;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[rt.warp0];
#pragma unroll 4
    for (int w = 1; w < rt.warps; w++) v += red[rt.warp0 + w];
    return v;
}

// fp16 -> fp64 without the conversion unit, which does 16 lanes a cycle where
// fp64 is involved: the fp16 bits are put at the top of an fp64 word by two or
// three integer instructions (sign in place, exponent and mantissa below a
// field of zeros).  That is the value times 2^-1008, exactly, zeros and
// subnormals included (they are fp64 subnormals of the same pattern).  An infinity
// comes out as 65536 of its sign, a NaN as more: who uses the values looks for
// those with OddTest and puts the result right with mend_odd.
constexpr double kHalfUp = 0x1p1008;
CQ_DEV double half_tiny(int top) {  // fp16 in the upper half of top
    return __hiloint2double((top >> 6) & 0x81fffc00, 0);
}
// 8 fp16 values, times 2^-1008
CQ_DEV void halves_tiny(const uint4 &u, double *v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = half_tiny((int)(w[i] << 16));
        v[2 * i + 1] = half_tiny((int)w[i]);
    }
}
// 8 fp16 values through fp32 (the conversion unit has room for some)
CQ_DEV void halves(const uint4 &u, double *v) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = __half22float2(h[i]);
        v[2 * i] = (double)f.x;
        v[2 * i + 1] = (double)f.y;
    }
}

// Whether some fp16 values hold an infinity or a NaN: the product with 0 is NaN then, else
// 0 (about 5 instructions for 8 values).  Looking costs 1 % with codes (4096 rows of 2048:
// 33.7 -> 34.0 us) and 3 % where a row has five fp16 operands (LayerNorm twice with a gate,
// 1021 x 4096: 25.4 -> 26.2).  Without branches, by a NaN in the factor that the values are
// used with, it costs as much (34.4 and 25.8) and spoils the channels beside them.
struct OddTest {
    uint32_t m = 0;
    CQ_DEV void add(const uint4 &u) {
        const __half2 *h = reinterpret_cast<const __half2 *>(&u);
        const __half2 z = __float2half2_rn(0.0f);
        const __half2 p = __hfma2(h[1], z, __hmul2(h[0], z)), q = __hfma2(h[3], z, __hmul2(h[2], z));
        m |= *reinterpret_cast<const uint32_t *>(&p) | *reinterpret_cast<const uint32_t *>(&q);
    }
    CQ_DEV bool odd() const { return __builtin_expect((m & 0x7fff7fffu) != 0, 0); }
};
CQ_DEV bool odd_half(unsigned h) { return (h & 0x7c00) == 0x7c00; }
// The E channels of v have been multiplied by (or, PLUS, had added) what half_tiny made of
// the fp16 values at p.  What is still to be done where one is not finite: a product with an
// infinity (its sign is v's already) or a NaN, or an addition of it.  The values are
// read again, so that the path that all calls take holds nothing for this.
template <int E, bool PLUS>
CQ_DEV void mend_odd(double (&v)[E], int nv, const __half *p) {
#pragma unroll
    for (int i = 0; i < E; i++)
        if (i < nv) {
            const unsigned short h = __half_as_ushort(p[i]);
            if (odd_half(h)) {
                const double o = (double)__half2float(__ushort_as_half(PLUS ? h : h & 0x7fff));
                v[i] = PLUS ? v[i] + o : v[i] * o;
            }
        }
}

// v = norm(v) over the row; nv of the thread's E channels exist, the others are
// 0 and stay 0.
template <int E>
CQ_DEV void norm_regs(double (&v)[E], int nv, const NormArgs &a, const __half *w, const __half *b,
                      int c0, RowThreads &rt) {
    if (a.layer) {
        double t = 0.0, u = 0.0;
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            t += v[i];
            u += v[i + 1];
        }
        // (corrected once: a row of one value has that mean exactly, and 0 is normed)
        const double sum = row_sum(t + u, rt), m0 = sum * a.inv_h;
        const double mean = fma(fma(-m0, a.h, sum), a.inv_h, m0);
#pragma unroll
        for (int c = 0; c < E; c += 8)
            if (c < nv) {
#pragma unroll
                for (int i = 0; i < 8; i++) v[c + i] -= mean;
            }
    }
    uint4 wv[E / 8];
    if (w) {
#pragma unroll
        for (int c = 0; c < E / 8; c++)
            wv[c] = 8 * c < nv ? *reinterpret_cast<const uint4 *>(w + c0 + 8 * c) : make_uint4(0, 0, 0, 0);
    }
    double t = 0.0, u = 0.0;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        t = fma(v[i], v[i], t);
        u = fma(v[i + 1], v[i + 1], u);
    }
    const double inv = rsqrt(fma(row_sum(t + u, rt), a.inv_h, a.eps));
    OddTest odd;
#pragma unroll
    for (int c = 0; c < E; c += 8) {
        if (w) {
            odd.add(wv[c / 8]);
            double f[8];
            halves_tiny(wv[c / 8], f);
#pragma unroll
            for (int i = 0; i < 8; i++) v[c + i] *= inv * (f[i] * kHalfUp);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) v[c + i] *= inv;
        }
    }
    if (odd.odd()) mend_odd<E, false>(v, nv, w + c0);
    if (!b) return;
    odd = OddTest{};
#pragma unroll
    for (int c = 0; c < E; c += 8) {
        if (c < nv) {
            const uint4 bv = *reinterpret_cast<const uint4 *>(b + c0 + c);
            odd.add(bv);
            double f[8];
            halves_tiny(bv, f);
#pragma unroll
            for (int i = 0; i < 8; i++) v[c + i] = fma(f[i], kHalfUp, v[c + i]);
        }
    }
    if (odd.odd()) mend_odd<E, true>(v, nv, b + c0);
}

// Butterfly levels [L0, N) over 2^N registers at v[0 .. 2^N)
template <int N, int L0 = 0>
CQ_DEV void butterflies(double *v) {
#pragma unroll
    for (int h = 1 << L0; h < (1 << N); h <<= 1)
#pragma unroll
        for (int i = 0; i < (1 << N); i++)
            if ((i & h) == 0) {
                const double x = v[i], y = v[i + h];
                v[i] = x + y;
                v[i + h] = x - y;
            }
}
// Levels [0, N) of values that are 2^-1008 of theirs: the first level scales.
template <int E, int N>
CQ_DEV void first_levels(double (&v)[E]) {
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        if (N == 0) {
            v[i] *= kHalfUp;
            v[i + 1] *= kHalfUp;
        } else {
            const double y = v[i + 1] * kHalfUp;
            v[i + 1] = fma(v[i], kHalfUp, -y);
            v[i] = fma(v[i], kHalfUp, y);
        }
    }
    if (N > 1) {
#pragma unroll
        for (int i = 0; i < E; i += 1 << N) butterflies<N, 1>(v + i);
    }
}

// f(Int<n>) for n in [N, MAX]
template <int N>
struct Int {
    static constexpr int v = N;
};
template <int N, int MAX, class F>
CQ_DEV void with_const(int n, F &&f) {
    if constexpr (N < MAX) {
        if (n == N)
            f(Int<N>{});
        else
            with_const<N + 1, MAX>(n, f);
    } else {
        f(Int<MAX>{});
    }
}

constexpr int log2_of(int e) { return e <= 1 ? 0 : 1 + log2_of(e / 2); }

// The exchange area holds position p of a row at p + p / E: one double of
// padding per E, so that threads writing E consecutive positions each hit
// different banks.  In the stage of index bits [S, S + N) (S >= log2 E) a thread
// holds columns c = j + k T of the row's H / 2^N, 2^N positions each, 2^S apart;
// T threads of a row have channels.
template <int E, int S, int N>
struct Stage {
    static constexpr int LE = log2_of(E);
    static constexpr int step = (1 << S) + (1 << (S - LE));  // places between a column's positions
    CQ_DEV static int place(int c) {
        const int hi = c >> S, lo = c & ((1 << S) - 1);
        return hi * (step << N) + lo + (lo >> LE);
    }
    CQ_DEV static int position(int c) { return ((c >> S) << (S + N)) + (c & ((1 << S) - 1)); }

    CQ_DEV static void run(double (&v)[E], double *xch, int j, int T, bool store) {
#pragma unroll
        for (int k = 0; k < (E >> N); k++) {
            double *col = xch + place(j + k * T);
#pragma unroll
            for (int m = 0; m < (1 << N); m++) v[(k << N) + m] = col[m * step];
            butterflies<N>(v + (k << N));
            if (store) {
#pragma unroll
                for (int m = 0; m < (1 << N); m++) col[m * step] = v[(k << N) + m];
            }
        }
    }
};

// The groups of index bits from S up, each ending in the exchange area.
template <int E, int S>
CQ_DEV void upper_groups(double (&v)[E], double *xch, int j, int T, int lb, bool mine) {
    constexpr int kTop = 13, LE = log2_of(E);  // blocks of at most 2^13
    if constexpr (S < kTop) {
        if (lb <= S) return;
        constexpr int NMAX = kTop - S < LE ? kTop - S : LE;
        if (mine)
            with_const<1, NMAX>(min(lb - S, LE),
                                [&](auto N) { Stage<E, S, N.v>::run(v, xch, j, T, true); });
        __syncthreads();
        upper_groups<E, S + LE>(v, xch, j, T, lb, mine);
    }
}

// 1 / A to about 1e-14 (A a positive rotated value: 2^-24 to 2^29): fp32, then
// one Newton step.  The codes need it to 1e-9 (see round_code).
CQ_DEV double recip(double A) {
    const double r = (double)(1.0f / (float)A);
    return r * fma(-A, r, 2.0);
}

// Code of a value: v R rounded to even by adding 1.5 * 2^52; within 5e-7 of a tie
// (near) the exact rational decides instead.
constexpr double kMagic = 6755399441055744.0;
CQ_DEV int round_code(double v, double R, bool &near) {
    const double big = fma(v, R, kMagic);
    const double r = fma(v, R, kMagic - big);
    near = (__double2hiint(r) & 0x7fffffff) >= 0x3fdffffe;
    return __double2loint(big);
}

// Writes the codes of a column of 2^N values 2^LE positions apart.
template <int E, int N>
CQ_DEV void put_columns(const double (&v)[E], int8_t *cb, int j, int T, double R, long long Ai,
                        int qmax) {
    constexpr int LE = log2_of(E);
    bool any = false;
#pragma unroll
    for (int k = 0; k < (E >> N); k++) {
        int8_t *col = cb + Stage<E, LE, N>::position(j + k * T);
#pragma unroll
        for (int m = 0; m < (1 << N); m++) {
            bool near;
            col[m << LE] = (int8_t)round_code(v[(k << N) + m], R, near);
            any = any || near;
        }
    }
    if (any) {
#pragma unroll
        for (int i = 0; i < E; i++) {
            bool near;
            round_code(v[i], R, near);
            if (near)
                cb[Stage<E, LE, N>::position(j + (i >> N) * T) + ((i & ((1 << N) - 1)) << LE)] =
                    (int8_t)quantize_tie(v[i], Ai, qmax);
        }
    }
}

// 4 codes as bytes -> nibbles 0-3 in bits 0-15 (low nibble first)
CQ_DEV uint32_t nibbles(uint32_t a) {
    a &= 0x0f0f0f0fu;
    return a | a >> 4;  // bytes 0 and 2 hold the pairs
}

// A later row's bytes, into the L2
CQ_DEV void prefetch_row(const void *p, int bytes, int j, int threads) {
    for (int i = 128 * j; i < bytes; i += 128 * threads)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char *>(p) + i));
}

// Rows in registers, E channels a thread.  The rotation's index bits are taken
// log2 E at a time: the lowest in the layout of the loads, each further group
// after an exchange through shared memory that puts the group's 2^N values into
// one thread (2 shared accesses a value for up to log2 E levels; a lane shuffle
// of an fp64 value costs 2 instructions a level).  The groups above the second
// come first and the second, [log2 E, ..), last, so the codes are made in one of
// few layouts; they go through shared memory once, as bytes, back to the layout
// of the loads.
template <int E, int REGS, bool R16, bool CODES>
__global__ void __maxnreg__(REGS) k_residual_norm(const NormArgs a) {
    extern __shared__ __align__(16) double xch_all[];
    __shared__ double red[64];
    __shared__ int s_hi[16];
    __shared__ unsigned s_lo[16];
    constexpr int LE = log2_of(E);
    constexpr int RS = R16 ? E / 8 : E / 4;  // 16-byte pieces of a thread's residual
    griddep_wait();
    griddep_launch();
    RowThreads rt;
    const int row = threadIdx.x / a.tpr;
    rt.j = threadIdx.x - row * a.tpr;
    rt.warps = a.tpr >> 5;
    rt.warp0 = row * rt.warps;
    rt.red = red;
    rt.flip = 0;
    if (threadIdx.x < 16) {  // in use after the barriers of the sums
        s_hi[threadIdx.x] = 0;
        s_lo[threadIdx.x] = 0;
    }
    const int H = a.H, j = rt.j, c0 = E * j;
    const int T = H / E;  // threads of the row with channels, where blocks go over E channels
    double *xch = xch_all + (size_t)row * (H + T);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const int64_t t = (int64_t)blockIdx.x * a.rpc + row;
    const int nv = t < a.T ? max(0, min(E, H - c0)) : 0;  // a multiple of 8
    const int64_t at = t * H + c0;

    if (!CODES && t + a.ahead < a.T) {
        const int64_t next = (t + a.ahead) * H;
        prefetch_row(reinterpret_cast<const char *>(a.resid) + next * (R16 ? 2 : 4), H * (R16 ? 2 : 4), rt.j, a.tpr);
        if (a.y) prefetch_row(a.y + next, H * 4, rt.j, a.tpr);
        if (a.gate_mode == CQ_GATE_ELEMENT) prefetch_row(a.gate + next, H * 2, rt.j, a.tpr);
    }
    double v[E];
    // everything the row reads once is requested before the first use
    uint4 rr[RS];
    if (R16) {
        const uint4 *src = reinterpret_cast<const uint4 *>(reinterpret_cast<const __half *>(a.resid) + at);
#pragma unroll
        for (int c = 0; c < E / 8; c++) rr[c] = 8 * c < nv ? __ldcs(src + c) : zero;
    } else {
        const uint4 *src = reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(a.resid) + at);
#pragma unroll
        for (int c = 0; c < E / 4; c++) rr[c] = 4 * c < nv ? __ldcs(src + c) : zero;
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
            OddTest odd;
#pragma unroll
            for (int c = 0; c < E; c += 8) {
                if (c < nv) {
                    const uint4 gv = *reinterpret_cast<const uint4 *>(gp + c);
                    odd.add(gv);
                    double f[8];
                    halves_tiny(gv, f);
#pragma unroll
                    for (int i = 0; i < 8; i++) v[c + i] *= f[i] * kHalfUp;
                }
            }
            if (odd.odd()) mend_odd<E, false>(v, nv, gp);
        }
    }
    // r' = round(resid_scale * r + block_scale * v)
    if (R16) {
#pragma unroll
        for (int c = 0; c < E / 8; c++) {
            if (a.y) {
                double f[8];
                halves(rr[c], f);
                __half2 *h = reinterpret_cast<__half2 *>(&rr[c]);
#pragma unroll
                for (int i = 0; i < 8; i += 2)
                    h[i / 2] = __halves2half2(
                        __double2half(fma(a.resid_scale, f[i], a.block_scale * v[8 * c + i])),
                        __double2half(fma(a.resid_scale, f[i + 1], a.block_scale * v[8 * c + i + 1])));
                if (8 * c < nv)
                    *reinterpret_cast<uint4 *>(reinterpret_cast<__half *>(a.resid_out) + at + 8 * c) = rr[c];
            }
            halves(rr[c], v + 8 * c);
        }
    } else {
#pragma unroll
        for (int c = 0; c < E / 4; c++) {
            float *f = reinterpret_cast<float *>(&rr[c]);
            if (a.y) {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    f[i] = __double2float_rn(
                        fma(a.resid_scale, (double)f[i], a.block_scale * v[4 * c + i]));
                if (4 * c < nv)
                    *reinterpret_cast<uint4 *>(reinterpret_cast<float *>(a.resid_out) + at + 4 * c) = rr[c];
            }
#pragma unroll
            for (int i = 0; i < 4; i++) v[4 * c + i] = (double)f[i];
        }
    }
    norm_regs<E>(v, nv, a, a.pre_w, a.pre_b, c0, rt);
    OddTest odd;
#pragma unroll
    for (int c = 0; c < E / 8; c++) {
        uint4 o;
        __half2 *h = reinterpret_cast<__half2 *>(&o);
#pragma unroll
        for (int i = 0; i < 8; i += 2)
            h[i / 2] = __halves2half2(__double2half(v[8 * c + i]), __double2half(v[8 * c + i + 1]));
        if (8 * c < nv) *reinterpret_cast<uint4 *>(a.x + at + 8 * c) = o;
        if (CODES) {
            odd.add(o);
            halves_tiny(o, v + 8 * c);
        }
    }
    if (!CODES) return;
    // a row whose x is not finite: the high word of a NaN as its largest magnitude, above
    // any value's, so its scale is NaN and its codes are 0
    if (odd.odd()) atomicMax(&s_hi[row], 0x7ff80000);

    // ---- rotation (channels beyond the row are zeros of whole blocks of 8)
    const int lb = a.log2b;
    with_const<0, LE>(min(lb, LE), [&](auto N) { first_levels<E, N.v>(v); });
    const bool mine = nv > 0;
    const int n2 = min(max(lb - LE, 0), LE);  // bits of the second group
    if (n2 > 0) {
        if (mine) {
#pragma unroll
            for (int i = 0; i < E; i++) xch[(E + 1) * j + i] = v[i];
        }
        __syncthreads();
        upper_groups<E, 2 * LE>(v, xch, j, T, lb, mine);
        if (mine)
            with_const<1, LE>(n2, [&](auto N) { Stage<E, LE, N.v>::run(v, xch, j, T, false); });
    }
    // ---- the row's largest magnitude.  fp64 comparisons run at 16 lanes a cycle:
    // the magnitudes are compared as integers, first the high words of all, then
    // the low words of those whose high word is the largest
    int mh = 0;
#pragma unroll
    for (int i = 0; i < E; i++) mh = max(mh, __double2hiint(v[i]) & 0x7fffffff);
    if (!mine) mh = 0;
    const int wh = __reduce_max_sync(0xffffffffu, mh);
    if ((threadIdx.x & 31) == 0) atomicMax(&s_hi[row], wh);
    __syncthreads();  // also: the exchange area is free
    const int top = s_hi[row];
    if (mine && mh == top) {
        unsigned ml = 0;
#pragma unroll
        for (int i = 0; i < E; i++)
            if ((__double2hiint(v[i]) & 0x7fffffff) == top) ml = max(ml, (unsigned)__double2loint(v[i]));
        atomicMax(&s_lo[row], ml);
    }
    __syncthreads();
    const double A = __hiloint2double(top, (int)s_lo[row]);
    const int qmax = (1 << (a.bits - 1)) - 1;
    const long long Ai = __double2ll_rn(A * 16777216.0);
    const double R = Ai > 0 ? (double)qmax * recip(A) : 0.0;
    // the steps of quant_scale, its root taken on the host
    if (j == 0 && mine)
        a.s[t] = __double2float_rn(__ddiv_rn(__ddiv_rn(A, a.sqrt_b), (double)qmax));
    int8_t *cb = reinterpret_cast<int8_t *>(xch);
    if (mine) {
        if (n2 == 0) {
            uint32_t w[E / 4];
#pragma unroll
            for (int i = 0; i < E; i++) {
                bool near;
                int c = round_code(v[i], R, near);
                if (near) c = quantize_tie(v[i], Ai, qmax);
                w[i / 4] = i % 4 ? w[i / 4] | (uint32_t)(c & 255) << (8 * (i % 4)) : (uint32_t)(c & 255);
            }
#pragma unroll
            for (int i = 0; i < E / 4; i++) *reinterpret_cast<uint32_t *>(cb + c0 + 4 * i) = w[i];
        } else {
            with_const<1, LE>(n2, [&](auto N) { put_columns<E, N.v>(v, cb, j, T, R, Ai, qmax); });
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; i += 8) {
        if (i < nv) {
            const uint2 u = *reinterpret_cast<const uint2 *>(cb + c0 + i);
            if (a.bits == 8)
                *reinterpret_cast<uint2 *>(a.q + t * a.ldq + c0 + i) = u;
            else
                *reinterpret_cast<uint32_t *>(a.q + t * a.ldq + (c0 + i) / 2) =
                    prmt(nibbles(u.x), nibbles(u.y), 0x6420);
        }
    }
}

template <int E, int REGS>
static cudaError_t launch_rows(NormArgs a, bool r16, cudaStream_t st) {
    const int T = (a.H + E - 1) / E;
    a.tpr = (T + 31) / 32 * 32;
    // short rows share a CTA of up to 128 threads
    a.rpc = (int)std::min<int64_t>(std::max(1, 128 / a.tpr), a.T);
    const bool codes = a.bits > 0;
    // A row fetches the one that takes its place where the arithmetic is short (4096 rows of
    // 2048, fp32 residual: 25.5 -> 22.8 us); with codes or a second norm that only adds
    // instructions (codes 33.6 -> 34.0).
    const int ctas = std::max(1, std::min(32, 65536 / (REGS * a.tpr * a.rpc)));
    a.ahead = codes || a.post_norm ? a.T : (int64_t)ctas * a.rpc * sm_count();
    const size_t smem = codes ? (size_t)a.rpc * (a.H + a.H / E) * sizeof(double) : 0;
    auto kern = r16 ? (codes ? k_residual_norm<E, REGS, true, true> : k_residual_norm<E, REGS, true, false>)
                    : (codes ? k_residual_norm<E, REGS, false, true>
                             : k_residual_norm<E, REGS, false, false>);
    count_launch();
    return launch_pdl(kern, dim3((unsigned)((a.T + a.rpc - 1) / a.rpc)), dim3(a.tpr * a.rpc), smem,
                      st, 1, a);
}

// Channels and registers a thread.  16 at 80 registers with codes: fewer channels
// are more exchanges, and more registers fewer rows at once (4096 rows of 2048: 33.4 us,
// 8 channels 41.7).  Else:
//  - rows over 6400 would be alone on their SM at 80 registers, and over 8192 need 64
//    anyway: 64, some of them spilled (2000 rows of 8192: 93 -> 70 us with codes,
//    60 -> 48 without; from 4096 up, 3 rows instead of 2: 2000 of 5120, codes 48.5 -> 43.9,
//    but with a post norm, which spills more, 61 -> 67).  One row an SM or less gains
//    nothing from room for a second (100 rows of 8192, codes: 7.4 and 7.8).
//  - few rows are paced by the length of a row's instruction stream: 8 channels (one row
//    of 2560: 3.7 us, and 4.7 with 16).
//  - without codes 8 channels, where a thread's fp32 pieces then are 32 bytes apart and not
//    64 (4096 rows of 2048, fp32 residual: 25.6 us, and 31.3 with 16; fp16, 1024: 10.3 and
//    10.9; all before rows were fetched ahead), but 16 for long rows of much arithmetic
//    (fp16, 2048: 21.0 and 20.0).
static cudaError_t launch_residual_norm(const NormArgs &a, bool r16, cudaStream_t st) {
    TimedScope ts(st, CQ_KERNEL_RESIDUAL_NORM);
    const bool codes = a.bits > 0, many = a.T > sm_count();
    if (a.H > 8192 || (many && (a.H > 6400 || (a.H > 4096 && codes && !a.post_norm))))
        return launch_rows<16, 64>(a, r16, st);
    if (a.H <= 4096 && (a.T <= 2 * sm_count() || (!codes && (a.H < 2048 || (!r16 && !a.post_norm)))))
        return launch_rows<8, 64>(a, r16, st);
    return launch_rows<16, 80>(a, r16, st);
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
    a.h = (double)d->H;
    a.inv_h = 1.0 / a.h;
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
    a.sqrt_b = std::sqrt((double)(b > 0 ? b : 1));
    try {
        return launch_residual_norm(a, d->resid_bits == 16, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? CQ_OK
                   : CQ_ERR_CUDA;
    } catch (...) {
        return CQ_ERR_CUDA;
    }
}

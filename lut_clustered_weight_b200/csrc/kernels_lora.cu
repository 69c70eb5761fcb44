// kernels_lora.cu -- cq_lora_add: low-rank adapters of many requests beside a
// shared projection, sm_100a.  out = y + scale * B (A x) with the adapter of
// each row.
//
// Rows of one adapter are gathered into tiles of up to TM rows; a cluster of
// CTAs works on a tile in one launch:
//   shrink  t = A x: the cluster's CTAs, and the warps of a CTA, split K; the
//           partial t are summed through shared and distributed shared memory
//           in a fixed order, so every CTA of the cluster has all of t
//   expand  out = y + scale * B t: the CTAs split the columns
// so t never goes to global memory and every CTA streams its part of A, x, B
// and y once.  Both products run on mma.sync m16n8k16: the op is bound by bytes (y
// is read and written in fp32), not by the tensor pipe (at rank 64 it does 16
// flops a byte).  The shrink's operands come by cp.async through a ring of stages,
// so that a CTA's whole part of K is on its way at once; the expansion's straight
// from global memory into fragments: a lane takes 16 bytes (8 consecutive k) of a
// row of B, which serves two k16 steps when both operands are permuted along k alike.
//
// t is fp32 and B is fp16: t is scaled by a power of two per row, so that its
// largest entry is in [1, 2), and split into two fp16 parts, t = hi + lo with
// an error of 2^-22 of that entry; one more MMA per tile keeps fp32-like sums
// (one fp16 part would leave 2^-11 of the update in an fp32 output).
#include <cooperative_groups.h>

#include <algorithm>

#include "cq_common.cuh"
#include "cq_internal.h"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace cq {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraMaxRank = 128;
// Up to this many rows (one a thread) every CTA finds its own tile in the ids;
// above, one CTA sorts the rows first (k_lora_plan).
constexpr int kLoraSmallM = kLoraThreads;

struct LoraTile {
    int id, start, rows, pad;  // rows perm[start, start + rows); id -1: no adapter
};

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
    // planned launches only (M > kLoraSmallM)
    const int *n_tiles;
    const LoraTile *tiles;
    const int *perm;
};

CQ_DEV int valid_id(int id, int n) { return (unsigned)id < (unsigned)n ? id : -1; }

// Elements k and up of an 8-element fp16 chunk zeroed (k may be <= 0 or >= 8).
CQ_DEV uint4 keep_first(uint4 v, int k) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] = k >= 2 * i + 2 ? w[i] : k == 2 * i + 1 ? w[i] & 0xffffu : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One k32 step of the expansion held as 16 bytes per lane and row: lane q of a row's four holds
// k 8q .. 8q + 7.  MMA step s takes elements 4s .. 4s + 3 as the fragment's k
// (2q, 2q + 1) and (2q + 8, 2q + 9), for both operands.
CQ_DEV uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Row i is thread i's (M <= kLoraThreads).  Rows of an adapter form tiles of TM in
// row order; the row that begins one leads it, and tile t is that of the t-th
// leading row.  False if there is none.  buf: 256 ints of shared memory.
CQ_DEV bool find_tile(const LoraArgs &p, int t, int TM, int *buf, int *s_rows, int *s_id,
                      int *s_count) {
    __shared__ int s_lead[kLoraWarps];
    __shared__ int s_first;
    const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
    const bool row = i < p.M;
    // -2: no row, and no adapter where such rows need nothing done (in place)
    int id = row ? valid_id(p.ids[i], p.n) : -2;
    if (id == -1 && p.y == p.out) id = -2;
    buf[i] = id;
    if (i == 0) *s_count = 0;
    __syncthreads();
    int before = __popc(__match_any_sync(0xffffffffu, id) & ((1u << lane) - 1u));
    const int4 *b4 = reinterpret_cast<const int4 *>(buf);
    for (int j = 0; j < 8 * warp; j++) {
        const int4 o = b4[j];
        before += (o.x == id) + (o.y == id) + (o.z == id) + (o.w == id);
    }
    const bool leads = id != -2 && before % TM == 0;
    const unsigned mask = __ballot_sync(0xffffffffu, leads);
    if (lane == 0) s_lead[warp] = __popc(mask);
    __syncthreads();
    int at = __popc(mask & ((1u << lane) - 1u)), total = 0;
#pragma unroll
    for (int w = 0; w < kLoraWarps; w++) {
        if (w < warp) at += s_lead[w];
        total += s_lead[w];
    }
    if (t >= total) return false;
    if (leads && at == t) {
        *s_id = id;
        s_first = before;
    }
    __syncthreads();
    const int place = before - s_first;
    const bool mine = id == *s_id && place >= 0 && place < TM;
    if (mine) s_rows[place] = i;
    const int count = __syncthreads_count(mine);
    // the places beyond the last row repeat it (their results are not stored)
    if (i >= count && i < TM) s_rows[i] = s_rows[count - 1];
    if (i == 0) *s_count = count;
    __syncthreads();
    return true;
}

CQ_DEV void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int TM, int R>
struct LoraShape {
    static constexpr int KC = TM == 64 ? 64 : 128;        // k of a stage
    static constexpr int pitch = 2 * KC + 16;             // bytes of a staged row (ldmatrix: no conflicts)
    static constexpr int rows = TM + R;                   // x rows, then A rows
    static constexpr int stage = rows * pitch;
    static constexpr int t_bytes = 2 * TM * (R + 8) * 2;  // hi, lo
    static constexpr int fit = (110 * 1024 - t_bytes) / stage;   // two CTAs an SM
    static constexpr int NS = fit > 6 ? 6 : fit < 2 ? 2 : fit;   // stages
    static constexpr int WK = TM == 16 ? kLoraWarps : 1;  // partial t of a CTA (warps along k)
    static constexpr int LDP = R + 8;                     // floats a row of the partial t
    static constexpr int LDT = R + 8;                     // halves a row of hi / lo
    static constexpr int part_bytes = WK * TM * LDP * 4;
    static constexpr int pool = NS * stage > part_bytes ? NS * stage : part_bytes;
    static constexpr size_t smem = (size_t)pool + t_bytes;
};

CQ_DEV void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// Partial t of this CTA: rows [0, TM) of the tile times A over k chunks [ch0, ch1)
// of KC.  x and A rows come by cp.async through a ring of stages, zero-filled
// beyond the tile's rows, the rank and K.  TM 64: warp = 16 rows x half the
// rank; TM 16: warp = one k16 step of each stage, summed at the end.  Leaves the sums
// in part [TM][LDP] (over the ring), after a barrier.
template <int TM, int R>
CQ_DEV void shrink(const LoraArgs &p, int id, int rows, int rank, const int *s_rows,
                   unsigned char *ring, float *part, int ch0, int ch1) {
    using S = LoraShape<TM, R>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int PR = S::KC / 8;                 // 16-byte pieces a row
    constexpr int RP = kLoraThreads / PR;         // rows a pass
    constexpr int PASSES = (S::rows + RP - 1) / RP;
    const int prow = tid / PR, pcol = 8 * (tid % PR);
    const __half *src[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; i++) {
        const int row = prow + i * RP;
        src[i] = nullptr;
        if (row < TM) {
            if (row < rows) src[i] = p.x + (int64_t)s_rows[row] * p.K + pcol;
        } else if (row - TM < rank) {
            src[i] = p.a + ((int64_t)id * p.r + row - TM) * p.K + pcol;
        }
    }
    auto fetch = [&](int ch, int slot) {
        const int k = ch * S::KC;
#pragma unroll
        for (int i = 0; i < PASSES; i++) {
            const int row = prow + i * RP;
            if (S::rows % RP == 0 || row < S::rows) {
                const bool in = src[i] != nullptr && k + pcol < p.K;
                cp_async16_zfill(ring + slot * S::stage + row * S::pitch + 2 * pcol,
                                 in ? src[i] + k : p.x, in ? 16 : 0);
            }
        }
    };
    constexpr int WN = TM == 64 ? 2 : 1;
    constexpr int NT = R / 8 / WN;                // n8 tiles of a warp
    const int wm = TM == 64 ? warp & 3 : 0, wn = TM == 64 ? warp >> 2 : 0;
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[j][e] = 0.0f;
    // ldmatrix rows of this lane: x rows, and n rows (two n8 tiles at once)
    const uint32_t ring0 = smem_u32(ring);
    const uint32_t xa = (16 * wm + (lane & 15)) * S::pitch + 16 * (lane >> 4);
    const uint32_t wa = (TM + 8 * NT * wn + (lane & 7) + 8 * (lane >> 4)) * S::pitch +
                        16 * ((lane >> 3) & 1);
#pragma unroll
    for (int i = 0; i < S::NS - 1; i++) {
        if (ch0 + i < ch1) fetch(ch0 + i, i);
        cp_async_commit_group();
    }
    int slot = 0;
    for (int ch = ch0; ch < ch1; ch++) {
        cp_async_wait_group<S::NS - 2>();
        __syncthreads();
        {
            const int next = ch + S::NS - 1;
            if (next < ch1) fetch(next, slot == 0 ? S::NS - 1 : slot - 1);
            cp_async_commit_group();
        }
        const uint32_t base = ring0 + slot * S::stage;
        constexpr int STEPS = TM == 64 ? S::KC / 16 : 1;
        if (TM == 16 || 16 * wm < rows) {
#pragma unroll
            for (int st = 0; st < STEPS; st++) {
                const uint32_t kb = 32 * (TM == 64 ? st : warp);
                uint32_t a[4];
                ldmatrix4(a, base + xa + kb);
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t b[4];
                    // (a single n8 tile: the second half of the lanes reads rows beyond it,
                    // inside the stage or the next one, and its result is not used)
                    ldmatrix4(b, base + wa + j * 8 * S::pitch + kb);
                    mma_16816(acc[j], a, b[0], b[1]);
                    if (j + 1 < NT) mma_16816(acc[j + 1], a, b[2], b[3]);
                }
            }
        }
        slot = slot + 1 == S::NS ? 0 : slot + 1;
    }
    cp_async_wait_group<0>();
    __syncthreads();  // the ring is free
    const int g = lane >> 2, q = lane & 3;
    float *pw = part + (TM == 64 ? 16 * wm * S::LDP + 8 * NT * wn : warp * TM * S::LDP);
#pragma unroll
    for (int j = 0; j < NT; j++) {
        *reinterpret_cast<float2 *>(pw + g * S::LDP + 8 * j + 2 * q) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2 *>(pw + (g + 8) * S::LDP + 8 * j + 2 * q) =
            make_float2(acc[j][2], acc[j][3]);
    }
    if (S::WK > 1) {
        __syncthreads();
        for (int i = tid; i < TM * R; i += kLoraThreads) {
            const int at = (i / R) * S::LDP + i % R;
            float v = part[at];
#pragma unroll
            for (int w = 1; w < S::WK; w++) v += part[w * TM * S::LDP + at];
            part[at] = v;
        }
    }
}

// t of the whole cluster, a warp per row, as hi + lo and the factor of the row.
template <int TM, int R>
CQ_DEV void gather_t(cg::cluster_group &cluster, float *part, int C, int rows, float sc, __half *th,
                     __half *tl, float *s_factor) {
    using S = LoraShape<TM, R>;
    constexpr int PER = (R + 31) / 32;
    constexpr int RB = TM == 16 || PER > 2 ? 2 : 4;  // rows a warp has in flight
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
    for (int r0 = warp; r0 < TM; r0 += RB * kLoraWarps) {
        float v[RB][PER];
#pragma unroll
        for (int b = 0; b < RB; b++)
#pragma unroll
            for (int i = 0; i < PER; i++) v[b][i] = 0.0f;
        if (r0 < rows) {
            for (int c = 0; c < C; c += 4) {  // C is a multiple of 4
                float u[4][RB][PER];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float *rp = cluster.map_shared_rank(part, c + k);
#pragma unroll
                    for (int b = 0; b < RB; b++)
#pragma unroll
                        for (int i = 0; i < PER; i++)
                            u[k][b][i] = R >= 32 || lane < R
                                             ? rp[(r0 + b * kLoraWarps) * S::LDP + lane + 32 * i]
                                             : 0.0f;
                }
#pragma unroll
                for (int k = 0; k < 4; k++)
#pragma unroll
                    for (int b = 0; b < RB; b++)
#pragma unroll
                        for (int i = 0; i < PER; i++) v[b][i] += u[k][b][i];
            }
        }
#pragma unroll
        for (int b = 0; b < RB; b++) {
            const int row = r0 + b * kLoraWarps;
            float mx = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; i++) mx = fmaxf(mx, fabsf(v[b][i]));
#pragma unroll
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // 2^-e and 2^e of the largest entry's exponent, both normal numbers
            const int e = min(max((__float_as_int(mx) >> 23) & 255, 1), 253);
            const float down = __int_as_float((254 - e) << 23), up = __int_as_float(e << 23);
#pragma unroll
            for (int i = 0; i < PER; i++) {
                const float t = v[b][i] * down;
                const __half hi = __float2half_rn(t);
                if (R >= 32 || lane < R) {
                    th[row * S::LDT + lane + 32 * i] = hi;
                    tl[row * S::LDT + lane + 32 * i] = __float2half_rn(t - __half2float(hi));
                }
            }
            if (lane == 0) s_factor[row] = sc * up;
        }
    }
}

// Expansion of a block of 8 NB columns: MMA column 2q + e of n8 tile j is column
// 2 NB q + 2j + e of the block, so a lane holds 2 NB consecutive columns of y.
template <int R, int NB>
struct Expand {
    static constexpr int KS = R >= 32 ? R / 32 : 1;   // 32-wide steps of the rank
    static constexpr int W = 8 * NB;                  // columns
    static constexpr int LDT = R + 8;
    struct B {
        uint4 w[NB][KS];
    };
    struct Y {
        float4 a[NB / 2], b[NB / 2];
    };

    CQ_DEV static void load_b(B &o, const LoraArgs &p, int id, int rank, int n0) {
        const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
        for (int j = 0; j < NB; j++) {
            const int col = n0 + 2 * NB * (g >> 1) + 2 * j + (g & 1);
            const __half *br = p.b + ((int64_t)id * p.N + min(col, p.N - 1)) * p.r;
#pragma unroll
            for (int s = 0; s < KS; s++) {
                o.w[j][s] = make_uint4(0, 0, 0, 0);
                if (R >= 32) {
                    const int k = 32 * s + 8 * q;
                    if (k < rank) o.w[j][s] = *reinterpret_cast<const uint4 *>(br + k);
                } else {  // 4 consecutive k a lane, one MMA step
                    const int k = 4 * q;
                    if (k < rank) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(br + k);
                        o.w[j][s].x = v.x;
                        o.w[j][s].y = v.y;
                    }
                }
            }
        }
    }
    // what lies beyond the rank in a chunk that holds its end is not used
    CQ_DEV static void cut_b(B &o, int rank) {
        const int q = threadIdx.x & 3;
#pragma unroll
        for (int j = 0; j < NB; j++)
#pragma unroll
            for (int s = 0; s < KS; s++)
                o.w[j][s] = keep_first(o.w[j][s], rank - (R >= 32 ? 32 * s + 8 * q : 4 * q));
    }
    CQ_DEV static void load_y(Y &o, const LoraArgs &p, const int *s_rows, int ra, int rows, int n0) {
        const int q = threadIdx.x & 3, c = n0 + 2 * NB * q, rb = ra + 8;
        const float *pa = p.y + (int64_t)s_rows[ra] * p.ldy + c;
        const float *pb = p.y + (int64_t)s_rows[rb] * p.ldy + c;
#pragma unroll
        for (int i = 0; i < NB / 2; i++) {
            const bool in = c + 4 * i < p.N;  // N % 8 == 0
            o.a[i] = in && ra < rows ? reinterpret_cast<const float4 *>(pa)[i] : make_float4(0, 0, 0, 0);
            o.b[i] = in && rb < rows ? reinterpret_cast<const float4 *>(pb)[i] : make_float4(0, 0, 0, 0);
        }
    }
    CQ_DEV static void run(const B &w, const Y &y, const LoraArgs &p, const int *s_rows,
                           const float *s_factor, const __half *th, const __half *tl, int ra,
                           int rows, int n0) {
        const int q = threadIdx.x & 3, rb = ra + 8, c = n0 + 2 * NB * q;
        float acc[NB][4];
#pragma unroll
        for (int j = 0; j < NB; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) acc[j][e] = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; s++) {
#pragma unroll
            for (int part_i = 0; part_i < 2; part_i++) {  // lo first, then hi
                const __half *tp = part_i ? th : tl;
                if (R >= 32) {
                    const uint4 va = *reinterpret_cast<const uint4 *>(tp + ra * LDT + 32 * s + 8 * q);
                    const uint4 vb = *reinterpret_cast<const uint4 *>(tp + rb * LDT + 32 * s + 8 * q);
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t a[4] = {word(va, 2 * h), word(vb, 2 * h), word(va, 2 * h + 1),
                                               word(vb, 2 * h + 1)};
#pragma unroll
                        for (int j = 0; j < NB; j++)
                            mma_16816(acc[j], a, word(w.w[j][s], 2 * h), word(w.w[j][s], 2 * h + 1));
                    }
                } else {
                    const uint2 va = *reinterpret_cast<const uint2 *>(tp + ra * LDT + 4 * q);
                    const uint2 vb = *reinterpret_cast<const uint2 *>(tp + rb * LDT + 4 * q);
                    const uint32_t a[4] = {va.x, vb.x, va.y, vb.y};
#pragma unroll
                    for (int j = 0; j < NB; j++) mma_16816(acc[j], a, w.w[j][s].x, w.w[j][s].y);
                }
            }
        }
        const float fa = s_factor[ra], fb = s_factor[rb];
        float *oa = p.out + (int64_t)s_rows[ra] * p.ldo + c;
        float *ob = p.out + (int64_t)s_rows[rb] * p.ldo + c;
#pragma unroll
        for (int i = 0; i < NB / 2; i++) {
            const float(&l)[4] = acc[2 * i], (&h)[4] = acc[2 * i + 1];
            if (c + 4 * i < p.N) {
                if (ra < rows)
                    reinterpret_cast<float4 *>(oa)[i] =
                        make_float4(y.a[i].x + fa * l[0], y.a[i].y + fa * l[1], y.a[i].z + fa * h[0],
                                    y.a[i].w + fa * h[1]);
                if (rb < rows)
                    reinterpret_cast<float4 *>(ob)[i] =
                        make_float4(y.b[i].x + fb * l[2], y.b[i].y + fb * l[3], y.b[i].z + fb * h[2],
                                    y.b[i].w + fb * h[3]);
            }
        }
    }
};

template <int TM, int R>
__global__ void __launch_bounds__(kLoraThreads, 2) k_lora(const LoraArgs p) {
    using S = LoraShape<TM, R>;
    constexpr int NB = TM == 16 && R <= 64 ? 4 : 2;  // n8 tiles of a column block
    using X = Expand<R, NB>;
    extern __shared__ __align__(16) unsigned char smem[];
    float *part = reinterpret_cast<float *>(smem);                // [WK][TM][LDP], over the ring
    __half *th = reinterpret_cast<__half *>(smem + S::pool);      // [TM][LDT]
    __half *tl = th + TM * S::LDT;
    __shared__ int s_rows[TM];
    __shared__ float s_factor[TM];
    __shared__ int s_id, s_count;

    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), crank = (int)cluster.block_rank();
    const int tile = blockIdx.x / C;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2;
    griddep_wait();
    griddep_launch();

    // ---- the tile: adapter and rows (the same for every CTA of the cluster)
    if (p.tiles) {
        if (tile >= *p.n_tiles) return;
        const LoraTile T = p.tiles[tile];
        for (int i = threadIdx.x; i < TM; i += kLoraThreads)
            s_rows[i] = p.perm[T.start + min(i, T.rows - 1)];
        if (threadIdx.x == 0) {
            s_id = T.id;
            s_count = T.rows;
        }
        __syncthreads();
    } else if (!find_tile(p, tile, TM, reinterpret_cast<int *>(smem), s_rows, &s_id, &s_count)) {
        return;
    }
    const int id = s_id, rows = s_count;
    const int rank = id < 0 ? 0 : p.ranks ? max(0, min(p.ranks[id], p.r)) : p.r;
    const float sc = id >= 0 && p.scale ? p.scale[id] : 1.0f;

    // columns of this CTA, in blocks of W
    const int nblk = (p.N + X::W - 1) / X::W;
    const int nb0 = (int)((int64_t)crank * nblk / C), nb1 = (int)((int64_t)(crank + 1) * nblk / C);
    const int c0 = nb0 * X::W, c1 = min(nb1 * X::W, p.N);
    if (rank == 0) {  // out = y
        if (p.y != p.out) {
            for (int i = warp; i < rows; i += kLoraWarps) {
                const float *src = p.y + (int64_t)s_rows[i] * p.ldy;
                float *dst = p.out + (int64_t)s_rows[i] * p.ldo;
                for (int c = c0 + 4 * lane; c < c1; c += 128)
                    *reinterpret_cast<float4 *>(dst + c) = *reinterpret_cast<const float4 *>(src + c);
            }
        }
        return;
    }
    // B's part for the expansion, into the L2 while the shrink runs
    {
        const char *bp = reinterpret_cast<const char *>(p.b + ((int64_t)id * p.N + c0) * p.r);
        const int bytes = (c1 - c0) * p.r * 2;
        for (int i = 128 * threadIdx.x; i < bytes; i += 128 * kLoraThreads) prefetch_l2(bp + i);
    }
    {
        const int chunks = (p.K + S::KC - 1) / S::KC;
        shrink<TM, R>(p, id, rows, rank, s_rows, smem, part, (int)((int64_t)crank * chunks / C),
                      (int)((int64_t)(crank + 1) * chunks / C));
    }
    // the first block's operands do not wait for t
    int nb = nb0 + warp;
    typename X::B w, wn;
    typename X::Y y, yn;
    if (nb < nb1) {
        X::load_b(w, p, id, rank, nb * X::W);
        X::load_y(y, p, s_rows, g, rows, nb * X::W);
    }
    cluster.sync();
    gather_t<TM, R>(cluster, part, C, rows, sc, th, tl, s_factor);
    __syncthreads();
    cluster.barrier_arrive();  // this CTA has read every partial t

    // ---- expand: a warp per column block, over the tile's rows 16 at a time, the
    // next y (and B) requested before this block's products
    const int mbs = (rows + 15) >> 4;
    for (; nb < nb1; nb += kLoraWarps) {
        const int nn = nb + kLoraWarps;
        const bool more = nn < nb1;
        if (more) X::load_b(wn, p, id, rank, nn * X::W);
        X::cut_b(w, rank);
        for (int mb = 0; mb < mbs; mb++) {
            if (mb + 1 < mbs)
                X::load_y(yn, p, s_rows, 16 * (mb + 1) + g, rows, nb * X::W);
            else if (more)
                X::load_y(yn, p, s_rows, g, rows, nn * X::W);
            X::run(w, y, p, s_rows, s_factor, th, tl, 16 * mb + g, rows, nb * X::W);
            y = yn;
        }
        w = wn;
    }
    __syncwarp();
    cluster.barrier_wait();  // no CTA leaves while another may read its partial t
}

// ---------------------------------------------------------------- rows by adapter
// One CTA: counts per adapter (slot n: no adapter), their offsets, the tile
// list and the permutation.  A row's place among its adapter's rows comes from
// the counting atomics: their order may change from call to call, and with it the
// rows of a tile, but a row's result does not depend on its place.
constexpr int kPlanThreads = 1024;
constexpr int kPlanRows = 8;  // rows a thread holds at once

// Exclusive scan over the CTA of (a, b); adds and advances the running totals.
CQ_DEV void scan_pair(int &a, int &b, int &ta, int &tb, int (*wsum)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int a0 = a, b0 = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    __syncthreads();  // wsum may still be read from the last scan
    if (lane == 31) {
        wsum[0][warp] = a;
        wsum[1][warp] = b;
    }
    __syncthreads();
    int wa = wsum[0][lane], wb = wsum[1][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, wa, o), y = __shfl_up_sync(0xffffffffu, wb, o);
        if (lane >= o) {
            wa += x;
            wb += y;
        }
    }
    const int pa = __shfl_sync(0xffffffffu, wa, (warp + 31) & 31);
    const int pb = __shfl_sync(0xffffffffu, wb, (warp + 31) & 31);
    a += ta - a0 + (warp ? pa : 0);
    b += tb - b0 + (warp ? pb : 0);
    ta += __shfl_sync(0xffffffffu, wa, 31);
    tb += __shfl_sync(0xffffffffu, wb, 31);
}

__global__ void __launch_bounds__(kPlanThreads)
k_lora_plan(const int32_t *__restrict__ ids, int M, int n, int TM, bool skip_none, int *n_tiles,
            LoraTile *tiles, int *perm, int *place) {
    extern __shared__ int cnt[];  // [n + 1] counts, then offsets
    __shared__ int wsum[2][32];
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, lane = tid & 31;
    int key[kPlanRows], at[kPlanRows];
    auto load = [&](int b0) {
#pragma unroll
        for (int u = 0; u < kPlanRows; u++) {
            const int i = b0 + u * kPlanThreads + tid;
            key[u] = i < M ? valid_id(ids[i], n) : -2;
        }
#pragma unroll
        for (int u = 0; u < kPlanRows; u++)
            if (key[u] == -1) key[u] = n;
    };
    load(0);
    for (int i = tid; i <= n; i += kPlanThreads) cnt[i] = 0;
    __syncthreads();
    const bool once = M <= kPlanRows * kPlanThreads;  // keys and places stay in registers
    for (int b0 = 0; b0 < M; b0 += kPlanRows * kPlanThreads) {
        if (b0) load(b0);
#pragma unroll
        for (int u = 0; u < kPlanRows; u++) {
            if (b0 + u * kPlanThreads >= M) break;
            // the lanes of a warp with the same adapter take one atomic
            const unsigned peers = __match_any_sync(0xffffffffu, key[u]);
            const int leader = __ffs(peers) - 1;
            int base = 0;
            if (lane == leader && key[u] >= 0) base = atomicAdd(&cnt[key[u]], __popc(peers));
            at[u] = __shfl_sync(0xffffffffu, base, leader) + __popc(peers & ((1u << lane) - 1u));
            const int i = b0 + u * kPlanThreads + tid;
            if (!once && i < M) place[i] = at[u];
        }
    }
    __syncthreads();
    int rows = 0, nt = 0;
    for (int b0 = 0; b0 <= n; b0 += kPlanThreads) {
        const int i = b0 + tid;
        const int c = i <= n ? cnt[i] : 0;
        const int t = i == n && skip_none ? 0 : (c + TM - 1) / TM;
        int start = c, first = t;
        scan_pair(start, first, rows, nt, wsum);
        if (i <= n) {
            cnt[i] = start;
            for (int k = 0; k < t; k++)
                tiles[first + k] = LoraTile{i == n ? -1 : i, start + k * TM, min(TM, c - k * TM), 0};
        }
    }
    if (tid == 0) *n_tiles = nt;
    __syncthreads();
    for (int b0 = 0; b0 < M; b0 += kPlanRows * kPlanThreads) {
        if (!once) load(b0);
#pragma unroll
        for (int u = 0; u < kPlanRows; u++) {
            const int i = b0 + u * kPlanThreads + tid;
            if (i < M) perm[cnt[key[u]] + (once ? at[u] : place[i])] = i;
        }
    }
}

// ---------------------------------------------------------------- host
static bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows of a tile: 16 (one MMA row block) while there are few, 64 for batches of
// many rows, where A and B are then re-read a quarter as often.
static int lora_tile_rows(int64_t M) { return M >= 2048 ? 64 : 16; }
static int64_t lora_max_tiles(int64_t M, int64_t n) {
    return M / lora_tile_rows(M) + std::min(n + 1, M);
}
// Scratch of a planned call: tile count, tile list, permutation, places.
struct LoraScratch {
    size_t tiles, perm, place, total;
};
static LoraScratch lora_scratch(int64_t M, int64_t n) {
    LoraScratch s{};
    s.tiles = 256;
    s.perm = s.tiles + align256(lora_max_tiles(M, n) * sizeof(LoraTile));
    s.place = s.perm + align256(M * sizeof(int));
    s.total = s.place + (M > kPlanRows * kPlanThreads ? align256(M * sizeof(int)) : 0);
    return s;
}

template <int TM, int R>
static cudaError_t launch_tiles(const LoraArgs &p, int64_t tiles, int C, cudaStream_t st) {
    count_launch();
    return launch_pdl(k_lora<TM, R>, dim3((unsigned)(tiles * C)), dim3(kLoraThreads),
                      LoraShape<TM, R>::smem, st, C, p);
}

template <int TM>
static cudaError_t launch_rank(const LoraArgs &p, int64_t tiles, int C, cudaStream_t st) {
    if (p.r <= 16) return launch_tiles<TM, 16>(p, tiles, C, st);
    if (p.r <= 32) return launch_tiles<TM, 32>(p, tiles, C, st);
    if (p.r <= 64) return launch_tiles<TM, 64>(p, tiles, C, st);
    return launch_tiles<TM, 128>(p, tiles, C, st);
}

static cudaError_t launch_lora(LoraArgs p, void *ws, cudaStream_t st) {
    TimedScope ts(st, CQ_KERNEL_LORA_ADD);
    const int64_t tiles = lora_max_tiles(p.M, p.n);
    if (p.M <= kLoraSmallM) return launch_rank<16>(p, tiles, 8, st);
    const LoraScratch s = lora_scratch(p.M, p.n);
    uint8_t *w = reinterpret_cast<uint8_t *>(ws);
    int *n_tiles = reinterpret_cast<int *>(w);
    LoraTile *list = reinterpret_cast<LoraTile *>(w + s.tiles);
    int *perm = reinterpret_cast<int *>(w + s.perm), *place = reinterpret_cast<int *>(w + s.place);
    const int TM = lora_tile_rows(p.M);
    count_launch();
    cudaError_t e = launch_pdl(k_lora_plan, dim3(1), dim3(kPlanThreads),
                               (size_t)(p.n + 1) * sizeof(int), st, 1, p.ids, p.M, p.n, TM,
                               p.y == p.out, n_tiles, list, perm, place);
    if (e != cudaSuccess) return e;
    p.n_tiles = n_tiles;
    p.tiles = list;
    p.perm = perm;
    return TM == 16 ? launch_rank<16>(p, tiles, 8, st) : launch_rank<64>(p, tiles, 4, st);
}

}  // namespace cq

extern "C" {

CQ_API size_t cq_lora_add_workspace_size(int64_t M, int64_t n_adapters) {
    using namespace cq;
    if (M <= kLoraSmallM || M > (int64_t(1) << 24) || n_adapters <= 0 || n_adapters > 4096)
        return 0;
    return lora_scratch(M, n_adapters).total;
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
        return launch_lora(p, workspace, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? CQ_OK
                   : CQ_ERR_CUDA;
    } catch (...) {
        return CQ_ERR_CUDA;
    }
}

}  // extern "C"

// kernels_lora.cu -- cq_lora_add: low-rank adapters of many requests beside a
// shared projection, sm_100a.  out = y + scale * B (A x) with the adapter of
// each row.
//
// Rows of one adapter are gathered into tiles of up to TM rows.  A tile's work is
//   shrink  t = A x: the CTAs of a cluster, and the warps of a CTA, split K; the
//           partial t are summed through shared and distributed shared memory
//           in a fixed order
//   expand  out = y + scale * B t: CTAs split the columns
// in one of two forms (lora_one_launch):
//   one launch (k_lora; up to 40 rows, and up to 256 where the work is small): every CTA
//           finds its tile in the ids, a cluster does both products of a tile and t stays
//           in its shared memory; B goes straight from global memory into fragments: a
//           lane takes 16 bytes (8 consecutive k) of a row of B, which serves two k16 steps
//           when both operands are permuted along k alike
//   planned (k_lora_plan, k_lora_t, k_lora_out): one CTA sorts the rows into tiles of the
//           workspace, clusters write t there, and the columns are a launch of their own,
//           with B and y through a ring of shared-memory stages
// Either way A, x, B and y are streamed once per tile, the shrink's operands by cp.async
// through a ring of stages, so that a CTA's part of K is on its way at once.  Both products
// run on mma.sync m16n8k16: the op is bound by bytes (y is read and written in fp32),
// not by the tensor pipe (at rank 64 it does 16 flops a byte).
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
// One launch in which every CTA finds its own tile in the ids: always up to kLoraOneM
// rows, by the work up to one row a thread (lora_one_launch).  Else one CTA sorts the rows
// first (k_lora_plan).
constexpr int kLoraOneM = 40;

struct LoraTile {
    int id, start, rows, rank;  // id -1: no adapter; start: of its rows among the sorted ones
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
    // planned launches only
    const int *n_tiles;
    const LoraTile *tiles;
    const int *list;  // rows of tile i at list[i * TM ..)
    __half *t;        // [2][M][R]: hi, lo of the sorted rows
    float *factor;    // [M]
    int splits;       // CTAs a tile's columns are shared out to (k_lora_out)
};

CQ_DEV int valid_id(int id, int n) { return (unsigned)id < (unsigned)n ? id : -1; }

// Elements k and up of an 8-element fp16 chunk zeroed (k may be <= 0 or >= 8).
CQ_DEV uint4 keep_first(uint4 v, int k) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] = k >= 2 * i + 2 ? w[i] : k == 2 * i + 1 ? w[i] & 0xffffu : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One k32 step of the expansion held as 16 bytes per lane and row: lane q of a row's
// four holds k 8q .. 8q + 7.  MMA step s takes elements 4s .. 4s + 3 as the fragment's
// k (2q, 2q + 1) and (2q + 8, 2q + 9), for both operands.
CQ_DEV uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// What a CTA of the one-launch form works on.
struct FoundTile {
    int id, rank, rows, first;  // first: place of the tile's first row among the adapter's rows
    float scale;
};

// Row i is thread i's (M <= kLoraThreads).  Rows of an adapter form tiles of TM in
// row order; the row that begins one leads it, and tile t is that of the t-th
// leading row.  False if there is none.  buf: 256 ints of shared memory.
CQ_DEV bool find_tile(const LoraArgs &p, int t, int TM, int *buf, int *s_rows, FoundTile *f) {
    __shared__ int s_lead[kLoraWarps];
    const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
    // -2: no row, and no adapter where such rows need nothing done (in place)
    int id = i < p.M ? valid_id(p.ids[i], p.n) : -2;
    if (id == -1 && p.y == p.out) id = -2;
    buf[i] = id;
    // the row's rank and scale come while the tile is looked for
    int rank = 0;
    float scale = 1.0f;
    if (id >= 0) {
        rank = p.ranks ? max(0, min(p.ranks[id], p.r)) : p.r;
        if (p.scale) scale = p.scale[id];
    }
    __syncthreads();
    // rows of the same adapter before this one (comparisons: __match_any takes a step
    // per different value)
    int before = 0;
    const int4 *b4 = reinterpret_cast<const int4 *>(buf);
    if (32 * warp < p.M) {
#pragma unroll 8
        for (int j = 0; j < 8 * warp; j++) {
            const int4 o = b4[j];
            before += (o.x == id) + (o.y == id) + (o.z == id) + (o.w == id);
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int4 o = b4[8 * warp + j];
            before += (o.x == id && 4 * j < lane) + (o.y == id && 4 * j + 1 < lane) +
                      (o.z == id && 4 * j + 2 < lane) + (o.w == id && 4 * j + 3 < lane);
        }
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
    if (leads && at == t) *f = FoundTile{id, rank, 0, before, scale};
    __syncthreads();
    const int place = before - f->first;
    const bool mine = id == f->id && place >= 0 && place < TM;
    if (mine) s_rows[place] = i;
    const int count = __syncthreads_count(mine);
    // the places beyond the last row repeat it (their results are not stored)
    if (i >= count && i < TM) s_rows[i] = s_rows[count - 1];
    if (i == 0) f->rows = count;
    __syncthreads();
    return true;
}

CQ_DEV void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int TM, int R>
struct LoraShape {
    static constexpr int WM = TM / 16;                    // warps along the rows
    static constexpr int WN = TM == 64 || R == 128 ? 2 : 1;  // along the rank
    static constexpr int WK = kLoraWarps / WM / WN;       // along k: partial t of a CTA
    // k of a stage (TM 64: fewer, longer stages where the rank is large: 2442 rows, K 6448, rank
    // 64 46.5 us, and 48.3 with 64; rank 16 27.8, and 23.2)
    static constexpr int KC = TM == 64 ? (R >= 64 ? 128 : 64) : 16 * WK;
    static constexpr int pitch = 2 * KC + 16;             // bytes of a staged row (ldmatrix: no conflicts)
    static constexpr int rows = TM + R;                   // x rows, then A rows
    static constexpr int stage = rows * pitch;
    // halves a row of hi / lo: 8 rows of a fragment load hit different banks (16-byte
    // loads: rows 64 bytes apart modulo 128; R 16, 8-byte loads: 32)
    static constexpr int LDT = R <= 32 ? R : R + 32;
    static constexpr int t_bytes = TM == 16 ? 2 * TM * LDT * 2 : 0;  // hi, lo (k_lora only)
    static constexpr int fit = (110 * 1024 - t_bytes) / stage;   // two CTAs an SM
    static constexpr int NS = fit > 4 ? 4 : fit < 2 ? 2 : fit;   // stages
    static constexpr int LDP = R + 8;                     // floats a row of the partial t
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
// rank; TM 16: warp = one k16 step of each stage (rank over 64: and half the rank),
// summed at the end.  Leaves the sums in part [TM][LDP] (over the ring); a barrier
// has to follow.
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
    constexpr int NT = R / 8 / S::WN;             // n8 tiles of a warp
    const int wm = warp % S::WM, wk = warp / S::WM % S::WK, wn = warp / (S::WM * S::WK);
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[j][e] = 0.0f;
    // ldmatrix rows of this lane: x rows, and n rows (two n8 tiles at once)
    const uint32_t ring0 = smem_u32(ring);
    const uint32_t xa = (16 * wm + (lane & 15)) * S::pitch + 16 * (lane >> 4);
    // (a warp with one n8 tile reads it twice)
    const uint32_t wa = (TM + 8 * NT * wn + (lane & 7) + (NT > 1 ? 8 * (lane >> 4) : 0)) * S::pitch +
                        16 * ((lane >> 3) & 1);
#pragma unroll 1
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
                const uint32_t kb = 32 * (TM == 64 ? st : wk);
                uint32_t a[4];
                ldmatrix4(a, base + xa + kb);
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t b[4];
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
    float *pw = part + (wk * TM + 16 * wm) * S::LDP + 8 * NT * wn;
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

// A warp's row of t as hi + lo in units of a power of two, and that unit times the
// adapter's scale.
template <int R>
CQ_DEV void split_row(const float (&v)[(R + 31) / 32], float sc, __half *hi, __half *lo,
                      float *factor) {
    constexpr int PER = (R + 31) / 32;
    const int lane = threadIdx.x & 31;
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; i++) mx = fmaxf(mx, fabsf(v[i]));
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // 2^-e and 2^e of the largest entry's exponent, both normal numbers
    const int e = min(max((__float_as_int(mx) >> 23) & 255, 1), 253);
    const float down = __int_as_float((254 - e) << 23), up = __int_as_float(e << 23);
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const float t = v[i] * down;
        const __half h = __float2half_rn(t);
        if (R >= 32 || lane < R) {
            hi[lane + 32 * i] = h;
            // (a finite t is below 4; an infinite one is hi alone)
            lo[lane + 32 * i] = __float2half_rn(fabsf(t) <= 4.0f ? t - __half2float(h) : 0.0f);
        }
    }
    if (lane == 0) *factor = sc * up;
}

// t of the whole cluster, a warp per row, as hi + lo and the factor of the row.  Beyond
// the rank it is 0 (the partial sums there are x times 0: NaN if x is infinite).
template <int TM, int R>
CQ_DEV void gather_t(cg::cluster_group &cluster, float *part, int C, int rows, int rank, float sc,
                     __half *th, __half *tl, float *s_factor) {
    using S = LoraShape<TM, R>;
    constexpr int PER = (R + 31) / 32;
    constexpr int RB = TM == 16 ? 2 : PER > 2 ? 4 : 8;  // rows a warp has in flight
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
                            u[k][b][i] = lane + 32 * i < rank
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
            split_row<R>(v[b], sc, th + row * S::LDT, tl + row * S::LDT, s_factor + row);
        }
    }
}

// Expansion.  A warp has 16 rows of the tile, whose t it keeps in fragments, and
// goes over column blocks of 8 NB: MMA column 2q + e of n8 tiles 2i and 2i + 1 is
// column 16 i + 4q + e, + 2 in the second, of the block, so a lane holds 4
// consecutive columns of y and four lanes 64 bytes of a row.
template <int R, int NB>
struct Expand {
    static constexpr int KS = R >= 32 ? R / 32 : 1;   // 32-wide steps of the rank
    static constexpr int W = 8 * NB;                  // columns
    struct T {
        uint4 a[2][KS], b[2][KS];  // rows g and g + 8 of lo, hi
    };
    // (hi0, lo0: row g; hi1, lo1: row g + 8)
    template <bool LO = true>
    CQ_DEV static void load_t(T &o, const __half *hi0, const __half *lo0, const __half *hi1,
                              const __half *lo1) {
        const int q = threadIdx.x & 3;
#pragma unroll
        for (int h = LO ? 0 : 1; h < 2; h++) {
            const __half *ta = h ? hi0 : lo0, *tb = h ? hi1 : lo1;
#pragma unroll
            for (int s = 0; s < KS; s++) {
                if (R >= 32) {
                    o.a[h][s] = *reinterpret_cast<const uint4 *>(ta + 32 * s + 8 * q);
                    o.b[h][s] = *reinterpret_cast<const uint4 *>(tb + 32 * s + 8 * q);
                } else {
                    const uint2 u = *reinterpret_cast<const uint2 *>(ta + 4 * q);
                    const uint2 v = *reinterpret_cast<const uint2 *>(tb + 4 * q);
                    o.a[h][s] = make_uint4(u.x, u.y, 0, 0);
                    o.b[h][s] = make_uint4(v.x, v.y, 0, 0);
                }
            }
        }
    }
    struct B {
        uint4 w[NB][KS];
    };
    struct Y {
        float4 a[NB / 2], b[NB / 2];
    };
    static constexpr int pieces = NB;  // 16-byte pieces of y a lane has per block and 16 rows

    // the row of B, in the block, that is row g of n8 tile j
    CQ_DEV static int b_row(int j, int g) { return 16 * (j >> 1) + 4 * (g >> 1) + 2 * (j & 1) + (g & 1); }
    CQ_DEV static void load_b(B &o, const LoraArgs &p, int id, int rank, int n0) {
        const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
        for (int j = 0; j < NB; j++) {
            const int col = n0 + b_row(j, g);
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
    // the same from the block's staged rows
    CQ_DEV static void take_b(B &o, const unsigned char *rows, int pitch) {
        const int q = threadIdx.x & 3, g = (threadIdx.x & 31) >> 2;
#pragma unroll
        for (int j = 0; j < NB; j++) {
            const unsigned char *at = rows + b_row(j, g) * pitch;
#pragma unroll
            for (int s = 0; s < KS; s++) {
                if (R >= 32) {
                    o.w[j][s] = *reinterpret_cast<const uint4 *>(at + 64 * s + 16 * q);
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(at + 8 * q);
                    o.w[j][s] = make_uint4(v.x, v.y, 0, 0);
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
    // y of a block and 16 rows into this thread's own pieces of a slot (256
    // pieces apart), and from there: no other thread reads them, so no barrier
    // (ya, yb: y at column 4q of the warp's rows g and g + 8, NULL: no row)
    CQ_DEV static void fetch_y(unsigned char *slot, const float *ya, const float *yb, int N, int n0) {
        const int c = n0 + 4 * (threadIdx.x & 3);
        unsigned char *dst = slot + 16 * threadIdx.x;
#pragma unroll
        for (int i = 0; i < NB / 2; i++) {
            const bool in = c + 16 * i < N;  // N % 8 == 0
            if (in && ya) cp_async16_zfill(dst + 2 * i * 16 * kLoraThreads, ya + n0 + 16 * i, 16);
            if (in && yb) cp_async16_zfill(dst + (2 * i + 1) * 16 * kLoraThreads, yb + n0 + 16 * i, 16);
        }
    }
    CQ_DEV static void take_y(Y &o, const unsigned char *slot) {
        const float4 *src = reinterpret_cast<const float4 *>(slot) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < NB / 2; i++) {
            o.a[i] = src[2 * i * kLoraThreads];
            o.b[i] = src[(2 * i + 1) * kLoraThreads];
        }
    }
    // LO false: t holds the high parts alone, the low ones are read from lo0 and lo1
    template <bool LO = true>
    CQ_DEV static void run(const B &w, const T &t, const Y &y, float fa, float fb, float *oa,
                           float *ob, int N, int n0, const __half *lo0 = nullptr,
                           const __half *lo1 = nullptr) {
        const int c = n0 + 4 * (threadIdx.x & 3);
        float acc[NB][4];
#pragma unroll
        for (int j = 0; j < NB; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) acc[j][e] = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; h++) {  // lo first, then hi
#pragma unroll
            for (int s = 0; s < KS; s++) {
                uint4 ta, tb;
                if (LO || h) {
                    ta = t.a[h][s];
                    tb = t.b[h][s];
                } else {
                    ta = *reinterpret_cast<const uint4 *>(lo0 + 32 * s + 8 * (threadIdx.x & 3));
                    tb = *reinterpret_cast<const uint4 *>(lo1 + 32 * s + 8 * (threadIdx.x & 3));
                }
#pragma unroll
                for (int m = 0; m < (R >= 32 ? 2 : 1); m++) {
                    const uint32_t a[4] = {word(ta, 2 * m), word(tb, 2 * m), word(ta, 2 * m + 1),
                                           word(tb, 2 * m + 1)};
#pragma unroll
                    for (int j = 0; j < NB; j++)
                        mma_16816(acc[j], a, word(w.w[j][s], 2 * m), word(w.w[j][s], 2 * m + 1));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NB / 2; i++) {
            const float(&l)[4] = acc[2 * i], (&h)[4] = acc[2 * i + 1];
            if (c + 16 * i < N) {
                if (oa)
                    *reinterpret_cast<float4 *>(oa + n0 + 16 * i) =
                        make_float4(y.a[i].x + fa * l[0], y.a[i].y + fa * l[1], y.a[i].z + fa * h[0],
                                    y.a[i].w + fa * h[1]);
                if (ob)
                    *reinterpret_cast<float4 *>(ob + n0 + 16 * i) =
                        make_float4(y.b[i].x + fb * l[2], y.b[i].y + fb * l[3], y.b[i].z + fb * h[2],
                                    y.b[i].w + fb * h[3]);
            }
        }
    }
};

// out = y for the columns [c0, c1) of a tile without an adapter.
CQ_DEV void copy_rows(const LoraArgs &p, const int *s_rows, int rows, int c0, int c1) {
    if (p.y == p.out || c1 <= c0) return;
    constexpr int U = 4;  // pieces of 4 columns a thread has on their way
    const int per = (c1 - c0) >> 2, total = rows * per;
    for (int i0 = threadIdx.x; i0 < total; i0 += U * kLoraThreads) {
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int i = i0 + u * kLoraThreads, row = i / per;
            if (i < total)
                v[u] = *reinterpret_cast<const float4 *>(p.y + (int64_t)s_rows[row] * p.ldy + c0 +
                                                         4 * (i - row * per));
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int i = i0 + u * kLoraThreads, row = i / per;
            if (i < total)
                *reinterpret_cast<float4 *>(p.out + (int64_t)s_rows[row] * p.ldo + c0 +
                                            4 * (i - row * per)) = v[u];
        }
    }
}

// ---------------------------------------------------------------- few rows: one launch
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
    __shared__ FoundTile s_tile;

    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), crank = (int)cluster.block_rank();
    const int tile = blockIdx.x / C;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2;
    griddep_wait();
    griddep_launch();

    // ---- the tile: adapter and rows (the same for every CTA of the cluster)
    if (!find_tile(p, tile, TM, reinterpret_cast<int *>(smem), s_rows, &s_tile)) return;
    const int id = s_tile.id, rows = s_tile.rows, rank = s_tile.rank;
    const float sc = s_tile.scale;

    // columns of this CTA, in blocks of W
    const int nblk = (p.N + X::W - 1) / X::W;
    const int nb0 = (int)((int64_t)crank * nblk / C), nb1 = (int)((int64_t)(crank + 1) * nblk / C);
    const int c0 = nb0 * X::W, c1 = min(nb1 * X::W, p.N);
    if (rank == 0) {
        copy_rows(p, s_rows, rows, c0, c1);
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
    // ---- expand.  y comes by cp.async, D blocks ahead, into slots behind the partial
    // t (which the other CTAs still read); the next block's B is requested a block
    // ahead
    constexpr int y_off = TM * S::LDP * 4, slot_bytes = X::pieces * 16 * kLoraThreads;
    constexpr int room = (S::pool - y_off) / slot_bytes;
    constexpr int D = room > 8 ? 8 : room;
    static_assert(D >= 1, "no room for y");
    constexpr int MB = TM / 16, WC = kLoraWarps / MB;  // warps along the rows, along the columns
    unsigned char *slots = smem + y_off;
    const int ra = 16 * (warp % MB) + g, rb = ra + 8, cq = 4 * (lane & 3);
    const bool busy = 16 * (warp % MB) < rows;
    const float *ya = ra < rows ? p.y + (int64_t)s_rows[ra] * p.ldy + cq : nullptr;
    const float *yb = rb < rows ? p.y + (int64_t)s_rows[rb] * p.ldy + cq : nullptr;
    float *oa = ra < rows ? p.out + (int64_t)s_rows[ra] * p.ldo + cq : nullptr;
    float *ob = rb < rows ? p.out + (int64_t)s_rows[rb] * p.ldo + cq : nullptr;
    int nb = busy ? nb0 + warp / MB : nb1;  // block of this step
    int fn = nb, fs = 0;                    // block and slot of the next request
    auto request = [&]() {
        if (fn < nb1) X::fetch_y(slots + fs * slot_bytes, ya, yb, p.N, fn * X::W);
        fn += WC;
        cp_async_commit_group();
        fs = fs + 1 == D ? 0 : fs + 1;
    };
    if (S::WK > 1) __syncthreads();  // the warps' sums are read
#pragma unroll 1
    for (int i = 0; i < D; i++) request();
    typename X::B w, wn;
    if (nb < nb1) X::load_b(w, p, id, rank, nb * X::W);
    cluster.sync();
    gather_t<TM, R>(cluster, part, C, rows, rank, sc, th, tl, s_factor);
    __syncthreads();
    cluster.barrier_arrive();  // this CTA has read every partial t

    typename X::T t;
    constexpr bool LO = R <= 64;  // (rank 128: the low parts stay in shared memory)
    const __half *la = tl + ra * S::LDT, *lb = tl + rb * S::LDT;
    X::template load_t<LO>(t, th + ra * S::LDT, la, th + rb * S::LDT, lb);
    const float fa = s_factor[ra], fb = s_factor[rb];
    int slot = 0;
    for (; nb < nb1; nb += WC) {
        // (rank over 32: no registers for a second B; spilling it cost 4 us at rank 64)
        if (R <= 32 && nb + WC < nb1) X::load_b(wn, p, id, rank, (nb + WC) * X::W);
        if (rank & 7) X::cut_b(w, rank);
        typename X::Y y;
        cp_async_wait_group<D - 1>();
        X::take_y(y, slots + slot * slot_bytes);
        X::template run<LO>(w, t, y, fa, fb, oa, ob, p.N, nb * X::W, la, lb);
        request();  // into the slot just taken
        slot = slot + 1 == D ? 0 : slot + 1;
        if (R <= 32)
            w = wn;
        else if (nb + WC < nb1)
            X::load_b(w, p, id, rank, (nb + WC) * X::W);
    }
    cp_async_wait_group<0>();
    __syncwarp();
    cluster.barrier_wait();  // no CTA leaves while another may read its partial t
}

// ---------------------------------------------------------------- many rows
// Where rows or work are many the two products are launches of their own: a tile's
// shrink is short and waits on latencies, its expansion streams y, and in one
// launch all CTAs would be in the same phase at the same time (4096 rows, K 2048,
// N 2816, rank 64: 20 of 45 us with y on its way).
// The tile's entry and rows, by loads that do not wait for one another and go past
// the L1 (k_lora_out reads them before its wait, and an earlier call may have left its
// own there).  s_rows beyond the tile's rows is not meaningful.
template <int TM>
CQ_DEV bool planned_tile(const LoraArgs &p, int tile, int *s_rows, LoraTile &T) {
    const int n = __ldcg(p.n_tiles);
    const int4 v = __ldcg(reinterpret_cast<const int4 *>(p.tiles + tile));
    if (threadIdx.x < TM) s_rows[threadIdx.x] = __ldcg(p.list + (int64_t)tile * TM + threadIdx.x);
    T = LoraTile{v.x, v.y, v.z, v.w};
    __syncthreads();
    return tile < n;
}

// t = A x of a tile by a cluster: the CTAs split K, then each sums the partial t of
// its share of the rows over the cluster and stores them as hi, lo and factor.
template <int TM, int R>
__global__ void __launch_bounds__(kLoraThreads, 2) k_lora_t(const LoraArgs p) {
    using S = LoraShape<TM, R>;
    extern __shared__ __align__(16) unsigned char smem[];
    float *part = reinterpret_cast<float *>(smem);
    __shared__ int s_rows[TM];
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), crank = (int)cluster.block_rank();
    griddep_wait();
    griddep_launch();
    LoraTile T;
    if (!planned_tile<TM>(p, blockIdx.x / C, s_rows, T)) return;
    const int rank = T.rank;
    if (rank == 0) return;
    const float sc = p.scale ? p.scale[T.id] : 1.0f;
    const int chunks = (p.K + S::KC - 1) / S::KC;
    shrink<TM, R>(p, T.id, T.rows, rank, s_rows, smem, part, (int)((int64_t)crank * chunks / C),
                  (int)((int64_t)(crank + 1) * chunks / C));
    cluster.sync();
    constexpr int PER = (R + 31) / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a warp's rows, RB of them in flight
    constexpr int RB = TM == 64 ? 2 : 1;  // (C 4 and 8: TM rows are C * 8 * RB)
    float v[RB][PER];
#pragma unroll
    for (int b = 0; b < RB; b++)
#pragma unroll
        for (int i = 0; i < PER; i++) v[b][i] = 0.0f;
    const int r0 = crank * kLoraWarps + warp;
    for (int c = 0; c < C; c += 4) {  // C is a multiple of 4
        float u[4][RB][PER];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const float *rp = cluster.map_shared_rank(part, c + k);
#pragma unroll
            for (int b = 0; b < RB; b++) {
                const int row = r0 + b * C * kLoraWarps;
#pragma unroll
                for (int i = 0; i < PER; i++)
                    u[k][b][i] = row < T.rows && lane + 32 * i < rank
                                     ? rp[row * S::LDP + lane + 32 * i]
                                     : 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < 4; k++)
#pragma unroll
            for (int b = 0; b < RB; b++)
#pragma unroll
                for (int i = 0; i < PER; i++) v[b][i] += u[k][b][i];
    }
    cluster.barrier_arrive();  // this CTA has read every partial t
#pragma unroll
    for (int b = 0; b < RB; b++) {
        const int row = r0 + b * C * kLoraWarps;
        const int64_t at = T.start + row;
        if (row < T.rows)
            split_row<R>(v[b], sc, p.t + at * R, p.t + ((int64_t)p.M + at) * R, p.factor + at);
    }
    __syncwarp();
    cluster.barrier_wait();  // no CTA leaves while another may read its partial t
}

// out = y + factor * B t of a tile's share of the columns.  A warp has 16 rows of the
// tile and a share of the columns of each step; a ring of stages holds a step's rows
// of B (shared by the warps of the same columns) and its y (every thread its own).
// Nothing before k_lora_t can still be running when this kernel starts (k_lora_t lets it
// start after its own wait), so the tile, y and B are requested before the wait for t.
template <int TM, int R>
struct OutShape {
    static constexpr int NB = TM == 64 && R <= 64 ? 4 : 2;    // n8 tiles of a warp's step
    static constexpr int MB = TM / 16, WC = kLoraWarps / MB;  // warps along the rows, along the columns
    static constexpr int W = WC * 8 * NB;                  // columns of a step
    // bytes of a staged row of B: the 8 rows of a fragment load hit different banks
    static constexpr int pitch = R >= 64 ? 2 * R + 64 : 2 * R;
    static constexpr int y_off = W * pitch;
    static constexpr int stage = y_off + NB * 16 * kLoraThreads;
    static constexpr int fit = 100 * 1024 / stage;         // two CTAs an SM
    static constexpr int D = fit > 8 ? 8 : fit < 2 ? 2 : fit;
};

template <int TM, int R>
__global__ void __launch_bounds__(kLoraThreads, 2) k_lora_out(const LoraArgs p) {
    using S = OutShape<TM, R>;
    using X = Expand<R, S::NB>;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int s_rows[TM];
    const int tile = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    LoraTile T;
    if (!planned_tile<TM>(p, tile, s_rows, T)) {
        griddep_wait();  // this kernel ends after k_lora_t, whatever its CTAs had to do
        return;
    }
    const int rows = T.rows, rank = T.rank;
    const int nblk = (p.N + S::W - 1) / S::W;
    const int nb0 = (int)((int64_t)split * nblk / p.splits);
    const int nb1 = (int)((int64_t)(split + 1) * nblk / p.splits);
    if (rank == 0) {
        griddep_wait();
        copy_rows(p, s_rows, rows, nb0 * S::W, min(nb1 * S::W, p.N));
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    const int ra = 16 * (warp % S::MB) + g, rb = ra + 8, wc = warp / S::MB;
    const int cw = wc * X::W;                   // the warp's columns in a step
    const bool busy = 16 * (warp % S::MB) < rows;
    const int cq = 4 * q;
    const float *ya = ra < rows ? p.y + (int64_t)s_rows[ra] * p.ldy + cq : nullptr;
    const float *yb = rb < rows ? p.y + (int64_t)s_rows[rb] * p.ldy + cq : nullptr;
    float *oa = ra < rows ? p.out + (int64_t)s_rows[ra] * p.ldo + cq : nullptr;
    float *ob = rb < rows ? p.out + (int64_t)s_rows[rb] * p.ldo + cq : nullptr;
    // 16-byte pieces of a step's rows of B: PR a row, up to r (zeros beyond the rank's
    // last piece)
    constexpr int PR = R / 8, PB = S::W * PR, PASSES = (PB + kLoraThreads - 1) / kLoraThreads;
    const __half *bbase = p.b + (int64_t)T.id * p.N * p.r;
    auto request = [&](int nb, int slot) {
        unsigned char *st = smem + slot * S::stage;
        if (nb < nb1) {
#pragma unroll
            for (int i = 0; i < PASSES; i++) {
                const int pc = tid + i * kLoraThreads;
                if (PB % kLoraThreads == 0 || pc < PB) {
                    const int row = pc / PR, k = 8 * (pc % PR), col = min(nb * S::W + row, p.N - 1);
                    const bool in = k < rank;
                    cp_async16_zfill(st + row * S::pitch + 2 * k,
                                     in ? bbase + (int64_t)col * p.r + k : p.b, in ? 16 : 0);
                }
            }
            X::fetch_y(st + S::y_off, ya, yb, p.N, nb * S::W + cw);
        }
        cp_async_commit_group();
    };
    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < S::D - 1; i++) request(nb0 + i, i);
    griddep_wait();
    griddep_launch();
    typename X::T t;
    const int64_t a0 = T.start + min(ra, rows - 1), b0 = T.start + min(rb, rows - 1);
    const __half *lo = p.t + (int64_t)p.M * R;
    X::load_t(t, p.t + a0 * R, lo + a0 * R, p.t + b0 * R, lo + b0 * R);
    const float fa = p.factor[a0], fb = p.factor[b0];
    for (int nb = nb0; nb < nb1; nb++) {
        cp_async_wait_group<S::D - 2>();
        __syncthreads();  // every thread's pieces are here; the slot taken last is free
        request(nb + S::D - 1, slot == 0 ? S::D - 1 : slot - 1);
        if (busy) {
            const unsigned char *st = smem + slot * S::stage;
            typename X::B w;
            X::take_b(w, st + cw * S::pitch, S::pitch);
            if (rank & 7) X::cut_b(w, rank);
            typename X::Y y;
            X::take_y(y, st + S::y_off);
            X::run(w, t, y, fa, fb, oa, ob, p.N, nb * S::W + cw);
        }
        slot = slot + 1 == S::D ? 0 : slot + 1;
    }
    cp_async_wait_group<0>();
}

// ---------------------------------------------------------------- rows by adapter
// One CTA: counts per adapter (slot n: no adapter), their offsets, the tiles and
// their rows.  A row's place among its adapter's rows comes from
// the counting atomics: their order may change from call to call, and with it the
// rows of a tile, but a row's result does not depend on its place.
constexpr int kPlanThreads = 1024;
constexpr int kPlanRows = 8;  // rows a thread holds at once

// Exclusive scan over a warp, and over the CTA, of (a, b); adds and advances the running
// totals.
CQ_DEV void warp_scan_pair(int &a, int &b, int &ta, int &tb) {
    const int lane = threadIdx.x & 31, a0 = a, b0 = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    const int sa = __shfl_sync(0xffffffffu, a, 31), sb = __shfl_sync(0xffffffffu, b, 31);
    a += ta - a0;
    b += tb - b0;
    ta += sa;
    tb += sb;
}
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
            LoraTile *tiles, int *list, int *place, const int32_t *__restrict__ ranks, int r_max) {
    extern __shared__ int cnt[];  // [n + 1] counts, then places in the list
    int *row0 = cnt + n + 1;      // [n + 1] first sorted row of each adapter
    int *tile0 = row0 + n + 1;    // [n + 2] first tile
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
            // a warp inside one request takes one atomic
            int same;
            __match_all_sync(0xffffffffu, key[u], &same);
            if (same) {
                int base = 0;
                if (lane == 0 && key[u] >= 0) base = atomicAdd(&cnt[key[u]], 32);
                at[u] = __shfl_sync(0xffffffffu, base, 0) + lane;
            } else {
                at[u] = key[u] >= 0 ? atomicAdd(&cnt[key[u]], 1) : 0;
            }
            const int i = b0 + u * kPlanThreads + tid;
            if (!once && i < M) place[i] = at[u];
        }
    }
    __syncthreads();
    // prefixes of rows and tiles over the adapters: one warp's scan up to 31 of them
    int rows = 0, nt = 0;
    for (int b0 = 0; b0 <= n; b0 += kPlanThreads) {
        const int i = b0 + tid;
        const int c = i <= n ? cnt[i] : 0;
        const int t = i == n && skip_none ? 0 : (c + TM - 1) / TM;
        int start = c, first = t;
        if (n >= 32)
            scan_pair(start, first, rows, nt, wsum);
        else if (tid < 32)
            warp_scan_pair(start, first, rows, nt);
        if (i <= n) {
            cnt[i] = first * TM;  // its tiles' places in the list
            row0[i] = start;
            tile0[i] = first;
            if (i == n) tile0[n + 1] = first + t;
        }
    }
    __syncthreads();
    nt = tile0[n + 1];
    if (tid == 0) *n_tiles = nt;
    for (int ti = tid; ti < nt; ti += kPlanThreads) {
        // the adapter whose tiles hold ti: the last with tile0 <= ti (those without
        // tiles have the next one's tile0)
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (tile0[mid] <= ti)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int k = ti - tile0[lo];
        const int rank = lo == n ? 0 : ranks ? max(0, min(ranks[lo], r_max)) : r_max;
        const int here = row0[lo] + k * TM;
        const int end = lo == n ? M : row0[lo + 1];
        tiles[ti] = LoraTile{lo == n ? -1 : lo, here, min(TM, end - here), rank};
    }
    for (int b0 = 0; b0 < M; b0 += kPlanRows * kPlanThreads) {
        if (!once) load(b0);
#pragma unroll
        for (int u = 0; u < kPlanRows; u++) {
            const int i = b0 + u * kPlanThreads + tid;
            if (i < M && !(skip_none && key[u] == n))
                list[cnt[key[u]] + (once ? at[u] : place[i])] = i;
        }
    }
}

// ---------------------------------------------------------------- host
static bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows of a tile: 16 (one MMA row block) while there are few, 64 for batches of
// many rows, where A and B are then re-read a quarter as often.  Measured, us, 16 and 64:
// K 2048, N 2816, 8 adapters of rank 64: 600 rows 15.0 and 17.3, 1500: 25.1 and 20.6, 3000:
// 42.7 and 33.2, 4096: 49.8 and 33.9; K = N = 4096, 16 of rank 16: 1024 rows 17.3 and 20.7,
// 2048: 24.4 and 29.1, 3000: 39.0 and 38.3; K 1024, N 2048, 4 of rank 128: 1024 rows 19.2
// and 19.3, 4096: 56.5 and 37.5.  The two cross between 1024 and 3000 rows.
static int lora_tile_rows(int64_t M) { return M >= 2048 ? 64 : 16; }
static int64_t lora_max_tiles(int64_t M, int64_t n) {
    return M / lora_tile_rows(M) + std::min(n + 1, M);
}
static int lora_rank(int64_t r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }
// The one-launch form has no sort before it (3 us) but does all of a tile in one cluster:
// it is behind where tiles are many waves of clusters or long.  Measured, us, one launch
// and planned: 64 rows, K = N = 4096, 32 adapters of rank 64: 14.0 and 15.8, 64 adapters:
// 27.1 and 23.8; 192 rows, 32 adapters: 19.0 and 17.3; 192 rows, K = N = 2048, 8 adapters
// of rank 64: 12.4 and 11.3, at K = N = 512: 7.3 and 9.9; 128 rows over 200 adapters of
// rank 16, K 2560, N 6144: 34 and 27.
static bool lora_one_launch(int64_t M, int64_t K, int64_t N, int64_t n, int64_t r) {
    if (M <= kLoraOneM || M > kLoraThreads) return M <= kLoraOneM;
    const int64_t tiles = lora_max_tiles(M, n), work = tiles * 16 * lora_rank(r) * (K + N);
    return work < 48000000 || (M <= 160 && tiles <= 80 && work < 350000000);
}
// Scratch of a planned call: tile count, tiles, their rows, places, t, factors.
struct LoraScratch {
    size_t tiles, list, place, t, factor, total;
};
static LoraScratch lora_scratch(int64_t M, int64_t n, int64_t r) {
    LoraScratch s{};
    s.tiles = 256;
    s.list = s.tiles + align256(lora_max_tiles(M, n) * sizeof(LoraTile));
    s.place = s.list + align256(lora_max_tiles(M, n) * lora_tile_rows(M) * sizeof(int));
    s.t = s.place + (M > kPlanRows * kPlanThreads ? align256(M * sizeof(int)) : 0);
    s.factor = s.t + align256(2 * M * lora_rank(r) * sizeof(__half));
    s.total = s.factor + align256(M * sizeof(float));
    return s;
}

// One cluster per tile: 8 CTAs, or 4 where a tile's A and B are small (12 KB: 6.5 us
// with 4, 7.3 with 8; 280 KB: 8.4 and 6.8).
template <int R>
static cudaError_t launch_small(const LoraArgs &p, cudaStream_t st) {
    const int C = ((int64_t)p.K + p.N) * p.r * 2 < 96 * 1024 ? 4 : 8;
    count_launch();
    return launch_pdl(k_lora<16, R>, dim3((unsigned)(lora_max_tiles(p.M, p.n) * C)),
                      dim3(kLoraThreads), LoraShape<16, R>::smem, st, C, p);
}

template <int TM, int R>
static cudaError_t launch_planned(LoraArgs p, cudaStream_t st) {
    // K over 8 CTAs instead of 4 where a CTA's part is still 16 stages or more and the
    // sums to be exchanged are small (2442 rows, K 6448, rank 16: 23.5 us, and 27.7
    // with 4; 4096 rows, K 2048, rank 64: 41 and 34)
    const int C = R <= 32 && p.K >= 64 * LoraShape<TM, R>::KC ? 8 : 4;
    const int64_t tiles = lora_max_tiles(p.M, p.n);
    count_launch(2);
    cudaError_t e = launch_pdl(k_lora_t<TM, R>, dim3((unsigned)(tiles * C)), dim3(kLoraThreads),
                               (size_t)LoraShape<TM, R>::pool, st, C, p);
    if (e != cudaSuccess) return e;
    // column shares of a tile: two CTAs an SM in all, of at least four steps each (a share
    // of fewer fills its ring for little: 517 rows, N 2560, rank 32 16.7 us, and 18.3 with
    // one step or two; of eight 19.6: too few CTAs)
    using S = OutShape<TM, R>;
    const int nblk = (p.N + S::W - 1) / S::W;
    const int64_t full = std::max<int64_t>(1, p.M / TM);
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(2LL * sm_count() / full, nblk / 4));
    return launch_pdl(k_lora_out<TM, R>, dim3((unsigned)(tiles * p.splits)), dim3(kLoraThreads),
                      (size_t)S::D * S::stage, st, 1, p);
}

static cudaError_t launch_lora(LoraArgs p, void *ws, cudaStream_t st) {
    TimedScope ts(st, CQ_KERNEL_LORA_ADD);
    const int R = lora_rank(p.r);
    if (lora_one_launch(p.M, p.K, p.N, p.n, p.r))
        return R == 16   ? launch_small<16>(p, st)
               : R == 32 ? launch_small<32>(p, st)
               : R == 64 ? launch_small<64>(p, st)
                         : launch_small<128>(p, st);
    const LoraScratch s = lora_scratch(p.M, p.n, p.r);
    uint8_t *w = reinterpret_cast<uint8_t *>(ws);
    int *n_tiles = reinterpret_cast<int *>(w);
    LoraTile *list = reinterpret_cast<LoraTile *>(w + s.tiles);
    int *rows = reinterpret_cast<int *>(w + s.list), *place = reinterpret_cast<int *>(w + s.place);
    const int TM = lora_tile_rows(p.M);
    count_launch();
    cudaError_t e = launch_pdl(k_lora_plan, dim3(1), dim3(kPlanThreads),
                               (size_t)(3 * p.n + 4) * sizeof(int), st, 1, p.ids, p.M, p.n, TM,
                               p.y == p.out, n_tiles, list, rows, place, p.ranks, p.r);
    if (e != cudaSuccess) return e;
    p.n_tiles = n_tiles;
    p.tiles = list;
    p.list = rows;
    p.t = reinterpret_cast<__half *>(w + s.t);
    p.factor = reinterpret_cast<float *>(w + s.factor);
    if (TM == 16)
        return R == 16   ? launch_planned<16, 16>(p, st)
               : R == 32 ? launch_planned<16, 32>(p, st)
               : R == 64 ? launch_planned<16, 64>(p, st)
                         : launch_planned<16, 128>(p, st);
    return R == 16   ? launch_planned<64, 16>(p, st)
           : R == 32 ? launch_planned<64, 32>(p, st)
           : R == 64 ? launch_planned<64, 64>(p, st)
                     : launch_planned<64, 128>(p, st);
}

}  // namespace cq

extern "C" {

CQ_API size_t cq_lora_add_workspace_size(int64_t M, int64_t n_adapters, int64_t r_max) {
    using namespace cq;
    if (M <= kLoraOneM || M > (int64_t(1) << 24) || n_adapters <= 0 || n_adapters > 4096 ||
        r_max <= 0 || r_max > kLoraMaxRank)
        return 0;
    return lora_scratch(M, n_adapters, r_max).total;
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
    const size_t need = cq_lora_add_workspace_size(M, n_adapters, r_max);
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

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
// and y once.  Both products run on mma.sync m16n8k16 with the operands loaded
// from global memory straight into fragments: a lane takes 16 bytes (8
// consecutive k) of a row, which serves two k16 steps when both operands are
// permuted along k alike, so there is no staging and no barrier in the loops.
// The op is bound by bytes (y is read and written in fp32), not by the tensor
// pipe: at rank 64 it does 16 flops a byte.
//
// t is fp32 and B is fp16: t is scaled by a power of two per row, so that its
// largest entry is in [1, 2), and split into two fp16 parts, t = hi + lo with
// an error of 2^-22 of that entry; one more MMA per tile keeps fp32-like sums
// (one fp16 part would leave 2^-11 of the update in an fp32 output).
#include <cooperative_groups.h>

#include <algorithm>

#include "cq_common.cuh"
#include "cq_internal.h"

namespace cg = cooperative_groups;

namespace cq {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraMaxRank = 128;
// Up to this many rows every cluster finds its own tile in the ids; above, one
// CTA sorts the rows first (k_lora_plan).
constexpr int kLoraSmallM = 512;

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

// One k32 step held as 16 bytes per lane and row: lane q of a row's four holds
// k 8q .. 8q + 7.  MMA step s takes elements 4s .. 4s + 3 as the fragment's k
// (2q, 2q + 1) and (2q + 8, 2q + 9), for both operands.
CQ_DEV uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int TM, int R>
struct LoraShape {
    static constexpr int WM = TM / 16;            // warps along the rows (shrink)
    static constexpr int WK = kLoraWarps / WM;    // warps along K
    static constexpr int LDP = R + 8;             // floats a row of the partial t
    static constexpr int LDT = R + 8;             // halves a row of hi / lo
    static constexpr size_t part_bytes = (size_t)WK * TM * LDP * sizeof(float);
    static constexpr size_t t_bytes = (size_t)2 * TM * LDT * sizeof(__half);
    static constexpr size_t smem = part_bytes + t_bytes;
};

template <int TM, int R>
__global__ void __launch_bounds__(kLoraThreads, 2) k_lora(const LoraArgs p) {
    using S = LoraShape<TM, R>;
    constexpr int KS = R / 32 > 0 ? R / 32 : 1;   // 32-wide steps of the rank
    extern __shared__ __align__(16) unsigned char smem[];
    float *part = reinterpret_cast<float *>(smem);                       // [WK][TM][LDP]
    __half *th = reinterpret_cast<__half *>(smem + S::part_bytes);       // [TM][LDT]
    __half *tl = th + TM * S::LDT;
    __shared__ int s_rows[TM];
    __shared__ float s_factor[TM];
    __shared__ int s_id, s_count;

    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), crank = (int)cluster.block_rank();
    const int tile = blockIdx.x / C;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, q = lane & 3;
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
    } else if (warp == 0) {
        // cluster `tile` stands for row `tile`: it leads a tile if the number of
        // earlier rows of the same adapter is a multiple of TM
        const int mine = valid_id(p.ids[tile], p.n);
        int before = 0, count = 0;
        for (int b0 = 0; b0 < p.M; b0 += 32) {
            const int i = b0 + lane;
            const bool same = i < p.M && valid_id(p.ids[i], p.n) == mine;
            before += __popc(__ballot_sync(0xffffffffu, same && i < tile));
            const unsigned after = __ballot_sync(0xffffffffu, same && i >= tile);
            const int at = count + __popc(after & ((1u << lane) - 1u));
            if (same && i >= tile && at < TM) s_rows[at] = i;
            count += __popc(after);
        }
        count = min(count, TM);
        __syncwarp();
        const int last = s_rows[count - 1];
        __syncwarp();
        for (int i = count + lane; i < TM; i += 32) s_rows[i] = last;
        if (lane == 0) {
            s_id = mine;
            s_count = before % TM == 0 ? count : 0;
        }
    }
    __syncthreads();
    const int id = s_id, rows = s_count;
    if (rows == 0) return;
    const int rank = id < 0 ? 0 : p.ranks ? max(0, min(p.ranks[id], p.r)) : p.r;

    // columns of this CTA, in blocks of 32
    const int nblk = (p.N + 31) >> 5;
    const int nb0 = (int)((int64_t)crank * nblk / C), nb1 = (int)((int64_t)(crank + 1) * nblk / C);
    if (rank == 0) {  // out = y
        if (p.y != p.out) {
            const int c0 = nb0 * 32, c1 = min(nb1 * 32, p.N);
            for (int i = warp; i < rows; i += kLoraWarps) {
                const float *src = p.y + (int64_t)s_rows[i] * p.ldy;
                float *dst = p.out + (int64_t)s_rows[i] * p.ldo;
                for (int c = c0 + 4 * lane; c < c1; c += 128)
                    *reinterpret_cast<float4 *>(dst + c) = *reinterpret_cast<const float4 *>(src + c);
            }
        }
        return;
    }

    // ---- shrink: warp (wm, wk) sums rows [16 wm, +16) over its part of K
    {
        const int wm = warp % S::WM, wk = warp / S::WM;
        const int steps = (p.K + 31) >> 5, parts = C * S::WK, me = crank * S::WK + wk;
        const int s0 = (int)((int64_t)me * steps / parts), s1 = (int)((int64_t)(me + 1) * steps / parts);
        float acc[R / 8][4];
#pragma unroll
        for (int j = 0; j < R / 8; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) acc[j][e] = 0.0f;
        if (16 * wm < rows) {
            const __half *x0 = p.x + (int64_t)s_rows[16 * wm + g] * p.K + 8 * q;
            const __half *x1 = p.x + (int64_t)s_rows[16 * wm + g + 8] * p.K + 8 * q;
            const __half *ab = p.a + ((int64_t)id * p.r + g) * p.K + 8 * q;
#pragma unroll 2
            for (int s = s0; s < s1; s++) {
                const int k = 32 * s;
                const bool in = k + 8 * q < p.K;
                const uint4 zero = make_uint4(0, 0, 0, 0);
                const uint4 xa = in ? *reinterpret_cast<const uint4 *>(x0 + k) : zero;
                const uint4 xb = in ? *reinterpret_cast<const uint4 *>(x1 + k) : zero;
                uint4 w[R / 8];
#pragma unroll
                for (int j = 0; j < R / 8; j++)
                    w[j] = in && 8 * j + g < rank
                               ? *reinterpret_cast<const uint4 *>(ab + (int64_t)8 * j * p.K + k)
                               : zero;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const uint32_t a[4] = {word(xa, 2 * h), word(xb, 2 * h), word(xa, 2 * h + 1),
                                           word(xb, 2 * h + 1)};
#pragma unroll
                    for (int j = 0; j < R / 8; j++)
                        mma_16816(acc[j], a, word(w[j], 2 * h), word(w[j], 2 * h + 1));
                }
            }
        }
        float *pw = part + ((size_t)wk * TM + 16 * wm) * S::LDP;
#pragma unroll
        for (int j = 0; j < R / 8; j++) {
            *reinterpret_cast<float2 *>(pw + g * S::LDP + 8 * j + 2 * q) =
                make_float2(acc[j][0], acc[j][1]);
            *reinterpret_cast<float2 *>(pw + (g + 8) * S::LDP + 8 * j + 2 * q) =
                make_float2(acc[j][2], acc[j][3]);
        }
    }
    __syncthreads();
    if (S::WK > 1) {
        for (int i = threadIdx.x; i < TM * R; i += kLoraThreads) {
            const int at = (i / R) * S::LDP + i % R;
            float v = part[at];
#pragma unroll
            for (int w = 1; w < S::WK; w++) v += part[(size_t)w * TM * S::LDP + at];
            part[at] = v;
        }
    }
    cluster.sync();
    // ---- t of the whole cluster, a warp per row, as two fp16 parts
    {
        constexpr int PER = (R + 31) / 32;
        const float sc = p.scale ? p.scale[id] : 1.0f;
        for (int row = warp; row < TM; row += kLoraWarps) {
            float v[PER];
            float mx = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; i++) v[i] = 0.0f;
            if (row < rows) {
                for (int c = 0; c < C; c++) {
                    const float *rp = cluster.map_shared_rank(part, c) + row * S::LDP;
#pragma unroll
                    for (int i = 0; i < PER; i++)
                        if (R >= 32 || lane < R) v[i] += rp[lane + 32 * i];
                }
            }
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
                const __half hi = __float2half_rn(t);
                if (R >= 32 || lane < R) {
                    th[row * S::LDT + lane + 32 * i] = hi;
                    tl[row * S::LDT + lane + 32 * i] = __float2half_rn(t - __half2float(hi));
                }
            }
            if (lane == 0) s_factor[row] = sc * up;
        }
    }
    __syncthreads();
    cluster.barrier_arrive();  // this CTA has read every partial t

    // ---- expand: a warp per 32 columns.  MMA column 2q + e of n8 tile j is
    // column 8q + 2j + e of the block, so a lane holds 8 consecutive columns
    for (int nb = nb0 + warp; nb < nb1; nb += kLoraWarps) {
        const int n0 = 32 * nb;
        uint4 bw[4][KS];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int col = n0 + 8 * (g >> 1) + 2 * j + (g & 1);
            const __half *br = p.b + ((int64_t)id * p.N + min(col, p.N - 1)) * p.r;
#pragma unroll
            for (int s = 0; s < KS; s++) {
                if (R >= 32) {
                    const int k = 32 * s + 8 * q;
                    bw[j][s] = k < rank ? keep_first(*reinterpret_cast<const uint4 *>(br + k), rank - k)
                                        : make_uint4(0, 0, 0, 0);
                } else {  // 4 consecutive k per lane, one MMA step
                    const int k = 4 * q;
                    uint2 v = make_uint2(0, 0);
                    if (k < rank) v = *reinterpret_cast<const uint2 *>(br + k);
                    bw[j][s] = keep_first(make_uint4(v.x, v.y, 0, 0), rank - k);
                }
            }
        }
        const int c = n0 + 8 * q;
        const bool in = c < p.N;  // N % 8 == 0: whole lanes
        for (int mb = 0; 16 * mb < rows; mb++) {
            const int ra = 16 * mb + g, rb = ra + 8;
            const bool la = in && ra < rows, lb = in && rb < rows;
            float4 ya[2] = {}, yb[2] = {};
            if (la) {
                const float4 *src = reinterpret_cast<const float4 *>(p.y + (int64_t)s_rows[ra] * p.ldy + c);
                ya[0] = src[0];
                ya[1] = src[1];
            }
            if (lb) {
                const float4 *src = reinterpret_cast<const float4 *>(p.y + (int64_t)s_rows[rb] * p.ldy + c);
                yb[0] = src[0];
                yb[1] = src[1];
            }
            float acc[4][4];
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[j][e] = 0.0f;
#pragma unroll
            for (int s = 0; s < KS; s++) {
#pragma unroll
                for (int part_i = 0; part_i < 2; part_i++) {  // lo first, then hi
                    const __half *tp = part_i ? th : tl;
                    if (R >= 32) {
                        const uint4 va = *reinterpret_cast<const uint4 *>(tp + ra * S::LDT + 32 * s + 8 * q);
                        const uint4 vb = *reinterpret_cast<const uint4 *>(tp + rb * S::LDT + 32 * s + 8 * q);
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const uint32_t a[4] = {word(va, 2 * h), word(vb, 2 * h),
                                                   word(va, 2 * h + 1), word(vb, 2 * h + 1)};
#pragma unroll
                            for (int j = 0; j < 4; j++)
                                mma_16816(acc[j], a, word(bw[j][s], 2 * h), word(bw[j][s], 2 * h + 1));
                        }
                    } else {
                        const uint2 va = *reinterpret_cast<const uint2 *>(tp + ra * S::LDT + 4 * q);
                        const uint2 vb = *reinterpret_cast<const uint2 *>(tp + rb * S::LDT + 4 * q);
                        const uint32_t a[4] = {va.x, vb.x, va.y, vb.y};
#pragma unroll
                        for (int j = 0; j < 4; j++) mma_16816(acc[j], a, bw[j][s].x, bw[j][s].y);
                    }
                }
            }
            if (la) {
                const float f = s_factor[ra];
                float4 *dst = reinterpret_cast<float4 *>(p.out + (int64_t)s_rows[ra] * p.ldo + c);
                dst[0] = make_float4(ya[0].x + f * acc[0][0], ya[0].y + f * acc[0][1],
                                     ya[0].z + f * acc[1][0], ya[0].w + f * acc[1][1]);
                dst[1] = make_float4(ya[1].x + f * acc[2][0], ya[1].y + f * acc[2][1],
                                     ya[1].z + f * acc[3][0], ya[1].w + f * acc[3][1]);
            }
            if (lb) {
                const float f = s_factor[rb];
                float4 *dst = reinterpret_cast<float4 *>(p.out + (int64_t)s_rows[rb] * p.ldo + c);
                dst[0] = make_float4(yb[0].x + f * acc[0][2], yb[0].y + f * acc[0][3],
                                     yb[0].z + f * acc[1][2], yb[0].w + f * acc[1][3]);
                dst[1] = make_float4(yb[1].x + f * acc[2][2], yb[1].y + f * acc[2][3],
                                     yb[1].z + f * acc[3][2], yb[1].w + f * acc[3][3]);
            }
        }
    }
    __syncwarp();
    cluster.barrier_wait();  // no CTA leaves while another may read its partial t
}

// ---------------------------------------------------------------- rows by adapter
// One CTA: counts per adapter (slot n: no adapter), their offsets, the tile
// list and the permutation.  The order of an adapter's rows inside its range is
// that of the atomics and may change from call to call; a row's result does not
// depend on its place in a tile.
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads)
k_lora_plan(const int32_t *__restrict__ ids, int M, int n, int TM, int *n_tiles, LoraTile *tiles,
            int *perm) {
    extern __shared__ int cnt[];  // [n + 1] counts, then next free place
    __shared__ int wsum[2][32];
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i <= n; i += kPlanThreads) cnt[i] = 0;
    __syncthreads();
    constexpr int U = 4;  // loads in flight per thread
    auto each = [&](auto &&f) {
        for (int b0 = 0; b0 < M; b0 += U * kPlanThreads) {
            int v[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int i = b0 + u * kPlanThreads + tid;
                v[u] = i < M ? valid_id(ids[i], n) : -2;
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int key = v[u] == -1 ? n : v[u];
                // the lanes of a warp with the same adapter take one atomic
                const unsigned peers = __match_any_sync(0xffffffffu, key);
                const int leader = __ffs(peers) - 1;
                f(b0 + u * kPlanThreads + tid, key, peers, leader);
            }
        }
    };
    each([&](int, int key, unsigned peers, int leader) {
        if (key >= 0 && lane == leader) atomicAdd(&cnt[key], __popc(peers));
    });
    __syncthreads();
    // exclusive prefixes of rows and tiles over the adapters
    int row0 = 0, tile0 = 0;
    for (int b0 = 0; b0 <= n; b0 += kPlanThreads) {
        const int i = b0 + tid;
        const int c = i <= n ? cnt[i] : 0, t = (c + TM - 1) / TM;
        int rs = c, ts = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, rs, o), b = __shfl_up_sync(0xffffffffu, ts, o);
            if (lane >= o) {
                rs += a;
                ts += b;
            }
        }
        if (lane == 31) {
            wsum[0][warp] = rs;
            wsum[1][warp] = ts;
        }
        __syncthreads();
        int rb = row0, tb = tile0, rt = 0, tt = 0;
        for (int w = 0; w < 32; w++) {
            if (w < warp) {
                rb += wsum[0][w];
                tb += wsum[1][w];
            }
            rt += wsum[0][w];
            tt += wsum[1][w];
        }
        const int start = rb + rs - c;
        if (i <= n) {
            cnt[i] = start;
            for (int k = 0; k < t; k++)
                tiles[tb + ts - t + k] =
                    LoraTile{i == n ? -1 : i, start + k * TM, min(TM, c - k * TM), 0};
        }
        row0 += rt;
        tile0 += tt;
        __syncthreads();
    }
    if (tid == 0) *n_tiles = tile0;
    each([&](int i, int key, unsigned peers, int leader) {
        int at = 0;
        if (key >= 0 && lane == leader) at = atomicAdd(&cnt[key], __popc(peers));
        at = __shfl_sync(0xffffffffu, at, leader);
        if (key >= 0) perm[at + __popc(peers & ((1u << lane) - 1u))] = i;
    });
}

// ---------------------------------------------------------------- host
static bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows of a tile: 16 (one MMA row block) while a tile's cost is its latency,
// 64 for batches of many rows, where A and B are then re-read a quarter as often.
static int lora_tile_rows(int64_t M) { return M > kLoraSmallM ? 64 : 16; }
static int64_t lora_max_tiles(int64_t M, int64_t n) {
    return M / lora_tile_rows(M) + std::min(n + 1, M);
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
    if (p.M <= kLoraSmallM) return launch_rank<16>(p, p.M, p.M <= 128 ? 8 : 4, st);
    const int64_t tiles = lora_max_tiles(p.M, p.n);
    int *n_tiles = reinterpret_cast<int *>(ws);
    LoraTile *list = reinterpret_cast<LoraTile *>(reinterpret_cast<uint8_t *>(ws) + 256);
    int *perm = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(list) +
                                        align256(tiles * sizeof(LoraTile)));
    count_launch();
    cudaError_t e = launch_pdl(k_lora_plan, dim3(1), dim3(kPlanThreads),
                               (size_t)(p.n + 1) * sizeof(int), st, 1, p.ids, p.M, p.n,
                               lora_tile_rows(p.M), n_tiles, list, perm);
    if (e != cudaSuccess) return e;
    p.n_tiles = n_tiles;
    p.tiles = list;
    p.perm = perm;
    return launch_rank<64>(p, tiles, 4, st);
}

}  // namespace cq

extern "C" {

CQ_API size_t cq_lora_add_workspace_size(int64_t M, int64_t n_adapters) {
    using namespace cq;
    if (M <= kLoraSmallM || M > (int64_t(1) << 24) || n_adapters <= 0 || n_adapters > 4096)
        return 0;
    return 256 + align256(lora_max_tiles(M, n_adapters) * sizeof(LoraTile)) +
           align256(M * sizeof(int));
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

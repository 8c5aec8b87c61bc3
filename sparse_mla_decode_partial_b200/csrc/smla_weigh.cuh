// smla_weigh.cuh -- the attention weight each cached position received:
//   acc[b, i] += sum over the query rows (t, h) of sequence b with i visible of
//     exp(scale q[b,t,h] . row_i - lse[b,t,h]).
// Only the score half of a decode, with the softmax's statistics known, so
// nothing is exchanged between positions: the work is reading the rows once.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "smla_indexer.cuh"
#include "smla_partial_q4.cuh"
#include "smla_q4.cuh"

namespace smla {

struct WeighParams {
    PartialParams p;      // q, cache, pages; seq_lens [B, dense_t], K = max_n, T = 1 unit of pack = dense_t tokens
    const float *lse;     // [B, T, H]
    float *acc;           // [B, max_n]
    int grid;             // CTAs that share the tiles
    int min_tiles;        // fewest tiles worth a CTA
};

// Query row r of sequence b: lse in log2 units as a sum of two floats (its
// rounding would otherwise scale every weight of the row) and the positions it
// sees, none for a row that attended to nothing (lse = -inf).
__device__ __forceinline__ void weigh_row(const WeighParams &a, int b, int r, float2 *l2, int *lim) {
    const PartialParams &p = a.p;
    const int rows = p.dense_t * p.dense_h;
    *l2 = make_float2(0.f, 0.f);
    *lim = 0;
    if (r >= rows) return;
    float l;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(l) : "l"(a.lse + (size_t)b * rows + r));
    const double x = (double)l * 1.4426950408889634074;
    l2->x = (float)x;
    l2->y = isfinite(l2->x) ? (float)(x - (double)l2->x) : 0.f;
    if (l != -INFINITY)
        *lim = min(max(ld_input(p.seq_lens + (size_t)b * p.dense_t + r / p.dense_h), 0), p.K);
}

// ---------------------------------------------------------------- 4-bit rows
// The dense decode's schedule and score product (smla_partial_q4.cuh): CTAs take
// equal runs of the batch's 64-position tiles, a page lands by one bulk copy,
// and each warp scores 16 of its rows against 16 G query rows at a time,
// decoding the codes once.  More query rows than 16 G go in further passes over
// the run's tiles by the same threads, so that every position is added to in a
// fixed order.
template <int G>
struct WeighQ4Cfg {
    static constexpr int kWarps = G == 4 ? 8 : 4;          // G = 4: one CTA per SM, so more warps in it
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kPages = kWarps / 4;              // pages of a tile
    static constexpr int kTile = 64 * kPages;
    static constexpr int kStages = 2;
    static constexpr int kStageBytes = kPages * Q4Cfg::kStageBytes;
    static constexpr int kOffQ = 0;
    static constexpr int kOffStage = 36 * G * 512;
    static constexpr int kOffRow = kOffStage + kStages * kStageBytes;  // float2 lse [16 G], int lim [16 G]
    static constexpr int kOffScratch = kOffRow + 16 * G * 12;          // int [48]
    static constexpr int kOffBar = kOffScratch + 192;
    static constexpr int kSmemBytes = kOffBar + 8 * kStages;
    static constexpr int kMinBlocks = G == 1 ? 3 : G == 2 ? 2 : 1;     // per SM
    static_assert(kMinBlocks * (kSmemBytes + 1024) <= 233472, "shared memory per SM");
};

template <int G>
__global__ void __launch_bounds__(WeighQ4Cfg<G>::kThreads, WeighQ4Cfg<G>::kMinBlocks)
    smla_weigh_q4_kernel(const WeighParams a) {
    using C = WeighQ4Cfg<G>;
    const PartialParams &p = a.p;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x, c = lane & 3, r = lane >> 2;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    float2 *lse_s = reinterpret_cast<float2 *>(smem + C::kOffRow);
    int *lim_s = reinterpret_cast<int *>(lse_s + 16 * G);
    const uint32_t sbase = smem_addr(smem);
    bool dead = false;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], C::kPages);
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Q4Run run = q4_find_run<C::kTile>(p, p.B, a.grid, a.min_tiles, nullptr,
                                            reinterpret_cast<int *>(smem + C::kOffScratch));
    const int rows = p.dense_t * p.dense_h;
    int b = run.unit, tile0 = run.tile, it = 0;
    for (long long at = run.begin; at < run.end; ++b, tile0 = 0) {
        const int len = q4_unit_len(p, b, false);
        const int tiles = (int)min((long long)((len + C::kTile - 1) / C::kTile - tile0), run.end - at);
        if (tiles <= 0) continue;
        at += tiles;
        const int *pt_b = p.page_table + (size_t)b * p.pt_stride;
        float *acc = a.acc + (size_t)b * p.K;
        auto page_of = [&](int pg) { return pg * 64 < len ? q4_page(pt_b, p.pt_stride, p.num_pages, pg) : -1; };
        auto issue = [&](int i, int t) {  // thread 0: tile t of the sequence into ring position i
#pragma unroll
            for (int k = 0; k < C::kPages; ++k)
                q4_copy_page(p, page_of(C::kPages * t + k),
                             smem + C::kOffStage + (i & 1) * C::kStageBytes + k * Q4Cfg::kStageBytes, &full[i & 1]);
        };
        for (int g0 = 0; g0 < rows; g0 += 16 * G) {
            __syncthreads();  // the previous pass is done with the ring, Q and the row data
            if (tid == 0) {
                issue(it, tile0);
                if (tiles > 1) issue(it + 1, tile0 + 1);
            }
            q4_stage_q<G, C::kThreads>(smem + C::kOffQ, p.q, (long long)b * rows + g0, rows - g0);
            if (tid < 16 * G) weigh_row(a, b, g0 + tid, &lse_s[tid], &lim_s[tid]);
            __syncthreads();
            for (int t = 0; t < tiles; ++t, ++it) {
                // lane (r, c), r < 4, adds up column 2 c + (r & 1) of n8 tile r >> 1
                const int page = C::kPages * (tile0 + t) + (warp >> 2);
                const int pos0 = page * 64 + 16 * (warp & 3);
                const bool mapped = page_of(page) >= 0;
                const int pos = pos0 + 8 * (r >> 1) + q4_row_of(2 * c + (r & 1));
                const bool mine = r < 4 && mapped && pos < len;
                float old = 0.f;
                if (mine) asm volatile("ld.global.f32 %0, [%1];" : "=f"(old) : "l"(acc + pos));
                mbar_wait(&full[it & 1], (it >> 1) & 1, dead);
                float s[G][2][4];
                q4_scores<G>(sbase + C::kOffQ,
                             sbase + C::kOffStage + (it & 1) * C::kStageBytes + 16 * warp * kQ4RowBytes, lane, s);
                __syncthreads();  // every warp is done with the tile
                if (tid == 0 && t + 2 < tiles) issue(it + 2, tile0 + t + 2);
                if (!mapped) {
                    if (g0 == 0 && lane < min(len - pos0, 16)) count_bad_index();
                    continue;
                }
                float w[4] = {0.f, 0.f, 0.f, 0.f};  // column 2 c + e of n8 tile i at [2 i + e]
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 l2 = lse_s[16 * g + 8 * h + r];
                        const int lim = lim_s[16 * g + 8 * h + r] - pos0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float x = fmaf(s[g][k >> 1][2 * h + (k & 1)], p.scale_log2, -l2.x) - l2.y;
                            w[k] += 8 * (k >> 1) + q4_row_of(2 * c + (k & 1)) < lim ? fast_exp2(x) : 0.f;
                        }
                    }
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] += __shfl_xor_sync(0xffffffffu, w[k], o);
                const float v = r == 0 ? w[0] : r == 1 ? w[1] : r == 2 ? w[2] : w[3];
                if (mine) acc[pos] = old + v;
            }
        }
    }
}

// ---------------------------------------------------------------- bf16 rows
struct WeighOld {
    const __nv_bfloat16 *q;   // [B, T, H, 576]
    const uint8_t *cache;     // bf16 rows of 1152 bytes
    long long num_pages;
    const int *page_table;    // [B, pt_stride]
    int pt_stride;
    const int *seq_lens;      // [B, T]
    const float *lse;         // [B, T, H]
    int B, T, H;
    float scale_log2;
    float *acc;               // [B, max_n]
    int max_n;
    int nchunk;               // CTAs per sequence
};

constexpr int kWeighWarps = 8;
constexpr int kWeighTile = 32;  // cache rows per warp and step

template <int HG>
struct WeighCfg {
    static constexpr int kRows = 16 * HG;  // query rows per pass
    static constexpr int kOffFrag = 0;     // uint4 [36][HG][32]: A fragments in lane order
    static constexpr int kOffLse = 36 * HG * 512;       // float2 [kRows]: lse in log2 units, high and low part
    static constexpr int kOffLim = kOffLse + kRows * 8;  // int [kRows]: visible positions
    static constexpr int kSmemBytes = kOffLim + kRows * 4;
};

// First of the four dims that lane column c feeds to k16 step s (dims +0, +1
// go to k = 2 c, 2 c + 1 and dims +2, +3 to k = 2 c + 8, 2 c + 9).  The sum
// over k does not care for the order of the dims, so each lane takes dims it
// can load as 16 consecutive bytes: 8 bf16 values (two steps) or one whole
// group of 32 codes (eight steps, one scale).
__device__ __forceinline__ int weigh_dim(int s, int c) { return 32 * (s >> 1) + 8 * c + 4 * (s & 1); }

// One warp: the scores of 32 cache rows (half a page, consecutive rows)
// against 16 HG query rows by mma.sync, the cache rows (N) straight from
// global memory into B fragments, the query rows (M) from shared memory.
template <int HG>
__device__ __forceinline__ void weigh_scores(const uint8_t *row0, const uint4 *frag, int lane,
                                             float (&s)[HG][4][4]) {
    const int c = lane & 3;
    constexpr int kRow = kRowBytes;
    const uint8_t *mine = row0 + (lane >> 2) * kRow;
#pragma unroll
    for (int g = 0; g < HG; ++g)
#pragma unroll
        for (int n = 0; n < 4; ++n) s[g][n][0] = s[g][n][1] = s[g][n][2] = s[g][n][3] = 0.f;
    auto step = [&](int st, const uint32_t (&b0)[4], const uint32_t (&b1)[4]) {
#pragma unroll
        for (int g = 0; g < HG; ++g) {
            const uint4 a = frag[(st * HG + g) * 32 + lane];
#pragma unroll
            for (int n = 0; n < 4; ++n) mma_bf16_16816(s[g][n], a.x, a.y, a.z, a.w, b0[n], b1[n]);
        }
    };
    auto chunk = [&](int st, const uint4 (&v)[4]) {  // 8 bf16 values per lane: two k16 steps
        const uint32_t x[4] = {v[0].x, v[1].x, v[2].x, v[3].x}, y[4] = {v[0].y, v[1].y, v[2].y, v[3].y};
        const uint32_t z[4] = {v[0].z, v[1].z, v[2].z, v[3].z}, w[4] = {v[0].w, v[1].w, v[2].w, v[3].w};
        step(st, x, y);
        step(st + 1, z, w);
    };
    {
#pragma unroll 1
        for (int j = 0; j < 18; j += 3) {
            uint4 v[3][4];
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int n = 0; n < 4; ++n) v[k][n] = ld_row16(mine + n * 8 * kRow + 64 * (j + k) + 16 * c);
#pragma unroll
            for (int k = 0; k < 3; ++k) chunk(2 * (j + k), v[k]);
        }
    }
}

template <int HG>
__global__ void __launch_bounds__(32 * kWeighWarps) smla_evict_weigh_kernel(const WeighOld p) {
    using C = WeighCfg<HG>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint4 *frag = reinterpret_cast<uint4 *>(smem + C::kOffFrag);
    float2 *lse_s = reinterpret_cast<float2 *>(smem + C::kOffLse);
    int *lim_s = reinterpret_cast<int *>(smem + C::kOffLim);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3;
    const int b = blockIdx.x / p.nchunk, part = blockIdx.x % p.nchunk;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    int len = 0;  // longest visible length of the sequence's query tokens
    for (int t = 0; t < p.T; ++t) {
        const int raw = ld_input(p.seq_lens + (size_t)b * p.T + t);
        len = max(len, min(max(raw, 0), p.max_n));
        if (part == 0 && threadIdx.x == t % blockDim.x && (raw < 0 || raw > p.max_n)) count_bad_index();
    }
    const int tiles = (len + kWeighTile - 1) / kWeighTile;
    const int *pt_b = p.page_table + (size_t)b * p.pt_stride;
    const int rows = p.T * p.H;
    constexpr int kRow = kRowBytes;

    for (int g0 = 0; g0 < rows; g0 += C::kRows) {
        __syncthreads();
        for (int i = threadIdx.x; i < 36 * HG * 32; i += blockDim.x) {
            const int l = i & 31, g = (i >> 5) % HG, st = i / (32 * HG);
            const int r = g0 + 16 * g + (l >> 2), d = weigh_dim(st, l & 3);
            const __nv_bfloat16 *q = p.q + ((size_t)b * rows + r) * kD + d;
            uint2 lo = make_uint2(0u, 0u), hi = lo;
            if (r < rows) lo = *reinterpret_cast<const uint2 *>(q);
            if (r + 8 < rows) hi = *reinterpret_cast<const uint2 *>(q + 8 * kD);
            frag[i] = make_uint4(lo.x, hi.x, lo.y, hi.y);
        }
        for (int i = threadIdx.x; i < C::kRows; i += blockDim.x) {
            const int r = g0 + i;
            float2 l2 = make_float2(0.f, 0.f);
            int lim = 0;
            if (r < rows) {
                const float l = p.lse[(size_t)b * rows + r];
                // lse in log2 units as a sum of two floats: its rounding would
                // otherwise scale every weight of the row
                const double x = (double)l * 1.4426950408889634074;
                l2.x = (float)x;
                l2.y = isfinite(l2.x) ? (float)(x - (double)l2.x) : 0.f;
                // a row that attended to nothing (lse = -inf) gives no weight
                lim = l == -INFINITY ? 0 : min(max(ld_input(p.seq_lens + (size_t)b * p.T + r / p.H), 0), p.max_n);
            }
            lse_s[i] = l2;
            lim_s[i] = lim;
        }
        __syncthreads();
        for (int tile = part * kWeighWarps + warp; tile < tiles; tile += p.nchunk * kWeighWarps) {
            const int pos0 = tile * kWeighTile;
            const long long row = paged_row(pt_b, p.pt_stride, p.num_pages, pos0);
            if (row < 0) {
                if (g0 == 0 && lane < min(kWeighTile, len - pos0)) count_bad_index();
                continue;
            }
            float s[HG][4][4];
            weigh_scores<HG>(p.cache + row * kRow, frag, lane, s);
            float w[8];  // column 8 n + 2 c + e at [2 n + e]
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = 0.f;
#pragma unroll
            for (int g = 0; g < HG; ++g) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = 16 * g + 8 * h + (lane >> 2);
                    const float2 l2 = lse_s[r];
                    const int lim = lim_s[r] - pos0 - 2 * c;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float x = fmaf(s[g][k >> 1][2 * h + (k & 1)], p.scale_log2, -l2.x) - l2.y;
                        w[k] += 8 * (k >> 1) + (k & 1) < lim ? fast_exp2(x) : 0.f;
                    }
                }
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] += __shfl_xor_sync(0xffffffffu, w[k], o);
            float v = w[0];
#pragma unroll
            for (int k = 1; k < 8; ++k) v = (lane >> 2) == k ? w[k] : v;
            const int pos = pos0 + 8 * (lane >> 3) + 2 * c + ((lane >> 2) & 1);
            if (pos < len) p.acc[(size_t)b * p.max_n + pos] += v;
        }
    }
}

}  // namespace smla

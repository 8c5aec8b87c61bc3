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
    PartialParams p;      // q, cache, pages; seq_lens [B, dense_t], K = max_n
    const float *lse;     // [B, T, H]
    float *acc;           // [B, max_n]
    int grid;             // CTAs that share the tiles
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

// ---------------------------------------------------------------- 4-bit rows, up to 16 query rows
// The dense decode's schedule and score product (smla_partial_q4.cuh): CTAs take
// equal runs of the batch's 64-position tiles, a page lands by one bulk copy,
// and each warp scores 16 of its rows against the 16 query rows.  Measured: 24
// sequences of 4635 to 64913 positions, 16 heads, 58 us on rows that are not in L2
// (4.0 TB/s; 36 us at the memory's rate), 51 us over and over on the same 236 MB, of
// which L2 keeps a part (70.9 by the kernel below).  Shared memory is 54% busy,
// issue slots 46%, the tensor pipe 34%, DRAM 51%: none is full.  Two pages per CTA
// are in flight, and the next is asked for behind a barrier of the whole CTA.
struct WeighQ4Cfg {
    static constexpr int kThreads = 128;
    static constexpr int kTile = 64;                       // one page
    static constexpr int kStages = 2;
    static constexpr int kStageBytes = Q4Cfg::kStageBytes;
    static constexpr int kOffQ = 0;
    static constexpr int kOffStage = 36 * 512;
    static constexpr int kOffRow = kOffStage + kStages * kStageBytes;  // float2 lse [16], int lim [16]
    static constexpr int kOffScratch = kOffRow + 16 * 12;          // int [48]
    static constexpr int kOffBar = kOffScratch + 192;
    static constexpr int kSmemBytes = kOffBar + 8 * kStages;
    static constexpr int kMinBlocks = 3;                   // per SM
    static_assert(kMinBlocks * (kSmemBytes + 1024) <= 233472, "shared memory per SM");
};

__global__ void __launch_bounds__(WeighQ4Cfg::kThreads, WeighQ4Cfg::kMinBlocks)
    smla_weigh_q4_kernel(const WeighParams a) {
    using C = WeighQ4Cfg;
    const PartialParams &p = a.p;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x, c = lane & 3, r = lane >> 2;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    float2 *lse_s = reinterpret_cast<float2 *>(smem + C::kOffRow);
    int *lim_s = reinterpret_cast<int *>(lse_s + 16);
    const uint32_t sbase = smem_addr(smem);
    bool dead = false;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Q4Run run = q4_find_run<C::kTile>(p, a.grid, 1, nullptr,
                                            reinterpret_cast<int *>(smem + C::kOffScratch));
    const int rows = p.dense_t * p.dense_h;
    int b = run.b, tile0 = run.tile, it = 0;
    for (long long at = run.begin; at < run.end && b < p.B; ++b, tile0 = 0) {
        const int len = at == run.begin ? run.len : q4_seq_len(p, b, false);
        const int tiles = (int)min((long long)((len + C::kTile - 1) / C::kTile - tile0), run.end - at);
        if (tiles <= 0) continue;
        at += tiles;
        const int *pt_b = p.page_table + (size_t)b * p.pt_stride;
        float *acc = a.acc + (size_t)b * p.K;
        auto page_of = [&](int t) { return q4_page(pt_b, p.pt_stride, p.num_pages, tile0 + t); };
        auto issue = [&](int i, int t) {  // thread 0: tile t of the run into ring position i
            q4_copy_page(p, page_of(t), smem + C::kOffStage + (i & 1) * C::kStageBytes, &full[i & 1]);
        };
        __syncthreads();  // the previous sequence is done with the ring, Q and the row data
        if (tid == 0) {
            issue(it, 0);
            if (tiles > 1) issue(it + 1, 1);
        }
        q4_stage_q<C::kThreads>(smem + C::kOffQ, p.q, (long long)b * rows, rows);
        if (tid < 16) weigh_row(a, b, tid, &lse_s[tid], &lim_s[tid]);
        __syncthreads();
        for (int t = 0; t < tiles; ++t, ++it) {
            // lane (r, c), r < 4, adds up column 2 c + (r & 1) of n8 tile r >> 1
            const int pos0 = (tile0 + t) * 64 + 16 * warp;
            const bool mapped = page_of(t) >= 0;
            const int pos = pos0 + 8 * (r >> 1) + q4_row_of(2 * c + (r & 1));
            const bool mine = r < 4 && mapped && pos < len;
            float old = 0.f;
            if (mine) asm volatile("ld.global.f32 %0, [%1];" : "=f"(old) : "l"(acc + pos));
            mbar_wait(&full[it & 1], (it >> 1) & 1, dead);
            float s[2][4];
            q4_scores(sbase + C::kOffQ,
                      sbase + C::kOffStage + (it & 1) * C::kStageBytes + 16 * warp * kQ4RowBytes, lane, s);
            __syncthreads();  // every warp is done with the tile
            if (tid == 0 && t + 2 < tiles) issue(it + 2, t + 2);
            if (!mapped) {
                if (lane < min(len - pos0, 16)) count_bad_index();
                continue;
            }
            float w[4] = {0.f, 0.f, 0.f, 0.f};  // column 2 c + e of n8 tile i at [2 i + e]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 l2 = lse_s[8 * h + r];
                const int lim = lim_s[8 * h + r] - pos0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x = fmaf(s[k >> 1][2 * h + (k & 1)], p.scale_log2, -l2.x) - l2.y;
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

// ---------------------------------------------------------------- bf16 rows, or more query rows
// 1152 bytes a row leave the tensor core about 50 cycles per row and SM, so the
// rows go through tcgen05 with up to 128 query rows at once, the indexer's way:
// the CACHE ROWS are M = 128 (two pages), the query rows N, and the accumulator
// holds one position per TMEM lane: the epilogue thread that owns a position adds
// up its columns alone.  A CTA (one per SM) takes an equal run of the batch's
// pages.  More query rows than 128 go in further passes over the run.
//   bf16 rows  boxes of 128 rows x 64 values by TMA (128B swizzle), A in shared
//              memory.
//   4-bit rows pages by bulk copies; the lane that owns a row decodes it into
//              TMEM, where it is the A operand: no decoded row passes through
//              shared memory.
// The MMA issuer takes three boxes of 64 values at a time: a wait, twelve MMAs, a
// commit.  Each such turn costs some 390 cycles beside its MMAs (about 60 each with
// A in TMEM), and one per box took 31 us where this took 22 (4-bit rows, 37
// sequences of 4096 positions).
// Warp 0 rows in, warp 1 TMEM owner and MMA issuer, warps 4-7 epilogue; 4-bit
// rows: warp 2 queries in, warps 8-15 decode.
// Measured: 72 query rows over 46089 positions, bf16 17.0 us on rows that are not in
// L2, 15.4 over and over on the same (8.2 us at the memory's rate, 43 us by mma.sync): 2.4 steps of 128 rows a CTA, so launch,
// queries and the first boxes are half of it; 4-bit 13.8 us (mma.sync in three
// passes 30.8).  37 sequences of 4096 positions, 4-bit rows: 24 query rows 23.4
// us, 64 24.7, 72 26.2 (mma.sync with 32, 64, 32 rows a pass: 23.0, 37.2, 63.3);
// bf16 rows: 16 to 64 query rows 30 us, 96 33.5 (27 us at the memory's rate), 128
// 50, where the queries leave the ring four boxes.
template <bool Q4>
struct WeighCfg {
    static constexpr int kThreads = Q4 ? 512 : 256;
    static constexpr int kMaxRows = 128;                  // query rows per pass (the MMA's N)
    // the ring: boxes of 128 cache rows x 64 values, or pages of 4-bit rows
    static constexpr int kStageBytes = Q4 ? 64 * kQ4RowBytes : 2 * 64 * 128;
    static constexpr int kMaxStages = Q4 ? 7 : 12;
    static constexpr int kChunks = 2;                     // Q4: decoded chunks in TMEM, of
    static constexpr int kChunkBoxes = 3;                 // three boxes (64 values: 32 columns) each
    static constexpr int kChunkCols = 32 * kChunkBoxes;
    // A score is added up in parts, of every second or third chunk each, which the
    // epilogue adds: the tensor core cuts partial sums towards zero, and 36 cuts in
    // one chain left weights 1.7e-6 off (bf16 rows; 0.5e-6 in three parts, where
    // plain fp32 sums are 0.2e-6 off; 4-bit rows 0.7e-6 in one, 0.4e-6 in two).  A
    // part is npad columns; steps alternate between two sets of parts where they fit.
    static constexpr int kTmemCols = 512;
    static constexpr int kChunkCol = kTmemCols - (Q4 ? kChunks * kChunkCols : 0);
    static constexpr int kMaxParts = Q4 ? 2 : 3;
    __host__ __device__ static constexpr int parts(int npad) { return 2 * kMaxParts * npad <= kChunkCol ? kMaxParts : 2; }
    __host__ __device__ static constexpr int sets(int npad) { return 2 * parts(npad) * npad <= kChunkCol ? 2 : 1; }
    // full[], empty[], q_full, q_empty, acc_full[2], acc_empty[2], chunk_full[], chunk_free[]
    static constexpr int kNumBars = 2 * kMaxStages + 6 + (Q4 ? 2 * kChunks : 0);
    static constexpr int kOffRow = 0;                     // float4 [kMaxRows]: lse (two parts), visible positions
    static constexpr int kOffBar = kOffRow + 16 * kMaxRows;
    static constexpr int kOffTmem = kOffBar + 8 * kNumBars;
    static constexpr int kOffScratch = kOffTmem + 16;     // int [48]
    static constexpr int kOffQ = (kOffScratch + 192 + 1023) / 1024 * 1024;  // [9][npad rows x 128 B], then the ring
    static constexpr int kSmemBytes = 232448;
    __host__ __device__ static constexpr int stages(int npad) {
        const int n = (kSmemBytes - 1024 - kOffQ - npad * kRowBytes) / kStageBytes;
        return n < kMaxStages ? n : kMaxStages;
    }
};
static_assert(WeighCfg<false>::stages(128) >= 4, "ring of boxes");
static_assert(WeighCfg<true>::stages(128) >= 3, "ring of pages");
static_assert(WeighCfg<false>::sets(128) == 2 && WeighCfg<true>::parts(128) * 128 <= WeighCfg<true>::kChunkCol,
              "parts of a score");

template <bool Q4>
__global__ void __launch_bounds__(WeighCfg<Q4>::kThreads, 1)
    smla_weigh_kernel(const __grid_constant__ CUtensorMap map_kv, const __grid_constant__ CUtensorMap map_q,
                      const WeighParams a) {
    using C = WeighCfg<Q4>;
    const PartialParams &p = a.p;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = p.dense_t * p.dense_h;
    const int npad = min((rows + 15) / 16 * 16, C::kMaxRows);
    const int nst = C::stages(npad), nset = C::sets(npad), parts = C::parts(npad);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar), *empty = full + C::kMaxStages;
    uint64_t *q_full = empty + C::kMaxStages, *q_empty = q_full + 1;
    uint64_t *acc_full = q_empty + 1, *acc_empty = acc_full + 2;
    uint64_t *chunk_full = acc_empty + 2, *chunk_free = chunk_full + C::kChunks;  // Q4
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffTmem);
    const uint32_t sbase = smem_addr(smem);
    const uint32_t q_addr = sbase + C::kOffQ, ring = q_addr + npad * kRowBytes;
    bool dead = false;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kMaxStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], Q4 ? 4 : 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 128);
        }
        if constexpr (Q4) {
            for (int i = 0; i < C::kChunks; ++i) {
                mbar_init(&chunk_full[i], 4);
                mbar_init(&chunk_free[i], 1);
            }
        }
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    const Q4Run run = q4_find_run<64>(p, a.grid, 2, nullptr, reinterpret_cast<int *>(smem + C::kOffScratch));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);

    // (A thread whose wait gave up goes on without waiting: one that left would
    // keep the others at their barriers.)
    // Every role walks the same pieces (a run of one sequence's pages), passes
    // (of kMaxRows query rows) and steps (of two pages).
    auto walk = [&](auto &&body) {
        int b = run.b, page0 = run.tile;
        for (long long at = run.begin; at < run.end && b < p.B; ++b, page0 = 0) {
            const int len = at == run.begin ? run.len : q4_seq_len(p, b, false);
            const int pages = (int)min((long long)((len + 63) / 64 - page0), run.end - at);
            if (pages <= 0) continue;
            at += pages;
            for (int g0 = 0; g0 < rows; g0 += C::kMaxRows) body(b, len, page0, pages, g0);
        }
    };

    // a pass's queries: nine boxes of npad rows x 64 values
    auto load_q = [&](int b, int g0, int &pass) {
        if (pass > 0) mbar_wait(q_empty, (pass - 1) & 1, dead);
        ++pass;
        mbar_arrive_expect_tx(q_full, (uint32_t)(npad * kRowBytes));
        const uint64_t keep = l2_policy_evict_last();
#pragma unroll 1
        for (int k = 0; k < 9; ++k) tma_load_2d(q_addr + k * npad * 128, &map_q, 64 * k, b * rows + g0, q_full, keep);
    };

    if (warp == 0) {
        // ============================================================ rows in
        if (lane == 0) {
            const uint64_t once = l2_policy_evict_first();
            int st = 0, round = 0, pass = 0;
            walk([&](int b, int len, int page0, int pages, int g0) {
                const int *pt_b = p.page_table + (size_t)b * p.pt_stride;
                if constexpr (Q4) {
                    for (int t = 0; t < pages && !dead; ++t) {
                        const int pg = q4_page(pt_b, p.pt_stride, p.num_pages, page0 + t);
                        if (round > 0) mbar_wait(&empty[st], (round - 1) & 1, dead);
                        q4_copy_page(p, pg, smem + (ring - sbase) + st * C::kStageBytes, &full[st]);
                        if (++st == nst) {
                            st = 0;
                            ++round;
                        }
                    }
                    return;
                }
                load_q(b, g0, pass);
                for (int t = 0; t < pages; t += 2) {
                    const int pg0 = q4_page(pt_b, p.pt_stride, p.num_pages, page0 + t);
                    const int pg1 = t + 1 < pages ? q4_page(pt_b, p.pt_stride, p.num_pages, page0 + t + 1) : -1;
                    const uint32_t bytes = (pg0 >= 0 ? 8192u : 0u) + (pg1 >= 0 ? 8192u : 0u);
#pragma unroll 1
                    for (int k = 0; k < 9; ++k) {
                        if (round > 0) mbar_wait(&empty[st], (round - 1) & 1, dead);
                        mbar_arrive_expect_tx(&full[st], bytes);
                        const uint32_t dst = ring + st * C::kStageBytes;
                        if (pg0 >= 0) tma_load_2d(dst, &map_kv, 64 * k, pg0 * 64, &full[st], once);
                        if (pg1 >= 0) tma_load_2d(dst + 8192, &map_kv, 64 * k, pg1 * 64, &full[st], once);
                        if (++st == nst) {
                            st = 0;
                            ++round;
                        }
                    }
                }
            });
        }
        __syncwarp();
    } else if (Q4 && warp == 2) {
        // ============================================================ queries in
        if (lane == 0) {
            int pass = 0;
            walk([&](int b, int, int, int, int g0) { load_q(b, g0, pass); });
        }
        __syncwarp();
    } else if (Q4 && warp >= 8) {
        // ============================================================ codes -> TMEM
        // Lane = cache row; warps 8, 9 and 12, 13 take a step's first page, the others
        // its second; warps 8-11 and 12-15 take turns at the chunks.
        // (A row that nobody sees, or that no page maps, is garbage in its own
        // lane alone.)
        const int w = warp & 3, half = w >> 1, turn = (warp - 8) >> 2;
        int idx = 0, c = 0;  // pages and chunks so far
        walk([&](int, int, int, int pages, int) {
            for (int t = 0; t < pages; t += 2) {
                const int page = idx + t + half, st = page % nst;
                const bool has = t + half < pages;
                if (has) mbar_wait(&full[st], (page / nst) & 1, dead);
                const uint32_t row = ring + st * C::kStageBytes + (32 * (w & 1) + lane) * kQ4RowBytes;
                uint32_t sc[8];
                if (has) {
                    const uint4 x = lds_16(row + kQ4OffScale), y = lds_16(row + kQ4OffScale + 16);
                    sc[0] = x.x, sc[1] = x.y, sc[2] = x.z, sc[3] = x.w;
                    sc[4] = y.x, sc[5] = y.y, sc[6] = y.z, sc[7] = y.w;
                }
#pragma unroll
                for (int j = 0; j < 9 / C::kChunkBoxes; ++j, ++c) {
                    if ((c & 1) != turn) continue;
                    if (c >= C::kChunks) mbar_wait(&chunk_free[turn], (c / C::kChunks - 1) & 1, dead);
                    tc_fence_after();
                    if (has) {
#pragma unroll
                        for (int k = C::kChunkBoxes * j; k < C::kChunkBoxes * (j + 1); ++k) {
                            uint32_t v[32];
                            if (k < 8) {
                                const uint4 a0 = lds_16(row + 32 * k), a1 = lds_16(row + 32 * k + 16);
                                const uint32_t word[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
                                for (int g = 0; g < 8; ++g) {
                                    const uint32_t s2 = __byte_perm(sc[k & 7], 0u, g < 4 ? 0x1010 : 0x3232);
                                    const uint4 x = q4_word(word[g], s2, q4_bias(s2));
                                    v[4 * g] = x.x, v[4 * g + 1] = x.y, v[4 * g + 2] = x.z, v[4 * g + 3] = x.w;
                                }
                            } else {
#pragma unroll
                                for (int g = 0; g < 8; ++g) {
                                    const uint4 x = lds_16(row + kQ4OffRope + 16 * g);
                                    v[4 * g] = x.x, v[4 * g + 1] = x.y, v[4 * g + 2] = x.z, v[4 * g + 3] = x.w;
                                }
                            }
                            tmem_st32(tmem + ((uint32_t)(32 * w) << 16) + C::kChunkCol + C::kChunkCols * turn +
                                          32 * (k % C::kChunkBoxes), v);
                        }
                        tmem_st_wait();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&chunk_full[turn]);
                }
                __syncwarp();
                if (has && lane == 0) mbar_arrive(&empty[st]);
            }
            idx += pages;
        });
        tc_fence_before();
    } else if (warp == 1) {
        // ============================================================ MMA issuer
        if (lane == 0) {
            const uint32_t idesc = idesc_bf16_f32(128, npad, false, false);
            const int n = Q4 ? C::kChunks : nst;
            uint64_t *in = Q4 ? chunk_full : full, *out = Q4 ? chunk_free : empty;
            int st = 0, round = 0, pass = 0, step = 0;
            walk([&](int, int, int, int pages, int) {
                mbar_wait(q_full, pass & 1, dead);
                ++pass;
                for (int t = 0; t < pages; t += 2, ++step) {
                    const int acc = step % nset;
                    if (step >= nset) mbar_wait(&acc_empty[acc], (step / nset - 1) & 1, dead);
                    tc_fence_after();
#pragma unroll 1
                    for (int k0 = 0; k0 < 9; k0 += C::kChunkBoxes) {
                        int box_st[C::kChunkBoxes];  // bf16: where the boxes are
#pragma unroll
                        for (int k = 0; k < (Q4 ? 1 : C::kChunkBoxes); ++k) {
                            mbar_wait(&in[st], round & 1, dead);
                            box_st[k] = st;
                            if (++st == n) {
                                st = 0;
                                ++round;
                            }
                        }
                        tc_fence_after();
                        const uint32_t d = tmem + (acc * parts + k0 / C::kChunkBoxes % parts) * npad;
                        const bool first = k0 < parts * C::kChunkBoxes;
#pragma unroll
                        for (int k = 0; k < C::kChunkBoxes; ++k) {
                            const uint64_t bd = smem_desc(q_addr + (k0 + k) * npad * 128, 16, 1024, kSwizzle128B);
                            const uint64_t ad = Q4 ? 0 : smem_desc(ring + box_st[k] * C::kStageBytes, 16, 1024, kSwizzle128B);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                const uint32_t add = first && (k | kk) == 0 ? 0u : 1u;
                                if constexpr (Q4)
                                    umma_bf16_ts(d, tmem + C::kChunkCol + C::kChunkCols * box_st[0] + 32 * k + 8 * kk, bd + 2 * kk,
                                                 idesc, add);
                                else
                                    umma_bf16(d, ad + 2 * kk, bd + 2 * kk, idesc, add);
                            }
                        }
#pragma unroll
                        for (int k = 0; k < (Q4 ? 1 : C::kChunkBoxes); ++k) umma_commit(&out[box_st[k]]);
                    }
                    umma_commit(&acc_full[acc]);
                }
                umma_commit(q_empty);
            });
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ============================================================ epilogue
        const int row = threadIdx.x - 128;  // TMEM lane: cache row of the step's two pages
        const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        float4 *row_s = reinterpret_cast<float4 *>(smem + C::kOffRow);
        int step = 0;
        walk([&](int b, int len, int page0, int pages, int g0) {
            named_bar_sync(1, 128);  // the previous pass is done with row_s
            {
                float2 l2;
                int lim;
                weigh_row(a, b, g0 + row, &l2, &lim);
                row_s[row] = make_float4(l2.x, l2.y, __int_as_float(lim), 0.f);
            }
            named_bar_sync(1, 128);
            const int *pt_b = p.page_table + (size_t)b * p.pt_stride;
            float *acc_b = a.acc + (size_t)b * p.K;
            for (int t = 0; t < pages; t += 2, ++step) {
                const int page = page0 + t + (row >> 6), pos = page * 64 + (row & 63);
                const bool mine = page < page0 + pages && pos < len;
                const bool mapped = mine && q4_page(pt_b, p.pt_stride, p.num_pages, page) >= 0;
                if (mine && !mapped && g0 == 0) count_bad_index();
                float old = 0.f;
                if (mapped) asm volatile("ld.global.f32 %0, [%1];" : "=f"(old) : "l"(acc_b + pos));
                mbar_wait(&acc_full[step % nset], (step / nset) & 1, dead);
                tc_fence_after();
                float w = 0.f;
#pragma unroll 1
                for (int n = 0; n < npad; n += 16) {
                    uint32_t s[C::kMaxParts][16];
#pragma unroll
                    for (int j = 0; j < C::kMaxParts; ++j)  // (a third part that is none: the second again)
                        tmem_ld_cols<16>(t_lane + (step % nset * parts + min(j, parts - 1)) * npad + n, s[j]);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float4 q = row_s[n + k];
                        float sum = __uint_as_float(s[0][k]) + __uint_as_float(s[1][k]);
                        if (C::kMaxParts == 3) sum = parts == 3 ? sum + __uint_as_float(s[C::kMaxParts - 1][k]) : sum;
                        const float x = fmaf(sum, p.scale_log2, -q.x) - q.y;
                        w += pos < __float_as_int(q.z) ? fast_exp2(x) : 0.f;
                    }
                }
                tc_fence_before();
                mbar_arrive(&acc_empty[step % nset]);
                if (mapped) acc_b[pos] = old + w;
            }
        });
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

}  // namespace smla

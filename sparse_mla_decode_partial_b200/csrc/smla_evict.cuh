// smla_evict.cuh -- eviction from the paged cache by accumulated attention
// weight: the weight every cached position has received is accumulated from a
// decode's queries and lse, the positions that received least are chosen, and
// the rows that stay fill the holes they leave.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "smla_indexer.cuh"
#include "smla_q4.cuh"

namespace smla {

// ---------------------------------------------------------------- accumulate
// acc[b, i] += sum over the query rows (t, h) of sequence b with i visible of
//   exp(scale q[b,t,h] . row_i - lse[b,t,h]).
struct WeighParams {
    const __nv_bfloat16 *q;   // [B, T, H, 576]
    const uint8_t *cache;     // bf16 rows of 1152 bytes or 4-bit rows of 416
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
template <bool Q4>
__device__ __forceinline__ int weigh_dim(int s, int c) {
    if (Q4 && s < 32) return 32 * (4 * (s >> 3) + c) + 8 * ((s & 7) >> 1) + 4 * (s & 1);
    return 32 * (s >> 1) + 8 * c + 4 * (s & 1);
}

// One warp: the scores of 32 cache rows (half a page, consecutive rows)
// against 16 HG query rows by mma.sync, the cache rows (N) straight from
// global memory into B fragments, the query rows (M) from shared memory.
template <bool Q4, int HG>
__device__ __forceinline__ void weigh_scores(const uint8_t *row0, const uint4 *frag, int lane,
                                             float (&s)[HG][4][4]) {
    const int c = lane & 3;
    constexpr int kRow = Q4 ? kQ4RowBytes : kRowBytes;
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
    if constexpr (Q4) {
        uint4 code[4], next[4];
        uint32_t sc[4], next_sc[4];
        auto load = [&](int j, uint4 (&d)[4], uint32_t (&s2)[4]) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                d[n] = ld_row16(mine + n * 8 * kRow + 16 * (4 * j + c));
                s2[n] = ld_scale(mine + n * 8 * kRow + kQ4OffScale + 2 * (4 * j + c));
            }
        };
        load(0, code, sc);
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
            if (j < 3) {
                load(j + 1, next, next_sc);
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n) next[n] = ld_row16(mine + n * 8 * kRow + kQ4OffRope + 16 * c);
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint4 v[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint32_t word = w == 0 ? code[n].x : w == 1 ? code[n].y : w == 2 ? code[n].z : code[n].w;
                    const uint32_t s2 = q4_scale2(sc[n]);
                    v[n] = q4_word(word, s2, q4_bias(s2));
                }
                chunk(8 * j + 2 * w, v);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                code[n] = next[n];
                sc[n] = next_sc[n];
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) next[n] = ld_row16(mine + n * 8 * kRow + kQ4OffRope + 64 + 16 * c);
        chunk(32, code);
        chunk(34, next);
    } else {
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

template <bool Q4, int HG>
__global__ void __launch_bounds__(32 * kWeighWarps) smla_evict_weigh_kernel(const WeighParams p) {
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
    constexpr int kRow = Q4 ? kQ4RowBytes : kRowBytes;

    for (int g0 = 0; g0 < rows; g0 += C::kRows) {
        __syncthreads();
        for (int i = threadIdx.x; i < 36 * HG * 32; i += blockDim.x) {
            const int l = i & 31, g = (i >> 5) % HG, st = i / (32 * HG);
            const int r = g0 + 16 * g + (l >> 2), d = weigh_dim<Q4>(st, l & 3);
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
            weigh_scores<Q4, HG>(p.cache + row * kRow, frag, lane, s);
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

// ---------------------------------------------------------------- plan
// Per sequence of n slots: the min(n, K) slots that stay, and for each slot
// i < min(n, K) the slot its row comes from (itself, or, for the j-th slot
// there that leaves, the j-th slot at or behind min(n, K) that stays).
struct EvictPlanParams {
    const float *acc;    // [B, max_n]
    const int *pos;      // [B, max_n] or null (slot i holds position i)
    const int *n;        // [B]
    int B, max_n, K, n_sink, n_recent;
    int *movers;         // [B, max_n] scratch
    int *src;            // [B, K]
    int *n_new;          // [B]
    float *acc_new;      // [B, max_n] or null
    int *pos_new;        // [B, max_n] or null
    int per;             // slots of a CTA: a multiple of 32
    int cached;          // their keys fit in shared memory
};

constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 2048;
constexpr int kPlanMaxCluster = 8;
// a histogram and two of sums, scan scratch and exchanged counts, two bitmaps and word
// prefixes, then (cached) the keys
__host__ __device__ constexpr int plan_fixed_bytes(int per) {
    return 3 * kPlanBins * 4 + 512 + 3 * 4 * (per / 32);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Barrier of the cluster; orders shared and global memory among its threads.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of shared memory at `p`'s place in CTA `rank` of the cluster.
__device__ __forceinline__ unsigned ld_cluster(const void *p, uint32_t rank) {
    uint32_t a;
    unsigned v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void add_cluster(const void *p, unsigned v, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Order-preserving key of a weight: larger stays; NaN counts as -inf, -0 as +0.
__device__ __forceinline__ uint32_t evict_key(float a) { return a != a ? 0x007FFFFFu : ix_key(a); }
__device__ __forceinline__ float ld_weight(const float *p) {
    float a;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(a) : "l"(p));
    return a;
}

// One cluster of CTAs per sequence, each CTA a run of its slots: radix
// selection of the K-th largest key (digits of 11, 11 and 10 bits, counts
// summed in the first CTA), bitmaps of the slots above and at it, ties to the
// smaller slot, then ranks of holes and movers by prefix sums.  A handful of
// block and cluster barriers with little work between them: latency bounds it.
__global__ void __launch_bounds__(kPlanThreads) smla_evict_plan_kernel(const EvictPlanParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int words = p.per / 32;
    unsigned *hist = reinterpret_cast<unsigned *>(smem);
    unsigned *sum2 = hist + kPlanBins;                                 // the cluster's counts (first CTA)
    int *scratch = reinterpret_cast<int *>(smem + 3 * kPlanBins * 4);  // 33 ints
    int *dec = scratch + 40;   // 4 ints
    int *xch = scratch + 48;   // counts that the cluster exchanges
    uint32_t *keep = reinterpret_cast<uint32_t *>(scratch + 128);
    uint32_t *tie = keep + words;
    int *pre = reinterpret_cast<int *>(tie + words);
    uint32_t *keys = reinterpret_cast<uint32_t *>(pre + words);
    const uint32_t nc = cluster_size(), rank = cluster_rank();
    const int b = blockIdx.x / nc, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t base = (size_t)b * p.max_n;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int raw = ld_input(p.n + b);
    const int n = min(max(raw, 0), p.max_n);
    if (tid == 0 && rank == 0 && raw != n) count_bad_index();
    const int m = min(n, p.K);
    if (tid == 0 && rank == 0) p.n_new[b] = m;
    int *src = p.src + (size_t)b * p.K;
    const int lo = (int)rank * p.per, hi = min(n, lo + p.per);  // this CTA's slots
    const bool cut = n > p.K;                                  // the same in the whole cluster
    if (cut) {
        for (int i = tid; i < 3 * kPlanBins; i += kPlanThreads) hist[i] = 0u;
        // weights in, and the newest position
        int top = INT_MIN;
#pragma unroll 4
        for (int i = lo + tid; i < hi; i += kPlanThreads) {
            if (p.pos != nullptr) top = max(top, ld_input(p.pos + base + i));
            if (p.cached) keys[i - lo] = evict_key(ld_weight(p.acc + base + i));
        }
        long long end = n;
        if (p.pos != nullptr) {
            top = __reduce_max_sync(0xffffffffu, top);
            if (lane == 0) scratch[warp] = top;
            __syncthreads();
            if (warp == 0) {
                top = __reduce_max_sync(0xffffffffu, scratch[lane]);
                if (lane == 0) xch[0] = top;
            }
            cluster_sync();
            top = INT_MIN;
            for (uint32_t r = 0; r < nc; ++r) top = max(top, (int)ld_cluster(&xch[0], r));
            end = (long long)top + 1;
        }
        const long long recent = end - p.n_recent;
        auto safe = [&](int i) {
            const int pos = p.pos != nullptr ? ld_input(p.pos + base + i) : i;
            return pos < p.n_sink || (long long)pos >= recent;
        };
        auto key_of = [&](int i) {
            if (p.cached) return keys[i - lo];
            return safe(i) ? 0xFFFFFFFFu : evict_key(ld_weight(p.acc + base + i));
        };
        if (p.cached && (p.n_sink > 0 || p.n_recent > 0)) {
#pragma unroll 4
            for (int i = lo + tid; i < hi; i += kPlanThreads)
                if (safe(i)) keys[i - lo] = 0xFFFFFFFFu;
        }
        cluster_sync();  // the cleared sums too

        uint32_t prefix = 0;  // the K-th largest key, digit by digit
        int need = p.K;
#pragma unroll 1
        for (int digit = 0; digit < 3; ++digit) {
            const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
            const int bits = digit == 2 ? 10 : 11;
            for (int i = lo + tid; i < hi; i += kPlanThreads) {
                const uint32_t k = key_of(i);
                if (digit == 0 || (k >> (shift + bits)) == (prefix >> (shift + bits)))
                    atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
            }
            __syncthreads();
            // The first CTA sums the counts and finds the bucket.  Only bins
            // that hold something travel (a few dozen): every CTA reading every
            // other's histogram took 6 us a digit.  Sums alternate between two
            // arrays, so that the next digit's never meet these.
            unsigned *sum = sum2 + (digit & 1) * kPlanBins;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const unsigned v = hist[tid + k * kPlanThreads];
                if (v) {
                    hist[tid + k * kPlanThreads] = 0u;
                    add_cluster(&sum[tid + k * kPlanThreads], v, 0);
                }
            }
            cluster_sync();
            if (rank == 0) {
                // thread t holds bins 2047 - 2 t and 2046 - 2 t: counts from the top
                const unsigned h1 = sum[kPlanBins - 1 - 2 * tid], h0 = sum[kPlanBins - 2 - 2 * tid];
                sum2[((digit & 1) ^ 1) * kPlanBins + tid] = 0u;
                sum2[((digit & 1) ^ 1) * kPlanBins + tid + kPlanThreads] = 0u;
                int total;
                const int incl = ix_block_scan((int)(h1 + h0), scratch, &total);
                const int excl = incl - (int)(h1 + h0);
                if (excl < need && need <= incl) {
                    const bool first = excl + (int)h1 >= need;
                    dec[0] = kPlanBins - (first ? 1 : 2) - 2 * tid;
                    dec[1] = need - excl - (first ? 0 : (int)h1);
                }
            }
            cluster_sync();
            prefix |= ld_cluster(&dec[0], 0) << shift;
            need = (int)ld_cluster(&dec[1], 0);
        }

        // bitmaps: slots above the K-th key, slots equal to it
        const int nw = hi > lo ? (hi - lo + 31) / 32 : 0;
        int equal_here = 0;
        for (int w = warp; w < nw; w += kPlanThreads / 32) {
            const int i = lo + 32 * w + lane;
            const uint32_t k = i < hi ? key_of(i) : 0u;
            const uint32_t above = __ballot_sync(0xffffffffu, i < hi && k > prefix);
            const uint32_t equal = __ballot_sync(0xffffffffu, i < hi && k == prefix);
            if (lane == 0) {
                keep[w] = above;
                tie[w] = equal;
                equal_here += __popc(equal);
            }
        }
        if (lane == 0) scratch[warp] = equal_here;
        __syncthreads();
        if (warp == 0) {
            const int x = __reduce_add_sync(0xffffffffu, scratch[lane]);
            if (lane == 0) xch[1] = x;
        }
        cluster_sync();
        // the first `need` ties stay
        int carry = 0;
        for (uint32_t r = 0; r < rank; ++r) carry += (int)ld_cluster(&xch[1], r);
        for (int w0 = 0; w0 < nw; w0 += kPlanThreads) {
            const int w = w0 + tid;
            const uint32_t t = w < nw ? tie[w] : 0u;
            int total;
            const int incl = ix_block_scan(__popc(t), scratch, &total);
            const int before = carry + incl - __popc(t);
            if (w < nw) {
                uint32_t left = t, got = 0u;
                for (int k = before; k < need && left; ++k) {
                    got |= left & (0u - left);
                    left &= left - 1u;
                }
                keep[w] |= got;
            }
            carry += total;
        }
        __syncthreads();
        // movers (slots at or behind m that stay) and holes (slots before m
        // that leave): a slot run lies on both sides of m in one word at most
        auto below = [&](int w) {
            const int s0 = lo + 32 * w;
            return s0 + 32 <= m ? 0xffffffffu : s0 >= m ? 0u : (1u << (m - s0)) - 1u;
        };
        int mv_here = 0, hole_here = 0;
        for (int w = tid; w < nw; w += kPlanThreads) {
            mv_here += __popc(keep[w] & ~below(w));
            hole_here += __popc(~keep[w] & below(w));
        }
        mv_here = __reduce_add_sync(0xffffffffu, mv_here);
        hole_here = __reduce_add_sync(0xffffffffu, hole_here);
        if (tid == 0) xch[2] = xch[3] = 0;
        __syncthreads();
        if (lane == 0 && (mv_here | hole_here)) {
            atomicAdd(&xch[2], mv_here);
            atomicAdd(&xch[3], hole_here);
        }
        cluster_sync();
        int mv = 0, hole = 0;
        for (uint32_t r = 0; r < rank; ++r) {
            mv += (int)ld_cluster(&xch[2], r);
            hole += (int)ld_cluster(&xch[3], r);
        }
        for (int w0 = 0; w0 < nw; w0 += kPlanThreads) {
            const int w = w0 + tid;
            const uint32_t mvs = w < nw ? keep[w] & ~below(w) : 0u, holes = w < nw ? ~keep[w] & below(w) : 0u;
            int total;
            const int mine = __popc(mvs);
            const int at_mv = ix_block_scan(mine, scratch, &total) - mine;
            int x = mv + at_mv;
            for (uint32_t left = mvs; left; left &= left - 1u) p.movers[base + x++] = lo + 32 * w + __ffs(left) - 1;
            mv += total;
            const int gone = __popc(holes);
            const int at_hole = ix_block_scan(gone, scratch, &total) - gone;
            if (w < nw) pre[w] = hole + at_hole;
            hole += total;
        }
        cluster_sync();  // the movers' list and pre are complete; no CTA leaves while another reads its counts
    }
    // this CTA's slots, then its share of what lies behind n
    auto put = [&](int i, int s) {
        if (i < p.K) src[i] = s;
        if (i < p.max_n) {
            if (p.acc_new != nullptr) p.acc_new[base + i] = s < 0 ? 0.f : ld_weight(p.acc + base + s);
            if (p.pos_new != nullptr)
                p.pos_new[base + i] = s < 0 ? -1 : p.pos != nullptr ? ld_input(p.pos + base + s) : s;
        }
    };
#pragma unroll 4
    for (int i = lo + tid; i < hi; i += kPlanThreads) {
        int s = i < m ? i : -1;
        if (cut && i < m) {
            const uint32_t k = keep[(i - lo) >> 5];
            if (!((k >> ((i - lo) & 31)) & 1u)) {
                const uint32_t lower = (1u << ((i - lo) & 31)) - 1u;
                s = ld_input(p.movers + base + pre[(i - lo) >> 5] + __popc(~k & lower));
            }
        }
        put(i, s);
    }
    for (long long i = n + (long long)rank * kPlanThreads + tid; i < max(p.K, p.max_n); i += nc * kPlanThreads)
        put((int)i, -1);
}

// ---------------------------------------------------------------- apply
// Row src[b, i] of each buffer moves to slot i where src[b, i] != i.  Sources
// lie at or behind the number of slots that stay and destinations before it,
// so the moves are independent of one another.
constexpr int kEvictBuffers = 4;
struct EvictApplyParams {
    const int *src;          // [B, K]
    int B, K;
    const int *page_table;   // [B, pt_stride]
    int pt_stride;
    long long num_pages;
    uint8_t *buf[kEvictBuffers];
    int pieces[kEvictBuffers];  // 16-byte pieces of a row
    int n_buf;
    int total;                  // pieces of a row over all buffers
};
constexpr int kApplyWarps = 8;
constexpr int kApplyDepth = 8;  // pieces in flight per lane
constexpr int kApplySlots = 16; // list entries per warp

// One warp per kApplySlots list entries.  It lists the moves among them, then its lanes
// walk the moves' 16-byte pieces, all buffers in a row, eight loads in flight
// each before the first store.  Bound by memory.
__global__ void __launch_bounds__(32 * kApplyWarps) smla_evict_apply_kernel(const EvictApplyParams p) {
    __shared__ int from_s[kApplyWarps][kApplySlots], to_s[kApplyWarps][kApplySlots];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long per = (p.K + kApplySlots - 1) / kApplySlots;
    const long long unit = (long long)blockIdx.x * kApplyWarps + warp;
    if (unit >= per * p.B) return;
    const int b = (int)(unit / per), i = (int)(unit % per) * kApplySlots + lane;
    const int s = lane < kApplySlots && i < p.K ? ld_input(p.src + (size_t)b * p.K + i) : -1;
    long long from = -1, to = -1;  // rows of the pool: below 2^31
    if (s != -1 && s != i) {
        const int *pt_b = p.page_table + (size_t)b * p.pt_stride;
        from = paged_row(pt_b, p.pt_stride, p.num_pages, s);
        to = paged_row(pt_b, p.pt_stride, p.num_pages, i);
        if (from < 0 || to < 0) count_bad_index();
    }
    const uint32_t moves = __ballot_sync(0xffffffffu, from >= 0 && to >= 0);
    if ((moves >> lane) & 1u) {
        const int k = __popc(moves & ((1u << lane) - 1u));
        from_s[warp][k] = (int)from;
        to_s[warp][k] = (int)to;
    }
    __syncwarp();
    const int n = __popc(moves);
    int move = 0, piece = lane;
    while (piece >= p.total) {
        piece -= p.total;
        ++move;
    }
    while (__any_sync(0xffffffffu, move < n)) {
        uint4 v[kApplyDepth];
        uint8_t *dst[kApplyDepth];
#pragma unroll
        for (int k = 0; k < kApplyDepth; ++k) {
            dst[k] = nullptr;
            if (move < n) {
                int x = piece, q = 0;
                while (x >= p.pieces[q]) x -= p.pieces[q++];
                const size_t row = (size_t)p.pieces[q] * 16;
                dst[k] = p.buf[q] + to_s[warp][move] * row + 16 * x;
                v[k] = ld_row16(p.buf[q] + from_s[warp][move] * row + 16 * x);
                piece += 32;
                while (piece >= p.total) {
                    piece -= p.total;
                    ++move;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kApplyDepth; ++k)
            if (dst[k] != nullptr) *reinterpret_cast<uint4 *>(dst[k]) = v[k];
    }
}

}  // namespace smla

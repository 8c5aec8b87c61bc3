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
                s2[n] = ld_scale2(mine + n * 8 * kRow + kQ4OffScale + 2 * (4 * j + c));
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
                    v[n] = q4_word(word, sc[n], q4_bias(sc[n]));
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
    int cached;          // keys fit in shared memory
};

constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 2048;
__host__ __device__ constexpr int plan_words(int max_n) { return (max_n + 31) / 32; }
// histogram, scan scratch, two bitmaps and word prefixes, then the keys
__host__ __device__ constexpr int plan_fixed_bytes(int max_n) {
    return kPlanBins * 4 + 256 + 3 * 4 * plan_words(max_n);
}

// Key of a slot: larger stays.  Protected slots above every weight; NaN counts
// as -inf; -0 equals +0.
__device__ __forceinline__ uint32_t evict_key(const EvictPlanParams &p, size_t base, int i, long long recent) {
    const int pos = p.pos != nullptr ? ld_input(p.pos + base + i) : i;
    if (pos < p.n_sink || (long long)pos >= recent) return 0xFFFFFFFFu;
    float a;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(a) : "l"(p.acc + base + i));
    return a != a ? 0x007FFFFFu : ix_key(a);
}

// One CTA per sequence: radix selection of the K-th largest key (digits of 11,
// 11 and 10 bits), bitmaps of the slots above and at it, ties to the smaller
// slot, then ranks of holes and movers by prefix sums over the bitmaps' words.
__global__ void __launch_bounds__(kPlanThreads) smla_evict_plan_kernel(const EvictPlanParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int words = plan_words(p.max_n);
    unsigned *hist = reinterpret_cast<unsigned *>(smem);
    int *scratch = reinterpret_cast<int *>(smem + kPlanBins * 4);  // 33 ints, then dec[4] at 40
    int *dec = scratch + 40;
    uint32_t *keep = reinterpret_cast<uint32_t *>(scratch + 64);
    uint32_t *tie = keep + words;
    int *pre = reinterpret_cast<int *>(tie + words);
    uint32_t *keys = reinterpret_cast<uint32_t *>(pre + words);
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t base = (size_t)b * p.max_n;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int raw = ld_input(p.n + b);
    const int n = min(max(raw, 0), p.max_n);
    if (tid == 0 && raw != n) count_bad_index();
    const int m = min(n, p.K);
    if (tid == 0) p.n_new[b] = m;
    int *src = p.src + (size_t)b * p.K;
    if (n > p.K) {
        long long end = n;
        if (p.pos != nullptr) {
            int top = INT_MIN;
            for (int i = tid; i < n; i += kPlanThreads) top = max(top, ld_input(p.pos + base + i));
            top = __reduce_max_sync(0xffffffffu, top);
            if (lane == 0) scratch[warp] = top;
            __syncthreads();
            top = scratch[lane];
            end = (long long)__reduce_max_sync(0xffffffffu, top) + 1;
            __syncthreads();
        }
        const long long recent = end - p.n_recent;
        if (p.cached)
            for (int i = tid; i < n; i += kPlanThreads) keys[i] = evict_key(p, base, i, recent);
        auto key_of = [&](int i) { return p.cached ? keys[i] : evict_key(p, base, i, recent); };

        uint32_t prefix = 0;  // the K-th largest key, digit by digit
        int need = p.K;
        for (int digit = 0; digit < 3; ++digit) {
            const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
            const int bits = digit == 2 ? 10 : 11;
            for (int i = tid; i < kPlanBins; i += kPlanThreads) hist[i] = 0u;
            __syncthreads();
            for (int i = tid; i < n; i += kPlanThreads) {
                const uint32_t k = key_of(i);
                if (digit == 0 || (k >> (shift + bits)) == (prefix >> (shift + bits)))
                    atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
            }
            __syncthreads();
            // thread t holds bins 2047 - 2 t and 2046 - 2 t: counts from the top
            const unsigned h1 = hist[kPlanBins - 1 - 2 * tid], h0 = hist[kPlanBins - 2 - 2 * tid];
            int total;
            const int incl = ix_block_scan((int)(h1 + h0), scratch, &total);
            const int excl = incl - (int)(h1 + h0);
            if (excl < need && need <= incl) {
                const bool first = excl + (int)h1 >= need;
                dec[0] = kPlanBins - (first ? 1 : 2) - 2 * tid;
                dec[1] = need - excl - (first ? 0 : (int)h1);
            }
            __syncthreads();
            prefix |= (uint32_t)dec[0] << shift;
            need = dec[1];
            __syncthreads();
        }

        // bitmaps: slots above the K-th key, slots equal to it
        const int nw = (n + 31) / 32;
        for (int w = warp; w < nw; w += kPlanThreads / 32) {
            const int i = 32 * w + lane;
            const uint32_t k = i < n ? key_of(i) : 0u;
            const uint32_t above = __ballot_sync(0xffffffffu, i < n && k > prefix);
            const uint32_t equal = __ballot_sync(0xffffffffu, i < n && k == prefix);
            if (lane == 0) {
                keep[w] = above;
                tie[w] = equal;
            }
        }
        __syncthreads();
        // the first `need` ties stay
        int carry = 0;
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
        // movers: slots at or behind m that stay, in order
        auto below = [&](int w) { return 32 * w + 32 <= m ? 0xffffffffu : 32 * w >= m ? 0u : (1u << (m - 32 * w)) - 1u; };
        carry = 0;
        for (int w0 = 0; w0 < nw; w0 += kPlanThreads) {
            const int w = w0 + tid;
            const uint32_t mv = w < nw ? keep[w] & ~below(w) : 0u;
            int total;
            const int incl = ix_block_scan(__popc(mv), scratch, &total);
            int at = carry + incl - __popc(mv);
            for (uint32_t left = mv; left; left &= left - 1u) p.movers[base + at++] = 32 * w + __ffs(left) - 1;
            carry += total;
        }
        // holes before each word
        carry = 0;
        for (int w0 = 0; w0 < nw; w0 += kPlanThreads) {
            const int w = w0 + tid;
            const uint32_t hole = w < nw ? ~keep[w] & below(w) : 0u;
            int total;
            const int incl = ix_block_scan(__popc(hole), scratch, &total);
            if (w < nw) pre[w] = carry + incl - __popc(hole);
            carry += total;
        }
        __syncthreads();  // the movers' list and pre are complete (one CTA wrote both)
    }
    for (int i = tid; i < max(p.K, p.max_n); i += kPlanThreads) {
        int s = -1;
        if (i < m) {
            s = i;
            if (n > p.K && !((keep[i >> 5] >> (i & 31)) & 1u)) {
                const uint32_t lower = (1u << (i & 31)) - 1u;
                s = ld_input(p.movers + base + pre[i >> 5] + __popc(~keep[i >> 5] & lower));
            }
        }
        if (i < p.K) src[i] = s;
        if (i < p.max_n) {
            if (p.acc_new != nullptr) {
                float a = 0.f;
                if (s >= 0) asm volatile("ld.global.f32 %0, [%1];" : "=f"(a) : "l"(p.acc + base + s));
                p.acc_new[base + i] = a;
            }
            if (p.pos_new != nullptr)
                p.pos_new[base + i] = s < 0 ? -1 : p.pos != nullptr ? ld_input(p.pos + base + s) : s;
        }
    }
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
    int row_bytes[kEvictBuffers];  // multiples of 16
    int n_buf;
};
constexpr int kApplyWarps = 8;

// One warp per 32 list entries; it copies the moved rows one after the other.
__global__ void __launch_bounds__(32 * kApplyWarps) smla_evict_apply_kernel(const EvictApplyParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long per = (p.K + 31) / 32;
    const long long unit = (long long)blockIdx.x * kApplyWarps + (threadIdx.x >> 5);
    if (unit >= per * p.B) return;
    const int b = (int)(unit / per), i = (int)(unit % per) * 32 + lane;
    const int s = i < p.K ? ld_input(p.src + (size_t)b * p.K + i) : -1;
    const bool moves = s != -1 && s != i;
    long long from = -1, to = -1;
    if (moves) {
        const int *pt_b = p.page_table + (size_t)b * p.pt_stride;
        from = paged_row(pt_b, p.pt_stride, p.num_pages, s);
        to = paged_row(pt_b, p.pt_stride, p.num_pages, i);
        if (from < 0 || to < 0) count_bad_index();
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, from >= 0 && to >= 0); todo; todo &= todo - 1u) {
        const int l = __ffs(todo) - 1;
        const long long f = __shfl_sync(0xffffffffu, from, l), t = __shfl_sync(0xffffffffu, to, l);
        for (int k = 0; k < p.n_buf; ++k) {
            const uint8_t *in = p.buf[k] + f * p.row_bytes[k];
            uint8_t *out = p.buf[k] + t * p.row_bytes[k];
            for (int x = 16 * lane; x < p.row_bytes[k]; x += 512)
                *reinterpret_cast<uint4 *>(out + x) = ld_row16(in + x);
        }
    }
}

}  // namespace smla

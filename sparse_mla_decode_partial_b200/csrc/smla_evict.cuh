// smla_evict.cuh -- eviction from the paged cache by accumulated attention
// weight: the positions that received least are chosen, and the rows that stay
// fill the holes they leave.  (smla_weigh.cuh accumulates the weights.)
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "smla_indexer.cuh"
#include "smla_q4.cuh"

namespace smla {

// ---------------------------------------------------------------- plan
// Per sequence of n slots: the min(n, K) slots that stay, and for each slot
// i < min(n, K) the slot its row comes from (itself, or, for the j-th slot
// there that leaves, the j-th slot at or behind min(n, K) that stays).
struct EvictPlanParams {
    const float *acc;    // [B, max_n]
    const int *pos;      // [B, max_n] or null (slot i holds position i)
    const int *n;        // [B]
    int B, max_n, K, n_sink, n_recent;
    int *movers;         // [B, max_n] scratch; null: what is behind slot m of pos_new serves until it is filled
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
// smaller slot, then ranks of holes and movers by prefix sums.  Block barriers of
// 1024 threads with little work between them: their chain bounds it.  Measured:
// 8448 slots 17.7 us, 16 sequences of 12132 to 29815 slots 25.0 us (with one CTA a
// sequence 23.6 and 46.5).  Cycles of the first, 34000 in all: keys in 2200,
// newest position and protected slots 3600, the three digits' counts 900, 560 and 630
// and their buckets 3600, 3900 and 4100 (about 3000 of each with one CTA to a
// sequence: the block scan), bitmaps 1100, ranks 8800 (5900), outputs 4700.
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
    int *movers = p.movers != nullptr ? p.movers + base : p.pos_new + base + m;
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
        if (p.pos == nullptr)
            cluster_sync();  // the sums are cleared (with pos, the exchange above saw to that)
        else
            __syncthreads();

        uint32_t prefix = 0;  // the K-th largest key, digit by digit
        int need = p.K, equal_all = 0;
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
                    dec[2] = (int)(first ? h1 : h0);
                }
            }
            cluster_sync();
            prefix |= ld_cluster(&dec[0], 0) << shift;
            need = (int)ld_cluster(&dec[1], 0);
            equal_all = (int)ld_cluster(&dec[2], 0);
        }
        const bool split = need < equal_all;  // not all slots at the K-th key stay

        // bitmaps: slots above the K-th key, slots equal to it
        const int nw = hi > lo ? (hi - lo + 31) / 32 : 0;
        int equal_here = 0;
        for (int w = warp; w < nw; w += kPlanThreads / 32) {
            const int i = lo + 32 * w + lane;
            const uint32_t k = i < hi ? key_of(i) : 0u;
            const uint32_t above = __ballot_sync(0xffffffffu, i < hi && k > prefix);
            const uint32_t equal = __ballot_sync(0xffffffffu, i < hi && k == prefix);
            if (lane == 0) {
                keep[w] = split ? above : above | equal;
                tie[w] = equal;
                equal_here += __popc(equal);
            }
        }
        if (split) {  // the first `need` of them do
            if (lane == 0) scratch[warp] = equal_here;
            __syncthreads();
            if (warp == 0) {
                const int x = __reduce_add_sync(0xffffffffu, scratch[lane]);
                if (lane == 0) xch[1] = x;
            }
            cluster_sync();
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
            for (uint32_t left = mvs; left; left &= left - 1u) movers[x++] = lo + 32 * w + __ffs(left) - 1;
            mv += total;
            const int gone = __popc(holes);
            const int at_hole = ix_block_scan(gone, scratch, &total) - gone;
            if (w < nw) pre[w] = hole + at_hole;
            hole += total;
        }
        cluster_sync();  // the movers' list and pre are complete; no CTA leaves while another reads its counts
    }
    // this CTA's slots below m, then its share of what lies behind
#pragma unroll 4
    for (int i = lo + tid; i < min(hi, m); i += kPlanThreads) {
        int s = i;
        if (cut) {
            const uint32_t k = keep[(i - lo) >> 5];
            if (!((k >> ((i - lo) & 31)) & 1u)) {
                const uint32_t lower = (1u << ((i - lo) & 31)) - 1u;
                s = ld_input(movers + pre[(i - lo) >> 5] + __popc(~k & lower));
            }
        }
        src[i] = s;
        if (p.acc_new != nullptr) p.acc_new[base + i] = ld_weight(p.acc + base + s);
        if (p.pos_new != nullptr) p.pos_new[base + i] = p.pos != nullptr ? ld_input(p.pos + base + s) : s;
    }
    // (no stores before this barrier that need not be: it waits for them; with
    // those of acc_new and src ahead of it 16 sequences took 41 us, not 26)
    if (cut) cluster_sync();  // the movers have been read
    for (long long i = m + (long long)rank * kPlanThreads + tid; i < max(p.K, p.max_n); i += nc * kPlanThreads) {
        if (i < p.K) src[i] = -1;
        if (i >= p.max_n) continue;
        if (p.acc_new != nullptr) p.acc_new[base + i] = 0.f;
        if (p.pos_new != nullptr) p.pos_new[base + i] = -1;
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
    int pieces[kEvictBuffers];  // 16-byte pieces of a row
    int n_buf;
    int total;                  // pieces of a row over all buffers
};

// One warp's share of the list entries [32 unit, 32 unit + 32) of the flattened
// (sequence, entry) groups: where the row of this lane's entry comes from and
// goes to, -1 where it stays.
struct EvictMove {
    long long from, to;  // rows of the pool: below 2^31
};
__device__ __forceinline__ int evict_entry(const EvictApplyParams &p, long long unit, long long per) {
    const int i = (int)(unit % per) * 32 + (int)(threadIdx.x & 31);
    return i < p.K ? ld_input(p.src + (size_t)(unit / per) * p.K + i) : -1;
}
__device__ __forceinline__ EvictMove evict_move(const EvictApplyParams &p, long long unit, long long per, int s) {
    const int b = (int)(unit / per), i = (int)(unit % per) * 32 + (int)(threadIdx.x & 31);
    EvictMove m{-1, -1};
    if (s == -1 || s == i) return m;
    const int *pt_b = p.page_table + (size_t)b * p.pt_stride;
    m.from = paged_row(pt_b, p.pt_stride, p.num_pages, s);
    m.to = paged_row(pt_b, p.pt_stride, p.num_pages, i);
    if (m.from < 0 || m.to < 0) {
        count_bad_index();
        m.from = m.to = -1;
    }
    return m;
}

// Rows that fit shared memory several times over (all real caches): one warp per
// CTA, a lane per move.  Each lane has its row's pieces copied in by bulk copies
// and, when the warp's have landed, out again: a few instructions per row, and
// 28 KB per CTA, seven CTAs per SM, in flight.  (Moving 16-byte pieces through
// registers took 65 instructions per 512 bytes, and 51 us where this takes 41,
// 80000 rows of 1408 bytes: 5.5 TB/s.  Eight CTAs of nineteen such rows: 41.3 us
// where seven of twenty take 40.6.)
constexpr int kApplyBulkBytes = 28160;  // twenty rows of 1152 + 256 bytes
constexpr int kApplyBlocks = 7;         // per SM; each with 128 bytes for the barrier
static_assert(kApplyBlocks * (kApplyBulkBytes + 128 + 1024) <= 233472 &&
              (kApplyBlocks + 1) * (kApplyBulkBytes + 128 + 1024) > 233472, "CTAs per SM");
__global__ void __launch_bounds__(32) smla_evict_apply_bulk_kernel(const EvictApplyParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bar;
    const int lane = threadIdx.x;
    if (lane == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    __syncwarp();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long per = (p.K + 31) / 32, units = per * p.B;
    const int row = 16 * p.total, most = kApplyBulkBytes / row;  // rows at a time
    bool dead = false;
    uint32_t phase = 0;
    int s = evict_entry(p, blockIdx.x, per);
    for (long long unit = blockIdx.x; unit < units && !dead; unit += gridDim.x) {
        const EvictMove m = evict_move(p, unit, per, s);
        if (unit + gridDim.x < units) s = evict_entry(p, unit + gridDim.x, per);
        const uint32_t moves = __ballot_sync(0xffffffffu, m.from >= 0);
        const int rank = __popc(moves & ((1u << lane) - 1u)), n = __popc(moves);
        for (int k0 = 0; k0 < n; k0 += most) {
            const bool mine = m.from >= 0 && rank >= k0 && rank < k0 + most;
            uint8_t *at = smem + (rank - k0) * row;
            if (lane == 0) mbar_arrive_expect_tx(&bar, (uint32_t)(min(most, n - k0) * row));
            __syncwarp();
            if (mine)
                for (int k = 0, off = 0; k < p.n_buf; ++k) {
                    const int bytes = 16 * p.pieces[k];
                    bulk_g2s(at + off, p.buf[k] + m.from * bytes, (uint32_t)bytes, &bar);
                    off += bytes;
                }
            mbar_wait(&bar, phase, dead);
            dead = __any_sync(0xffffffffu, dead);  // the warp stays together
            phase ^= 1u;
            if (mine && !dead) {
                for (int k = 0, off = 0; k < p.n_buf; ++k) {
                    const int bytes = 16 * p.pieces[k];
                    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                     __cvta_generic_to_global(p.buf[k] + m.to * bytes)),
                                 "r"(smem_addr(at + off)), "r"(bytes)
                                 : "memory");
                    off += bytes;
                }
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();  // the rows may be overwritten
        }
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

constexpr int kApplyWarps = 8;
constexpr int kApplyDepth = 8;  // pieces in flight per lane

// Longer rows.  One warp per 32 list entries: it lists the moves among them, then
// its lanes walk the moves' 16-byte pieces, all buffers in a row, eight loads in
// flight each before the first store.
__global__ void __launch_bounds__(32 * kApplyWarps) smla_evict_apply_kernel(const EvictApplyParams p) {
    __shared__ int from_s[kApplyWarps][32], to_s[kApplyWarps][32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long per = (p.K + 31) / 32;
    const long long unit = (long long)blockIdx.x * kApplyWarps + warp;
    if (unit >= per * p.B) return;
    const EvictMove m = evict_move(p, unit, per, evict_entry(p, unit, per));
    const uint32_t moves = __ballot_sync(0xffffffffu, m.from >= 0);
    if ((moves >> lane) & 1u) {
        const int k = __popc(moves & ((1u << lane) - 1u));
        from_s[warp][k] = (int)m.from;
        to_s[warp][k] = (int)m.to;
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

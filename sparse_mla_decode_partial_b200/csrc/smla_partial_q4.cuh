// smla_partial_q4.cuh -- split-K partial pass over 4-bit cache rows for up to
// 16 query rows (heads of one token, or of all tokens of a sequence that share
// a dense prefix), and the combine of the dense schedule's pieces.
//
// At 416 bytes a row the memory can deliver one row per SM about every 18
// cycles, so what counts is the work per row: decoding 512 codes, 2 * 16 * 1088
// flop, and the shared-memory traffic of both.  Writing decoded bf16 rows to
// shared memory for the tensor core to read (as the tcgen05 kernel does) costs
// 9 cycles of store and 17 of operand reads per row and leaves 3/4 of its M
// rows empty; here the codes stay packed in shared memory and are decoded in
// registers, straight into mma.sync B fragments, once per product:
//   S = Q K^T   A = 16 query rows (fragments in shared memory, in lane order),
//               B = 8 cache rows: a lane takes a whole group of 32 codes of one
//               row (one 16-byte load, one scale) for eight k16 steps; the
//               order of the dims within the sum is free.
//   O += P C    B = 16 cache rows x 8 columns: a lane takes 16 columns of four
//               rows; two byte permutes interleave the codes of two rows, and
//               the same and/or + fma as above then gives row pairs.
// A CTA is four warps and works on tiles of 64 rows.  Warp w scores rows 16 w
// .. 16 w + 15 alone (all 576 dims: no exchange of partial scores) and leaves
// P as an A fragment in its own rows' spent rope bytes; after one barrier every
// warp reads all four fragments and accumulates its 128 output columns.
// Running maxima: each warp keeps one per query row over its own rows, rounded
// up to an integer (log2 units), so that bringing its P to the common maximum
// is a multiplication by a power of two, exact in bf16: P is rounded once.
// The output is divided by the sum of the rounded P (lse is that of the others),
// so that a row which dominates is not off by its P's rounding, whatever the
// list's width or the bound K.  One row comes out bit for bit; lists of 513, 1024
// and 2048 rows whose softmax has a few large weights are off by 1.32e-3, 0.90e-3
// and 0.61e-3 of o (relative L2) where division by the sum of the others leaves
// 1.43e-3, 1.08e-3 and 1.20e-3, and o's own rounding is 1.07e-3, 0.75e-3 and
// 0.53e-3.  A product with ones adds them up, relative to the warp's own maximum:
// 110.9 us where the sum of the others alone takes 108.5 (32 sequences as below;
// adding up in registers 113.1), 37.1 and 36.9 (64 lists).
// Rows 416 bytes apart: the lane-to-row map below keeps every shared load free
// of bank conflicts without padding, so a page of the cache lands by one bulk
// copy.
// What bounds it: per 64-row tile an SM quarter spends about 1096 cycles on its
// 137 products (eight each) and 970 on the integer half of decoding, and the two
// hardly overlap: 2080 cycles in all in a loop with everything resident.  A full
// dense launch takes 2730 cycles a tile and SM at 1.6 GHz (issue slots 48% taken,
// integer pipe 42%, tensor pipe 37%, shared memory 41%) and about 3100 at 1.965
// GHz: the rest, 0.4 to 0.5 us a tile, does not shrink with the clock, so it is
// waiting, not issue; for what (pages, or the two barriers a tile) is not known.
// Lists take about 4200 cycles a tile on the SMs with the most (16 tiles; 40 of
// 148 SMs have 8): there the warps also issue the rows, 13 cp.async a thread and
// tile with a division each.  Measured with the combine: 32 sequences of 4329 to
// 65378 positions, 16 heads, 110.9 us (2.4 TB/s of rows; 40 us at the memory's
// rate); 64 lists of 2048 rows 37.1 us; one list 8.9 us.  Slower, beside 108.5
// us with fewer products: eight warps a tile (137 us for the
// first), one CTA of three groups per SM and a ring of seven pages (124), the
// score half on tcgen05 with rows decoded into tensor memory (181).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "smla_indexer.cuh"
#include "smla_q4.cuh"
#include "smla_tc_ptx.cuh"

namespace smla {

struct Q4Cfg {
    static constexpr int kThreads = 128;
    static constexpr int kRows = 16;                       // query rows (the mma's M)
    static constexpr int kTile = 64;                       // cache rows: one page
    static constexpr int kStages = 3;
    static constexpr int kStageBytes = kTile * kQ4RowBytes;  // 26624
    static constexpr int kResolve = 512;                   // list entries resolved at a time
    static constexpr int kOffQ = 0;                        // uint4 [36][32]
    static constexpr int kOffStage = 36 * 512;
    static constexpr int kOffRows = kOffStage + kStages * kStageBytes;  // int [kResolve]
    static constexpr int kOffBar = kOffRows + kResolve * 4;
    static constexpr int kSmemBytes = kOffBar + 8 * kStages;
    static constexpr int kMinBlocks = 2;                   // per SM: 2 x (100 + 1) KB
};
static_assert(Q4Cfg::kMinBlocks * (Q4Cfg::kSmemBytes + 1024) <= 233472, "shared memory per SM");

// The dense schedule: sequence b has ceil(its longest visible length / 64)
// tiles; CTA c of `grid` takes an equal run of the flattened tiles and writes
// one piece per sequence it meets, piece (c, b) at slot c + b (c + b grows
// strictly along the run, so slots are distinct).
struct Q4Params {
    PartialParams p;   // dense_t tokens of dense_h heads, at most 16 rows together
    int grid;          // CTAs that share the tiles
    int *prefix;       // [B + 1] tiles before each sequence, written by CTA 0
    float *piece_o;    // [grid + B, 16, 512]
    float2 *piece_ml;  // [grid + B, 16]: (max, lse) in log2 units
};

// Cache row (0..7 of its n8 tile) that column n of a B fragment stands for.
// With rows 416 = 3 * 128 + 32 bytes apart, rows 2 m and 2 m + 1 of the score
// product lie 64 bytes apart modulo 128, and rows 0, 2, 4, 6 (or 1, 3, 5, 7) of
// the output product in four different 32-byte quarters.
__device__ __forceinline__ int q4_row_of(int n) {
    const int c = n >> 1;
    return (n & 1) ? 4 + ((c + 2) & 3) : c;
}

// First of the four dims that lane column c feeds to k16 step s of the score
// product (dims +0, +1 at k = 2 c, 2 c + 1 and +2, +3 at k = 2 c + 8, 2 c + 9).
__device__ __forceinline__ int q4_dim_of(int s, int c) {
    return s < 32 ? 32 * (4 * (s >> 3) + c) + 8 * ((s & 7) >> 1) + 4 * (s & 1)
                  : 32 * (s >> 1) + 8 * c + 4 * (s & 1);
}

__device__ __forceinline__ uint32_t lds_u16x2(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return (uint32_t)v * 0x00010001u;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint4 lds_16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds_8(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ float lds_f(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts_f(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void sts_16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 2^d as a pair of bf16 for an integer-valued d <= 0 (0 below 2^-126, and for
// d = -inf or NaN, which stand for a side that has seen nothing).
__device__ __forceinline__ uint32_t bf16x2_pow2(float d) {
    const int e = 127 + (int)fmaxf(d, -127.f);
    return (uint32_t)(e << 7) * 0x00010001u;
}

// Raw scores of 16 cache rows (those at `rows`, 416 bytes apart) against the 16
// query rows, whose A fragments are uint4 [36][32] at q.  s[i]: query rows r,
// r + 8 against columns 2 c, 2 c + 1 of the i-th n8 tile.
__device__ __forceinline__ void q4_scores(uint32_t q, uint32_t rows, int lane, float (&s)[2][4]) {
    const int c = lane & 3;
    const uint32_t row = rows + q4_row_of(lane >> 2) * kQ4RowBytes;
    q += 16 * lane;
    // Even and odd steps keep accumulators of their own: two chains of 36
    // dependent products left the pipe waiting for their latency.
    float odd[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        odd[i][0] = odd[i][1] = odd[i][2] = odd[i][3] = 0.f;
        s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
    }
    auto steps = [&](int st, const uint4 (&v)[2]) {  // k16 steps st, st + 1
        const uint4 a0 = lds_16(q + st * 512), a1 = lds_16(q + (st + 1) * 512);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mma_bf16_16816(s[i], a0.x, a0.y, a0.z, a0.w, v[i].x, v[i].y);
            mma_bf16_16816(odd[i], a1.x, a1.y, a1.z, a1.w, v[i].z, v[i].w);
        }
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t s2[2], bias[2];
        uint4 code[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            code[i] = lds_16(row + i * 8 * kQ4RowBytes + 16 * (4 * j + c));
            s2[i] = lds_u16x2(row + i * 8 * kQ4RowBytes + kQ4OffScale + 2 * (4 * j + c));
            bias[i] = q4_bias(s2[i]);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint4 v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t word = w == 0 ? code[i].x : w == 1 ? code[i].y : w == 2 ? code[i].z : code[i].w;
                v[i] = q4_word(word, s2[i], bias[i]);
            }
            steps(8 * j + 2 * w, v);
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint4 v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = lds_16(row + i * 8 * kQ4RowBytes + kQ4OffRope + 64 * j + 16 * c);
        steps(32 + 2 * j, v);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[i][k] += odd[i][k];
}

// One warp's share of a CTA: scores of 16 rows, 128 output columns.
struct Q4Consumer {
    int warp, lane, r, c;
    float oacc[16][4];
    float mw0, mw1;    // running max (an integer or -inf) of query rows r, r + 8 over this warp's cache rows
    float l0, l1;      // this lane's part of sum exp2(s - mw)
    float racc[4];     // sums of this warp's rounded P relative to mw: query row r at [0], r + 8 at [2]
    float M0, M1;      // the CTA's running max, what oacc is relative to

    __device__ __forceinline__ void init(int warp_, int lane_) {
        warp = warp_;
        lane = lane_;
        r = lane >> 2;
        c = lane & 3;
        reset();
    }
    __device__ __forceinline__ void reset() {
        mw0 = mw1 = M0 = M1 = -INFINITY;
        l0 = l1 = 0.f;
        racc[0] = racc[1] = racc[2] = racc[3] = 0.f;
#pragma unroll
        for (int n = 0; n < 16; ++n) oacc[n][0] = oacc[n][1] = oacc[n][2] = oacc[n][3] = 0.f;
    }

    // Masked scores (log2 units, -inf where masked) -> P in this warp's rows'
    // rope bytes: its A fragment, and the maxima it is relative to.
    __device__ __forceinline__ void softmax(uint32_t tile, float (&s)[2][4]) {
        float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
        const float n0 = fmaxf(mw0, ceilf(x0)), n1 = fmaxf(mw1, ceilf(x1));
        const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
        const float f0 = fast_exp2(mw0 - u0), f1 = fast_exp2(mw1 - u1);  // 2^-inf = 0 before the first visible row
        l0 *= f0;
        l1 *= f1;
        racc[0] *= f0;
        racc[2] *= f1;
        mw0 = n0;
        mw1 = n1;
        uint32_t a[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float p00 = fast_exp2(s[i][0] - u0), p01 = fast_exp2(s[i][1] - u0);
            const float p10 = fast_exp2(s[i][2] - u1), p11 = fast_exp2(s[i][3] - u1);
            l0 += p00 + p01;
            l1 += p10 + p11;
            a[2 * i] = pack_bf16x2(p00, p01);
            a[2 * i + 1] = pack_bf16x2(p10, p11);
        }
        mma_bf16_16816(racc, a[0], a[1], a[2], a[3], 0x3F803F80u, 0x3F803F80u);  // a product with ones adds them up
        __syncwarp();  // every lane has read the rope bytes
        const uint32_t mine = tile + 16 * warp * kQ4RowBytes + kQ4OffRope;
        sts_16(mine + (lane >> 1) * kQ4RowBytes + 16 * (lane & 1), a[0], a[1], a[2], a[3]);
        if (c == 0) {
            sts_f(mine + r * kQ4RowBytes + 32, mw0);
            sts_f(mine + (r + 8) * kQ4RowBytes + 32, mw1);
        }
    }

    // O += P C over the tile's 64 rows, this warp's 128 columns.
    __device__ __forceinline__ void output(uint32_t tile) {
        float m0[4], m1[4];
        float n0 = M0, n1 = M1;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t at = tile + 16 * w * kQ4RowBytes + kQ4OffRope + 32;
            m0[w] = lds_f(at + r * kQ4RowBytes);
            m1[w] = lds_f(at + (r + 8) * kQ4RowBytes);
            n0 = fmaxf(n0, m0[w]);
            n1 = fmaxf(n1, m1[w]);
        }
        if (__any_sync(0xffffffffu, n0 != M0 || n1 != M1)) {
            const float a0 = n0 == M0 ? 1.f : fast_exp2(M0 - n0), a1 = n1 == M1 ? 1.f : fast_exp2(M1 - n1);
#pragma unroll
            for (int n = 0; n < 16; ++n) {
                oacc[n][0] *= a0;
                oacc[n][1] *= a0;
                oacc[n][2] *= a1;
                oacc[n][3] *= a1;
            }
            M0 = n0;
            M1 = n1;
        }
        const int ra = q4_row_of(2 * c), rb = q4_row_of(2 * c + 1);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t base = tile + 16 * w * kQ4RowBytes;
            const uint4 pf = lds_16(base + (lane >> 1) * kQ4RowBytes + kQ4OffRope + 16 * (lane & 1));
            const uint32_t f0 = bf16x2_pow2(m0[w] - M0), f1 = bf16x2_pow2(m1[w] - M1);
            const uint32_t a0 = bf16x2_mul(pf.x, f0), a1 = bf16x2_mul(pf.y, f1);
            const uint32_t a2 = bf16x2_mul(pf.z, f0), a3 = bf16x2_mul(pf.w, f1);
            const uint32_t at_a = base + ra * kQ4RowBytes, at_b = base + rb * kQ4RowBytes;
            const uint32_t col = 64 * warp + 8 * r, grp = kQ4OffScale + 2 * (4 * warp + (r >> 1));
            const uint2 wa = lds_8(at_a + col), wb = lds_8(at_b + col);
            const uint2 va = lds_8(at_a + 8 * kQ4RowBytes + col), vb = lds_8(at_b + 8 * kQ4RowBytes + col);
            const uint32_t s2 = lds_u16(at_a + grp) | lds_u16(at_b + grp) << 16;
            const uint32_t t2 = lds_u16(at_a + 8 * kQ4RowBytes + grp) | lds_u16(at_b + 8 * kQ4RowBytes + grp) << 16;
            const uint32_t sb = q4_bias(s2), tb = q4_bias(t2);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t x = i ? wa.y : wa.x, y = i ? wb.y : wb.x;
                const uint32_t z = i ? va.y : va.x, u = i ? vb.y : vb.x;
                // low halves: values 0, 2, 4, 6 of both rows; high halves: 1, 3, 5, 7
                const uint32_t e0 = __byte_perm(x, y, 0x5410), o0 = __byte_perm(x, y, 0x7632);
                const uint32_t e1 = __byte_perm(z, u, 0x5410), o1 = __byte_perm(z, u, 0x7632);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mma_bf16_16816(oacc[8 * i + 2 * k], a0, a1, a2, a3, q4_pair(e0 >> (4 * k), s2, sb),
                                   q4_pair(e1 >> (4 * k), t2, tb));
                    mma_bf16_16816(oacc[8 * i + 2 * k + 1], a0, a1, a2, a3, q4_pair(o0 >> (4 * k), s2, sb),
                                   q4_pair(o1 >> (4 * k), t2, tb));
                }
            }
        }
    }

    // Total weight of query rows r, r + 8 relative to M, the same in every lane
    // of a row, and that of the rounded P.  scratch: float2 [2][4][16] in shared
    // memory; the CTA synchronises.
    __device__ __forceinline__ void totals(float2 *scratch, float &t0, float &t1, float &u0, float &u1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (c == 0) {
            scratch[16 * warp + r] = make_float2(mw0, l0);
            scratch[16 * warp + r + 8] = make_float2(mw1, l1);
            scratch[64 + 16 * warp + r] = make_float2(racc[0], racc[2]);
        }
        __syncthreads();
        t0 = t1 = u0 = u1 = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float2 x = scratch[16 * w + r], y = scratch[16 * w + r + 8], z = scratch[64 + 16 * w + r];
            // a warp that saw nothing has sums of 0; one whose every score was
            // NaN keeps its NaN
            const float f0 = x.x == -INFINITY ? 1.f : fast_exp2(x.x - M0), f1 = y.x == -INFINITY ? 1.f : fast_exp2(y.x - M1);
            t0 += x.y * f0;
            t1 += y.y * f1;
            u0 += z.x * f0;
            u1 += z.y * f1;
        }
    }
};

// Stage 16 query rows (row0 .. row0 + nrows - 1 of q; the rest zero) as A
// fragments in lane order, by NT threads.
template <int NT>
__device__ __forceinline__ void q4_stage_q(uint8_t *dst, const __nv_bfloat16 *q, long long row0, int nrows) {
    uint4 *frag = reinterpret_cast<uint4 *>(dst);
#pragma unroll
    for (int k = 0; k < 36 * 32 / NT; ++k) {
        const int i = threadIdx.x + NT * k, l = i & 31, st = i >> 5, r = l >> 2;
        const __nv_bfloat16 *src = q + (row0 + r) * kD + q4_dim_of(st, l & 3);
        uint2 lo = make_uint2(0u, 0u), hi = lo;
        if (r < nrows)
            asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(lo.x), "=r"(lo.y) : "l"(src));
        if (r + 8 < nrows)
            asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(hi.x), "=r"(hi.y) : "l"(src + 8 * kD));
        frag[i] = make_uint4(lo.x, hi.x, lo.y, hi.y);
    }
}

// ---------------------------------------------------------------- sparse lists
// One CTA = one (query token, split).  Equal splits; the partials go to
// part_o / part_m / part_lse [B, T, H, S] (DIRECT: o, lse).  Rows come by 16-byte
// cp.async (64 lists of 2048: 37 us; by one bulk copy a row 39.6).  Equal runs over
// the batch as in the dense schedule took 47 us: a run that goes on in the next
// list starts its pipeline anew.  A cluster of four splits that merge in
// distributed shared memory took 35.8, but of two 60.8 against 43.7 and of sixteen
// (15 lists) 23.5 against 14.9.
template <bool DIRECT>
__global__ void __launch_bounds__(Q4Cfg::kThreads, Q4Cfg::kMinBlocks) smla_q4_sparse_kernel(const PartialParams p) {
    using C = Q4Cfg;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int s = blockIdx.x % p.nsplit, bt = blockIdx.x / p.nsplit;
    const int j0 = (int)min((long long)s * p.kc, (long long)p.K);
    const int len = (int)min((long long)p.kc, (long long)p.K - j0);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    int *rows_s = reinterpret_cast<int *>(smem + C::kOffRows);
    const uint32_t sbase = smem_addr(smem);
    bool dead = false;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], C::kThreads);
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint8_t *cache = reinterpret_cast<const uint8_t *>(p.cache);

    // 26 16-byte pieces per row, 13 per thread and tile; padding slots are
    // zero-filled (scale 0: they decode to zeros)
    auto issue = [&](int it, int t, int n) {
        const uint32_t dst = sbase + C::kOffStage + it % C::kStages * C::kStageBytes;
#pragma unroll
        for (int k = 0; k < 13; ++k) {
            const int e = tid + 128 * k, row = e / 26, ch = e - 26 * row;
            const int j = t * C::kTile + row;
            const int at = j < n ? rows_s[j] : -1;
            const uint8_t *src = cache + (size_t)(at >= 0 ? at : 0) * kQ4RowBytes + 16 * ch;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * e), "l"(src),
                         "r"(at >= 0 ? 16u : 0u)
                         : "memory");
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&full[it % C::kStages]))
                     : "memory");
    };

    Q4Consumer w;
    w.init(warp, lane);
    bool staged = false;
    int it = 0;  // tiles so far: ring position
    for (int base = 0; base < len; base += C::kResolve) {
        const int n = min(C::kResolve, len - base);
        __syncthreads();  // the ring and rows_s are free
        resolve_rows<4>(p, bt, j0, base, n, rows_s, tid, C::kThreads);
        __syncthreads();
        const int tiles = (n + C::kTile - 1) / C::kTile;
        for (int t = 0; t < min(C::kStages, tiles); ++t) issue(it + t, t, n);
        if (!staged) {
            q4_stage_q<C::kThreads>(smem + C::kOffQ, p.q, (long long)bt * p.H, p.H);
            staged = true;
            __syncthreads();
        }
        for (int t = 0; t < tiles; ++t, ++it) {
            const uint32_t tile = sbase + C::kOffStage + it % C::kStages * C::kStageBytes;
            mbar_wait(&full[it % C::kStages], (it / C::kStages) & 1, dead);
            float sc[2][4];
            q4_scores(sbase + C::kOffQ, tile + 16 * warp * kQ4RowBytes, lane, sc);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = t * C::kTile + 16 * warp + 8 * i + q4_row_of(2 * w.c + e);
                    const bool on = j < n && rows_s[j] >= 0;
                    sc[i][e] = on ? sc[i][e] * p.scale_log2 : -INFINITY;
                    sc[i][2 + e] = on ? sc[i][2 + e] * p.scale_log2 : -INFINITY;
                }
            }
            w.softmax(tile, sc);
            __syncthreads();  // P complete; every warp is done with the previous tile
            if (t >= 1 && t - 1 + C::kStages < tiles) issue(it - 1 + C::kStages, t - 1 + C::kStages, n);
            w.output(tile);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float t0, t1, u0, u1;
    w.totals(reinterpret_cast<float2 *>(smem + C::kOffStage), t0, t1, u0, u1);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int h = w.r + 8 * half;
        if (h >= p.H) continue;
        const float tot = half ? t1 : t0, M = half ? w.M1 : w.M0;
        const bool some = !(tot == 0.f);  // NaN counts
        const size_t row = (size_t)bt * p.H + h;
        const float sum = half ? u1 : u0;  // what the output is divided by
        const float inv = !some ? 0.f : DIRECT ? 1.f / sum : tot / sum;
        // n8 tile n of the accumulators is column 128 warp + 16 (2 c + e) + n
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int col = 128 * warp + 32 * w.c + 16 * e;
            if (DIRECT) {
#pragma unroll
                for (int n = 0; n < 16; n += 8) {
                    uint32_t x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[k] = pack_bf16x2(w.oacc[n + 2 * k][2 * half + e] * inv, w.oacc[n + 2 * k + 1][2 * half + e] * inv);
                    *reinterpret_cast<uint4 *>(p.o + row * kDc + col + n) = make_uint4(x[0], x[1], x[2], x[3]);
                }
            } else {
#pragma unroll
                for (int n = 0; n < 16; n += 4)
                    *reinterpret_cast<float4 *>(p.part_o + (row * p.nsplit + s) * kDc + col + n) =
                        make_float4(w.oacc[n][2 * half + e] * inv, w.oacc[n + 1][2 * half + e] * inv,
                                    w.oacc[n + 2][2 * half + e] * inv, w.oacc[n + 3][2 * half + e] * inv);
            }
        }
        if (warp == 0 && w.c == 0) {
            const float base = M == -INFINITY ? 0.f : M;
            const float lse = some ? (base + log2f(tot)) * kLn2 : -INFINITY;
            if (DIRECT) {
                p.lse[row] = lse;
            } else {
                p.part_m[row * p.nsplit + s] = some ? base * kLn2 : -INFINITY;
                p.part_lse[row * p.nsplit + s] = lse;
            }
        }
    }
}

// ---------------------------------------------------------------- dense prefixes
// Longest visible length of sequence b's query tokens; lengths outside [0, K]
// are clamped (and counted when `count`).
__device__ __forceinline__ int q4_seq_len(const PartialParams &p, int b, bool count) {
    int len = 0;
    for (int t = 0; t < p.dense_t; ++t) {
        const int raw = ld_input(p.seq_lens + (size_t)b * p.dense_t + t);
        if (count && (raw < 0 || raw > p.K)) count_bad_index();
        len = max(len, min(max(raw, 0), p.K));
    }
    return len;
}

// CTAs that share `total` tiles, min_tiles or more each.
__host__ __device__ __forceinline__ int q4_sharers(int grid, int min_tiles, long long total) {
    const long long most = (total + min_tiles - 1) / min_tiles;
    return (int)(most < 1 ? 1 : most < grid ? most : grid);
}

// A CTA's run [begin, end) of the flattened tiles of TILE positions: total
// first, then the sequence (b, of length len) and the tile it starts in.  Who
// walks the run stops at the last sequence too: lengths that someone writes
// during the launch must not send it on for ever.  Every thread calls it;
// scratch holds 48 ints of shared memory.  The first CTA counts bad lengths.
struct Q4Run {
    long long total, begin, end;
    int b, len, tile;
};
template <int TILE>
__device__ __forceinline__ Q4Run q4_find_run(const PartialParams &p, int grid, int min_tiles, int *prefix,
                                             int *scratch) {
    const bool first_cta = blockIdx.x == 0;
    Q4Run r{};
    int len = 0, tiles = 0, incl = 0, sum = 0;
    for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        len = b < p.B ? q4_seq_len(p, b, first_cta) : 0;
        tiles = (len + TILE - 1) / TILE;
        incl = ix_block_scan(tiles, scratch, &sum);
        if (prefix != nullptr && first_cta && b < p.B) prefix[b] = (int)r.total + incl - tiles;
        r.total += sum;
    }
    if (prefix != nullptr && first_cta && threadIdx.x == 0) prefix[p.B] = (int)r.total;
    const int sharers = q4_sharers(grid, min_tiles, r.total);
    if ((int)blockIdx.x >= sharers || r.total == 0) return r;
    r.begin = r.total * blockIdx.x / sharers;
    r.end = r.total * (blockIdx.x + 1) / sharers;
    long long before = 0;
    if (p.B > (int)blockDim.x && threadIdx.x == 0) scratch[40] = p.B;  // (none, should the lengths change meanwhile)
    for (int b0 = 0; b0 < p.B && before <= r.begin; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        if (p.B > (int)blockDim.x) {  // else the counts above are still those of this chunk
            len = b < p.B ? q4_seq_len(p, b, false) : 0;
            tiles = (len + TILE - 1) / TILE;
            incl = ix_block_scan(tiles, scratch, &sum);
        }
        const long long first = before + incl - tiles;
        if (first <= r.begin && r.begin < first + tiles) {
            scratch[40] = b;
            scratch[41] = (int)(r.begin - first);
            scratch[42] = len;
        }
        before += sum;
    }
    __syncthreads();
    r.b = scratch[40];
    r.tile = scratch[41];
    r.len = scratch[42];
    return r;
}

// Page of tile t of the sequence whose page-table row is pt_b; -1 where none is mapped.
__device__ __forceinline__ int q4_page(const int *pt_b, int pt_stride, long long num_pages, int t) {
    if (t >= pt_stride) return -1;
    const int pg = ld_input(pt_b + t);
    return (pg >= 0 && (long long)pg < num_pages) ? pg : -1;
}

// Thread 0: copy a page of 4-bit rows to shared memory at dst, or (no page)
// complete its barrier at once.
__device__ __forceinline__ void q4_copy_page(const PartialParams &p, int pg, uint8_t *dst, uint64_t *bar) {
    if (pg < 0) {
        mbar_arrive(bar);
        return;
    }
    mbar_arrive_expect_tx(bar, (uint32_t)Q4Cfg::kStageBytes);
    bulk_g2s(dst, reinterpret_cast<const uint8_t *>(p.cache) + (size_t)pg * Q4Cfg::kStageBytes,
             (uint32_t)Q4Cfg::kStageBytes, bar);
}

__global__ void __launch_bounds__(Q4Cfg::kThreads, Q4Cfg::kMinBlocks) smla_q4_dense_kernel(const Q4Params a) {
    using C = Q4Cfg;
    const PartialParams &p = a.p;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    int *scratch = reinterpret_cast<int *>(smem + C::kOffRows);  // scan scratch, then what the scan found
    const uint32_t sbase = smem_addr(smem);
    bool dead = false;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const Q4Run run = q4_find_run<C::kTile>(p, a.grid, 1, a.prefix, scratch);
    const int nrows = p.dense_t * p.dense_h;
    int b = run.b, tile0 = run.tile;
    Q4Consumer w;
    w.init(warp, lane);
    int it = 0;
    for (long long at = run.begin; at < run.end && b < p.B; ++b, tile0 = 0) {
        const int len = q4_seq_len(p, b, false);  // (run.len in a register through the loop: 110.6 us where this takes 108.4)
        const int tiles = (int)min((long long)((len + C::kTile - 1) / C::kTile - tile0), run.end - at);
        if (tiles <= 0) continue;  // a sequence that sees nothing
        at += tiles;
        const int *pt_b = p.page_table + (size_t)b * p.pt_stride;
        auto page_of = [&](int t) { return q4_page(pt_b, p.pt_stride, p.num_pages, t); };
        auto issue = [&](int i, int pg) {  // thread 0
            q4_copy_page(p, pg, smem + C::kOffStage + i % C::kStages * C::kStageBytes, &full[i % C::kStages]);
        };
        fence_proxy_async_smem();
        __syncthreads();  // the previous piece is done with the ring and with Q
        if (tid == 0) {
            for (int t = 0; t < min(C::kStages, tiles); ++t) issue(it + t, page_of(tile0 + t));
        }
        q4_stage_q<C::kThreads>(smem + C::kOffQ, p.q, (long long)b * nrows, nrows);
        // visible positions of this lane's two query rows
        int lim0 = 0, lim1 = 0;
        if (w.r < nrows)
            lim0 = min(max(ld_input(p.seq_lens + (size_t)b * p.dense_t + w.r / p.dense_h), 0), p.K);
        if (w.r + 8 < nrows)
            lim1 = min(max(ld_input(p.seq_lens + (size_t)b * p.dense_t + (w.r + 8) / p.dense_h), 0), p.K);
        w.reset();
        __syncthreads();
        for (int t = 0; t < tiles; ++t, ++it) {
            const uint32_t tile = sbase + C::kOffStage + it % C::kStages * C::kStageBytes;
            const int pos0 = (tile0 + t) * C::kTile;
            const bool mapped = page_of(tile0 + t) >= 0;
            int next = -1;
            if (tid == 0 && t >= 1 && t - 1 + C::kStages < tiles) next = page_of(tile0 + t - 1 + C::kStages);
            mbar_wait(&full[it % C::kStages], (it / C::kStages) & 1, dead);
            // rows that no query token sees may hold anything: scale 0 makes
            // them decode to zeros (0 * P = 0)
            const int live = mapped ? min(len - pos0, C::kTile) : 0;
            if (live < C::kTile) {
                if (!mapped && tid < min(len - pos0, C::kTile)) count_bad_index();
                if (tid >= live && tid < C::kTile) {
                    const uint32_t sc = tile + tid * kQ4RowBytes + kQ4OffScale;
                    sts_16(sc, 0u, 0u, 0u, 0u);
                    sts_16(sc + 16, 0u, 0u, 0u, 0u);
                }
                __syncthreads();
            }
            float sc[2][4];
            q4_scores(sbase + C::kOffQ, tile + 16 * warp * kQ4RowBytes, lane, sc);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = 16 * warp + 8 * i + q4_row_of(2 * w.c + e);
                    const int pos = j < live ? pos0 + j : INT_MAX;
                    sc[i][e] = pos < lim0 ? sc[i][e] * p.scale_log2 : -INFINITY;
                    sc[i][2 + e] = pos < lim1 ? sc[i][2 + e] * p.scale_log2 : -INFINITY;
                }
            }
            w.softmax(tile, sc);
            fence_proxy_async_smem();  // P and cleared scales, before a later bulk copy writes there
            __syncthreads();  // P complete; every warp is done with the previous tile
            if (tid == 0 && t >= 1 && t - 1 + C::kStages < tiles) issue(it - 1 + C::kStages, next);
            w.output(tile);
        }
        // ---- the piece
        __syncthreads();
        float t0, t1, u0, u1;
        w.totals(reinterpret_cast<float2 *>(smem + C::kOffStage), t0, t1, u0, u1);
        const size_t slot = (size_t)blockIdx.x + b;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int h = w.r + 8 * half;
            if (h >= nrows) continue;
            const float tot = half ? t1 : t0;
            const bool some = !(tot == 0.f);
            const float inv = some ? tot / (half ? u1 : u0) : 0.f;
            float *dst = a.piece_o + (slot * C::kRows + h) * kDc + 128 * warp + 32 * w.c;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int n = 0; n < 16; n += 4)
                    *reinterpret_cast<float4 *>(dst + 16 * e + n) =
                        make_float4(w.oacc[n][2 * half + e] * inv, w.oacc[n + 1][2 * half + e] * inv,
                                    w.oacc[n + 2][2 * half + e] * inv, w.oacc[n + 3][2 * half + e] * inv);
            if (warp == 0 && w.c == 0) {
                const float M = half ? w.M1 : w.M0;
                const float base = M == -INFINITY ? 0.f : M;
                a.piece_ml[slot * C::kRows + h] =
                    some ? make_float2(base, base + log2f(tot)) : make_float2(-INFINITY, -INFINITY);
            }
        }
    }
}

// ---------------------------------------------------------------- combine of pieces
// For each query row o = sum_c 2^(m_c - M) O_c / L, L = sum_c 2^(lse_c - M),
// lse = M + log2 L, over the pieces c that the sequence was cut into.  PARTS
// CTAs per row share its 512 columns: 128 / PARTS threads hold a CTA's columns
// as float4, and 4 PARTS groups of them take every (4 PARTS)-th piece and meet
// in shared memory.  PARTS is 4 while rows are at most half the SMs.  With 4 and
// with 1 (both kernels): one sequence of 37888 positions, 16 rows, 18.1 and 24.8
// us; four of 64000, 64 rows, 51.4 and 52.8; five of 51200, 80 rows, 54.9 and
// 54.1; nine of 19200, 144 rows, 43.3 and 41.8.
constexpr int kQ4CombineThreads = 512;
template <int PARTS>
__global__ void __launch_bounds__(kQ4CombineThreads) smla_q4_combine_kernel(const Q4Params a) {
    constexpr int kCols = 128 / PARTS, kGroups = kQ4CombineThreads / kCols;
    __shared__ float4 part[kGroups - 1][kCols];
    __shared__ float warp_max[16], warp_sum[16], weight[kQ4CombineThreads];
    constexpr int kAhead = 4;
    const PartialParams &p = a.p;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long row = blockIdx.x / PARTS;  // of [B, T, H]
    const int col0 = blockIdx.x % PARTS * kCols;
    const int nrows = p.dense_t * p.dense_h, b = (int)(row / nrows), r = (int)(row - (long long)b * nrows);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long first = ld_input(a.prefix + b), last = ld_input(a.prefix + b + 1);
    const long long total = ld_input(a.prefix + p.B);
    const int sharers = q4_sharers(a.grid, 1, total);
    // CTA of flattened tile x: the c with total c / sharers <= x < total (c + 1) / sharers
    int c0 = 0, n = 0;
    if (last > first) {
        c0 = (int)(((first + 1) * sharers - 1) / total);
        n = (int)((last * sharers - 1) / total) - c0 + 1;
    }
    const float2 *ml = a.piece_ml + ((size_t)c0 + b) * Q4Cfg::kRows + r;
    const float *po = a.piece_o + (((size_t)c0 + b) * Q4Cfg::kRows + r) * kDc;
    // The first loads of the pieces go out beside those of their maxima.
    const int g = tid / kCols, col = tid % kCols;
    auto piece = [&](int c) {
        return c < n ? __ldcg(reinterpret_cast<const float4 *>(po + (size_t)c * Q4Cfg::kRows * kDc) + col0 + col)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 ahead[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) ahead[k] = piece(g + k * kGroups);
    const float2 none = make_float2(-INFINITY, -INFINITY);
    auto max_lse = [&](int c) { return c < n ? __ldcg(ml + (size_t)c * Q4Cfg::kRows) : none; };
    const float2 mine = max_lse(tid);
    float M = mine.x;
    for (int c = tid + kQ4CombineThreads; c < n; c += kQ4CombineThreads) M = fmaxf(M, max_lse(c).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) warp_max[warp] = M;
    __syncthreads();
    M = warp_max[lane & 15];
#pragma unroll
    for (int o = 8; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    __nv_bfloat16 *out = p.o + row * kDc;
    if (M == -INFINITY) {  // nothing attended to
        if (tid < kCols) *reinterpret_cast<uint2 *>(out + 4 * (col0 + tid)) = make_uint2(0u, 0u);
        if (tid == 0 && col0 == 0) p.lse[row] = -INFINITY;
        return;
    }
    weight[tid] = mine.x == -INFINITY ? 0.f : exp2f(mine.x - M);  // 0: an empty piece, or none
    float L = mine.y == -INFINITY ? 0.f : exp2f(mine.y - M);
    for (int c = tid + kQ4CombineThreads; c < n; c += kQ4CombineThreads) {
        const float v = max_lse(c).y;
        if (v != -INFINITY) L += exp2f(v - M);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) warp_sum[warp] = L;
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int c, const float4 &v) {
        const float f = c < kQ4CombineThreads ? weight[c] : exp2f(max_lse(c).x - M);
        if (f == 0.f) return;  // (what an empty piece holds is undefined)
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) add(min(g + k * kGroups, kQ4CombineThreads - 1), ahead[k]);
#pragma unroll 4
    for (int c = g + kAhead * kGroups; c < n; c += kGroups) add(c, piece(c));
    if (g > 0) part[g - 1][col] = acc;
    __syncthreads();
    if (g > 0) return;
    L = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) L += warp_sum[w];
#pragma unroll
    for (int k = 0; k < kGroups - 1; ++k) {
        const float4 v = part[k][col];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
    }
    const float inv = 1.f / L;
    *reinterpret_cast<uint2 *>(out + 4 * (col0 + col)) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (tid == 0 && col0 == 0) p.lse[row] = (M + log2f(L)) * kLn2;
}

}  // namespace smla

// smla_q4.cuh -- the 4-bit latent cache: its row format, the kernel that
// quantises new rows into the paged cache, and the kernel that reads rows
// back as bf16.
//
// A row of 576 values takes 416 bytes (13 sectors of 32 bytes):
//   bytes [0, 256)    codes of the 512 latents, 4 bits each
//   bytes [256, 288)  16 bf16 scales, one per group of 32 latents
//   bytes [288, 416)  the 64 rope values, bf16, unchanged
// Latent d of group g = d / 32 reads back as (code - 8) * scale[g], code in
// 1 .. 15.  The scale is the smallest number of four significant bits that is
// at least max|x| / 7, and the code rounds x / scale to the nearest integer
// (ties to even), so |error| <= scale / 2 and nothing clips.
// Why four bits: (code - 8) has at most three significant bits and 136 * scale
// = 17 * 8 * scale at most eight, so both (code - 8) * scale and -136 * scale
// are bf16 numbers, and a kernel gets the value with one exact bf16 fma:
//   (128 + code) * scale - 136 * scale,
// where 128 + code is the bf16 bit pattern 0x4300 | code.  Decoding costs one
// and/or, one fma and (for three of four pairs) one shift per two values, and
// adds no rounding to the quantiser's.
// A group whose largest magnitude is below 2^-118 is stored as zeros.  A group
// holding NaN or a magnitude of 2^120 or more (infinities too) is stored as
// zeros and the row's 64 rope values become NaN: every score against the row
// is then NaN, while 0 * (row) stays 0 for query tokens that do not attend to
// it (rope values never enter the output).
// Eight codes share a little-endian 32-bit word: nibble k < 4 is value 2 k of
// the eight and nibble k + 4 value 2 k + 1, so (word >> 4 k) & 0x000f000f holds
// neighbours in the low and the high half.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "smla_partial_mma.cuh"

namespace smla {

constexpr int kQ4Group = 32;
constexpr int kQ4Groups = kDc / kQ4Group;             // 16
constexpr int kQ4OffScale = kDc / 2;                  // 256
constexpr int kQ4OffRope = kQ4OffScale + 2 * kQ4Groups;  // 288
constexpr int kQ4RowBytes = kQ4OffRope + 2 * kDr;     // 416

// ---------------------------------------------------------------- decoding
__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// (scale, scale) -> (-136 scale, -136 scale); exact for a stored scale.
__device__ __forceinline__ uint32_t q4_bias(uint32_t s2) { return bf16x2_mul(s2, 0xC308C308u); }
// Codes in bits 0-3 and 16-19 -> their two values.  The and/or is one lop3
// with both constants in registers: as two immediates it became two
// instructions, and the integer pipe (half rate) is what decoding waits for.
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, uint32_t s2, uint32_t bias2) {
    uint32_t v, mask, magic;
    asm("mov.b32 %0, 0x000F000F;" : "=r"(mask));
    asm("mov.b32 %0, 0x43004300;" : "=r"(magic));
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w), "r"(mask), "r"(magic));
    return bf16x2_fma(v, s2, bias2);
}
// One word -> its eight values in order.
__device__ __forceinline__ uint4 q4_word(uint32_t w, uint32_t s2, uint32_t bias2) {
    return make_uint4(q4_pair(w, s2, bias2), q4_pair(w >> 4, s2, bias2), q4_pair(w >> 8, s2, bias2),
                      q4_pair(w >> 12, s2, bias2));
}

// Weak loads that bypass L1 (rows may be written by the kernel this grid is a
// programmatic dependent of; see ld_input).
__device__ __forceinline__ uint4 ld_row16(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
// A group's scale, as loaded; q4_scale2 makes it (scale, scale).  Kept apart: a
// load meant to run ahead must not be followed by arithmetic on its result.
__device__ __forceinline__ uint32_t ld_scale(const uint8_t *p) {
    uint16_t v;
    asm volatile("ld.global.cg.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t q4_scale2(uint32_t scale) { return __byte_perm(scale, scale, 0x1010); }

__device__ __forceinline__ void count_bad_index() {
    atomicOr(&g_status_flags, kFlagIndexRange);
    atomicAdd(&g_bad_index_count, 1ull);
}

// Physical row of position pos of the sequence whose page-table row is pt_b;
// -1 where no page of the pool maps it.
__device__ __forceinline__ long long paged_row(const int *pt_b, int pt_stride, long long num_pages,
                                               long long pos) {
    if (pos < 0 || pos >= (long long)pt_stride * kPage) return -1;
    const int pg = ld_input(pt_b + (int)(pos >> 6));
    return (pg >= 0 && (long long)pg < num_pages) ? (long long)pg * kPage + (pos & (kPage - 1)) : -1;
}

// ---------------------------------------------------------------- quantise and append
struct Q4AppendParams {
    const __nv_bfloat16 *rows;  // [n_rows, 576]
    int n_rows;
    const int *cu_rows;         // [B + 1]: sequence b's rows are [cu_rows[b], cu_rows[b + 1])
    const int *start;           // [B]: position of its first one
    int B;
    const int *page_table;      // [B, pt_stride]
    int pt_stride;
    long long num_pages;
    uint8_t *cache;             // [num_pages * 64, 416]
};

// Smallest number of four significant bits >= a / 7 (a in [2^-118, 2^120), eight
// significant bits).  a / 7 either is such a number or differs from every one of
// them by 2^-12 of itself at least, so a / 7 less 2^-20 of itself (one product,
// its rounding included) lies above exactly the candidates below a / 7; rounding
// its mantissa up to three bits then gives the answer.
__device__ __forceinline__ float q4_scale_of(float a) {
    const uint32_t u = __float_as_uint(__fmul_rn(a, (float)((1.0 - 0x1p-20) / 7.0)));
    return __uint_as_float((u + 0x000FFFFFu) & 0xFFF00000u);
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

constexpr int kQ4Warps = 8;

// x / scale rounded to the nearest integer, ties to even, plus 8: a code, as the
// low bits of kQ4CodeBits + code.  inv is 1 / scale to within 2^-22 of itself, so
// x inv is off by 2^-18 at most (|x / scale| <= 7).  x has eight significant bits and scale
// four, so x / scale is either a half integer or at least 2^-10 away from one:
// rounding to a multiple of 2^-11 first (the fma onto 1.5 * 2^12) gives half
// integers exactly and moves nothing else across one.  The addition then rounds
// to an integer, which stands in the low mantissa bits of 1.5 * 2^23 + code.
// Two float operations where a true division takes about twenty instructions.
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr uint32_t kQ4CodeBits = 0x4B400000u;  // 1.5 * 2^23
__device__ __forceinline__ uint32_t q4_code(float x, float inv) {
    return __float_as_uint(__fadd_rn(__fmaf_rn(x, inv, 6144.f), 12582912.f + 8.f - 6144.f));
}

// One warp per RPW rows, all their loads in flight at once: lane l quantises
// words l and l + 32 of each (eight latents a word, four lanes a group), lanes
// 0-7 also carry its rope values, and the warp finds where the rows go.
// Every access covers whole 128-byte lines.  1152 bytes in, 416 out per row.
// Measured, with the read below behind it: 46080 rows of seven prompts 35.2 us
// (144 MB, 4.1 TB/s, where 6.6 is the most), 64 rows of a decode step 3.7 us.
// Memory latency bounds both: issue slots are 58% and 44% taken, and the bytes in
// flight are what registers hold (69 and 48 a thread).  Rows through shared memory
// by bulk copies, as the moves of an eviction go, were not tried.
template <int RPW>
__global__ void __launch_bounds__(32 * kQ4Warps) smla_q4_append_kernel(const Q4AppendParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long i0 = ((long long)blockIdx.x * kQ4Warps + (threadIdx.x >> 5)) * RPW;
    if (i0 >= p.n_rows) return;
    const int rows = (int)min((long long)RPW, p.n_rows - i0);
    uint4 in[RPW][2], rope[RPW];
#pragma unroll
    for (int k = 0; k < RPW; ++k) {
        const uint4 *src = reinterpret_cast<const uint4 *>(p.rows + (i0 + (k < rows ? k : 0)) * kD);
        in[k][0] = ld_input(src + lane);
        in[k][1] = ld_input(src + 32 + lane);
        rope[k] = ld_input(src + kDc / 8 + (lane & 7));
    }
    // The sequence of row i0, the last one with cu_rows[b] <= i0: the warp tries
    // 32 boundaries at a time, so that up to 32 sequences cost one round trip.
    const int end = ld_input(p.cu_rows + p.B);
    int lo = 0;
    for (int n = p.B; n > 1;) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const bool before = lane * step < n && ld_input(p.cu_rows + at) <= i0;
        const uint32_t v = __ballot_sync(0xffffffffu, before);
        const int k = v ? 31 - __clz(v) : 0;
        n = min(n - k * step, step);
        lo += k * step;
    }
    long long where = -1;  // lane k: row of the pool that row i0 + k goes to
    if (lane < rows && i0 + lane < end) {  // rows behind the last sequence go nowhere
        const long long i = i0 + lane;
        int first = ld_input(p.cu_rows + lo), next = ld_input(p.cu_rows + lo + 1);
        while (i >= next && lo + 1 < p.B) {  // the next sequences may be empty
            ++lo;
            first = next;
            next = ld_input(p.cu_rows + lo + 1);
        }
        if (first >= 0 && first <= i && i < next)
            where = paged_row(p.page_table + (size_t)lo * p.pt_stride, p.pt_stride, p.num_pages,
                              (long long)ld_input(p.start + lo) + (i - first));
        if (where < 0) count_bad_index();
    }
#pragma unroll
    for (int k = 0; k < RPW; ++k) {
        const long long row = __shfl_sync(0xffffffffu, where, k);
        if (row < 0) continue;
        uint8_t *dst = p.cache + row * kQ4RowBytes;
        bool bad = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t v[4] = {in[k][h].x, in[k][h].y, in[k][h].z, in[k][h].w};
            // largest magnitude of the group (bit patterns of magnitudes order
            // as integers, infinities and NaN above every finite value)
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) top = __vmaxu2(top, v[j] & 0x7FFF7FFFu);
            top = max(top & 0xFFFFu, top >> 16);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float most = __uint_as_float(top << 16);
            const bool finite = most < 0x1p120f;
            const bool live = finite && most >= 0x1p-118f;
            bad = bad || !finite;
            const float scale = live ? q4_scale_of(most) : 0.f;
            const float inv = live ? fast_rcp(scale) : 0.f;
            // kQ4CodeBits shifted to every nibble and added up, taken off beforehand
            uint32_t w = 0u - kQ4CodeBits * 0x11111111u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = finite ? v[j] : 0u;  // (inf * 0 would be no code)
                w += q4_code(bf16_lo(x), inv) << (4 * j);
                w += q4_code(bf16_hi(x), inv) << (4 * j + 16);
            }
            *reinterpret_cast<uint32_t *>(dst + 128 * h + 4 * lane) = w;
            if ((lane & 3) == 0)
                *reinterpret_cast<uint16_t *>(dst + kQ4OffScale + 16 * h + (lane >> 1)) =
                    (uint16_t)(__float_as_uint(scale) >> 16);
        }
        const bool poison = __any_sync(0xffffffffu, bad);
        if (lane < 8)
            *reinterpret_cast<uint4 *>(dst + kQ4OffRope + 16 * lane) =
                poison ? make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu) : rope[k];
    }
}

// ---------------------------------------------------------------- read back
struct Q4ReadParams {
    const uint8_t *cache;   // [num_pages * 64, 416]
    long long num_pages;
    const int *page_table;  // [B, pt_stride]
    int pt_stride;
    const int *positions;   // [B, K], -1 = none
    int B, K;
    __nv_bfloat16 *out;     // [B, K, 576]
};

// One warp per RPW listed positions, all their loads in flight at once: lane l
// decodes words l and l + 32 of each, lanes 0-7 copy the rope values.  416 bytes
// in, 1152 out per row (measured with the append above).
template <int RPW>
__global__ void __launch_bounds__(32 * kQ4Warps) smla_q4_read_kernel(const Q4ReadParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long n = (long long)p.B * p.K;
    const long long i0 = ((long long)blockIdx.x * kQ4Warps + (threadIdx.x >> 5)) * RPW;
    if (i0 >= n) return;
    long long where = -1;
    if (lane < RPW && i0 + lane < n) {
        const long long i = i0 + lane;
        const int pos = ld_input(p.positions + i);
        if (pos != -1) {
            where = paged_row(p.page_table + (size_t)(i / p.K) * p.pt_stride, p.pt_stride, p.num_pages, pos);
            if (where < 0) count_bad_index();
        }
    }
    uint32_t w[RPW][2], scale[RPW][2];
    uint4 rope[RPW];
#pragma unroll
    for (int k = 0; k < RPW; ++k) {
        const long long row = __shfl_sync(0xffffffffu, where, k);
        rope[k] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[k][h] = scale[k][h] = 0u;  // no row: zeros
            if (row >= 0) {
                const uint8_t *src = p.cache + row * kQ4RowBytes;
                asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(w[k][h]) : "l"(src + 128 * h + 4 * lane));
                scale[k][h] = ld_scale(src + kQ4OffScale + 16 * h + 2 * (lane >> 2));
            }
        }
        if (row >= 0) rope[k] = ld_row16(p.cache + row * kQ4RowBytes + kQ4OffRope + 16 * (lane & 7));
    }
#pragma unroll
    for (int k = 0; k < RPW; ++k) {
        if (i0 + k >= n) break;
        uint4 *dst = reinterpret_cast<uint4 *>(p.out + (i0 + k) * kD);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t s2 = q4_scale2(scale[k][h]);
            dst[32 * h + lane] = q4_word(w[k][h], s2, q4_bias(s2));
        }
        if (lane < 8) dst[kDc / 8 + lane] = rope[k];
    }
}

// Rows per warp: four keep more loads in flight, once there are rows enough
// for every SM to hold several such warps; below that, one row per warp has the
// shorter chain.  (Append + read, us, with one row per warp: 512 rows 1.9 + 1.9,
// 4736 2.7 + 2.7, 9472 3.9 + 3.6, 14208 5.4 + 4.5, 18944 6.6 + 5.6, 28416 9.3 +
// 7.4, 46080 14.4 + 11.1; with four: 2.9 + 2.5, 3.1 + 2.5, 4.6 + 4.3, 4.9 + 4.9, 6.4
// + 5.8, 8.0 + 7.0, 12.3 + 10.1; rows in L2.  18944 is where four begin.)
__host__ inline bool q4_many_rows(long long rows, int sms) { return rows >= (long long)sms * kQ4Warps * 4 * 4; }

}  // namespace smla

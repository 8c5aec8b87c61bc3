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
__device__ __forceinline__ uint2 ld_row8(const uint8_t *p) {
    uint2 v;
    asm volatile("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
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

// Smallest number of four significant bits >= a / 7 (a in [2^-118, 2^120)).
// a and 7 s are multiples of a common step that is at least 2^-12 of them, so
// the correctly rounded quotient is above, at or below a candidate exactly
// when the real one is.
__device__ __forceinline__ float q4_scale_of(float a) {
    const uint32_t u = __float_as_uint(__fdiv_rn(a, 7.f));
    return __uint_as_float((u + 0x000FFFFFu) & 0xFFF00000u);
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

constexpr int kQ4Warps = 8;  // rows per CTA, one warp each

// One warp per row: lane l quantises latents 16 l .. 16 l + 15 (half a group),
// lanes 0-7 also carry the rope values.  Bound by memory: 1152 bytes in, 416
// out per row.
__global__ void __launch_bounds__(32 * kQ4Warps) smla_q4_append_kernel(const Q4AppendParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long i = (long long)blockIdx.x * kQ4Warps + (threadIdx.x >> 5);
    if (i >= p.n_rows) return;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.rows + i * kD);
    const uint4 a = ld_input(src + 2 * lane), b4 = ld_input(src + 2 * lane + 1);
    uint4 rope = make_uint4(0u, 0u, 0u, 0u);
    if (lane < 8) rope = ld_input(src + kDc / 8 + lane);
    if (i >= ld_input(p.cu_rows + p.B)) return;  // rows behind the last sequence
    int lo = 0, hi = p.B - 1;                    // the last sequence with cu_rows[b] <= i
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ld_input(p.cu_rows + mid) <= i) lo = mid; else hi = mid - 1;
    }
    const int first = ld_input(p.cu_rows + lo);
    long long row = -1;
    if (first >= 0 && first <= i && i < ld_input(p.cu_rows + lo + 1))
        row = paged_row(p.page_table + (size_t)lo * p.pt_stride, p.pt_stride, p.num_pages,
                        (long long)ld_input(p.start + lo) + (i - first));
    if (row < 0) {
        if (lane == 0) count_bad_index();
        return;
    }
    const uint32_t v[8] = {a.x, a.y, a.z, a.w, b4.x, b4.y, b4.z, b4.w};
    // largest magnitude of the group (bit patterns of magnitudes order as
    // integers, infinities and NaN above every finite value)
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, max(v[k] & 0x7FFFu, (v[k] >> 16) & 0x7FFFu));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const float most = __uint_as_float(top << 16);
    const bool bad = !(most < 0x1p120f);
    const bool live = !bad && most >= 0x1p-118f;
    const float scale = live ? q4_scale_of(most) : 0.f;
    uint32_t w[2] = {0x88888888u, 0x88888888u};
    if (live) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            w[k] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c0 = (int)rintf(__fdiv_rn(bf16_lo(v[4 * k + j]), scale)) + 8;
                const int c1 = (int)rintf(__fdiv_rn(bf16_hi(v[4 * k + j]), scale)) + 8;
                w[k] |= (uint32_t)c0 << (4 * j) | (uint32_t)c1 << (4 * j + 16);
            }
        }
    }
    uint8_t *dst = p.cache + row * kQ4RowBytes;
    *reinterpret_cast<uint2 *>(dst + 8 * lane) = make_uint2(w[0], w[1]);
    if ((lane & 1) == 0)
        *reinterpret_cast<uint16_t *>(dst + kQ4OffScale + lane) = (uint16_t)(__float_as_uint(scale) >> 16);
    if (__any_sync(0xffffffffu, bad)) rope = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
    if (lane < 8) *reinterpret_cast<uint4 *>(dst + kQ4OffRope + 16 * lane) = rope;
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

// One warp per listed position: lane l decodes latents 16 l .. 16 l + 15,
// lanes 0-7 copy the rope values.  Bound by memory: 416 bytes in, 1152 out.
__global__ void __launch_bounds__(32 * kQ4Warps) smla_q4_read_kernel(const Q4ReadParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long i = (long long)blockIdx.x * kQ4Warps + (threadIdx.x >> 5);
    if (i >= (long long)p.B * p.K) return;
    const int pos = ld_input(p.positions + i);
    long long row = -1;
    if (pos != -1) {
        row = paged_row(p.page_table + (size_t)(i / p.K) * p.pt_stride, p.pt_stride, p.num_pages, pos);
        if (row < 0 && lane == 0) count_bad_index();
    }
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo, rope = lo;
    if (row >= 0) {
        const uint8_t *src = p.cache + row * kQ4RowBytes;
        const uint2 w = ld_row8(src + 8 * lane);
        const uint32_t s2 = q4_scale2(ld_scale(src + kQ4OffScale + (lane & ~1)));
        if (lane < 8) rope = ld_row16(src + kQ4OffRope + 16 * lane);
        const uint32_t bias = q4_bias(s2);
        lo = q4_word(w.x, s2, bias);
        hi = q4_word(w.y, s2, bias);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + i * kD);
    dst[2 * lane] = lo;
    dst[2 * lane + 1] = hi;
    if (lane < 8) dst[kDc / 8 + lane] = rope;
}

}  // namespace smla

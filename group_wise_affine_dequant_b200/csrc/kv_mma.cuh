// Code -> fp16 converters of the attention kernels. fp16 holds every int8 and
// E4M3 code exactly and rounds a softmax weight to 11 bits (bf16: 8), so both
// products run in fp16: keys times queries scaled by a power of two, weights
// times values.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "kv.cuh"
#include "tc_common.cuh"

namespace nvq {

// (v0, v1) of the low or high two bytes of w as a half2.
//   int8: 1024 + (c ^ 0x80) is an fp16 whose low byte is c + 128; subtracting 1152 is exact.
//   E4M3: the hardware conversion, exact.
template <int MODE>
__device__ __forceinline__ uint32_t prepare_word(uint32_t w) {
    return MODE == NV_KV_INT8 ? w ^ 0x80808080u : w;
}
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <int MODE>
__device__ __forceinline__ uint32_t pair_lo_h2(uint32_t w) {  // w after prepare_word
    if constexpr (MODE == NV_KV_INT8) {
        return h2_sub(tc::prmt(w, 0x64646464u, 0x4140), 0x64806480u);
    } else {
        uint32_t d;
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(w));
        return d;
    }
}
template <int MODE>
__device__ __forceinline__ uint32_t pair_hi_h2(uint32_t w) {
    if constexpr (MODE == NV_KV_INT8) {
        return h2_sub(tc::prmt(w, 0x64646464u, 0x4342), 0x64806480u);
    } else {
        uint32_t d;
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(d) : "r"(w));
        return d;
    }
}
__device__ __forceinline__ uint32_t f2_to_h2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A query row's power of two: with ex = the biased exponent of its largest magnitude, q *
// 2^(127 - ex) is below 2 and exact in fp16 down to 2^-24. Rows of 2^7 and more come out up to 2^15
// (fp16 ends at 2^16) instead, so that what their scores get back times the scale of keys near the largest
// number stays finite: where the codes beside such a key are 0, so are their scores. Rows below
// 2^-119 come out as multiples of 2^-14, which their last bit is. Both powers of two are normal fp32 numbers.
__device__ __forceinline__ uint32_t row_exponent(uint32_t max_abs_bits) {
    const uint32_t ex = max_abs_bits >> 23;
    return ex < 8u ? 8u : ex <= 133u ? ex : ex <= 147u ? 133u : ex <= 254u ? ex - 14u : 240u;
}
__device__ __forceinline__ float pow2_bits(uint32_t biased) { return __uint_as_float(biased << 23); }

// Weights are kept as 2^(z + lg - M + kLift): lg = log2 of the block's value
// scale over the item's largest, M a reference that the running maximum of
// z + lg may pass by kSlack before the sums are rescaled. So weights reach at most
// 2^15 in fp16 and lose bits only 2^-(14 + kLift) below the reference.
// The sum of weights without value scales adds w * 2^-lg.
// Blocks of zeros take lg = kLgZero: such weights are far below every other's, yet their part of
// that sum is kept wherever it matters (2^-54 of it is lost at most) and does not overflow it.
// Where value scales are further apart than 2^kLgWide, the smaller blocks' weights have no bits beside those of a
// block whose codes are zeros next to one large value (in another column, or not seen). Such items are
// wide and go row by row through plain_row. (2^24 apart, 2^-33 of the larger is 2^-9 of the smaller: bf16's rounding.)
constexpr float kLift = 8.f, kSlack = 7.f, kLgZero = -80.f, kLgWide = -24.f;
constexpr float kLog2e = 1.4426950408889634f;

// One block's constants in shared memory.
struct BlockScales {
    float ks;      // key scale; negative: the page is out of range, the block is not seen
    float lg;      // log2(value scale / largest of the item), kLgZero where the scale is 0
    float inv;     // 2^-lg
    int page;
};

}  // namespace nvq

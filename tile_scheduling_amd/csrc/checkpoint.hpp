// Rows kept in 8 bits: what a forward pass keeps for its backward pass.
//
//   32 neighbours of a row are a block, with one step 2^e: e the least for which the largest of
//   them is at most 127 steps, rounded; a value is round(x / 2^e) steps, off by half a step at most.
//   A row of N: 32 ceil(N / 32) int8 values (zero behind column N), then one byte e + 127 for
//   each block.  255: the block held an infinity or a NaN, and all of it stands for NaN.
//
// A power of two divides exactly, so every kernel that forms a block forms the same bytes, in 2
// instructions a value; the least step is 2^-126, and below half of it a value becomes zero.  Blocks
// of 32 keep the step near the values (of normal ones a block's largest is 2.1 deviations, a row's of
// 4096 3.7 or an outlier) and are a lane pair's share of a 32 x 32 accumulator block.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ts {

constexpr int kBlock = 32;
// Bytes of values in a row, which is where its exponents begin, and of the whole row.
__host__ __device__ constexpr long long kept_values(long long n) { return (n + kBlock - 1) / kBlock * kBlock; }
__host__ __device__ constexpr long long kept_row(long long n) { return kept_values(n) + kept_values(n) / kBlock; }

// The exponent byte of a block from the bits of its largest |x| (a NaN's are above infinity's).
// Largest values from 127.5 / 128 of a power of two on would round to 128 steps: they carry over.
__device__ __forceinline__ uint32_t block_exponent(uint32_t max_bits) {
    const uint32_t e = (max_bits + 0x10000u) >> 23;
    return max_bits >= 0x7f800000u ? 255u : e > 7u ? e - 6u : 1u;
}
// 2^-e of an exponent byte, 0 for a block without a step.
__device__ __forceinline__ float step_inverse(uint32_t e) { return __builtin_bit_cast(float, e == 255u ? 0u : (254u - e) << 23); }
// 2^e, NaN for a block without a step.
__device__ __forceinline__ float step_of(uint32_t e) { return __builtin_bit_cast(float, e == 255u ? 0x7fc00000u : e << 23); }

// Four values as bytes: adding 1.5 2^23 leaves the nearest whole number (ties to even) in the low
// bits, in two's complement.  The product is exact, so this is the one rounding.  (In a block without a
// step the bytes are anything.)
__device__ __forceinline__ uint32_t kept_pack4(const float* x, float inv) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __builtin_bit_cast(uint32_t, __builtin_fmaf(x[i], inv, 12582912.0f));
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
    return lo | hi;
}
__device__ __forceinline__ void kept_unpack4(uint32_t w, float step, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w >> (8 * i)) * step;
}
// A block whose largest value lies between 255/256 of a power of two and the power keeps it as the power,
// 64 steps, which its type does not hold where it is the type's last: 2^128 of bf16 and fp32, 2^16 of fp16.  2^128
// is read as the largest bf16 number, that border itself and a quarter of a step below, and by kernels that write fp16
// (F16) 2^16 as the largest fp16 number: finite rows come back finite, within half a step.
constexpr float kLastStep = 0x1p122f, kLastValue = 0x1.fep127f, kLastStepF16 = 0x1p10f, kLastValueF16 = 65504.0f;
template <int E, bool F16>
__device__ __forceinline__ void kept_last(float step, float* v) {
    if (step == kLastStep || (F16 && step == kLastStepF16)) {
        const bool f16 = step != kLastStep;
        const float power = f16 ? 0x1p16f : __builtin_inff(), last = f16 ? kLastValueF16 : kLastValue;
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = __builtin_fabsf(v[i]) == power ? __builtin_copysignf(last, v[i]) : v[i];
    }
}
// The step for values that only slopes are formed of, which do not change any more that far out: 2^121 in place of
// 2^122 keeps them finite, without a branch (in the products' epilogue kept_last costs 10 us of 490, 4096 x 16384 x 4096).
__device__ __forceinline__ float slope_step_of(uint32_t e) { return step_of(e == 255u || e < 248u ? e : 248u); }
// Largest over lanes l, l ^ 1, l ^ 2, l ^ 3.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    const uint32_t a = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true);   // 1 0 3 2
    v = a > v ? a : v;
    const uint32_t b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true);   // 2 3 0 1
    return b > v ? b : v;
}
// Larger of lanes l and l ^ 32.
__device__ __forceinline__ uint32_t halves_max(uint32_t v) {
    // the upper half of the first operand changes places with the lower half of the second
    const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return s[0] > s[1] ? s[0] : s[1];
}
// Eight columns n .. n + 7 of a row (n a multiple of 8) whose exponents begin at `values`; none
// where n is at or behind N.
struct Kept8 {
    uint32_t w[2], e;
    __device__ __forceinline__ void load(const uint8_t* row, long long values, long long n, bool any) {
        w[0] = w[1] = 0;
        e = 1;
        if (any) {
            const uint2 t = *reinterpret_cast<const uint2*>(row + n);
            w[0] = t.x;
            w[1] = t.y;
            e = row[values + n / kBlock];
        }
    }
    template <bool F16 = false>
    __device__ __forceinline__ void unpack(float* v) const {
        const float step = step_of(e);
        kept_unpack4(w[0], step, v);
        kept_unpack4(w[1], step, v + 4);
        kept_last<8, F16>(step, v);
    }
};

}  // namespace ts

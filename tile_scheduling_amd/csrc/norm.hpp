// What the kernels over rows share: 8-bit outputs with a scale per row, shapes of workgroups, launches.
#pragma once

#include <hip/hip_runtime.h>

#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/tsgemm.h"
#include "plan.hpp"
#include "rows.hpp"

namespace ts {

// 8-bit outputs with a scale per row.
enum : int { Q_NONE = 0, Q_E4M3 = 1, Q_I8 = 2 };
constexpr float kE4M3Max = 448.0f, kInt8Max = 127.0f;
constexpr float kMinScale = 0x1p-100f;   // keeps 1 / scale finite; rows of zeros take it

// Eight floats to e4m3 (round to nearest even; |v| <= 448 up to the rounding of the scale,
// which rounds back to 448).
__device__ __forceinline__ u32x2 pack8_e4m3(const float* v) {
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
    return u32x2{(uint32_t)lo, (uint32_t)hi};
}
// Eight floats of at most 127 to int8: adding 1.5 2^23 leaves the nearest whole number (ties to even)
// in the low byte.
__device__ __forceinline__ u32x2 pack8_i8(const float* v) {
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = __builtin_bit_cast(uint32_t, v[e] + 12582912.0f);
    u32x2 w;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w[h] = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0c0c0400u) | __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000c0cu);
    return w;
}
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
template <int Q>
__device__ __forceinline__ void store8_q(uint8_t* p, int valid, const float* v) {
    const u32x2 w = Q == Q_I8 ? pack8_i8(v) : pack8_e4m3(v);
    if (valid >= 8) {
        *reinterpret_cast<u32x2_a1*>(p) = w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) p[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
}
// Largest |v| as its bits, so that a NaN wins.
__device__ __forceinline__ uint32_t max8_bits(const float* v, uint32_t m) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v[e]) & 0x7fffffffu;
        m = b > m ? b : m;
    }
    return m;
}
template <int Q>
__device__ __forceinline__ float row_scale(uint32_t max_bits) {
    const float s = __builtin_bit_cast(float, max_bits) / (Q == Q_I8 ? kInt8Max : kE4M3Max);
    return s < kMinScale ? kMinScale : s;   // NaN stays NaN
}

// y / scale with one rounding: the product with the reciprocal, off by up to a step and a half of
// fp32, and one correction by its remainder.  (The product alone puts values next to the middle between
// two e4m3 numbers on the wrong side.)  An infinite scale has the reciprocal 0 and no remainder, so
// that finite values become 0.
struct Quotient {
    float inv, scale;
    __device__ __forceinline__ explicit Quotient(float s)
        : inv(1.0f / s), scale(s > 3.4028234e38f ? 0.0f : s) {}
    __device__ __forceinline__ float operator()(float v) const {
        const float q = v * inv;
        return __builtin_fmaf(__builtin_fmaf(-q, scale, v), inv, q);
    }
};

constexpr int kLongThreads = 1024;   // a workgroup of rows too long for its registers

// Shapes of the register kernels: threads a row and groups of eight columns a thread.
struct Shape {
    int t, c;
};

// Fewest threads a row whose four groups cover it; with few rows (fewer than would give
// every CU a workgroup) one group a thread where the workgroup allows it.  {0, 0}: a long
// row.
inline Shape norm_shape(int64_t M, int64_t N, int most) {
    const int64_t groups = (N + 7) / 8;
    static const int kThreads[] = {16, 64, 256, 1024};
    for (int t : kThreads) {
        const int limit = t == 1024 ? most : 4;
        const int want = t < 1024 && M * t < 256 * 256 ? 1 : limit;
        if (groups > (int64_t)t * want) continue;
        int c = 1;
        while ((int64_t)t * c < groups) c *= 2;
        return Shape{t, c};
    }
    return Shape{0, 0};
}

inline bool row_type(int32_t t) { return t == TS_F16 || t == TS_BF16 || t == TS_F32; }
inline int type_size(int32_t t) { return t == TS_F32 ? 4 : t == TS_E4M3 || t == TS_I8 || t == TS_Q8 ? 1 : 2; }

inline ts_status norm_sizes(int64_t M, int64_t N) {
    if (M < 0 || N < 0) return TS_ERR_INVALID_ARG;
    if (M > INT_MAX / 2 || N >= 1 << 26) return TS_ERR_UNSUPPORTED;   // N: threads of the launches over columns
    return TS_OK;
}

inline ts_status have_device() {
    int dev;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return TS_ERR_NO_DEVICE;
    }
    return TS_OK;
}

inline ts_status launch(const void* fn, int64_t gx, int64_t gy, int threads, void* args, hipStream_t stream) {
    void* argv[] = {args};
    return enqueue(fn, gx, threads, argv, stream, gy) ? TS_OK : TS_ERR_HIP;
}

// One workgroup for every few rows: a launch holds fewer than 2^32 threads, so many rows take
// more than one.
template <class Args>
ts_status launch_rows(const void* fn, int64_t blocks, int threads, Args& g, hipStream_t stream) {
    const int64_t most = (1LL << 31) / threads;
    for (g.first = 0; g.first < blocks; g.first += most) {
        const ts_status st = launch(fn, std::min<int64_t>(blocks - g.first, most), 1, threads, &g, stream);
        if (st != TS_OK) return st;
    }
    return TS_OK;
}

}  // namespace ts

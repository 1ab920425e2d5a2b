// What layer norm and its gradients share.
#pragma once

#include <hip/hip_runtime.h>

#include "checkpoint.hpp"
#include "norm.hpp"

namespace ts {

// Sums of K values over the T threads of a row, as row_sum; one pair of barriers for all of them.
template <int T, int K>
__device__ __forceinline__ void row_sums(float* v, float (*lds)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lanes_sum<(T < 64 ? T : 64)>(v[k]);
    if constexpr (T > 64) {
        __syncthreads();   // the words' last readers are done
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) lds[threadIdx.x >> 6][k] = v[k];
        }
        __syncthreads();
        // a lane takes one wave's words (all of them in every lane: 16 waves' cost 16 K registers)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = lanes_sum<T / 64>(lds[threadIdx.x & (T / 64 - 1)][k]);
    }
}
// 1 / deviation from the sums of d and d^2; a variance that rounds below zero is zero (NaN stays).
__device__ __forceinline__ float inverse_deviation(float sd, float sdd, float n, float eps) {
    const float e = sd / n, var = __builtin_fmaf(-e, e, sdd / n);
    return 1.0f / __builtin_sqrtf((var < 0.0f ? 0.0f : var) + eps);
}
// Weight or bias of eight columns; `none` where there is no vector.
template <class TX>
__device__ __forceinline__ void columns8(const void* p, int type, long long n, int valid, float none, float* v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = none;
    if (p) load8_vec<TX>(p, type, n, valid, v);
}

// Eight columns of a row as they lie in memory.
template <class TX>
struct Raw8 {
    u32x4 v[Elt<TX>::E == 8 ? 1 : 2];
    __device__ __forceinline__ void load(const void* base, long long m, long long ld, long long n, int N, int valid) {
        (void)N;
        const typename Elt<TX>::T* p = static_cast<const typename Elt<TX>::T*>(base) + m * ld + n;
        v[0] = load_row<TX>(p, valid);
        if constexpr (Elt<TX>::E == 4) v[1] = load_row<TX>(p + 4, valid - 4);
    }
    // Values unpacked before are not held in registers until the next time.
    __device__ __forceinline__ void renew() {
        if constexpr (Elt<TX>::E == 8) asm volatile("" : "+v"(v[0]));
    }
    __device__ __forceinline__ void unpack(float* f, int valid) const {
        (void)valid;
        unpack_row<TX>(v[0], f);
        if constexpr (Elt<TX>::E == 4) unpack_row<TX>(v[1], f + 4);
    }
};
struct RawKept {
    Kept8 k;
    __device__ __forceinline__ void load(const void* base, long long m, long long ld, long long n, int N, int valid) {
        k.load(static_cast<const uint8_t*>(base) + m * ld, kept_values(N), n, valid > 0);
    }
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(k.w[0]), "+v"(k.w[1])); }
    __device__ __forceinline__ void unpack(float* f, int valid) const {
        k.unpack(f);
        if (valid < 8) {   // whatever lies behind column N
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = e < valid ? f[e] : 0.0f;
        }
    }
};
}  // namespace ts

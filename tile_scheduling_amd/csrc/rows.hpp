// Groups of eight columns of a row, and sums over rows and columns: shared by the norm and
// the activation gradient.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "epilogue.hpp"

namespace ts {

// Whether an output at `out` may lie on an input at `in`: not on it at all, or element on element
// (each is read before it is written, by the same thread), so of one type and row stride.
inline bool in_place_ok(const void* out, const void* in, bool same_type, int64_t M, int64_t ld_out, int64_t ld_in) {
    return !out || out != in || (same_type && (M <= 1 || ld_out == ld_in));
}

// Eight consecutive elements of a row <-> eight floats, whatever the type: one 16-byte
// access (two for fp32) at element alignment; `valid` < 8 at the end of a row.
template <class TO>
__device__ __forceinline__ void load8(const typename Elt<TO>::T* p, int valid, float* v) {
    if constexpr (Elt<TO>::E == 8) {
        unpack_row<TO>(load_row<TO>(p, valid), v);
    } else {
        unpack_row<TO>(load_row<TO>(p, valid), v);
        unpack_row<TO>(load_row<TO>(p + 4, valid - 4), v + 4);
    }
}
template <class TO>
__device__ __forceinline__ void store8(typename Elt<TO>::T* p, int valid, const float* v) {
    store_row<TO>(p, pack_row<TO>(v), valid);
    if constexpr (Elt<TO>::E == 4) store_row<TO>(p + 4, pack_row<TO>(v + 4), valid - 4);
}
// Eight elements of a vector of either the rows' type or fp32.
template <class TO>
__device__ __forceinline__ void load8_vec(const void* p, int type, long long i, int valid, float* v) {
    if (type == ELT_F32)
        load8<OutF32>(static_cast<const float*>(p) + i, valid, v);
    else
        load8<TO>(static_cast<const typename Elt<TO>::T*>(p) + i, valid, v);
}
__device__ __forceinline__ void store_any(void* p, int type, long long i, float v) {
    if (type == ELT_F32) static_cast<float*>(p)[i] = v;
    else if (type == ELT_F16) static_cast<_Float16*>(p)[i] = (_Float16)v;
    else static_cast<__bf16*>(p)[i] = (__bf16)v;
}

// Butterfly sums and maxima over T lanes (T a power of two up to 64): every lane ends with
// the same bits.
template <int T>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = T / 2; d > 0; d /= 2) v += __shfl_xor(v, d, 64);
    return v;
}
template <int T>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
    for (int d = T / 2; d > 0; d /= 2) {
        const uint32_t o = __shfl_xor(v, d, 64);
        v = o > v ? o : v;
    }
    return v;
}
// The same over the T threads of a row (T <= 64: a part of a wave; else the workgroup, through
// `lds`, T / 64 words, between two barriers).
template <int T>
__device__ __forceinline__ float row_sum(float v, float* lds) {
    v = lanes_sum<(T < 64 ? T : 64)>(v);
    if constexpr (T > 64) {
        __syncthreads();   // the words' last readers are done
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = lds[0];
#pragma unroll
        for (int w = 1; w < T / 64; ++w) v += lds[w];
    }
    return v;
}
template <int T>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float* lds) {
    v = lanes_max<(T < 64 ? T : 64)>(v);
    if constexpr (T > 64) {
        uint32_t* l = reinterpret_cast<uint32_t*>(lds);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) l[threadIdx.x >> 6] = v;
        __syncthreads();
        v = l[0];
#pragma unroll
        for (int w = 1; w < T / 64; ++w) v = l[w] > v ? l[w] : v;
    }
    return v;
}

// Column sums of `rows` fp32 rows of N (the partial sums of workgroups, in their order) into
// N elements of any type.  A workgroup takes 16 columns (with 64, too few workgroups for short
// rows: 1024 rows of 4096 17.3 us, now 6); 64 lanes take every 64th row of a column and are added in a
// fixed order, so the result does not depend on timing.
__global__ void reduce_columns_kernel(const float* part, int rows, int N, void* out, int type);

// Enqueues reduce_columns_kernel; false if that failed.
bool launch_reduce_columns(const float* part, int rows, int N, void* out, int type, hipStream_t stream);

}  // namespace ts

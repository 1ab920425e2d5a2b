// Rows into 8 bits and back (checkpoint.hpp): what a forward pass keeps, and what the backward pass
// makes of it.  Both are bound by memory: a thread takes 16 columns, half a block, in 16-byte accesses.
// 4096 x 16384 bf16 packed 41 us (203 MB, 5.0 TB/s).
#include <hip/hip_runtime.h>

#include "checkpoint.hpp"
#include "norm.hpp"

namespace ts {

struct CheckpointArgs {
    const void* in;
    void* out;
    int M, N, act;
    uint32_t halves;        // 16 columns each, of a row
    long long ld_in, ld_out;
    long long first;        // row of the launch's first workgroup
    uint32_t rows;          // rows of the launch
};
__device__ __forceinline__ bool half_of(const CheckpointArgs& g, long long* m, int* n) {
    const uint32_t id = blockIdx.x * 256u + threadIdx.x, r = id / g.halves;
    *m = g.first + r;
    *n = 16 * (int)(id - r * g.halves);
    return r < g.rows;
}

template <class TX>
__global__ void __launch_bounds__(256) checkpoint_pack_kernel(CheckpointArgs g) {
    typedef typename Elt<TX>::T X;
    long long m;
    int n;
    if (!half_of(g, &m, &n)) return;   // whole blocks: their two lanes stay or go together
    const X* x = static_cast<const X*>(g.in) + m * g.ld_in + n;
    float v[16];
    load8<TX>(x, g.N - n, v);
    load8<TX>(x + 8, g.N - n - 8, v + 8);
    uint32_t most = max8_bits(v + 8, max8_bits(v, 0));
    const uint32_t other = (uint32_t)__builtin_amdgcn_mov_dpp((int)most, 0xb1, 0xf, 0xf, true);   // the block's other half
    const uint32_t e = block_exponent(other > most ? other : most);
    const float inv = step_inverse(e);
    uint8_t* row = static_cast<uint8_t*>(g.out) + m * g.ld_out;
    *reinterpret_cast<u32x4*>(row + n) = u32x4{kept_pack4(v, inv), kept_pack4(v + 4, inv), kept_pack4(v + 8, inv), kept_pack4(v + 12, inv)};
    if (n % kBlock == 0) row[kept_values(g.N) + n / kBlock] = (uint8_t)e;
}

template <class TY>
__global__ void __launch_bounds__(256) checkpoint_unpack_kernel(CheckpointArgs g) {
    typedef typename Elt<TY>::T Y;
    long long m;
    int n;
    if (!half_of(g, &m, &n)) return;
    const uint8_t* row = static_cast<const uint8_t*>(g.in) + m * g.ld_in;
    const u32x4 w = *reinterpret_cast<const u32x4*>(row + n);
    const float step = step_of(row[kept_values(g.N) + n / kBlock]);
    float v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) kept_unpack4(w[i], step, v + 4 * i);
    kept_last<16, std::is_same<TY, OutF16>::value>(step, v);
    act_values<16>(g.act, v);
    Y* y = static_cast<Y*>(g.out) + m * g.ld_out + n;
    store8<TY>(y, g.N - n, v);
    store8<TY>(y + 8, g.N - n - 8, v + 8);
}

namespace {

ts_status run(const void* fn, CheckpointArgs& g, hipStream_t stream) {
    g.halves = (uint32_t)(kept_values(g.N) / 16);
    // threads are counted in 31 bits
    const int64_t most = std::max<int64_t>(1, ((1LL << 31) - 256) / g.halves);
    for (g.first = 0; g.first < g.M; g.first += most) {
        g.rows = (uint32_t)std::min<int64_t>(g.M - g.first, most);
        const ts_status st = launch(fn, ((int64_t)g.rows * g.halves + 255) / 256, 1, 256, &g, stream);
        if (st != TS_OK) return st;
    }
    return TS_OK;
}

ts_status check(const void* x, const void* kept, int64_t M, int64_t N, int64_t stride_x, int64_t stride_kept, int32_t dtype) {
    if (!x || !kept || x == kept) return TS_ERR_INVALID_ARG;
    if (M > 1 && (stride_x < N || stride_kept < kept_row(N) || stride_kept % 16 != 0)) return TS_ERR_INVALID_ARG;
    if ((uintptr_t)x % type_size(dtype) || (uintptr_t)kept % 16) return TS_ERR_ALIGNMENT;
    return have_device();
}

}  // namespace
}  // namespace ts

using namespace ts;

extern "C" int64_t ts_checkpoint_row_bytes(int64_t N) {
    if (N < 0) return TS_ERR_INVALID_ARG;
    if (N >= 1 << 26) return TS_ERR_UNSUPPORTED;
    return (kept_row(N) + 15) / 16 * 16;
}

extern "C" ts_status ts_checkpoint_pack(const void* x, void* kept, int64_t M, int64_t N, int64_t stride_x,
                                        int64_t stride_kept, int32_t x_dtype, void* stream) {
    ts_status st = norm_sizes(M, N);
    if (st != TS_OK) return st;
    if (!row_type(x_dtype)) return TS_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return TS_OK;
    st = check(x, kept, M, N, stride_x, stride_kept, x_dtype);
    if (st != TS_OK) return st;
    CheckpointArgs g = {x, kept, (int)M, (int)N, 0, 0, stride_x, stride_kept, 0, 0};
    const void* fn = x_dtype == TS_F16    ? reinterpret_cast<const void*>(&checkpoint_pack_kernel<OutF16>)
                     : x_dtype == TS_BF16 ? reinterpret_cast<const void*>(&checkpoint_pack_kernel<OutBF16>)
                                          : reinterpret_cast<const void*>(&checkpoint_pack_kernel<OutF32>);
    return run(fn, g, static_cast<hipStream_t>(stream));
}

extern "C" ts_status ts_checkpoint_unpack(const void* kept, void* y, int64_t M, int64_t N, int64_t stride_kept,
                                          int64_t stride_y, int32_t y_dtype, int32_t activation, void* stream) {
    ts_status st = norm_sizes(M, N);
    if (st != TS_OK) return st;
    if (!row_type(y_dtype) || activation < TS_ACT_NONE || activation > TS_ACT_SILU) return TS_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return TS_OK;
    st = check(y, kept, M, N, stride_y, stride_kept, y_dtype);
    if (st != TS_OK) return st;
    CheckpointArgs g = {kept, y, (int)M, (int)N, activation, 0, stride_kept, stride_y, 0, 0};
    const void* fn = y_dtype == TS_F16    ? reinterpret_cast<const void*>(&checkpoint_unpack_kernel<OutF16>)
                     : y_dtype == TS_BF16 ? reinterpret_cast<const void*>(&checkpoint_unpack_kernel<OutBF16>)
                                          : reinterpret_cast<const void*>(&checkpoint_unpack_kernel<OutF32>);
    return run(fn, g, static_cast<hipStream_t>(stream));
}

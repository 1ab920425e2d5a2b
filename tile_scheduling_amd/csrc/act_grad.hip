// Gradient of the fused epilogue in front of the two products of the backward pass:
//   dZ = dC * act'(Z)   and   dbias = column sums of dZ,
// both from one read of dC and Z.  The column sums are taken over the unrounded fp32
// products: each workgroup sums its rows of a strip of 256 columns into one partial row,
// and a second small launch adds the partial rows in order (no atomics: the same bits on
// every run); up to 16 rows are one group, whose sums are dbias itself.  Bound by memory:
// 4096 x 8192 bf16 42 us (201 MB, 4.8 TB/s), and 4.7 us for the second launch.
// KEPT: Z in 8 bits (checkpoint.hpp).  VALUE: act(Z) too, an operand of the next weight's gradient, which
// the forward pass then need not keep.  Both: 4096 x 16384 bf16 104 us (489 MB, 4.7 TB/s).
#include <hip/hip_runtime.h>

#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/tsgemm.h"
#include "checkpoint.hpp"
#include "plan.hpp"
#include "rows.hpp"

namespace ts {

struct ActGradArgs {
    const void *dc, *z;
    void* dz;       // or null
    float* part;    // one row of N per row group, or null
    void* dbias;    // with one row group: the sums themselves, or null
    int M, N, act, rows, bias_type;   // rows of a row group
    long long ldc, ldz, ldo;   // (KEPT: ldz in bytes)
    void* value;    // VALUE: act(z), or null
    long long ldv;
};

// 256 threads: 32 strips of eight columns x 8 rows; blockIdx.y is the row group.
template <class TI, class TO, bool KEPT = false, bool VALUE = false>
__global__ void __launch_bounds__(256) act_grad_kernel(ActGradArgs g) {
    typedef typename Elt<TI>::T I;
    typedef typename Elt<TO>::T O;
    constexpr int RL = 8;
    __shared__ float sums[RL][32][8 + 1];
    const int strip = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const long long n = ((long long)blockIdx.x * 32 + strip) * 8;
    const int valid = (int)std::min<long long>(g.N - n, 8);
    const long long m0 = (long long)blockIdx.y * g.rows;
    const long long m1 = std::min<long long>(m0 + g.rows, g.M);
    float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (valid > 0) {
        for (long long m = m0 + rl; m < m1; m += RL) {   // (two rows in flight: 4096 x 8192 42 -> 51 us)
            float v[8], z[8];
            load8<TI>(static_cast<const I*>(g.dc) + m * g.ldc + n, valid, v);
            if (KEPT || g.z) {
                if constexpr (KEPT) {
                    Kept8 k;
                    k.load(static_cast<const uint8_t*>(g.z) + m * g.ldz, kept_values(g.N), n, true);
                    k.unpack<std::is_same<TO, OutF16>::value>(z);
                } else {
                    load8<TI>(static_cast<const I*>(g.z) + m * g.ldz + n, valid, z);
                }
                act_slopes<8>(g.act, v, z);
                if (VALUE && g.value) {
                    act_values<8>(g.act, z);
                    store8<TO>(static_cast<O*>(g.value) + m * g.ldv + n, valid, z);
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += v[e];
            if (g.dz) store8<TO>(static_cast<O*>(g.dz) + m * g.ldo + n, valid, v);
        }
    }
    if (!g.part && !g.dbias) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[rl][strip][e] = s[e];
    __syncthreads();
    const int c = threadIdx.x & 255;   // one column a thread
    const long long col = (long long)blockIdx.x * 256 + c;
    float t = sums[0][c >> 3][c & 7];
#pragma unroll
    for (int r = 1; r < RL; ++r) t += sums[r][c >> 3][c & 7];
    if (col >= g.N) return;
    if (g.dbias)
        store_any(g.dbias, g.bias_type, col, t);
    else
        g.part[(long long)blockIdx.y * g.N + col] = t;
}

namespace {

// Row groups: enough workgroups to fill the chip eight times over, of at least 16 rows.
int64_t group_rows(int64_t M, int64_t N) {
    const int64_t strips = (N + 255) / 256;
    const int64_t groups = std::max<int64_t>(1, std::min<int64_t>((M + 15) / 16, (2048 + strips - 1) / strips));
    return std::max<int64_t>(1, (M + groups - 1) / groups);
}
int64_t num_groups(int64_t M, int64_t N) {
    const int64_t rows = group_rows(M, N);
    return (M + rows - 1) / rows;
}

bool row_type(int32_t t) { return t == TS_F16 || t == TS_BF16 || t == TS_F32; }
int type_size(int32_t t) { return t == TS_F32 ? 4 : 2; }

template <bool KEPT = false, bool VALUE = false>
const void* kernel_of(int32_t in, int32_t out) {
    if (in == TS_F16) return reinterpret_cast<const void*>(&act_grad_kernel<OutF16, OutF16, KEPT, VALUE>);
    if (in == TS_BF16) return reinterpret_cast<const void*>(&act_grad_kernel<OutBF16, OutBF16, KEPT, VALUE>);
    if (out == TS_F16) return reinterpret_cast<const void*>(&act_grad_kernel<OutF32, OutF16, KEPT, VALUE>);
    if (out == TS_BF16) return reinterpret_cast<const void*>(&act_grad_kernel<OutF32, OutBF16, KEPT, VALUE>);
    return reinterpret_cast<const void*>(&act_grad_kernel<OutF32, OutF32, KEPT, VALUE>);
}

}  // namespace
}  // namespace ts

using namespace ts;

extern "C" int64_t ts_act_grad_workspace(int64_t M, int64_t N) {
    if (M < 0 || N < 0) return TS_ERR_INVALID_ARG;
    if (M > INT_MAX / 2 || N >= 1 << 26) return TS_ERR_UNSUPPORTED;   // N: threads of the sum over the groups
    if (N == 0) return 0;   // no strips to deal the groups over
    const int64_t groups = num_groups(M, N);
    return groups > 1 ? groups * N * 4 : 0;
}

namespace {

ts_status run(const void* dc, const void* preact, void* dz, void* value, void* dbias, int64_t M, int64_t N, int64_t stride_dc,
              int64_t stride_pm, int64_t stride_dz, int64_t stride_v, int32_t in_dtype, bool kept, int32_t out_dtype,
              int32_t bias_dtype, int32_t activation, void* stream, void* workspace, int64_t workspace_bytes) {
    const int64_t need = ts_act_grad_workspace(M, N);
    if (need < 0) return (ts_status)need;
    if (!row_type(in_dtype) || !row_type(out_dtype) || (dbias && !row_type(bias_dtype)) || workspace_bytes < 0 ||
        activation < TS_ACT_NONE || activation > TS_ACT_SILU)
        return TS_ERR_INVALID_ARG;
    if ((dz || value) && in_dtype != TS_F32 && out_dtype != in_dtype) return TS_ERR_UNSUPPORTED;
    if (N == 0 || (M == 0 && !dbias) || (!dz && !dbias && !value)) return TS_OK;
    const bool reads = activation != TS_ACT_NONE || value;
    if (M > 0 && (!dc || (reads && !preact))) return TS_ERR_INVALID_ARG;
    if (!reads) {
        preact = nullptr;
        kept = false;
    }
    if (M > 1 && (stride_dc < N || (preact && !kept && stride_pm < N) || (dz && stride_dz < N) || (value && stride_v < N) ||
                  (kept && (stride_pm < kept_row(N) || stride_pm % 16 != 0))))
        return TS_ERR_INVALID_ARG;
    if ((uintptr_t)dc % type_size(in_dtype) || (uintptr_t)preact % (kept ? 16 : type_size(in_dtype)) ||
        (uintptr_t)dz % type_size(out_dtype) || (uintptr_t)value % type_size(out_dtype) ||
        (dbias && (uintptr_t)dbias % type_size(bias_dtype)))
        return TS_ERR_ALIGNMENT;
    const bool same = out_dtype == in_dtype;
    if ((value && value == dz) || !in_place_ok(dz, dc, same, M, stride_dz, stride_dc) ||
        !in_place_ok(dz, preact, same && !kept, M, stride_dz, stride_pm) ||
        !in_place_ok(value, dc, same, M, stride_v, stride_dc) ||
        !in_place_ok(value, preact, same && !kept, M, stride_v, stride_pm))
        return TS_ERR_INVALID_ARG;
    if (dbias && need > 0 && (!workspace || workspace_bytes < need || (uintptr_t)workspace % 256)) return TS_ERR_INVALID_ARG;
    int dev;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return TS_ERR_NO_DEVICE;
    }
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    const int64_t groups = num_groups(M, N);
    if (M > 0) {
        ActGradArgs g = {dc, preact, dz, dbias && groups > 1 ? static_cast<float*>(workspace) : nullptr,
                         groups > 1 ? nullptr : dbias, (int)M, (int)N, activation, (int)group_rows(M, N), bias_dtype,
                         stride_dc, stride_pm, stride_dz, value, stride_v};
        void* args[] = {&g};
        const int32_t out = dz || value ? out_dtype : in_dtype;
        const void* fn = kept ? kernel_of<true, true>(in_dtype, out)
                         : value ? kernel_of<false, true>(in_dtype, out) : kernel_of<false, false>(in_dtype, out);
        if (!enqueue(fn, (N + 255) / 256, 256, args, hs, groups)) return TS_ERR_HIP;
    }
    if (dbias && groups != 1 && !launch_reduce_columns(static_cast<float*>(workspace), (int)groups, (int)N, dbias, bias_dtype, hs))
        return TS_ERR_HIP;
    return TS_OK;
}

}  // namespace

extern "C" ts_status ts_act_grad(const void* dc, const void* preact, void* dz, void* dbias, int64_t M, int64_t N,
                                 int64_t stride_dc, int64_t stride_pm, int64_t stride_dz, int32_t in_dtype,
                                 int32_t out_dtype, int32_t bias_dtype, int32_t activation, void* stream,
                                 void* workspace, int64_t workspace_bytes) {
    return run(dc, preact, dz, nullptr, dbias, M, N, stride_dc, stride_pm, stride_dz, N, in_dtype, false, out_dtype,
               bias_dtype, activation, stream, workspace, workspace_bytes);
}

extern "C" ts_status ts_act_grad_value(const void* dc, const void* preact, void* dz, void* value, void* dbias, int64_t M,
                                       int64_t N, int64_t stride_dc, int64_t stride_pm, int64_t stride_dz,
                                       int64_t stride_v, int32_t in_dtype, int32_t preact_dtype, int32_t out_dtype,
                                       int32_t bias_dtype, int32_t activation, void* stream, void* workspace,
                                       int64_t workspace_bytes) {
    if (preact_dtype != in_dtype && preact_dtype != TS_Q8) return TS_ERR_INVALID_ARG;
    return run(dc, preact, dz, value, dbias, M, N, stride_dc, stride_pm, stride_dz, stride_v, in_dtype,
               preact_dtype == TS_Q8, out_dtype, bias_dtype, activation, stream, workspace, workspace_bytes);
}

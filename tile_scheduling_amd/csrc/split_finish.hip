// Sums of a product's splits along K, in order, and the epilogue of the joined sums: eight
// columns of a row a thread.  The sums lie in whole tiles, so only C's side has edges.  Bound
// by the splits x M x N x 4 bytes just written, which the memory-side cache still holds: 4 splits
// of 1000 x 512 4.2 us, most of it the launch.
#include <hip/hip_runtime.h>

#include "plan.hpp"
#include "rows.hpp"
#include "split.hpp"

namespace ts {

template <class TO>
__global__ void __launch_bounds__(256) split_finish_kernel(SplitArgs g) {
    typedef typename Elt<TO>::T T;
    const int strips = (g.N + 7) / 8;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    if (id >= (long long)g.M * strips) return;
    const int m = (int)(id / strips), n = 8 * (int)(id - (long long)m * strips);
    const int valid = g.N - n < 8 ? g.N - n : 8;
    const f32x4* s = reinterpret_cast<const f32x4*>(g.sums + m * g.ld_sums + n);
    f32x4 a = s[0], b = s[1];
#pragma unroll 4
    for (int i = 1; i < g.splits; ++i) {
        s = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(s) + g.split_stride);
        a += s[0];
        b += s[1];
    }
    float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    if (g.scale_a || g.scale_b) {
        const float sa = g.scale_a ? g.scale_a[m] : 1.0f;
        float sb[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
        if (g.scale_b) load8<OutF32>(g.scale_b + n, valid, sb);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * sa * sb[e];
    }
    if (g.bias) {
        float bias[8];
        load_columns<8>(g.bias, g.bias_type, n, valid, bias);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += e < valid ? bias[e] : 0.0f;
    }
    if (g.aux_out) store8<TO>(static_cast<T*>(g.aux_out) + m * g.ld_out + n, valid, v);
    float w[8];
    if (g.aux_in) load8<TO>(static_cast<const T*>(g.aux_in) + m * g.ld_in + n, valid, w);
    if (g.grad) {
        act_slopes<8>(g.act, v, w);
    } else {
        act_values<8>(g.act, v);
        if (g.aux_in) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += w[e];
        }
    }
    store8<TO>(static_cast<T*>(g.C) + m * g.ldc + n, valid, v);
}

bool launch_split_finish(SplitArgs& g, int c, hipStream_t stream) {
    const long long threads = (long long)g.M * ((g.N + 7) / 8);
    const void* fn = c == ELT_F32   ? reinterpret_cast<const void*>(&split_finish_kernel<OutF32>)
                     : c == ELT_F16 ? reinterpret_cast<const void*>(&split_finish_kernel<OutF16>)
                                    : reinterpret_cast<const void*>(&split_finish_kernel<OutBF16>);
    void* args[] = {&g};
    return enqueue(fn, (threads + 255) / 256, 256, args, stream);
}

}  // namespace ts

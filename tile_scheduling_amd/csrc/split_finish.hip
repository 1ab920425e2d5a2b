// Sums of a product's splits along K, in order, and the epilogue of the joined sums: eight
// columns of a row a thread.  The sums lie in whole tiles, so only C's side has edges.  Bound
// by the splits x M x N x 4 bytes just written, which the memory-side cache still holds: 4 splits
// of 1000 x 512 4.2 us, most of it the launch.
#include <hip/hip_runtime.h>

#include "checkpoint.hpp"
#include "plan.hpp"
#include "rows.hpp"
#include "split.hpp"

namespace ts {

// INTS: int32 sums.  KEPT: preact in 8 bits (g.kept); four threads then hold a block of 32 columns, the
// last ones of a row perhaps none that exist.
template <class TO, bool INTS, bool KEPT>
__global__ void __launch_bounds__(256) split_finish_kernel(SplitArgs g) {
    typedef typename Elt<TO>::T T;
    const int strips = KEPT ? (int)(kept_values(g.N) / 8) : (g.N + 7) / 8;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    if (id >= (long long)g.M * strips) return;
    const int m = (int)(id / strips), n = 8 * (int)(id - (long long)m * strips);
    const int valid = g.N - n < 8 ? g.N - n : 8;   // KEPT: perhaps none
    const f32x4* s = reinterpret_cast<const f32x4*>(g.sums + m * g.ld_sums + n);
    f32x4 a = s[0], b = s[1];
#pragma unroll 4
    for (int i = 1; i < g.splits; ++i) {
        s = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(s) + g.split_stride);
        if constexpr (INTS) {
            a = __builtin_bit_cast(f32x4, __builtin_bit_cast(i32x4, a) + __builtin_bit_cast(i32x4, s[0]));
            b = __builtin_bit_cast(f32x4, __builtin_bit_cast(i32x4, b) + __builtin_bit_cast(i32x4, s[1]));
        } else {
            a += s[0];
            b += s[1];
        }
    }
    float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    if constexpr (INTS) {   // rounded as on tiles
        float sa = 1.0f, sb[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f}, bias[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (g.scale_a) sa = g.scale_a[m];
        if (g.scale_b) load8<OutF32>(g.scale_b + n, valid, sb);
        if (g.bias) load_columns<8>(g.bias, g.bias_type, n, valid, bias);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = scaled_apart((float)__builtin_bit_cast(int, v[e]), sa, sb[e], bias[e]);
    } else {
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
    }
    uint8_t* kept = KEPT ? g.kept + m * g.ld_kept : nullptr;
    if (KEPT && !g.grad) {
        uint32_t most = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = e < valid ? v[e] : 0.0f;   // the sums of columns behind N are anything
            const uint32_t x = __builtin_bit_cast(uint32_t, v[e]) & 0x7fffffffu;
            most = x > most ? x : most;
        }
        const uint32_t ex = block_exponent(quad_max(most));
        const float inv = step_inverse(ex);
        *reinterpret_cast<uint2*>(kept + n) = make_uint2(kept_pack4(v, inv), kept_pack4(v + 4, inv));
        if (n % kBlock == 0) kept[kept_values(g.N) + n / kBlock] = (uint8_t)ex;
    }
    if (g.aux_out) store8<TO>(static_cast<T*>(g.aux_out) + m * g.ld_out + n, valid, v);
    float w[8];
    if (g.aux_in) load8<TO>(static_cast<const T*>(g.aux_in) + m * g.ld_in + n, valid, w);
    if constexpr (KEPT) {
        if (g.grad) {
            Kept8 k;
            k.load(kept, kept_values(g.N), n, true);
            k.unpack(w);
        }
    }
    if (g.grad) {
        act_slopes<8>(g.act, v, w);
    } else {
        if constexpr (INTS) values_apart<8>(g.act, v);
        else act_values<8>(g.act, v);
        if (g.aux_in) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = INTS ? sum_apart(v[e], w[e]) : v[e] + w[e];
        }
    }
    store8<TO>(static_cast<T*>(g.C) + m * g.ldc + n, valid, v);
}

namespace {
template <bool INTS, bool KEPT>
const void* finish_kernel(int c) {
    return c == ELT_F32   ? reinterpret_cast<const void*>(&split_finish_kernel<OutF32, INTS, KEPT>)
           : c == ELT_F16 ? reinterpret_cast<const void*>(&split_finish_kernel<OutF16, INTS, KEPT>)
                          : reinterpret_cast<const void*>(&split_finish_kernel<OutBF16, INTS, KEPT>);
}
}  // namespace

bool launch_split_finish(SplitArgs& g, int ab, int c, hipStream_t stream) {
    const long long threads = (long long)g.M * (g.kept ? kept_values(g.N) / 8 : (g.N + 7) / 8);
    const void* fn = ab == ELT_I8 ? finish_kernel<true, false>(c) : g.kept ? finish_kernel<false, true>(c) : finish_kernel<false, false>(c);
    void* args[] = {&g};
    return enqueue(fn, (threads + 255) / 256, 256, args, stream);
}

}  // namespace ts

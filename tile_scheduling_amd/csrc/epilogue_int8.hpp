// The fused epilogue of int8 products for one activation family and 16-bit C, on the 256 tile: straight
// code as SpecialStore's (see there), for tiles inside M x N.
#pragma once

#include "epilogue.hpp"
#include "internal.hpp"

namespace ts {

// The scales and biases of a lane's 32 columns are held in registers (64) and z is formed where it is used:
// accumulators that are changed in place spill 80 to 300 registers.  (With the rows of a residual ahead 18 to
// 22 are, none inside the K loop.)  Against FusedStore, bf16 C, with bias, us: 4096 x 16384 x 4096 none 237 / 252, silu
// 254 / 268, residual 262 / 281; 5000 x 12290 x 1000 91 / 107, 106 / 124, 123 / 133; 4096 x 4096 x 8192 residual 120 / 126.
template <int FAM, bool RESIDUAL>
struct SpecialInt8Store {
    typedef EpiArgs Args;
    typedef FusedStore G;
    typedef SpecialStore<FAM, AUX_NONE> S;
    static constexpr int MIN_WAVES = 2;
    static constexpr bool RENEW = true;
    static __device__ __forceinline__ void start(const EpiArgs& g) { G::start(g); }
    static constexpr int NQ = G::NQ, NU = G::NU;

    template <bool PARTS, class E>
    static __device__ __forceinline__ void store(E& e, const EpiArgs& g0, int m0, int n0, const typename E::Parts& pt) {
        const EpiArgs& g = fresh_args();
        typedef typename E::OutType TO;
        typedef typename Elt<TO>::T T;
        static_assert(sizeof(T) == 2 && E::FN == 2 && E::INTS, "both blocks of a row staged together");
        if (m0 + E::BM > g.M || n0 + E::BN > g.N) {
            G::store<PARTS>(e, g0, m0, n0, pt);
            return;
        }
        const G::Tile t = G::tile_of(e, g, m0, n0);
        typename S::template Walk<E> in(t, g.aux_in, g.ld_in), w(t, g.C, g.ldc);
        u32x4 rows[NU];
        if constexpr (RESIDUAL) {
            in.fetch(rows);
            in.next(0);
        }
        float sb[E::FN * NQ][4], bias[E::FN * NQ][4], sa[E::FM];
#pragma unroll
        for (int j = 0; j < E::FN; ++j) G::template columns<E>(g, t, j, sb + j * NQ, bias + j * NQ);
#pragma unroll
        for (int i = 0; i < E::FM; ++i) sa[i] = g.scale_a ? g.scale_a[t.m + 32 * i + t.r32] : 1.0f;
        const Sigmoid coeff = sigmoid_of(g.act);
#pragma unroll
        for (int i = 0; i < E::FM; ++i) {
            if constexpr (RESIDUAL) {
#pragma unroll
                for (int u = 0; u < NU; ++u) *reinterpret_cast<u32x4*>(G::unit_lds(t, u)) = rows[u];
                if (i + 1 < E::FM) {
                    in.fetch(rows);
                    in.next(i + 1);
                }
            }
#pragma unroll
            for (int x = 0; x < E::FN * NQ; ++x) {
                char* at = G::quad_lds(t, (4 * t.hk + 32 * (x / NQ) + 8 * (x % NQ)) * 2);
                float v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float sum = e.acc[i][x / NQ][4 * (x % NQ) + c];   // (a bit cast of the vector's element takes its first)
                    v[c] = value_apart<FAM>(scaled_apart((float)__builtin_bit_cast(int, sum), sa[i], sb[x][c], bias[x][c]), coeff);
                }
                if constexpr (RESIDUAL) {
                    float f[8];
                    const u32x2 h = *reinterpret_cast<const u32x2*>(at);
                    unpack_row<TO>(u32x4{h[0], h[1], 0, 0}, f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] = sum_apart(v[c], f[c]);
                }
                Out<TO>::store4(reinterpret_cast<T*>(at), v, 4, true);
            }
            w.store(t);
            w.next(i);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

template <class TO, bool RESIDUAL>
const void* epi_int8_special(int fam) {
    switch (fam) {
        case FAM_RELU: return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg256w8, InI8, TO, PATH_EDGE_BT, false, SpecialInt8Store<FAM_RELU, RESIDUAL>>);
        case FAM_ERF: return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg256w8, InI8, TO, PATH_EDGE_BT, false, SpecialInt8Store<FAM_ERF, RESIDUAL>>);
        case FAM_SIGMOID: return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg256w8, InI8, TO, PATH_EDGE_BT, false, SpecialInt8Store<FAM_SIGMOID, RESIDUAL>>);
        default: return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg256w8, InI8, TO, PATH_EDGE_BT, false, SpecialInt8Store<FAM_NONE, RESIDUAL>>);
    }
}

}  // namespace ts

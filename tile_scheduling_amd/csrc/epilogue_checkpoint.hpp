// The fused epilogue with preact in 8 bits (checkpoint.hpp): written from the fp32 z in front of C,
// or read where C is a gradient.
#pragma once

#include "checkpoint.hpp"
#include "epilogue.hpp"

namespace ts {

// As FusedStore, whose parts it uses, in one or two rolled loops over the 32 x 32 blocks.  In a
// block the 32 columns of a row are the registers of lanes l and l + 32, so a block's largest
// value takes 16 maxima and one exchange, and its bytes are staged as those of C are: 64
// columns of a row, 64 bytes.
struct CheckpointStore {
    typedef EpiArgs Args;
    typedef FusedStore G;
    static constexpr int MIN_WAVES = G::MIN_WAVES;
    static constexpr bool RENEW = true;
    static __device__ __forceinline__ void start(const EpiArgs& g) { G::start(g); }
    static constexpr int NQ = G::NQ;

    // Staged bytes of 64 columns: chunk c (16 bytes) of row r.
    static __device__ __forceinline__ char* chunk(const G::Tile& t, int r, int c) {
        return t.st + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    }
    template <class E>
    static __device__ __forceinline__ void keep(const E& e, const EpiArgs& g, const G::Tile& t) {
        const long long values = kept_values(t.N);
        uint32_t left = 0;   // exponent of the block to the left
#pragma unroll 1
        for (int b = 0; b < E::FM * E::FN; ++b) {
            const int j = b % E::FN, m = t.m + 32 * (b / E::FN);
            float v[NQ][4];
            G::take_any(b, e, v, std::make_integer_sequence<int, E::FM * E::FN>{});
            if (!t.whole) {   // columns behind N hold anything
#pragma unroll
                for (int q = 0; q < NQ; ++q)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (t.n + 32 * j + 8 * q + 4 * t.hk + c >= t.N) v[q][c] = 0.0f;
            }
            uint32_t most = 0;
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t a = __builtin_bit_cast(uint32_t, v[q][c]) & 0x7fffffffu;
                    most = a > most ? a : most;
                }
            const uint32_t other = __shfl_xor(most, 32, 64);
            const uint32_t ex = block_exponent(other > most ? other : most);
            const float inv = step_inverse(ex);
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int at = 32 * j + 8 * q + 4 * t.hk;
                *reinterpret_cast<uint32_t*>(chunk(t, t.r32, at >> 4) + (at & 15)) = kept_pack4(v[q], inv);
            }
            if (j == 0) {
                left = ex;
                continue;
            }
            // 64 columns: two 16-byte pieces a lane; the row's values end at a multiple of 32
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = 16 * u + (t.ln >> 2), c = t.ln & 3;
                const u32x4 w = *reinterpret_cast<const u32x4*>(chunk(t, r, c));
                if (m + r < t.M && t.n + 16 * c < values)
                    *reinterpret_cast<u32x4*>(g.kept + (m + r) * g.ld_kept + t.n + 16 * c) = w;
            }
            if (t.hk == 0 && m + t.r32 < t.M && t.n < t.N) {
                uint8_t* p = g.kept + (m + t.r32) * g.ld_kept + values + t.n / kBlock;
                if (t.n + 32 < t.N)
                    *reinterpret_cast<uint16_t*>(p) = (uint16_t)(left | ex << 8);
                else
                    *p = (uint8_t)left;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // Four columns of z at n, nothing at or behind column N.
    static __device__ __forceinline__ void kept_quad(const G::Tile& t, const uint8_t* row, float step, int n,
                                                     float* w) {
        uint32_t x = 0;
        if (n < t.N) x = *reinterpret_cast<const uint32_t*>(row + n);
        kept_unpack4(x, step, w);
    }
    template <bool PARTS, class E>
    static __device__ __forceinline__ void store(E& e, const EpiArgs&, int m0, int n0, const typename E::Parts& pt) {
        const EpiArgs& g = fresh_args();
        typedef typename E::Config Cfg;
        typedef typename E::OutType TO;
        typedef typename Elt<TO>::T T;
        constexpr int OSZ = sizeof(T);
        constexpr int JB = OSZ == 2 ? 2 : 1;               // blocks staged together
        const G::Tile t = G::tile_of(e, g, m0, n0);
        G::template finish_sums<PARTS>(e, g, t, pt);
        if (!g.grad) keep(e, g, t);
        const Sigmoid coeff = sigmoid_of(g.act);
        const bool read = g.aux_in != nullptr;
        const long long values = kept_values(t.N);
#pragma unroll 1
        for (int b = 0; b < Cfg::FM * Cfg::FN; ++b) {
            const int j = b % Cfg::FN;
            const int m = t.m + 32 * (b / Cfg::FN), n = JB == 2 ? t.n : t.n + 32 * j;   // of the staged part
            if (read && b % JB == 0) {
                u32x4 rows[G::NU];
                G::fetch<TO>(t, g.aux_in, g.ld_in, m, n, rows);
#pragma unroll
                for (int u = 0; u < G::NU; ++u) *reinterpret_cast<u32x4*>(G::unit_lds(t, u)) = rows[u];
            }
            float v[NQ][4];
            G::take_any(b, e, v, std::make_integer_sequence<int, Cfg::FM * Cfg::FN>{});
            const int at0 = 4 * t.hk * OSZ + (JB == 2 ? 32 * j * OSZ : 0);
            if (g.grad) {
                const int nb = t.n + 32 * j;
                const bool in = m + t.r32 < t.M && nb < t.N;
                const uint8_t* row = g.kept + (in ? (long long)(m + t.r32) * g.ld_kept : 0);
                const float step = step_of(in ? row[values + nb / kBlock] : 1u);
                float w[NQ][4];
#pragma unroll
                for (int q = 0; q < NQ; ++q) kept_quad(t, row, step, in ? nb + 8 * q + 4 * t.hk : t.N, w[q]);
                with_family(g.act, [&](auto fam) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
#pragma unroll
                        for (int c = 0; c < 4; ++c) v[q][c] *= fam_slope<decltype(fam)::value>(w[q][c], coeff);
                });
            } else {
                with_family(g.act, [&](auto fam) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
#pragma unroll
                        for (int c = 0; c < 4; ++c) v[q][c] = fam_value<decltype(fam)::value>(v[q][c], coeff);
                });
            }
            if (read) {
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    float f[8];
                    if constexpr (OSZ == 4) {
                        unpack_row<TO>(*reinterpret_cast<const u32x4*>(G::quad_lds(t, at0 + 8 * q * OSZ)), f);
                    } else {
                        const u32x2 h = *reinterpret_cast<const u32x2*>(G::quad_lds(t, at0 + 8 * q * OSZ));
                        unpack_row<TO>(u32x4{h[0], h[1], 0, 0}, f);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[q][c] += f[c];
                }
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                Out<TO>::store4(reinterpret_cast<T*>(G::quad_lds(t, at0 + 8 * q * OSZ)), v[q], 4, true);
            if (b % JB == JB - 1) G::flush<TO>(t, g.C, g.ldc, m, n);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

template <class Cfg, class TI, class TO>
const void* epi_checkpoint(int path) {
    if (path == PATH_EDGE_BT) return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH_EDGE_BT, false, CheckpointStore>);
    return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH_EDGE_NN, false, CheckpointStore>);
}

}  // namespace ts

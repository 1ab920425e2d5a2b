// The fused epilogue with preact in 8 bits (checkpoint.hpp): written from the fp32 z in front of C,
// or read where C is a gradient.
#pragma once

#include "checkpoint.hpp"
#include "epilogue.hpp"
#include "internal.hpp"

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
            const uint32_t ex = block_exponent(halves_max(most));
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
                const float step = slope_step_of(in ? row[values + nb / kBlock] : 1u);
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

// The forward form for one activation family, 16-bit C and no residual, on either tile: straight code as
// SpecialStore's (see there), for tiles inside M x N.  Against CheckpointStore, bf16, gelu, 4096 x 8192 x 4096
// 234 / 262 us; against preact in 16 bits 4096 x 8192 x 4096 234 / 226, 4096 x 16384 x 1024 182 / 168.
template <int FAM>
struct SpecialCheckpointStore {
    typedef EpiArgs Args;
    typedef FusedStore G;
    typedef SpecialStore<FAM, AUX_NONE> S;
    static constexpr int MIN_WAVES = 2;
    static constexpr bool RENEW = true;
    static __device__ __forceinline__ void start(const EpiArgs& g) { G::start(g); }
    static constexpr int NQ = G::NQ;

    template <bool PARTS, class E>
    static __device__ __forceinline__ void store(E& e, const EpiArgs& g0, int m0, int n0, const typename E::Parts& pt) {
        const EpiArgs& g = fresh_args();
        typedef typename E::OutType TO;
        typedef typename Elt<TO>::T T;
        static_assert(sizeof(T) == 2 && E::FN == 2, "both blocks of a row staged together");
        if (m0 + E::BM > g.M || n0 + E::BN > g.N) {
            CheckpointStore::store<PARTS>(e, g0, m0, n0, pt);
            return;
        }
        const G::Tile t = G::tile_of(e, g, m0, n0);
        typename S::template Walk<E> w(t, g.C, g.ldc);
        // the rows' values, 16 rows an access, and their exponents, one row a lane
        const uint32_t ld = (uint32_t)g.ld_kept;   // 16 rows of it fit in 31 bits (host)
        uint8_t* kv = g.kept + t.m * g.ld_kept + t.n;
        uint8_t* ke = g.kept + t.m * g.ld_kept + kept_values(t.N) + t.n / kBlock;
        const uint32_t lane_v = (uint32_t)(t.ln >> 2) * ld + (uint32_t)(t.ln & 3) * 16u, lane_e = (uint32_t)t.r32 * ld;
        float bias[E::FN * NQ][4], one[NQ][4];
#pragma unroll
        for (int j = 0; j < E::FN; ++j) G::template columns<E>(g, t, j, one, bias + j * NQ);
        const Sigmoid coeff = sigmoid_of(g.act);
#pragma unroll
        for (int i = 0; i < E::FM; ++i) {
            uint32_t ex[E::FN];
#pragma unroll
            for (int j = 0; j < E::FN; ++j) {
                float v[NQ][4];
                uint32_t most = 0;
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    S::z_of(e, i, j, q, bias, v[q]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t a = __builtin_bit_cast(uint32_t, v[q][c]) & 0x7fffffffu;
                        most = a > most ? a : most;
                    }
                }
                ex[j] = block_exponent(halves_max(most));
                const float inv = step_inverse(ex[j]);
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    const int at = 32 * j + 8 * q + 4 * t.hk;
                    *reinterpret_cast<uint32_t*>(CheckpointStore::chunk(t, t.r32, at >> 4) + (at & 15)) = kept_pack4(v[q], inv);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
                *reinterpret_cast<u32x4*>(kv + (uint32_t)u * 16u * ld + lane_v) =
                    *reinterpret_cast<const u32x4*>(CheckpointStore::chunk(t, 16 * u + (t.ln >> 2), t.ln & 3));
            if (t.hk == 0) *reinterpret_cast<uint16_t*>(ke + lane_e) = (uint16_t)(ex[0] | ex[1] << 8);
            kv += 32 * g.ld_kept;
            ke += 32 * g.ld_kept;
            asm volatile("" : "+s"(kv), "+s"(ke));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int x = 0; x < E::FN * NQ; ++x) {
                float v[4];
                S::z_of(e, i, x / NQ, x % NQ, bias, v);
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = fam_value<FAM>(v[c], coeff);
                Out<TO>::store4(reinterpret_cast<T*>(G::quad_lds(t, (4 * t.hk + 32 * (x / NQ) + 8 * (x % NQ)) * 2)), v, 4, true);
            }
            w.store(t);
            w.next(i);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

template <class Cfg, class TI, class TO>
const void* epi_checkpoint(int path) {
    if (path == PATH_EDGE_BT) return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH_EDGE_BT, false, CheckpointStore>);
    if (path == PATH_EDGE_AT) return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH_EDGE_AT, false, CheckpointStore>);
    if (path == PATH_EDGE_ATBT) return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH_EDGE_ATBT, false, CheckpointStore>);
    return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH_EDGE_NN, false, CheckpointStore>);
}
template <class Cfg, class TI, class TO, int PATH>
const void* epi_checkpoint_special(int fam) {
    switch (fam) {
        case FAM_RELU: return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH, false, SpecialCheckpointStore<FAM_RELU>>);
        case FAM_ERF: return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH, false, SpecialCheckpointStore<FAM_ERF>>);
        case FAM_SIGMOID: return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH, false, SpecialCheckpointStore<FAM_SIGMOID>>);
        default: return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH, false, SpecialCheckpointStore<FAM_NONE>>);
    }
}

}  // namespace ts

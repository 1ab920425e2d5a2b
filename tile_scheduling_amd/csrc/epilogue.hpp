// The fused epilogue of the tiled product: bias, activation, residual and the scales of
// 8-bit operands, applied to the fp32 accumulators before their one rounding, and the
// activations with their derivatives.
//
//   z = acc * scale_a[m] * scale_b[n] + bias[n]        (scales: 8-bit operands only)
//   forward   preact = z;  C = act(z) + residual
//   gradient  C = z * act'(preact)
//
// Every term is formed in fp32; preact and C are each rounded once, to C's type.
#pragma once

#include "gemm_kernel.hpp"

namespace ts {

// Activations (same numbering as TS_ACT_* in tsgemm.h).
enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };
// Element types (same numbering as TS_F16, TS_BF16, TS_F32, TS_E4M3); 0 = absent.
enum : int { ELT_NONE = 0, ELT_F16 = 1, ELT_BF16 = 2, ELT_F32 = 3, ELT_E4M3 = 4 };

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(-kLog2e * x); }   // e^-x
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_neg(x)); }

// Upper tail of the normal distribution times e^(x^2/2), x >= 0: a degree 8 polynomial
// without constant term in t = 1 / (1 + 0.305 x), fitted to 0.5 erfcx(x / sqrt 2) by
// reweighted least squares (relative error 9.4e-8 over x in [0, 13], 3.9e-7 evaluated
// in fp32).  One reciprocal and 8 fused multiply-adds; 0.5 (1 + erf) would lose every
// digit of the tail.
__device__ __forceinline__ float tail_scaled(float x) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.305f, x, 1.0f));
    float p = 0x1.2ca3eap-5f;
    p = __builtin_fmaf(p, t, -0x1.395214p-3f);
    p = __builtin_fmaf(p, t, 0x1.7c5962p-3f);
    p = __builtin_fmaf(p, t, -0x1.371c1ep-5f);
    p = __builtin_fmaf(p, t, 0x1.efb4aep-4f);
    p = __builtin_fmaf(p, t, 0x1.a79c90p-4f);
    p = __builtin_fmaf(p, t, 0x1.f59fc8p-4f);
    p = __builtin_fmaf(p, t, 0x1.f23c82p-4f);
    return p * t;
}

// gelu(z) = z Phi(z); gelu_tanh(z) = z sigmoid(w), w = sqrt(8/pi) (z + 0.044715 z^3), the
// same function as 0.5 z (1 + tanh(w / 2)); silu(z) = z sigmoid(z).
constexpr float kTanhW0 = 1.59576912160573071176f;             // sqrt(8 / pi)
constexpr float kTanhW1 = 1.59576912160573071176f * 0.044715f;
constexpr float kInvSqrt2Pi = 0.39894228040143267794f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == ACT_RELU) return z < 0.0f ? 0.0f : z;   // NaN stays NaN
    if constexpr (ACT == ACT_GELU) {
        const float x = __builtin_fabsf(z);
        const float q = tail_scaled(x) * __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z);
        return z * (z < 0.0f ? q : 1.0f - q);
    }
    if constexpr (ACT == ACT_GELU_TANH) return z * sigmoid(z * __builtin_fmaf(kTanhW1 * z, z, kTanhW0));
    if constexpr (ACT == ACT_SILU) return z * sigmoid(z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    if constexpr (ACT == ACT_GELU) {
        const float x = __builtin_fabsf(z);
        const float e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z);
        const float q = tail_scaled(x) * e;
        return __builtin_fmaf(z * kInvSqrt2Pi, e, z < 0.0f ? q : 1.0f - q);
    }
    if constexpr (ACT == ACT_GELU_TANH) {
        const float g = sigmoid(z * __builtin_fmaf(kTanhW1 * z, z, kTanhW0));
        return __builtin_fmaf(z * (g * (1.0f - g)), __builtin_fmaf(3.0f * kTanhW1 * z, z, kTanhW0), g);
    }
    if constexpr (ACT == ACT_SILU) {
        const float g = sigmoid(z);
        return g * __builtin_fmaf(z, 1.0f - g, 1.0f);
    }
    return 1.0f;
}

// The activation is one wave-uniform number: a scalar branch per group of E values.
template <int E>
__device__ __forceinline__ void act_values(int act, float* v) {
    switch (act) {
        case ACT_RELU:
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = act_value<ACT_RELU>(v[e]);
            break;
        case ACT_GELU:
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = act_value<ACT_GELU>(v[e]);
            break;
        case ACT_GELU_TANH:
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = act_value<ACT_GELU_TANH>(v[e]);
            break;
        case ACT_SILU:
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = act_value<ACT_SILU>(v[e]);
            break;
        default: break;
    }
}
// v[e] *= act'(z[e])
template <int E>
__device__ __forceinline__ void act_slopes(int act, float* v, const float* z) {
    switch (act) {
        case ACT_RELU:
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] *= act_slope<ACT_RELU>(z[e]);
            break;
        case ACT_GELU:
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] *= act_slope<ACT_GELU>(z[e]);
            break;
        case ACT_GELU_TANH:
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] *= act_slope<ACT_GELU_TANH>(z[e]);
            break;
        case ACT_SILU:
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] *= act_slope<ACT_SILU>(z[e]);
            break;
        default: break;
    }
}

// ---- rows of C's type, any alignment -----------------------------------------------------

// 16 bytes at the alignment of their elements: global accesses of gfx950 need no more
// (the compiler emits one 16-byte instruction).
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

template <class TO> struct Elt;   // TO: OutF16, OutBF16, OutF32
template <> struct Elt<OutF16> {
    typedef _Float16 T;
    typedef u32x4_a2 V;
    static constexpr int E = 8, CODE = ELT_F16;
};
template <> struct Elt<OutBF16> {
    typedef __bf16 T;
    typedef u32x4_a2 V;
    static constexpr int E = 8, CODE = ELT_BF16;
};
template <> struct Elt<OutF32> {
    typedef float T;
    typedef u32x4_a4 V;
    static constexpr int E = 4, CODE = ELT_F32;
};

// Elements p[0 .. E) as one 16-byte vector, those at or past `valid` zero.
template <class TO>
__device__ __forceinline__ u32x4 load_row(const typename Elt<TO>::T* p, int valid) {
    typedef Elt<TO> L;
    if (valid >= L::E) return *reinterpret_cast<const typename L::V*>(p);
    u32x4 r = {0, 0, 0, 0};
    if constexpr (L::E == 8) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = e < valid ? q[e] : 0u;
        r = u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
    } else {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = e < valid ? q[e] : 0u;
        r = u32x4{h[0], h[1], h[2], h[3]};
    }
    return r;
}
template <class TO>
__device__ __forceinline__ void unpack_row(u32x4 r, float* v) {
    if constexpr (std::is_same<TO, OutF32>::value) {
        const f32x4 f = __builtin_bit_cast(f32x4, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = f[e];
    } else if constexpr (std::is_same<TO, OutF16>::value) {
        const f16x8 f = __builtin_bit_cast(f16x8, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)f[e];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __builtin_bit_cast(float, r[e] << 16);
            v[2 * e + 1] = __builtin_bit_cast(float, r[e] & 0xffff0000u);
        }
    }
}
// Round to nearest even.
template <class TO>
__device__ __forceinline__ u32x4 pack_row(const float* v) {
    if constexpr (std::is_same<TO, OutF32>::value) {
        const f32x4 f = {v[0], v[1], v[2], v[3]};
        return __builtin_bit_cast(u32x4, f);
    } else if constexpr (std::is_same<TO, OutF16>::value) {
        const f16x8 f = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3],
                         (_Float16)v[4], (_Float16)v[5], (_Float16)v[6], (_Float16)v[7]};
        return __builtin_bit_cast(u32x4, f);
    } else {
        const bf16x8 f = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3],
                          (__bf16)v[4], (__bf16)v[5], (__bf16)v[6], (__bf16)v[7]};
        return __builtin_bit_cast(u32x4, f);
    }
}
template <class TO>
__device__ __forceinline__ void store_row(typename Elt<TO>::T* p, u32x4 r, int valid) {
    typedef Elt<TO> L;
    if (valid >= L::E) {
        *reinterpret_cast<typename L::V*>(p) = r;
    } else if constexpr (L::E == 8) {
        uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) q[e] = (uint16_t)(r[e >> 1] >> (16 * (e & 1)));
    } else {
        uint32_t* q = reinterpret_cast<uint32_t*>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < valid) q[e] = r[e];
    }
}
// One element of any of the three types.
__device__ __forceinline__ float load_any(const void* p, int type, long long i) {
    if (type == ELT_F32) return static_cast<const float*>(p)[i];
    if (type == ELT_F16) return (float)static_cast<const _Float16*>(p)[i];
    return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// ---- the tile epilogue -------------------------------------------------------------------

struct EpiArgs : GemmArgs {
    const void* bias;       // N elements of bias_type, or null
    const void* aux_in;     // residual (forward) or preact (gradient), C's type, or null
    void* aux_out;          // preact (forward), C's type, or null
    long long ld_in, ld_out;
    const float *scale_a, *scale_b;   // 8-bit operands: M and N fp32 (null: 1)
    int bias_type, act, grad;
};

// E consecutive columns of one row: v holds z (see the top), `in` the row's aux_in
// elements.  Returns C's elements and, in *pre, preact's.
template <class TO>
__device__ __forceinline__ u32x4 epilogue_row(const EpiArgs& g, float* v, u32x4 in, u32x4* pre) {
    constexpr int E = Elt<TO>::E;
    if (g.grad) {
        float z[E];
        unpack_row<TO>(in, z);
        act_slopes<E>(g.act, v, z);
    } else {
        if (g.aux_out) *pre = pack_row<TO>(v);
        act_values<E>(g.act, v);
        if (g.aux_in) {
            float r[E];
            unpack_row<TO>(in, r);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] += r[e];
        }
    }
    return pack_row<TO>(v);
}

// Store of one tile.  Each wave stages 16 rows x 64 columns of fp32 at a time through its
// own 4 KiB of LDS (the plain store's staging area, 16-byte chunks XOR-swizzled by row)
// and reads them back row-major, 16 bytes of C's type per lane, so that bias, residual,
// preact and C all move as whole row segments of 128 or 256 bytes; staging fp32 rather than
// C's type keeps the epilogue on unrounded sums.  aux_in's rows of a pass are loaded before
// the pass is staged.  The passes are one rolled loop whose staging part alone is
// instantiated per pass (its accumulators are fixed registers): with every activation
// in every pass the code is too long to unroll, and the accumulators end up in memory.
struct FusedStore {
    typedef EpiArgs Args;
    static constexpr int RS = 16;   // rows a pass

    // Accumulators of pass P (rows 16 P .. 16 P + 15 of the wave's sub-tile) into staging.
    template <int P, bool PARTS, class E>
    static __device__ __forceinline__ void stage(E& e, char* st, int r32, int hk, int tt, const typename E::Parts& pt) {
        typedef typename E::Config Cfg;
        constexpr int i = P / 2, h = P % 2;
        const int r = r32 - h * RS;
        // the empty asm statements keep the compiler from merging the passes' code, which
        // would select their accumulators by address, in memory
        asm volatile("" ::"n"(P));
        if (r >= 0 && r < RS) {
#pragma unroll
        for (int j = 0; j < Cfg::FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int ch = (8 * j + 2 * q + hk) ^ r;   // columns 32 j + 8 q + 4 hk .. + 3
                float v[4] = {e.acc[i][j][4 * q], e.acc[i][j][4 * q + 1], e.acc[i][j][4 * q + 2],
                              e.acc[i][j][4 * q + 3]};
                if (PARTS) e.add_parts(v, pt, (i * Cfg::FN + j) * 4 + q, tt);
                *reinterpret_cast<f32x4*>(st + r * 256 + ch * 16) = f32x4{v[0], v[1], v[2], v[3]};
            }
        }
        asm volatile("" ::"n"(P));
    }
    template <bool PARTS, class E, int... P>
    static __device__ __forceinline__ void stage_any(E& e, int p, char* st, int r32, int hk, int tt,
                                                     const typename E::Parts& pt, std::integer_sequence<int, P...>) {
        ((p == P ? stage<P, PARTS>(e, st, r32, hk, tt, pt) : (void)0), ...);
    }

    // What a lane holds for its E columns (n .. n + E - 1 of the tile, `valid` of them
    // before N) over the passes of a tile.
    template <class E>
    struct Columns {
        typedef Elt<typename E::OutType> L;
        typedef typename L::T T;
        static constexpr int LPR = 64 / L::E, RPU = 64 / LPR;   // lanes a row, rows a store instruction
        static constexpr int NU = RS / RPU;                     // store instructions a pass
        int row, col, n, valid;
        float bias[L::E], sb[L::E];
        const T* in;
        T *out, *C;
        u32x4 rows[NU];                                         // aux_in's rows of the pass
    };

    // Store instruction U of a pass: row m of C, staged row rp.
    template <int U, class E>
    static __device__ __forceinline__ void row_step(const EpiArgs& g, const Columns<E>& k, const char* st, int mp) {
        typedef Columns<E> K;
        typedef typename K::L L;
        typedef typename E::OutType TO;
        const int rp = U * K::RPU + k.row;
        const long long m = mp + U * K::RPU;
        if (m >= g.M) return;
        const float sa = E::PAIRS && g.scale_a ? g.scale_a[m] : 1.0f;
        if (k.valid >= L::E) {
            float v[L::E];
#pragma unroll
            for (int c = 0; c < L::E / 4; ++c) {
                const f32x4 f = *reinterpret_cast<const f32x4*>(st + rp * 256 + ((k.col / 4 + c) ^ rp) * 16);
#pragma unroll
                for (int w = 0; w < 4; ++w) v[4 * c + w] = f[w];
            }
#pragma unroll
            for (int c = 0; c < L::E; ++c) v[c] = (E::PAIRS ? v[c] * (sa * k.sb[c]) : v[c]) + k.bias[c];
            u32x4 pre;
            const u32x4 w = epilogue_row<TO>(g, v, k.rows[U], &pre);
            if (g.aux_out) *reinterpret_cast<typename L::V*>(k.out + m * g.ld_out) = pre;
            *reinterpret_cast<typename L::V*>(k.C + m * g.ldc) = w;
        } else {   // the columns before N of a chunk that crosses it, one by one
#pragma unroll 1
            for (int c = 0; c < k.valid; ++c) {
                float v = *reinterpret_cast<const float*>(st + rp * 256 + (((k.col + c) / 4) ^ rp) * 16 +
                                                          ((k.col + c) & 3) * 4);
                if (E::PAIRS) v *= sa * (g.scale_b ? g.scale_b[k.n + c] : 1.0f);
                if (g.bias) v += load_any(g.bias, g.bias_type, k.n + c);
                const float a = g.aux_in ? (float)k.in[m * g.ld_in + c] : 0.0f;
                if (g.grad) {
                    act_slopes<1>(g.act, &v, &a);
                } else {
                    if (g.aux_out) k.out[m * g.ld_out + c] = (typename K::T)v;
                    act_values<1>(g.act, &v);
                    v += a;
                }
                k.C[m * g.ldc + c] = (typename K::T)v;
            }
        }
    }
    template <class E, int... U>
    static __device__ __forceinline__ void pass_steps(const EpiArgs& g, const Columns<E>& k, const char* st, int mp,
                                                      std::integer_sequence<int, U...>) {
        (row_step<U, E>(g, k, st, mp), ...);
    }

    template <bool PARTS, class E>
    static __device__ __forceinline__ void store(E& e, const EpiArgs& g, int m0, int n0,
                                                 const typename E::Parts& pt) {
        typedef typename E::Config Cfg;
        typedef Columns<E> K;
        typedef typename K::L L;
        static_assert(Cfg::TN == 64 && Cfg::STAGE_W == RS * 256, "staging shape");
        int ln = e.lane, tt = e.tid;   // opaque: addresses are formed here, not hoisted over the K loop
        asm volatile("" : "+v"(ln));
        if (PARTS) asm volatile("" : "+v"(tt));
        char* st = e.ldsc + e.wave * Cfg::STAGE_W;
        K k;
        k.row = ln / K::LPR;
        k.col = (ln % K::LPR) * L::E;
        k.n = n0 + e.wn * Cfg::TN + k.col;
        k.valid = g.N - k.n;
        k.in = static_cast<const typename K::T*>(g.aux_in) + k.n;
        k.out = static_cast<typename K::T*>(g.aux_out) + k.n;
        k.C = static_cast<typename K::T*>(g.C) + k.n;
#pragma unroll
        for (int c = 0; c < L::E; ++c) {
            k.bias[c] = g.bias && c < k.valid ? load_any(g.bias, g.bias_type, k.n + c) : 0.0f;
            k.sb[c] = E::PAIRS && g.scale_b && c < k.valid ? g.scale_b[k.n + c] : 1.0f;
        }
        const int mw = m0 + e.wm * Cfg::TM + k.row;
#pragma unroll 1
        for (int p = 0; p < 2 * Cfg::FM; ++p) {
            const int mp = mw + p * RS;
#pragma unroll
            for (int u = 0; u < K::NU; ++u) {
                const long long m = mp + u * K::RPU;
                k.rows[u] = u32x4{0, 0, 0, 0};
                if (g.aux_in && m < g.M && k.valid >= L::E)
                    k.rows[u] = *reinterpret_cast<const typename L::V*>(k.in + m * g.ld_in);
            }
            stage_any<PARTS>(e, p, st, ln & 31, ln >> 5, tt, pt, std::make_integer_sequence<int, 2 * Cfg::FM>{});
            pass_steps<E>(g, k, st, mp, std::make_integer_sequence<int, K::NU>{});
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

// Kernel instances with the fused epilogue.  The edge paths only (they differ from the
// whole-tile paths by a compare and a select per load), and two loops: stream-K, and the
// nested cross-tile loop for every other mode (a program of one tile is its tiled form).
enum : int { EPI_STREAMK = 1, EPI_XTILE = 2 };   // kernel kinds

template <class Cfg, class TI, class TO, int PATH>
const void* epi_kernel_by_kind(int kind) {
    if (kind == EPI_STREAMK)
        return reinterpret_cast<const void*>(&gemm_tiles_kernel<Cfg, TI, TO, PATH, MODE_STREAMK, FusedStore>);
    return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH, false, FusedStore>);
}

// One function per tile configuration and input type, each in its own translation unit.
const void* epi_kernels_cfg128_f16(int out_f32, int path, int kind);
const void* epi_kernels_cfg128_bf16(int out_f32, int path, int kind);
const void* epi_kernels_cfg128_e4m3(int out, int path, int kind);
const void* epi_kernels_cfg256w8_f16(int out_f32, int path, int kind);
const void* epi_kernels_cfg256w8_bf16(int out_f32, int path, int kind);
const void* epi_kernels_cfg256w8_e4m3(int out, int path, int kind);

template <class Cfg, class TI, class TO>
const void* epi_kernel(int path, int kind) {
    if constexpr (std::is_same<TI, InE4M3>::value) {
        return epi_kernel_by_kind<Cfg, TI, TO, PATH_EDGE_BT>(kind);
    } else {
        switch (path) {
            case PATH_EDGE_BT: return epi_kernel_by_kind<Cfg, TI, TO, PATH_EDGE_BT>(kind);
            case PATH_EDGE_AT: return epi_kernel_by_kind<Cfg, TI, TO, PATH_EDGE_AT>(kind);
            case PATH_EDGE_ATBT: return epi_kernel_by_kind<Cfg, TI, TO, PATH_EDGE_ATBT>(kind);
            default: return epi_kernel_by_kind<Cfg, TI, TO, PATH_EDGE>(kind);
        }
    }
}

}  // namespace ts

// The fused epilogue of the tiled product: bias, activation, residual and the scales of
// 8-bit operands, applied to the fp32 accumulators before their one rounding, and the
// activations with their derivatives.
//
//   z = (acc * scale_a[m]) * scale_b[n] + bias[n]      (scales: 8-bit operands only; in this order
//                                                       on every path, as their own product may
//                                                       leave the range)
//   forward   preact = z;  C = act(z) + residual
//   gradient  C = z * act'(preact)
//
// Every term is formed in fp32; preact and C are each rounded once, to C's type.
#pragma once

#include <limits.h>

#include "gemm_kernel.hpp"

namespace ts {

// Activations (same numbering as TS_ACT_* in tsgemm.h).
enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };
// Element types (same numbering as TS_F16, TS_BF16, TS_F32, TS_E4M3, TS_I8, TS_Q8); 0 = absent.
enum : int { ELT_NONE = 0, ELT_F16 = 1, ELT_BF16 = 2, ELT_F32 = 3, ELT_E4M3 = 4, ELT_I8 = 5, ELT_Q8 = 6 };

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

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

// The activation is one wave-uniform number; silu and gelu_tanh are one function with
// different coefficients: z sigmoid(z (w0 + w1 z^2)).  Calls f(tag) with the family's tag.
enum : int { FAM_NONE = 0, FAM_RELU = 1, FAM_ERF = 2, FAM_SIGMOID = 3 };
// The coefficients carry the -log2(e) of the exponential: 1 / (1 + 2^(z (e0 + e1 z^2))).
struct Sigmoid {
    float e0, e1;
};
// From here on the sigmoid of both is 1 in fp32; the argument stops there, as silu's e1 z would be
// 0 times infinity at the end of the range.  NaN comes back through the factor z.
constexpr float kSaturated = 64.0f;
__device__ __forceinline__ Sigmoid sigmoid_of(int act) {
    return act == ACT_SILU ? Sigmoid{-kLog2e, 0.0f} : Sigmoid{-kLog2e * kTanhW0, -kLog2e * kTanhW1};
}
__device__ __forceinline__ float sigmoid(float z, Sigmoid c) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * __builtin_fmaf(c.e1 * z, z, c.e0)));
}
template <int FAM>
__device__ __forceinline__ float fam_value(float z, Sigmoid c) {
    if constexpr (FAM == FAM_RELU) return z < 0.0f ? 0.0f : z;   // NaN stays NaN
    if constexpr (FAM == FAM_ERF) {
        const float q = tail_scaled(__builtin_fabsf(z)) * __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z);
        return z * (z < 0.0f ? q : 1.0f - q);
    }
    if constexpr (FAM == FAM_SIGMOID) return z * sigmoid(__builtin_fminf(z, kSaturated), c);
    return z;
}
template <int FAM>
__device__ __forceinline__ float fam_slope(float z, Sigmoid c) {
    if constexpr (FAM == FAM_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    if constexpr (FAM == FAM_ERF) {
        const float e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z);
        const float q = tail_scaled(__builtin_fabsf(z)) * e;
        return __builtin_fmaf(z * kInvSqrt2Pi, e, z < 0.0f ? q : 1.0f - q);
    }
    if constexpr (FAM == FAM_SIGMOID) {
        const float g = sigmoid(z, c);
        // where z^2 overflows, g (1 - g) is 0: the factor beside it stays finite
        const float d = -kLn2 * __builtin_fmaxf(__builtin_fmaf(3.0f * c.e1 * z, z, c.e0), -1e30f);
        return __builtin_fmaf(z * (g * (1.0f - g)), d, g);
    }
    return 1.0f;
}
template <class F>
__device__ __forceinline__ void with_family(int act, F&& f) {
    if (act == ACT_RELU) f(std::integral_constant<int, FAM_RELU>{});
    else if (act == ACT_GELU) f(std::integral_constant<int, FAM_ERF>{});
    else if (act != ACT_NONE) f(std::integral_constant<int, FAM_SIGMOID>{});
}
template <int E>
__device__ __forceinline__ void act_values(int act, float* v) {
    const Sigmoid c = sigmoid_of(act);
    with_family(act, [&](auto fam) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = fam_value<decltype(fam)::value>(v[e], c);
    });
}
// v[e] *= act'(z[e])
template <int E>
__device__ __forceinline__ void act_slopes(int act, float* v, const float* z) {
    const Sigmoid c = sigmoid_of(act);
    with_family(act, [&](auto fam) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= fam_slope<decltype(fam)::value>(z[e], c);
    });
}

// ---- int8 products -----------------------------------------------------------------------
//
// Their sums are exact, so with every later term rounded on its own, and in the same order, all schedules, K
// splits, row counts and tiles (inside C and on its edge) give the same bits: z is one product and one fused
// multiply-add, a missing scale 1 and a missing bias 0.  Left to itself the compiler joins terms where it sees them
// in one piece of code: gelu's 1 - q, z gate + residual, what comes last with the conversion to fp16.
__device__ __forceinline__ float scaled_apart(float sum, float scale_a, float scale_b, float bias) {
    float z = __builtin_fmaf(sum * scale_a, scale_b, bias);
    asm("" : "+v"(z));
    return z;
}
// fam_value of such a z.
template <int FAM>
__device__ __forceinline__ float value_apart(float z, Sigmoid coeff) {
    if constexpr (FAM == FAM_ERF) {
#pragma clang fp contract(off)
        const float q = tail_scaled(__builtin_fabsf(z)) * __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z);
        const float r = 1.0f - q;
        z = z * (z < 0.0f ? q : r);
    } else {
        z = fam_value<FAM>(z, coeff);
    }
    asm("" : "+v"(z));
    return z;
}
template <int E>
__device__ __forceinline__ void values_apart(int act, float* v) {
    const Sigmoid c = sigmoid_of(act);
    with_family(act, [&](auto fam) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = value_apart<decltype(fam)::value>(v[e], c);
    });
}
__device__ __forceinline__ float sum_apart(float a, float b) {
#pragma clang fp contract(off)
    float s = a + b;
    asm("" : "+v"(s));
    return s;
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

// E (4 or 8) consecutive elements of a vector of any type; those at or past `valid` keep v.
template <int E, class TO>
__device__ __forceinline__ void load_columns_of(const void* p, long long n, int valid, float* v) {
    constexpr int STEP = Elt<TO>::E < E ? Elt<TO>::E : E;   // 4 or 8 elements an access
    const typename Elt<TO>::T* q = static_cast<const typename Elt<TO>::T*>(p) + n;
    float t[8];
    if (valid >= E) {
        if constexpr (Elt<TO>::E == 8 && E == 4) {   // 8 bytes
            typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
            const u32x2 w = *reinterpret_cast<const u32x2_a2*>(q);
            unpack_row<TO>(u32x4{w[0], w[1], 0, 0}, t);
        } else {
#pragma unroll
            for (int c = 0; c < E; c += STEP) unpack_row<TO>(load_row<TO>(q + c, STEP), t + c);
        }
#pragma unroll
        for (int c = 0; c < E; ++c) v[c] = t[c];
    } else {
#pragma unroll
        for (int c = 0; c < E; ++c)
            if (c < valid) v[c] = (float)q[c];
    }
}
template <int E>
__device__ __forceinline__ void load_columns(const void* p, int type, long long n, int valid, float* v) {
    if (type == ELT_F32) load_columns_of<E, OutF32>(p, n, valid, v);
    else if (type == ELT_F16) load_columns_of<E, OutF16>(p, n, valid, v);
    else load_columns_of<E, OutBF16>(p, n, valid, v);
}

// ---- the tile epilogue -------------------------------------------------------------------

struct EpiArgs : GemmArgs {
    const void* bias;       // N elements of bias_type, or null
    const void* aux_in;     // residual (forward) or preact (gradient), C's type, or null
    void* aux_out;          // preact (forward), C's type, or null
    long long ld_in, ld_out;
    const float *scale_a, *scale_b;   // 8-bit operands: M and N fp32 (null: 1)
    int bias_type, act, grad;
    int stagger;            // sleeps (320 clocks) between the starts of consecutive groups of programs
    // preact as rows of 8-bit values and exponents (checkpoint.hpp), written (forward) or read (gradient)
    // by CheckpointStore and split_finish_kernel in place of aux_out and aux_in; null elsewhere
    uint8_t* kept;
    long long ld_kept;      // bytes
};

// The launch's arguments, read anew from the kernel argument segment: scalars that only the
// epilogue needs are then not held (spilled to vector registers) through the K loop.
__device__ __forceinline__ const EpiArgs& fresh_args() {
    typedef const __attribute__((address_space(4))) EpiArgs* P;
    P p = (P)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const EpiArgs*)p;
}
// A constant in a register that is not held between its uses.
__device__ __forceinline__ float fresh(float c) {
    asm volatile("" : "+v"(c));
    return c;
}

// Epilogue and store of one tile, in the accumulators' own layout: a lane holds, in block
// (i, j) of its wave's sub-tile, columns 32 j + 8 q + 4 hk .. + 3 (q = 0 .. 3) of row
// 32 i + r32.  Scales and bias are applied in place; then a block is taken to 16 registers of
// its own, worked on there, and staged, rounded, in the wave's 4 KiB of LDS: 32 rows of 128 bytes,
// the 64 columns of a row of blocks in 16 bits, or 32 columns in fp32, 16-byte chunks
// XOR-swizzled by row.  From there it leaves as whole 128-byte row segments, 16 bytes a lane;
// a matrix that is read (residual, preact) comes the other way through the same bytes.
// The blocks are one rolled loop, in which only the taking of accumulators (fixed registers)
// has a copy per block: unrolled, with every activation in every copy, the code is too
// long, and accumulators changed in place behind branches end up spilled.  (An earlier form
// staged fp32 for all types and decided per row segment on the way out: a dozen branches and
// twice the LDS traffic per segment, 5 us a 256 x 256 tile.)
struct FusedStore {
    typedef EpiArgs Args;
    static constexpr int MIN_WAVES = 2;   // two workgroups of the 128 tile, or one of the 256 tile, on a CU
    static constexpr bool RENEW = true;
    // Programs start in eight groups, g.stagger sleeps apart (see stagger_sleeps).
    static __device__ __forceinline__ void start(const EpiArgs& g) {
        const int n = ((blockIdx.x >> 3) & 7) * g.stagger;
        for (int i = 0; i < n; ++i) __builtin_amdgcn_s_sleep(5);
    }
    static constexpr int NQ = 4;   // quads of a lane in a block
    static constexpr int NU = 4;   // 16-byte accesses of a lane to the staged 4 KiB

    // What the blocks of a tile share.
    struct Tile {
        char* st;         // the wave's staging area
        int ln, r32, hk;
        int m, n;         // first row and column of the wave's sub-tile
        int M, N;
        bool whole;       // its 64 columns are all before N (wave-uniform)
    };
    static __device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }
    // Staged bytes: unit u of this lane (row 8 u + ln / 8, chunk ln mod 8), and `bytes` at
    // byte `at` of row r32.
    static __device__ __forceinline__ char* unit_lds(const Tile& t, int u) {
        const int row = 8 * u + (t.ln >> 3);
        return t.st + row * 128 + (((t.ln & 7) ^ swz(row)) << 4);
    }
    static __device__ __forceinline__ char* quad_lds(const Tile& t, int at) {
        return t.st + t.r32 * 128 + (((at >> 4) ^ swz(t.r32)) << 4) + (at & 15);
    }
    // Unit u in a matrix of C's type whose staged part begins at row m, column n: that address
    // is scalar, the lane's offset 32 bits wide (the host keeps row strides below 2^26).
    template <class T>
    static __device__ __forceinline__ T* unit_at(const Tile& t, const void* base, long long ld, int m, int n, int u) {
        char* p = static_cast<char*>(const_cast<void*>(base)) + ((m + 8 * u) * ld + n) * (long long)sizeof(T);
        return reinterpret_cast<T*>(p + ((uint32_t)(t.ln >> 3) * (uint32_t)ld * (uint32_t)sizeof(T) + (uint32_t)(t.ln & 7) * 16u));
    }

    template <class E>
    static __device__ __forceinline__ Tile tile_of(const E& e, const EpiArgs& g, int m0, int n0) {
        Tile t;
        t.ln = E::fresh_lane();   // addresses are formed here, not hoisted over the K loop
        t.st = e.ldsc + e.wave * E::Config::STAGE_W;
        t.r32 = t.ln & 31;
        t.hk = t.ln >> 5;
        t.m = m0 + e.wm * E::Config::TM;
        t.n = n0 + e.wn * E::Config::TN;
        t.M = g.M;
        t.N = g.N;
        t.whole = t.n + E::Config::TN <= g.N;
        return t;
    }

    // Block B (i = B / FN, j = B mod FN) of the accumulators.  The empty asm statements keep
    // the compiler from merging the copies for different B, which would select the
    // accumulators by address, in memory.
    template <int B, class E>
    static __device__ __forceinline__ void take(const E& e, float (*v)[4]) {
        constexpr int i = B / E::FN, j = B % E::FN;
        asm volatile("" ::"n"(B));
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int c = 0; c < 4; ++c) v[q][c] = e.acc[i][j][4 * q + c];
        asm volatile("" ::"n"(B));
    }
    template <class E, int... B>
    static __device__ __forceinline__ void take_any(int b, const E& e, float (*v)[4], std::integer_sequence<int, B...>) {
        ((b == B ? take<B>(e, v) : (void)0), ...);
    }
    // Scales and bias of this lane's columns in block column j.
    template <class E>
    static __device__ __forceinline__ void columns(const EpiArgs& g, const Tile& t, int j, float (*sb)[4], float (*bias)[4]) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const int n = t.n + 4 * t.hk + 32 * j + 8 * q;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sb[q][c] = E::PAIRS ? fresh(1.0f) : 1.0f;
                bias[q][c] = fresh(0.0f);
            }
            if (E::PAIRS && g.scale_b) load_columns<4>(g.scale_b, ELT_F32, n, t.whole ? 4 : g.N - n, sb[q]);
            if (g.bias) load_columns<4>(g.bias, g.bias_type, n, t.whole ? 4 : g.N - n, bias[q]);
        }
    }
    // z in place of the sums, in straight runs (no branch around them): partial sums of a
    // split tile, scales, bias.
    template <bool PARTS, class E>
    static __device__ __forceinline__ void finish_sums(E& e, const EpiArgs& g, const Tile& t, const typename E::Parts& pt) {
        float sa[E::FM];
#pragma unroll
        for (int i = 0; i < E::FM; ++i) {
            const int m = t.m + 32 * i + t.r32;
            sa[i] = E::PAIRS && g.scale_a && m < g.M ? g.scale_a[m] : 1.0f;
        }
        const int tt = e.wave * 64 + t.ln;
#pragma unroll
        for (int j = 0; j < E::FN; ++j) {
            float sb[NQ][4], bias[NQ][4];
            columns<E>(g, t, j, sb, bias);
#pragma unroll
            for (int i = 0; i < E::FM; ++i)
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    float a[4] = {e.acc[i][j][4 * q], e.acc[i][j][4 * q + 1], e.acc[i][j][4 * q + 2], e.acc[i][j][4 * q + 3]};
                    if (PARTS) e.add_parts(a, pt, (i * E::FN + j) * 4 + q, tt);
                    if (E::INTS) {   // one rounding of the exact sum (none below 2^24)
#pragma unroll
                        for (int c = 0; c < 4; ++c) a[c] = (float)__builtin_bit_cast(int, a[c]);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        e.acc[i][j][4 * q + c] = E::PAIRS ? __builtin_fmaf(a[c] * sa[i], sb[q][c], bias[q][c]) : a[c] + bias[q][c];
                }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // The staged part of a matrix that begins at (m, n), one unit per u.
    template <class TO>
    static __device__ __forceinline__ void fetch(const Tile& t, const void* base, long long ld, int m, int n, u32x4* rows) {
        typedef typename Elt<TO>::T T;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const T* s = unit_at<T>(t, base, ld, m, n, u);
            rows[u] = u32x4{0, 0, 0, 0};
            if (m + 8 * u + (t.ln >> 3) < t.M)
                rows[u] = t.whole ? *reinterpret_cast<const typename Elt<TO>::V*>(s)
                                  : load_row<TO>(s, t.N - (n + (t.ln & 7) * Elt<TO>::E));
        }
    }
    template <class TO>
    static __device__ __forceinline__ void flush(const Tile& t, void* base, long long ld, int m, int n) {
        typedef typename Elt<TO>::T T;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(unit_lds(t, u));
            if (m + 8 * u + (t.ln >> 3) < t.M) {
                T* p = unit_at<T>(t, base, ld, m, n, u);
                if (t.whole)
                    *reinterpret_cast<typename Elt<TO>::V*>(p) = w;
                else
                    store_row<TO>(p, w, t.N - (n + (t.ln & 7) * Elt<TO>::E));
            }
        }
    }

    // The sums themselves, fp32, to a matrix of whole tiles.
    template <class E>
    static __device__ __forceinline__ void store_sums(E& e, const EpiArgs& g, int m0, int n0, float* base, long long ld) {
        Tile t = tile_of(e, g, m0, n0);
        t.M = INT_MAX;
        t.whole = true;
#pragma unroll
        for (int i = 0; i < E::FM; ++i)
#pragma unroll
            for (int j = 0; j < E::FN; ++j) {
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    const float v[4] = {e.acc[i][j][4 * q], e.acc[i][j][4 * q + 1], e.acc[i][j][4 * q + 2], e.acc[i][j][4 * q + 3]};
                    Out<OutF32>::store4(reinterpret_cast<float*>(quad_lds(t, 16 * t.hk + 32 * q)), v, 4, true);
                }
                flush<OutF32>(t, base, ld, t.m + 32 * i, t.n + 32 * j);
                __builtin_amdgcn_sched_barrier(0);
            }
    }
    template <bool PARTS, class E>
    static __device__ __forceinline__ void store(E& e, const EpiArgs&, int m0, int n0, const typename E::Parts& pt) {
        const EpiArgs& g = fresh_args();
        typedef typename E::Config Cfg;
        typedef typename E::OutType TO;
        typedef typename Elt<TO>::T T;
        static_assert(Cfg::TN == 64 && Cfg::STAGE_W == 4096 && Cfg::FN == 2, "staging shape");
        constexpr int OSZ = sizeof(T);
        constexpr int JB = OSZ == 2 ? 2 : 1;               // blocks staged together
        const Tile t = tile_of(e, g, m0, n0);
        finish_sums<PARTS>(e, g, t, pt);
        const Sigmoid coeff = sigmoid_of(g.act);
        // preact first (where it is wanted), then C
#pragma unroll 1
        for (int out = g.aux_out ? 0 : 1; out < 2; ++out) {
            void* base = out ? g.C : g.aux_out;
            const long long ld = out ? g.ldc : g.ld_out;
            const bool read = out && g.aux_in;
#pragma unroll 1
            for (int b = 0; b < Cfg::FM * Cfg::FN; ++b) {
                const int j = b % Cfg::FN;
                const int m = t.m + 32 * (b / Cfg::FN), n = JB == 2 ? t.n : t.n + 32 * j;   // of the staged part
                if (read && b % JB == 0) {
                    u32x4 rows[NU];
                    fetch<TO>(t, g.aux_in, g.ld_in, m, n, rows);
#pragma unroll
                    for (int u = 0; u < NU; ++u) *reinterpret_cast<u32x4*>(unit_lds(t, u)) = rows[u];
                }
                float v[NQ][4];
                take_any(b, e, v, std::make_integer_sequence<int, Cfg::FM * Cfg::FN>{});
                const int at0 = 4 * t.hk * OSZ + (JB == 2 ? 32 * j * OSZ : 0);
                if (out && !g.grad)
                    with_family(g.act, [&](auto fam) {
#pragma unroll
                        for (int q = 0; q < NQ; ++q)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                v[q][c] = E::INTS ? value_apart<decltype(fam)::value>(v[q][c], coeff)
                                                  : fam_value<decltype(fam)::value>(v[q][c], coeff);
                    });
                if (read) {
                    float w[NQ][4];
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        float f[8];
                        if constexpr (OSZ == 4) {
                            unpack_row<TO>(*reinterpret_cast<const u32x4*>(quad_lds(t, at0 + 8 * q * OSZ)), f);
                        } else {
                            const u32x2 h = *reinterpret_cast<const u32x2*>(quad_lds(t, at0 + 8 * q * OSZ));
                            unpack_row<TO>(u32x4{h[0], h[1], 0, 0}, f);
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c) w[q][c] = f[c];
                    }
                    if (g.grad) {
                        with_family(g.act, [&](auto fam) {
#pragma unroll
                            for (int q = 0; q < NQ; ++q)
#pragma unroll
                                for (int c = 0; c < 4; ++c) v[q][c] *= fam_slope<decltype(fam)::value>(w[q][c], coeff);
                        });
                    } else {
#pragma unroll
                        for (int q = 0; q < NQ; ++q)
#pragma unroll
                            for (int c = 0; c < 4; ++c) v[q][c] = E::INTS ? sum_apart(v[q][c], w[q][c]) : v[q][c] + w[q][c];
                    }
                }
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                    Out<TO>::store4(reinterpret_cast<T*>(quad_lds(t, at0 + 8 * q * OSZ)), v[q], 4, true);
                if (b % JB == JB - 1) flush<TO>(t, base, ld, m, n);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
};

// K of a product with few tiles, split: program (split, tile) sums the K steps
// [ks split / splits, ks (split + 1) / splits) of one tile and stores the fp32 sums, in whole
// tiles, to a matrix of its split's own; split_finish_kernel (split_finish.hip) adds them in
// order of the splits and applies the epilogue.  Programs that share a column panel of B (the
// tiles of one tile column, one split) are neighbours on one XCD.
struct SplitArgs : EpiArgs {
    float* sums;              // [splits][rows of whole tiles][ld_sums]
    long long ld_sums, split_stride;   // fp32 elements
    int splits;
};
template <class Cfg, class TI, class TO, int PATH>
__global__ void __launch_bounds__(Cfg::NT) __attribute__((amdgpu_waves_per_eu(2)))
gemm_split_kernel(SplitArgs g) {
    __shared__ __attribute__((aligned(16))) char lds_a0[Cfg::A_SLOT], lds_a1[Cfg::A_SLOT];
    __shared__ __attribute__((aligned(16))) char lds_b0[Cfg::B_SLOT], lds_b1[Cfg::B_SLOT];
    __shared__ __attribute__((aligned(16))) char lds_c[Cfg::C_BYTES > 0 ? Cfg::C_BYTES : 16];
    typedef Engine<Cfg, TI, TO, PATH> E;
    E e(g, lds_a0, lds_a1, lds_b0, lds_b1, lds_c);
    const int p = xcd_remap(blockIdx.x, gridDim.x, g.s.xcds);
    const int col = p / g.s.nm, tm = p - col * g.s.nm;
    const int split = col / g.s.nn, tn = col - split * g.s.nn;
    const int m0 = tm * Cfg::BM, n0 = tn * Cfg::BN;
    const int k0 = (int)((long long)g.s.ks * split / g.splits), k1 = (int)((long long)g.s.ks * (split + 1) / g.splits);
    e.zero_acc();
    e.template tile_mainloop<true>(m0, n0, k0, k1);
    FusedStore::store_sums(e, g, m0, n0, g.sums + split * g.split_stride, g.ld_sums);
    e.drain();
}

// The same for one activation family and one use of aux_in, for the 256 tile: a tile inside
// M x N runs as one straight piece of code in which every accumulator, wait and store is fixed
// at compile time.  A load's wait then leaves the stores issued after it in flight (loads
// and stores retire in order on one counter; behind a branch the compiler has to wait for
// all of them), so the rows of aux_in are fetched one staged part ahead.  Tiles on the edge
// take FusedStore.  Against it, us, 4096 x 16384, bf16 C: K = 1024 none 124 / 133, gelu 156 / 169, residual
// 143 / 165, with relu 142 / 165, gelu with preact 163 / 187, relu's gradient 146 / 170; K = 4096 3 to 27 less in
// 420 to 480; fp32 C level without aux_in, with residual and relu 172 / 214 (K = 1024) and 469 / 510 (4096).
// AUX_LINES: preact and C in 16 bits, rows of whole 128-byte lines: stored past the caches, so that
// the two streams do not push the operands out of them (4096 x 16384 x 4096 gelu 464 -> 440 us, 16384 x
// 8192 x 2048 530 -> 503; with rows that share lines such stores cost 170 -> 211 us, 5000 x 12290 x 1000,
// and without preact they gain nothing).
enum : int { AUX_NONE = 0, AUX_RESIDUAL = 1, AUX_GRAD = 2, AUX_PREACT = 3, AUX_LINES = 4 };
template <int FAM, int AUX>
struct SpecialStore {
    typedef EpiArgs Args;
    static constexpr int MIN_WAVES = 2;
    static constexpr bool RENEW = true;
    typedef FusedStore G;
    static __device__ __forceinline__ void start(const EpiArgs& g) { G::start(g); }
    static constexpr int NQ = G::NQ, NU = G::NU;
    static constexpr bool IN = AUX == AUX_RESIDUAL || AUX == AUX_GRAD;   // aux_in is read
    static constexpr bool PRE = AUX == AUX_PREACT || AUX == AUX_LINES;   // preact is written

    // A walk over the staged parts of a matrix of C's type: the address of the part's first
    // row is scalar and moves on from part to part (opaque, or the addresses of all parts are
    // formed at once and spilled), the lane's offset 32 bits wide.
    template <class E>
    struct Walk {
        typedef typename E::OutType TO;
        typedef typename Elt<TO>::T T;
        static constexpr int OSZ = sizeof(T), JB = OSZ == 2 ? 2 : 1;   // blocks in a part
        static constexpr int NP = E::FM * E::FN / JB;                  // parts of a tile
        char* p;
        long long row8;
        uint32_t lane;
        __device__ __forceinline__ Walk(const G::Tile& t, const void* base, long long ld)
            : p(static_cast<char*>(const_cast<void*>(base)) + (t.m * ld + t.n) * (long long)OSZ), row8(8 * ld * OSZ),
              lane((uint32_t)(t.ln >> 3) * (uint32_t)ld * (uint32_t)OSZ + (uint32_t)(t.ln & 7) * 16u) {}
        __device__ __forceinline__ typename Elt<TO>::V* unit(int u) const {
            return reinterpret_cast<typename Elt<TO>::V*>(p + u * row8 + lane);
        }
        // to part q + 1 from part q
        __device__ __forceinline__ void next(int q) {
            if (JB == 2 || q % E::FN == E::FN - 1)
                p += 4 * row8 - (JB == 1 ? 128 * (E::FN - 1) : 0);
            else
                p += 128;   // 32 fp32 columns on
            asm volatile("" : "+s"(p));
        }
        __device__ __forceinline__ void fetch(u32x4* rows) const {
#pragma unroll
            for (int u = 0; u < NU; ++u) rows[u] = *unit(u);
        }
        __device__ __forceinline__ void store(const G::Tile& t) const {
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const typename Elt<TO>::V v = *reinterpret_cast<const u32x4*>(G::unit_lds(t, u));
                if constexpr (AUX == AUX_LINES)
                    __builtin_nontemporal_store(v, unit(u));
                else
                    *unit(u) = v;
            }
        }
    };
    // z of quad q of block (i, j).
    template <class E>
    static __device__ __forceinline__ void z_of(const E& e, int i, int j, int q, const float (*bias)[4], float* v) {
        static_assert(!E::PAIRS, "16-bit operands (the scales of 8-bit ones cost the registers this form needs)");
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = e.acc[i][j][4 * q + c] + bias[j * NQ + q][c];
    }
    // fp32 C beside a matrix that is read: parts of 16 rows of the wave's 64 columns, 256 bytes a
    // row.  Lanes of the other 16 rows of a block skip the write of a part, and aux_in is joined
    // on the way out, where a lane holds the same 16 bytes of it, so it needs no way through LDS;
    // its rows are fetched one part ahead, past the caches (they are read once).  Where C's rows
    // are not whole lines, a line that two segments share leaves the L2 in one piece only if both come
    // soon after another: with segments of 128 bytes, a block's time between neighbours, and the
    // residual passing through the L2 besides, 5000 x 12290 x 1000 took 250 us, now 215 (B [N][K] 253,
    // 208); 4096 x 16384 x 256 125, now 102.  Without aux_in the two forms are level.
    template <class E>
    struct WideWalk {
        char* p;
        long long row4;
        uint32_t lane;
        __device__ __forceinline__ WideWalk(const G::Tile& t, const void* base, long long ld)
            : p(static_cast<char*>(const_cast<void*>(base)) + (t.m * ld + t.n) * 4), row4(16 * ld),
              lane((uint32_t)(t.ln >> 4) * (uint32_t)ld * 4u + (uint32_t)(t.ln & 15) * 16u) {}
        __device__ __forceinline__ u32x4_a4* unit(int u) const { return reinterpret_cast<u32x4_a4*>(p + u * row4 + lane); }
        __device__ __forceinline__ void next() {
            p += 4 * row4;
            asm volatile("" : "+s"(p));
        }
        __device__ __forceinline__ void fetch(u32x4* rows) {
#pragma unroll
            for (int u = 0; u < NU; ++u) rows[u] = __builtin_nontemporal_load(unit(u));
            next();
        }
    };
    template <class E>
    static __device__ __forceinline__ void store_wide(E& e, const EpiArgs& g, const G::Tile& t) {
        static_assert(E::FN == 2, "64 columns of a wave");
        constexpr int NP = 2 * E::FM;
        WideWalk<E> in(t, g.aux_in, g.ld_in), w(t, g.C, g.ldc);
        u32x4 rows[2][NU];
        in.fetch(rows[0]);
        float bias[E::FN * NQ][4], one[NQ][4];
        if constexpr (AUX == AUX_RESIDUAL) {
#pragma unroll
            for (int j = 0; j < E::FN; ++j) G::template columns<E>(g, t, j, one, bias + j * NQ);
        }
        const Sigmoid coeff = sigmoid_of(g.act);
        const int r16 = t.r32 & 15;
        char* wr = t.st + r16 * 256;
        const char* rd = t.st + (t.ln >> 4) * 256;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int i = p / 2;
            float v[E::FN * NQ][4];
#pragma unroll
            for (int x = 0; x < E::FN * NQ; ++x)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float a = e.acc[i][x / NQ][4 * (x % NQ) + c];
                    if (p % 2 == 0 && AUX == AUX_RESIDUAL) a = fam_value<FAM>(a + bias[x][c], coeff);
                    e.acc[i][x / NQ][4 * (x % NQ) + c] = a;
                    v[x][c] = a;
                }
            if ((t.r32 >> 4) == p % 2) {
#pragma unroll
                for (int x = 0; x < E::FN * NQ; ++x)
                    Out<OutF32>::store4(reinterpret_cast<float*>(wr + (((2 * x + t.hk) ^ r16) << 4)), v[x], 4, true);
            }
            if (p + 1 < NP) in.fetch(rows[(p + 1) % 2]);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                f32x4 c = __builtin_bit_cast(f32x4, *reinterpret_cast<const u32x4*>(rd + u * 1024 + (((t.ln & 15) ^ (4 * u + (t.ln >> 4))) << 4)));
                const f32x4 r = __builtin_bit_cast(f32x4, rows[p % 2][u]);
#pragma unroll
                for (int k = 0; k < 4; ++k) c[k] = AUX == AUX_GRAD ? c[k] * fam_slope<FAM>(r[k], coeff) : c[k] + r[k];
                *w.unit(u) = __builtin_bit_cast(u32x4, c);
            }
            w.next();
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    template <bool PARTS, class E>
    static __device__ __forceinline__ void store(E& e, const EpiArgs&, int m0, int n0, const typename E::Parts& pt) {
        const EpiArgs& g = fresh_args();
        typedef typename E::OutType TO;
        typedef typename Elt<TO>::T T;
        typedef Walk<E> K;
        if (m0 + E::BM > g.M || n0 + E::BN > g.N) {
            G::store<PARTS>(e, g, m0, n0, pt);
            return;
        }
        const G::Tile t = G::tile_of(e, g, m0, n0);
        if constexpr (K::OSZ == 4 && IN) {
            store_wide(e, g, t);
            return;
        }
        K in(t, g.aux_in, g.ld_in), pre(t, g.aux_out, g.ld_out), w(t, g.C, g.ldc);
        u32x4 rows[NU];
        if constexpr (IN) {
            in.fetch(rows);
            in.next(0);
        }
        float bias[E::FN * NQ][4], one[NQ][4];
#pragma unroll
        for (int j = 0; j < E::FN; ++j) G::template columns<E>(g, t, j, one, bias + j * NQ);
        const Sigmoid coeff = sigmoid_of(g.act);
#pragma unroll
        for (int p = 0; p < K::NP; ++p) {
            const int i = p * K::JB / E::FN, j0 = (p * K::JB) % E::FN;
            if constexpr (IN) {
#pragma unroll
                for (int u = 0; u < NU; ++u) *reinterpret_cast<u32x4*>(G::unit_lds(t, u)) = rows[u];
                if (p + 1 < K::NP) {
                    in.fetch(rows);
                    in.next(p + 1);
                }
            }
            if constexpr (PRE) {
#pragma unroll
                for (int x = 0; x < K::JB * NQ; ++x) {
                    float v[4];
                    z_of(e, i, j0 + x / NQ, x % NQ, bias, v);
                    Out<TO>::store4(reinterpret_cast<T*>(G::quad_lds(t, (4 * t.hk + 32 * (x / NQ) + 8 * (x % NQ)) * K::OSZ)), v, 4, true);
                }
                pre.store(t);
                pre.next(p);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int x = 0; x < K::JB * NQ; ++x) {
                float v[4];
                z_of(e, i, j0 + x / NQ, x % NQ, bias, v);
                char* at = G::quad_lds(t, (4 * t.hk + 32 * (x / NQ) + 8 * (x % NQ)) * K::OSZ);
                if constexpr (AUX != AUX_GRAD) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] = fam_value<FAM>(v[c], coeff);
                }
                if constexpr (IN) {
                    float f[8];
                    if constexpr (K::OSZ == 4) {
                        unpack_row<TO>(*reinterpret_cast<const u32x4*>(at), f);
                    } else {
                        const u32x2 h = *reinterpret_cast<const u32x2*>(at);
                        unpack_row<TO>(u32x4{h[0], h[1], 0, 0}, f);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] = AUX == AUX_GRAD ? v[c] * fam_slope<FAM>(f[c], coeff) : v[c] + f[c];
                }
                Out<TO>::store4(reinterpret_cast<T*>(at), v, 4, true);
            }
            w.store(t);
            w.next(p);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

// Kernel instances with the fused epilogue.  The edge paths only (they differ from the
// whole-tile paths by a compare and a select per load), and two loops: stream-K, and the
// nested cross-tile loop for every other mode (a program of one tile is its tiled form); and
// the 128 tile with K split.
// The special forms of the epilogue are kinds of the second.
enum : int { EPI_STREAMK = 1, EPI_XTILE = 2, EPI_SPLIT = 3, EPI_SPECIAL = 8 };   // EPI_SPECIAL + 4 * AUX_* + FAM_*

template <class Cfg, class TI, class TO, int PATH, int FAM, int AUX>
const void* epi_special() {
    return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH, false, SpecialStore<FAM, AUX>>);
}
// Two outputs in 16 bits; in fp32 the general form is faster (5000 x 12290 x 1000 relu 252 / 281 us,
// 4096 x 16384 x 1024 209 / 220).
template <class Cfg, class TI, class TO, int PATH, int FAM, int AUX>
const void* epi_special_two() {
    if constexpr (std::is_same<TO, OutF32>::value) return nullptr;
    else return epi_special<Cfg, TI, TO, PATH, FAM, AUX>();
}
// The special instances of one type and layout (null: none for this kind).
template <class Cfg, class TI, class TO, int PATH>
const void* epi_special_by_kind(int kind) {
    switch (kind) {
        case EPI_SPECIAL + 4 * AUX_NONE + FAM_NONE: return epi_special<Cfg, TI, TO, PATH, FAM_NONE, AUX_NONE>();
        case EPI_SPECIAL + 4 * AUX_NONE + FAM_RELU: return epi_special<Cfg, TI, TO, PATH, FAM_RELU, AUX_NONE>();
        case EPI_SPECIAL + 4 * AUX_NONE + FAM_ERF: return epi_special<Cfg, TI, TO, PATH, FAM_ERF, AUX_NONE>();
        case EPI_SPECIAL + 4 * AUX_NONE + FAM_SIGMOID: return epi_special<Cfg, TI, TO, PATH, FAM_SIGMOID, AUX_NONE>();
        case EPI_SPECIAL + 4 * AUX_RESIDUAL + FAM_NONE: return epi_special<Cfg, TI, TO, PATH, FAM_NONE, AUX_RESIDUAL>();
        case EPI_SPECIAL + 4 * AUX_RESIDUAL + FAM_RELU: return epi_special<Cfg, TI, TO, PATH, FAM_RELU, AUX_RESIDUAL>();
        case EPI_SPECIAL + 4 * AUX_RESIDUAL + FAM_ERF: return epi_special<Cfg, TI, TO, PATH, FAM_ERF, AUX_RESIDUAL>();
        case EPI_SPECIAL + 4 * AUX_RESIDUAL + FAM_SIGMOID: return epi_special<Cfg, TI, TO, PATH, FAM_SIGMOID, AUX_RESIDUAL>();
        case EPI_SPECIAL + 4 * AUX_PREACT + FAM_NONE: return epi_special_two<Cfg, TI, TO, PATH, FAM_NONE, AUX_PREACT>();
        case EPI_SPECIAL + 4 * AUX_PREACT + FAM_RELU: return epi_special_two<Cfg, TI, TO, PATH, FAM_RELU, AUX_PREACT>();
        case EPI_SPECIAL + 4 * AUX_PREACT + FAM_ERF: return epi_special_two<Cfg, TI, TO, PATH, FAM_ERF, AUX_PREACT>();
        case EPI_SPECIAL + 4 * AUX_PREACT + FAM_SIGMOID: return epi_special_two<Cfg, TI, TO, PATH, FAM_SIGMOID, AUX_PREACT>();
        case EPI_SPECIAL + 4 * AUX_LINES + FAM_ERF: return epi_special_two<Cfg, TI, TO, PATH, FAM_ERF, AUX_LINES>();
        case EPI_SPECIAL + 4 * AUX_LINES + FAM_SIGMOID: return epi_special_two<Cfg, TI, TO, PATH, FAM_SIGMOID, AUX_LINES>();
        case EPI_SPECIAL + 4 * AUX_GRAD + FAM_RELU: return epi_special<Cfg, TI, TO, PATH, FAM_RELU, AUX_GRAD>();
        case EPI_SPECIAL + 4 * AUX_GRAD + FAM_ERF: return epi_special<Cfg, TI, TO, PATH, FAM_ERF, AUX_GRAD>();
        case EPI_SPECIAL + 4 * AUX_GRAD + FAM_SIGMOID: return epi_special<Cfg, TI, TO, PATH, FAM_SIGMOID, AUX_GRAD>();
        default: return nullptr;
    }
}
// Each in its own translation unit: the 8-wave 256 tile, A [M][K] and B [K][N] or [N][K].
const void* epi_special_f16_nn(int out_f32, int kind);
const void* epi_special_f16_nt(int out_f32, int kind);
const void* epi_special_bf16_nn(int out_f32, int kind);
const void* epi_special_f16_tn(int out_f32, int kind);
const void* epi_special_bf16_tn(int out_f32, int kind);
const void* epi_special_bf16_nt(int out_f32, int kind);
const void* epi_special_i8(int out, int fam, int residual);   // epilogue_int8.hpp

template <class Cfg, class TI, class TO, int PATH>
const void* epi_kernel_by_kind(int kind) {
    if (kind == EPI_STREAMK)
        return reinterpret_cast<const void*>(&gemm_tiles_kernel<Cfg, TI, TO, PATH, MODE_STREAMK, FusedStore>);
    if constexpr (Cfg::BM == 128) {
        // the sums are fp32 whatever C's type, which for 8-bit operands still chooses the products
        // (int8: int32, the same for every type of C)
        typedef typename std::conditional<std::is_same<TI, InE4M3>::value && !std::is_same<TO, OutF32>::value, OutBF16, OutF32>::type TS;
        if (kind == EPI_SPLIT) return reinterpret_cast<const void*>(&gemm_split_kernel<Cfg, TI, TS, PATH>);
    }
    return reinterpret_cast<const void*>(&gemm_xtile_kernel<Cfg, TI, TO, PATH, false, FusedStore>);
}

// One function per tile configuration and input type, each in its own translation unit.
const void* epi_kernels_cfg128_f16(int out_f32, int path, int kind);
const void* epi_kernels_cfg128_bf16(int out_f32, int path, int kind);
const void* epi_kernels_cfg128_e4m3(int out, int path, int kind);
const void* epi_kernels_cfg256w8_f16(int out_f32, int path, int kind);
const void* epi_kernels_cfg256w8_bf16(int out_f32, int path, int kind);
const void* epi_kernels_cfg256w8_e4m3(int out, int path, int kind);
const void* epi_kernels_cfg128_i8(int out, int path, int kind);
const void* epi_kernels_cfg256w8_i8(int out, int path, int kind);
// With CheckpointStore (epilogue_checkpoint.hpp), or its special form for a family (-1: none): 16-bit
// operands.
const void* epi_checkpoint_f16(int cfg, int out_f32, int path, int fam);
const void* epi_checkpoint_bf16(int cfg, int out_f32, int path, int fam);

template <class Cfg, class TI, class TO>
const void* epi_kernel(int path, int kind) {
    if constexpr (is_8bit<TI>()) {
        return epi_kernel_by_kind<Cfg, TI, TO, PATH_EDGE_BT>(kind);
    } else {
        switch (path) {
            case PATH_EDGE_BT: return epi_kernel_by_kind<Cfg, TI, TO, PATH_EDGE_BT>(kind);
            case PATH_EDGE_AT: return epi_kernel_by_kind<Cfg, TI, TO, PATH_EDGE_AT>(kind);
            case PATH_EDGE_ATBT: return epi_kernel_by_kind<Cfg, TI, TO, PATH_EDGE_ATBT>(kind);
            default: return epi_kernel_by_kind<Cfg, TI, TO, PATH_EDGE_NN>(kind);
        }
    }
}

}  // namespace ts

// Layer norm of rows with the residual's addition in front of it, and rows rounded to 8 bits without a
// norm.
//
//   h = x + residual,  u = (h - mean(h)) r,  r = 1 / sqrt(var(h) + eps),  y = u w + b
//
// The variance is that of the differences d = h - mean, from registers, and both its sums correct
// for the rounding of the mean: with e = mean(d), var = mean(d^2) - e^2 and d - e is what counts, so a mean
// a thousand times the deviation costs no digits that h still has.
//
// Bound by memory: a row is read once, into registers.  Measured, bf16: 5000 x 8192 with residual to e4m3 51 us (287
// MB, 5.7 TB/s); 2048 x 4096 to int8 11 us; one row of 4096 4.3 us, rounded without a norm 2.7.
#include "layernorm.hpp"

namespace ts {

struct LayerArgs {
    const void *x, *residual, *weight, *bias;
    void *y, *h;
    float* scale;
    uint8_t* kept;     // h in 8 bits, or null
    int M, N, w_type;
    long long ldx, ldr, ldy, ldh, ld_kept;
    float eps;
    long long first;   // workgroups before this launch's
};

// Eight columns at n of a row, kept: the four threads of a block of 32 call it together.
__device__ __forceinline__ void keep8(uint8_t* row, int N, long long n, const float* v) {
    const uint32_t e = block_exponent(quad_max(max8_bits(v, 0)));
    const float inv = step_inverse(e);
    if (n >= kept_values(N)) return;
    *reinterpret_cast<u32x2*>(row + n) = u32x2{kept_pack4(v, inv), kept_pack4(v + 4, inv)};
    if (n % kBlock == 0) row[kept_values(N) + n / kBlock] = (uint8_t)e;
}

// T threads a row (T <= 256: 256 / T rows a workgroup), up to C groups of eight columns a
// thread, T * C * 8 >= N.  Weights and biases (of type W) are loaded with the row and held as they lie in
// memory: loaded where they are used, behind the sums, each row waits for them a second time (5000 x 8192
// with residual to e4m3 75 us, now 56).  Workgroups that walk rows, the weights in registers and the next row on
// its way, gain nothing more (58 to 62).  NORM false: y = x, rounded to 8 bits.
template <class TX, class W, int Q, bool NORM, int T, int C>
__global__ void __launch_bounds__(T < 256 ? 256 : T) layernorm_kernel(LayerArgs g) {
    typedef typename Elt<TX>::T X;
    constexpr int RPW = T < 256 ? 256 / T : 1;
    __shared__ float lds[T > 64 ? T / 64 : 1][2];
    const long long m = (g.first + blockIdx.x) * RPW + threadIdx.x / T;
    const int t = threadIdx.x % T;
    if (m >= g.M) return;   // T <= 64 only: whole rows of lanes
    Raw8<W> w[NORM ? C : 1], b[NORM ? C : 1];
    Raw8<TX> x[C], res[NORM ? C : 1];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int n = (c * T + t) * 8, valid = g.N - n;
        x[c].load(g.x, m, g.ldx, n, g.N, valid);
        if constexpr (NORM)
            if (g.residual) res[c].load(g.residual, m, g.ldr, n, g.N, valid);
    }
    if constexpr (NORM) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = (c * T + t) * 8, valid = g.N - n;
            if (g.weight) w[c].load(g.weight, 0, 0, n, g.N, valid);
            if (g.bias) b[c].load(g.bias, 0, 0, n, g.N, valid);
        }
    }
    float v[C][8];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int n = (c * T + t) * 8, valid = g.N - n;
        x[c].unpack(v[c], valid);
        if constexpr (NORM) {
            if (g.residual) {
                float r[8];
                res[c].unpack(r, valid);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[c][e] += r[e];
                if (valid > 0) store8<TX>(static_cast<X*>(g.h) + m * g.ldh + n, valid, v[c]);
            }
            if (g.kept) keep8(g.kept + m * g.ld_kept, g.N, n, v[c]);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += v[c][e];
        }
    }
    if constexpr (NORM) {
        row_sums<T, 2>(s, lds);   // (the second is not used here)
        const float mean = s[0] / (float)g.N;
        s[0] = s[1] = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int valid = g.N - (c * T + t) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] -= mean;
            if (valid < 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[c][e] = e < valid ? v[c][e] : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[0] += v[c][e];
                s[1] = __builtin_fmaf(v[c][e], v[c][e], s[1]);
            }
        }
        row_sums<T, 2>(s, lds);
        const float r = inverse_deviation(s[0], s[1], (float)g.N, g.eps), off = s[0] / (float)g.N;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = (c * T + t) * 8, valid = g.N - n;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] = (v[c][e] - off) * r;
            if (g.weight) {
                float f[8];
                w[c].renew();
                w[c].unpack(f, valid);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[c][e] *= f[e];
            }
            if (g.bias) {
                float f[8];
                b[c].renew();
                b[c].unpack(f, valid);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[c][e] += f[e];
            }
            if constexpr (Q == Q_NONE) {
                if (valid > 0) store8<TX>(static_cast<X*>(g.y) + m * g.ldy + n, valid, v[c]);
            }
        }
    }
    if constexpr (Q != Q_NONE) {
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int valid = g.N - (c * T + t) * 8;
            if (valid < 8) {   // columns past N count for nothing
#pragma unroll
                for (int e = 0; e < 8; ++e) v[c][e] = e < valid ? v[c][e] : 0.0f;
            }
            most = max8_bits(v[c], most);
        }
        const float sc = row_scale<Q>(row_max<T>(most, &lds[0][0]));
        const Quotient by(sc);
        if (t == 0) g.scale[m] = sc;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = (c * T + t) * 8, valid = g.N - n;
            if (valid <= 0) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] = by(v[c][e]);
            store8_q<Q>(static_cast<uint8_t*>(g.y) + m * g.ldy + n, valid, v[c]);
        }
    }
}

// Rows too long for the registers of a workgroup: the row is read again for each step.  h is
// written last, by the thread that reads its element, so it may take the place of x or the
// residual.
template <class TX, int Q, bool NORM>
__global__ void __launch_bounds__(kLongThreads) layernorm_long_kernel(LayerArgs g) {
    typedef typename Elt<TX>::T X;
    __shared__ float lds[kLongThreads / 64][2];
    const long long m = g.first + blockIdx.x;
    const X* x = static_cast<const X*>(g.x) + m * g.ldx;
    auto load_h = [&](long long n, int valid, float* v) {
        load8<TX>(x + n, valid, v);
        if (NORM && g.residual) {
            float r[8];
            load8<TX>(static_cast<const X*>(g.residual) + m * g.ldr + n, valid, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += r[e];
        }
    };
    auto valid_of = [&](long long n) { return (int)std::min<long long>(g.N - n, 8); };
    float mean = 0.0f, off = 0.0f, r = 1.0f;
    if constexpr (NORM) {
        float s[2] = {0.0f, 0.0f};
        for (long long n = threadIdx.x * 8; n < kept_values(g.N); n += kLongThreads * 8) {   // whole blocks of 32
            float v[8];
            load_h(n, valid_of(n), v);
            if (g.kept) keep8(g.kept + m * g.ld_kept, g.N, n, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += v[e];
        }
        row_sums<kLongThreads, 2>(s, lds);
        mean = s[0] / (float)g.N;
        s[0] = s[1] = 0.0f;
        for (long long n = threadIdx.x * 8; n < g.N; n += kLongThreads * 8) {
            const int valid = valid_of(n);
            float v[8];
            load_h(n, valid, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = e < valid ? v[e] - mean : 0.0f;
                s[0] += d;
                s[1] = __builtin_fmaf(d, d, s[1]);
            }
        }
        row_sums<kLongThreads, 2>(s, lds);
        r = inverse_deviation(s[0], s[1], (float)g.N, g.eps);
        off = s[0] / (float)g.N;
    }
    auto output = [&](long long n, int valid, float* v) {
        if constexpr (NORM) {
            float w[8], b[8];
            columns8<TX>(g.weight, g.w_type, n, valid, 1.0f, w);
            columns8<TX>(g.bias, g.w_type, n, valid, 0.0f, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(((v[e] - mean) - off) * r, w[e], b[e]);
        }
    };
    Quotient by(1.0f);
    if constexpr (Q != Q_NONE) {
        uint32_t most = 0;
        for (long long n = threadIdx.x * 8; n < g.N; n += kLongThreads * 8) {
            const int valid = valid_of(n);
            float v[8];
            load_h(n, valid, v);
            output(n, valid, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < valid ? v[e] : 0.0f;
            most = max8_bits(v, most);
        }
        const float sc = row_scale<Q>(row_max<kLongThreads>(most, &lds[0][0]));
        by = Quotient(sc);
        if (threadIdx.x == 0) g.scale[m] = sc;
    }
    for (long long n = threadIdx.x * 8; n < g.N; n += kLongThreads * 8) {
        const int valid = valid_of(n);
        float v[8];
        load_h(n, valid, v);
        if (NORM && g.residual) store8<TX>(static_cast<X*>(g.h) + m * g.ldh + n, valid, v);
        output(n, valid, v);
        if constexpr (Q != Q_NONE) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = by(v[e]);
            store8_q<Q>(static_cast<uint8_t*>(g.y) + m * g.ldy + n, valid, v);
        } else {
            store8<TX>(static_cast<X*>(g.y) + m * g.ldy + n, valid, v);
        }
    }
}

namespace {

template <class TX, class W, int Q, bool NORM>
const void* kernel_of(Shape s) {
#define TS_NORM(T, C) \
    if (s.t == T && s.c == C) return reinterpret_cast<const void*>(&layernorm_kernel<TX, W, Q, NORM, T, C>)
    TS_NORM(16, 1); TS_NORM(16, 2); TS_NORM(16, 4);
    TS_NORM(64, 1); TS_NORM(64, 2); TS_NORM(64, 4);
    TS_NORM(256, 1); TS_NORM(256, 2); TS_NORM(256, 4);
    TS_NORM(1024, 1); TS_NORM(1024, 2); TS_NORM(1024, 4);
    if constexpr (!NORM) { TS_NORM(1024, 8); }
#undef TS_NORM
    return reinterpret_cast<const void*>(&layernorm_long_kernel<TX, Q, NORM>);
}
template <class TX, class W, bool NORM>
ts_status run(LayerArgs& g, int32_t y_dtype, hipStream_t stream) {
    const Shape s = norm_shape(g.M, g.N, NORM ? 4 : 8);   // (eight groups a thread spill 11 to 600 registers)
    const void* fn;
    if (y_dtype == TS_E4M3) fn = kernel_of<TX, W, Q_E4M3, NORM>(s);
    else if (y_dtype == TS_I8) fn = kernel_of<TX, W, Q_I8, NORM>(s);
    else fn = kernel_of<TX, W, Q_NONE, true>(s);
    if (s.t == 0) return launch_rows(fn, g.M, kLongThreads, g, stream);
    const int rpw = s.t < 256 ? 256 / s.t : 1;
    return launch_rows(fn, ((int64_t)g.M + rpw - 1) / rpw, std::max(s.t, 256), g, stream);
}
template <class TX, bool NORM>
ts_status run_w(LayerArgs& g, int32_t y_dtype, hipStream_t stream) {
    if constexpr (NORM && Elt<TX>::E == 8)
        if (g.w_type == ELT_F32 && (g.weight || g.bias)) return run<TX, OutF32, NORM>(g, y_dtype, stream);
    return run<TX, TX, NORM>(g, y_dtype, stream);
}
template <bool NORM>
ts_status run_any(LayerArgs& g, int32_t x_dtype, int32_t y_dtype, hipStream_t stream) {
    if (x_dtype == TS_F16) return run_w<OutF16, NORM>(g, y_dtype, stream);
    if (x_dtype == TS_BF16) return run_w<OutBF16, NORM>(g, y_dtype, stream);
    return run_w<OutF32, NORM>(g, y_dtype, stream);
}

bool eight_bit(int32_t t) { return t == TS_E4M3 || t == TS_I8; }

}  // namespace
}  // namespace ts

using namespace ts;

extern "C" ts_status ts_layernorm(const void* x, const void* residual, const void* weight, const void* bias, void* y,
                                  void* h, float* scale, void* kept, int64_t M, int64_t N, int64_t stride_x,
                                  int64_t stride_r, int64_t stride_y, int64_t stride_h, int64_t stride_kept,
                                  int32_t x_dtype, int32_t w_dtype, int32_t y_dtype, float eps, void* stream) {
    ts_status st = norm_sizes(M, N);
    if (st != TS_OK) return st;
    const bool vectors = weight || bias;
    if (!row_type(x_dtype) || (vectors && !row_type(w_dtype)) || !(row_type(y_dtype) || eight_bit(y_dtype)) ||
        !(eps >= 0.0f) || eps > 3.4e38f)
        return TS_ERR_INVALID_ARG;
    const bool q = eight_bit(y_dtype);
    if ((!q && y_dtype != x_dtype) || (vectors && w_dtype != x_dtype && w_dtype != TS_F32)) return TS_ERR_UNSUPPORTED;
    if (M == 0 || (N == 0 && !q)) return TS_OK;
    // rows without elements still have their scale, the least one
    if (q && !scale) return TS_ERR_INVALID_ARG;
    if (N > 0 && (!x || !y || (residual && !h) || (!residual && h))) return TS_ERR_INVALID_ARG;
    if (N > 0 && M > 1 && (stride_x < N || stride_y < N || (residual && (stride_r < N || stride_h < N)) ||
                           (kept && (stride_kept < kept_row(N) || stride_kept % 16 != 0))))
        return TS_ERR_INVALID_ARG;
    const int xs = type_size(x_dtype);
    if ((uintptr_t)x % xs || (uintptr_t)residual % xs || (uintptr_t)h % xs || (uintptr_t)y % type_size(y_dtype) ||
        (vectors && ((uintptr_t)weight % type_size(w_dtype) || (uintptr_t)bias % type_size(w_dtype))) ||
        (uintptr_t)scale % 4 || (uintptr_t)kept % 16)
        return TS_ERR_ALIGNMENT;
    if (N > 0 && (y == h || !in_place_ok(h, x, true, M, stride_h, stride_x) ||
                  !in_place_ok(h, residual, true, M, stride_h, stride_r) ||
                  !in_place_ok(y, x, !q, M, stride_y, stride_x) || !in_place_ok(y, residual, !q, M, stride_y, stride_r) ||
                  (kept && (kept == x || kept == residual || kept == y || kept == h))))
        return TS_ERR_INVALID_ARG;
    st = have_device();
    if (st != TS_OK) return st;
    LayerArgs g = {x, residual, weight, bias, y, h, scale, N > 0 ? static_cast<uint8_t*>(kept) : nullptr, (int)M, (int)N,
                   w_dtype, stride_x, stride_r, stride_y, stride_h, stride_kept, eps, 0};
    return run_any<true>(g, x_dtype, y_dtype, static_cast<hipStream_t>(stream));
}

extern "C" ts_status ts_quantize_rows(const void* x, void* y, float* scale, int64_t M, int64_t N, int64_t stride_x,
                                      int64_t stride_y, int32_t x_dtype, int32_t y_dtype, void* stream) {
    ts_status st = norm_sizes(M, N);
    if (st != TS_OK) return st;
    if (!row_type(x_dtype) || !eight_bit(y_dtype)) return TS_ERR_INVALID_ARG;
    if (M == 0) return TS_OK;
    if (!scale || (N > 0 && (!x || !y || x == y))) return TS_ERR_INVALID_ARG;
    if (N > 0 && M > 1 && (stride_x < N || stride_y < N)) return TS_ERR_INVALID_ARG;
    if ((uintptr_t)x % type_size(x_dtype) || (uintptr_t)scale % 4) return TS_ERR_ALIGNMENT;
    st = have_device();
    if (st != TS_OK) return st;
    LayerArgs g = {x, nullptr, nullptr, nullptr, y, nullptr, scale, nullptr, (int)M, (int)N, TS_F32, stride_x, 0, stride_y,
                   0, 0, 0.0f, 0};
    return run_any<false>(g, x_dtype, y_dtype, static_cast<hipStream_t>(stream));
}

// Layer norm of rows with the residual's addition in front of it, its gradients, and rows rounded to
// 8 bits without a norm.
//
//   h = x + residual,  u = (h - mean(h)) r,  r = 1 / sqrt(var(h) + eps),  y = u w + b
//   g = w dy:  dx = r (g - mean(g)) - u (r mean(g u)) + dh,  dw = sum over rows of dy u,  db = of dy
//
// The variance is that of the differences d = h - mean, from registers, and both its sums correct
// for the rounding of the mean: with e = mean(d), var = mean(d^2) - e^2 and d - e is what counts, so a mean
// a thousand times the deviation costs no digits that h still has.
//
// Bound by memory: a row is read once into registers; the gradients hold h and dy as they lie in memory
// (half the registers in 16 bits, a quarter for h kept in 8) and the running sums of dw and db.
#include <hip/hip_runtime.h>

#include "checkpoint.hpp"
#include "norm.hpp"

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

// Sums of K values over the T threads of a row, as row_sum; one pair of barriers for all of them.
template <int T, int K>
__device__ __forceinline__ void row_sums(float* v, float (*lds)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lanes_sum<(T < 64 ? T : 64)>(v[k]);
    if constexpr (T > 64) {
        __syncthreads();   // the words' last readers are done
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) lds[threadIdx.x >> 6][k] = v[k];
        }
        __syncthreads();
        // a lane takes one wave's words (all of them in every lane: 16 waves' cost 16 K registers)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = lanes_sum<T / 64>(lds[threadIdx.x & (T / 64 - 1)][k]);
    }
}
// 1 / deviation from the sums of d and d^2; a variance that rounds below zero is zero (NaN stays).
__device__ __forceinline__ float inverse_deviation(float sd, float sdd, float n, float eps) {
    const float e = sd / n, var = __builtin_fmaf(-e, e, sdd / n);
    return 1.0f / __builtin_sqrtf((var < 0.0f ? 0.0f : var) + eps);
}
// Weight or bias of eight columns; `none` where there is no vector.
template <class TX>
__device__ __forceinline__ void columns8(const void* p, int type, long long n, int valid, float none, float* v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = none;
    if (p) load8_vec<TX>(p, type, n, valid, v);
}
// Eight columns at n of a row, kept: the four threads of a block of 32 call it together.
__device__ __forceinline__ void keep8(uint8_t* row, int N, long long n, const float* v) {
    const uint32_t e = block_exponent(quad_max(max8_bits(v, 0)));
    const float inv = step_inverse(e);
    if (n >= kept_values(N)) return;
    *reinterpret_cast<u32x2*>(row + n) = u32x2{kept_pack4(v, inv), kept_pack4(v + 4, inv)};
    if (n % kBlock == 0) row[kept_values(N) + n / kBlock] = (uint8_t)e;
}

// T threads a row (T <= 256: 256 / T rows a workgroup), up to C groups of eight columns a
// thread, T * C * 8 >= N.  NORM false: y = x, rounded to 8 bits.
template <class TX, int Q, bool NORM, int T, int C>
__global__ void __launch_bounds__(T < 256 ? 256 : T) layernorm_kernel(LayerArgs g) {
    typedef typename Elt<TX>::T X;
    constexpr int RPW = T < 256 ? 256 / T : 1;
    __shared__ float lds[T > 64 ? T / 64 : 1][2];
    const long long m = (g.first + blockIdx.x) * RPW + threadIdx.x / T;
    const int t = threadIdx.x % T;
    if (m >= g.M) return;   // T <= 64 only: whole rows of lanes
    const X* x = static_cast<const X*>(g.x) + m * g.ldx;
    float v[C][8];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int n = (c * T + t) * 8, valid = g.N - n;
        load8<TX>(x + n, valid, v[c]);
        if constexpr (NORM) {
            if (g.residual) {
                float r[8];
                load8<TX>(static_cast<const X*>(g.residual) + m * g.ldr + n, valid, r);
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
            float w[8], b[8];
            columns8<TX>(g.weight, g.w_type, n, valid, 1.0f, w);
            columns8<TX>(g.bias, g.w_type, n, valid, 0.0f, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] = __builtin_fmaf((v[c][e] - off) * r, w[e], b[e]);
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

// ---- gradients ---------------------------------------------------------------------------

struct LayerGradArgs {
    const void *dy, *h, *weight, *dh;
    void* dx;
    float* part;    // partial sums, one row of N of dw and one of db per workgroup, or null
    float* stats;   // long rows: mean, r, r mean(g) and r mean(g u) of every row
    int M, N, w_type;
    long long ldy, ldh, lds, ldx;   // (h in 8 bits: ldh in bytes)
    float eps;
    long long first;   // workgroups before this launch's (the launches of one workgroup a row)
};

// Eight columns of a row as they lie in memory.
template <class TX>
struct Raw8 {
    u32x4 v[Elt<TX>::E == 8 ? 1 : 2];
    __device__ __forceinline__ void load(const void* base, long long m, long long ld, long long n, int N, int valid) {
        (void)N;
        const typename Elt<TX>::T* p = static_cast<const typename Elt<TX>::T*>(base) + m * ld + n;
        v[0] = load_row<TX>(p, valid);
        if constexpr (Elt<TX>::E == 4) v[1] = load_row<TX>(p + 4, valid - 4);
    }
    // Values unpacked before are not held in registers until the next time.
    __device__ __forceinline__ void renew() {
        if constexpr (Elt<TX>::E == 8) asm volatile("" : "+v"(v[0]));
    }
    __device__ __forceinline__ void unpack(float* f, int valid) const {
        (void)valid;
        unpack_row<TX>(v[0], f);
        if constexpr (Elt<TX>::E == 4) unpack_row<TX>(v[1], f + 4);
    }
};
struct RawKept {
    Kept8 k;
    __device__ __forceinline__ void load(const void* base, long long m, long long ld, long long n, int N, int valid) {
        k.load(static_cast<const uint8_t*>(base) + m * ld, kept_values(N), n, valid > 0);
    }
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(k.w[0]), "+v"(k.w[1])); }
    __device__ __forceinline__ void unpack(float* f, int valid) const {
        k.unpack(f);
        if (valid < 8) {   // whatever lies behind column N
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = e < valid ? f[e] : 0.0f;
        }
    }
};
template <class TX, bool HK>
using HRow = typename std::conditional<HK, RawKept, Raw8<TX>>::type;

// T threads a row, C groups of eight columns a thread, as above; a workgroup walks rows
// (its row groups: row, row + groups, ...), each thread holding the weights and the running
// sums of dw and db of its own columns in registers.  HK: h kept in 8 bits.
template <class TX, bool HK, int T, int C>
__global__ void __launch_bounds__(T < 256 ? 256 : T) layernorm_grad_kernel(LayerGradArgs g) {
    typedef typename Elt<TX>::T X;
    constexpr int RPW = T < 256 ? 256 / T : 1;
    __shared__ float lds1[T > 64 ? T / 64 : 1][2], lds2[T > 64 ? T / 64 : 1][3];
    const int groups = gridDim.x * RPW;
    const int group = blockIdx.x * RPW + threadIdx.x / T;
    const int t = threadIdx.x % T;
    const float rn = 1.0f / (float)g.N;
    float w[C][8], dw[C][8], db[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int n = (c * T + t) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[c][e] = db[c][e] = 0.0f;
        columns8<TX>(g.weight, g.w_type, n, g.N - n, 1.0f, w[c]);
    }
    for (long long m = group; m < g.M; m += groups) {   // T > 64: one row a workgroup, so m is uniform
        HRow<TX, HK> h[C];
        Raw8<TX> dy[C];
        float a[2] = {0.0f, 0.0f};   // sums of h and g
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = (c * T + t) * 8, valid = g.N - n;
            h[c].load(g.h, m, g.ldh, n, g.N, valid);
            dy[c].load(g.dy, m, g.ldy, n, g.N, valid);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int valid = g.N - (c * T + t) * 8;
            float x[8], y[8];
            h[c].unpack(x, valid);
            dy[c].unpack(y, valid);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                a[0] += x[e];
                a[1] = __builtin_fmaf(w[c][e], y[e], a[1]);
            }
        }
        row_sums<T, 2>(a, lds1);
        const float mean = a[0] * rn;
        float b[3] = {0.0f, 0.0f, 0.0f};   // sums of d, d^2 and g d
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int valid = g.N - (c * T + t) * 8;
            float x[8], y[8];
            h[c].renew();
            dy[c].renew();
            h[c].unpack(x, valid);
            dy[c].unpack(y, valid);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] -= mean;
            if (valid < 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = e < valid ? x[e] : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                b[0] += x[e];
                b[1] = __builtin_fmaf(x[e], x[e], b[1]);
                b[2] = __builtin_fmaf(w[c][e] * y[e], x[e], b[2]);
            }
        }
        row_sums<T, 3>(b, lds2);
        const float r = inverse_deviation(b[0], b[1], (float)g.N, g.eps), off = b[0] * rn;
        const float k1 = r * (a[1] * rn);
        const float k2 = r * (r * (__builtin_fmaf(-off, a[1], b[2]) * rn));
        const float center = mean + off;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = (c * T + t) * 8, valid = g.N - n;
            if (valid <= 0) continue;
            float x[8], y[8], d[8];
            h[c].renew();
            dy[c].renew();
            h[c].unpack(x, valid);
            dy[c].unpack(y, valid);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float unit = (x[e] - center) * r;
                dw[c][e] = __builtin_fmaf(y[e], unit, dw[c][e]);
                db[c][e] += y[e];
                d[e] = __builtin_fmaf(-unit, k2, __builtin_fmaf(r * w[c][e], y[e], -k1));
            }
            if (g.dh) {
                float f[8];
                load8<TX>(static_cast<const X*>(g.dh) + m * g.lds + n, valid, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] += f[e];
            }
            store8<TX>(static_cast<X*>(g.dx) + m * g.ldx + n, valid, d);
        }
    }
    if (!g.part) return;
    float* part = g.part + (long long)blockIdx.x * 2 * g.N;
    if constexpr (RPW == 1) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = (c * T + t) * 8, valid = g.N - n;
            if (valid > 0) {
                store8<OutF32>(part + n, valid, dw[c]);
                store8<OutF32>(part + g.N + n, valid, db[c]);
            }
        }
    } else {   // the workgroup's row groups first, in order
        __shared__ float sums[256][17];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            __syncthreads();   // the last readers are done
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sums[threadIdx.x][e] = dw[c][e];
                sums[threadIdx.x][8 + e] = db[c][e];
            }
            __syncthreads();
            for (int k = threadIdx.x; k < 16 * T; k += 256) {
                const int which = k / (8 * T), j = k % (8 * T);
                float s = 0.0f;
#pragma unroll
                for (int r = 0; r < RPW; ++r) s += sums[r * T + j / 8][8 * which + j % 8];
                const int n = c * T * 8 + j;
                if (n < g.N) part[(long long)which * g.N + n] = s;
            }
        }
    }
}

// Long rows, in three steps: the four numbers of each row, the partial sums of dw and db by strips
// of columns, and dx element by element (last: dx may take the place of dy or dh).
template <class TX, bool HK>
__global__ void __launch_bounds__(kLongThreads) layernorm_grad_stats_kernel(LayerGradArgs g) {
    __shared__ float lds1[kLongThreads / 64][2], lds2[kLongThreads / 64][3];
    const long long m = g.first + blockIdx.x;
    const float rn = 1.0f / (float)g.N;
    auto each = [&](auto&& f) {
        for (long long n = threadIdx.x * 8; n < g.N; n += kLongThreads * 8) {
            const int valid = (int)std::min<long long>(g.N - n, 8);
            HRow<TX, HK> h;
            Raw8<TX> dy;
            float x[8], y[8], w[8];
            h.load(g.h, m, g.ldh, n, g.N, valid);
            dy.load(g.dy, m, g.ldy, n, g.N, valid);
            h.unpack(x, valid);
            dy.unpack(y, valid);
            columns8<TX>(g.weight, g.w_type, n, valid, 1.0f, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) f(x[e], w[e] * y[e], e < valid);
        }
    };
    float a[2] = {0.0f, 0.0f}, b[3] = {0.0f, 0.0f, 0.0f};
    each([&](float x, float gy, bool) {
        a[0] += x;
        a[1] += gy;
    });
    row_sums<kLongThreads, 2>(a, lds1);
    const float mean = a[0] * rn;
    each([&](float x, float gy, bool in) {
        const float d = in ? x - mean : 0.0f;
        b[0] += d;
        b[1] = __builtin_fmaf(d, d, b[1]);
        b[2] = __builtin_fmaf(gy, d, b[2]);
    });
    row_sums<kLongThreads, 3>(b, lds2);
    if (threadIdx.x == 0) {
        const float r = inverse_deviation(b[0], b[1], (float)g.N, g.eps), off = b[0] * rn;
        g.stats[4 * m] = mean + off;
        g.stats[4 * m + 1] = r;
        g.stats[4 * m + 2] = r * (a[1] * rn);
        g.stats[4 * m + 3] = r * (r * (__builtin_fmaf(-off, a[1], b[2]) * rn));
    }
}
// 256 threads: 64 strips of eight columns x 4 rows; blockIdx.y is the row group.
template <class TX, bool HK>
__global__ void __launch_bounds__(256) layernorm_grad_columns_kernel(LayerGradArgs g) {
    __shared__ float sums[3][64][16];
    const long long n = ((long long)blockIdx.x * 64 + (threadIdx.x & 63)) * 8;
    const int rl = threadIdx.x >> 6;
    const int valid = (int)std::min<long long>(g.N - n, 8);
    float s[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = 0.0f;
    if (valid > 0) {
        for (long long m = (long long)blockIdx.y * 4 + rl; m < g.M; m += (long long)gridDim.y * 4) {
            HRow<TX, HK> h;
            Raw8<TX> dy;
            float x[8], y[8];
            h.load(g.h, m, g.ldh, n, g.N, valid);
            dy.load(g.dy, m, g.ldy, n, g.N, valid);
            h.unpack(x, valid);
            dy.unpack(y, valid);
            const float mean = g.stats[4 * m], r = g.stats[4 * m + 1];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[e] = __builtin_fmaf(y[e], (x[e] - mean) * r, s[e]);
                s[8 + e] += y[e];
            }
        }
    }
    if (rl > 0)
#pragma unroll
        for (int e = 0; e < 16; ++e) sums[rl - 1][threadIdx.x & 63][e] = s[e];
    __syncthreads();
    if (rl == 0 && valid > 0) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            s[e] = ((s[e] + sums[0][threadIdx.x][e]) + sums[1][threadIdx.x][e]) + sums[2][threadIdx.x][e];
        float* part = g.part + (long long)blockIdx.y * 2 * g.N + n;
        store8<OutF32>(part, valid, s);
        store8<OutF32>(part + g.N, valid, s + 8);
    }
}
template <class TX, bool HK>
__global__ void __launch_bounds__(kLongThreads) layernorm_grad_dx_kernel(LayerGradArgs g) {
    typedef typename Elt<TX>::T X;
    const long long m = g.first + blockIdx.x;
    const float mean = g.stats[4 * m], r = g.stats[4 * m + 1], k1 = g.stats[4 * m + 2], k2 = g.stats[4 * m + 3];
    for (long long n = threadIdx.x * 8; n < g.N; n += kLongThreads * 8) {
        const int valid = (int)std::min<long long>(g.N - n, 8);
        HRow<TX, HK> h;
        Raw8<TX> dy;
        float x[8], y[8], w[8], a[8];
        h.load(g.h, m, g.ldh, n, g.N, valid);
        dy.load(g.dy, m, g.ldy, n, g.N, valid);
        h.unpack(x, valid);
        dy.unpack(y, valid);
        columns8<TX>(g.weight, g.w_type, n, valid, 1.0f, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = 0.0f;
        if (g.dh) load8<TX>(static_cast<const X*>(g.dh) + m * g.lds + n, valid, a);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += __builtin_fmaf(-((x[e] - mean) * r), k2, __builtin_fmaf(r * w[e], y[e], -k1));
        store8<TX>(static_cast<X*>(g.dx) + m * g.ldx + n, valid, a);
    }
}

namespace {

template <class TX, int Q, bool NORM>
const void* kernel_of(Shape s) {
#define TS_NORM(T, C) \
    if (s.t == T && s.c == C) return reinterpret_cast<const void*>(&layernorm_kernel<TX, Q, NORM, T, C>)
    TS_NORM(16, 1); TS_NORM(16, 2); TS_NORM(16, 4);
    TS_NORM(64, 1); TS_NORM(64, 2); TS_NORM(64, 4);
    TS_NORM(256, 1); TS_NORM(256, 2); TS_NORM(256, 4);
    TS_NORM(1024, 1); TS_NORM(1024, 2); TS_NORM(1024, 4);
    if constexpr (!NORM) { TS_NORM(1024, 8); }
#undef TS_NORM
    return reinterpret_cast<const void*>(&layernorm_long_kernel<TX, Q, NORM>);
}
// Threads and groups of columns of the gradients: up to two groups a thread with 1024 threads, whose 128
// registers hold no more sums.
constexpr int kGradMost = 2;
template <class TX, bool HK>
const void* grad_kernel_of(Shape s) {
#define TS_NORM(T, C) \
    if (s.t == T && s.c == C) return reinterpret_cast<const void*>(&layernorm_grad_kernel<TX, HK, T, C>)
    TS_NORM(16, 1); TS_NORM(16, 2); TS_NORM(16, 4);
    TS_NORM(64, 1); TS_NORM(64, 2); TS_NORM(64, 4);
    TS_NORM(256, 1); TS_NORM(256, 2); TS_NORM(256, 4);
    TS_NORM(1024, 1); TS_NORM(1024, 2);
#undef TS_NORM
    return nullptr;
}

int64_t grad_groups(int64_t M, int64_t N) {
    const Shape s = norm_shape(M, N, kGradMost);
    if (s.t == 0) return std::max<int64_t>(1, std::min<int64_t>((M + 63) / 64, 64));
    const int rpw = s.t < 256 ? 256 / s.t : 1;
    return std::min<int64_t>((M + rpw - 1) / rpw, 1024);
}

template <class TX, bool NORM>
ts_status run(LayerArgs& g, int32_t y_dtype, hipStream_t stream) {
    const Shape s = norm_shape(g.M, g.N, NORM ? 4 : 8);   // (eight groups a thread spill 11 to 600 registers)
    const void* fn;
    if (y_dtype == TS_E4M3) fn = kernel_of<TX, Q_E4M3, NORM>(s);
    else if (y_dtype == TS_I8) fn = kernel_of<TX, Q_I8, NORM>(s);
    else fn = kernel_of<TX, Q_NONE, true>(s);
    if (s.t == 0) return launch_rows(fn, g.M, kLongThreads, g, stream);
    const int rpw = s.t < 256 ? 256 / s.t : 1;
    return launch_rows(fn, ((int64_t)g.M + rpw - 1) / rpw, std::max(s.t, 256), g, stream);
}
template <bool NORM>
ts_status run_any(LayerArgs& g, int32_t x_dtype, int32_t y_dtype, hipStream_t stream) {
    if (x_dtype == TS_F16) return run<OutF16, NORM>(g, y_dtype, stream);
    if (x_dtype == TS_BF16) return run<OutBF16, NORM>(g, y_dtype, stream);
    return run<OutF32, NORM>(g, y_dtype, stream);
}

template <class TX, bool HK>
ts_status run_grad(LayerGradArgs& g, int64_t groups, hipStream_t stream) {
    const Shape s = norm_shape(g.M, g.N, kGradMost);
    if (s.t != 0) return launch(grad_kernel_of<TX, HK>(s), groups, 1, std::max(s.t, 256), &g, stream);
    ts_status st = launch_rows(reinterpret_cast<const void*>(&layernorm_grad_stats_kernel<TX, HK>), g.M, kLongThreads, g, stream);
    if (st == TS_OK && g.part)
        st = launch(reinterpret_cast<const void*>(&layernorm_grad_columns_kernel<TX, HK>), ((int64_t)g.N + 511) / 512,
                    groups, 256, &g, stream);
    if (st == TS_OK)
        st = launch_rows(reinterpret_cast<const void*>(&layernorm_grad_dx_kernel<TX, HK>), g.M, kLongThreads, g, stream);
    return st;
}

// Two sums a column: half as many columns as the launches over columns take.
ts_status grad_sizes(int64_t M, int64_t N) {
    const ts_status st = norm_sizes(M, N);
    return st == TS_OK && N >= 1 << 25 ? TS_ERR_UNSUPPORTED : st;
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

// Bytes: the partial sums of dw and db, then (long rows) four numbers per row.
extern "C" int64_t ts_layernorm_backward_workspace(int64_t M, int64_t N) {
    ts_status st = grad_sizes(M, N);
    if (st != TS_OK) return st;
    if (M == 0 || N == 0) return 0;
    const int64_t part = (grad_groups(M, N) * 2 * N * 4 + 255) / 256 * 256;
    return part + (norm_shape(M, N, kGradMost).t == 0 ? M * 16 : 0);
}

extern "C" ts_status ts_layernorm_backward(const void* dy, const void* h, const void* weight, const void* dh, void* dx,
                                           void* dweight, void* dbias, int64_t M, int64_t N, int64_t stride_dy,
                                           int64_t stride_h, int64_t stride_dh, int64_t stride_dx, int32_t dtype,
                                           int32_t h_dtype, int32_t w_dtype, float eps, void* stream, void* workspace,
                                           int64_t workspace_bytes) {
    ts_status st = grad_sizes(M, N);
    if (st != TS_OK) return st;
    const bool sums = dweight || dbias, vectors = weight || sums;
    if (!row_type(dtype) || (h_dtype != dtype && h_dtype != TS_Q8) || (vectors && !row_type(w_dtype)) || !(eps >= 0.0f) ||
        eps > 3.4e38f)
        return TS_ERR_INVALID_ARG;
    if (vectors && w_dtype != dtype && w_dtype != TS_F32) return TS_ERR_UNSUPPORTED;
    if (workspace_bytes < 0) return TS_ERR_INVALID_ARG;
    if (N == 0 || (M == 0 && !sums)) return TS_OK;
    const bool kept = h_dtype == TS_Q8;
    if (M > 0 && (!dy || !h || !dx)) return TS_ERR_INVALID_ARG;
    if (M > 1 && (stride_dy < N || stride_dx < N || (dh && stride_dh < N) || (!kept && stride_h < N) ||
                  (kept && (stride_h < kept_row(N) || stride_h % 16 != 0))))
        return TS_ERR_INVALID_ARG;
    const int xs = type_size(dtype), ws = type_size(w_dtype);
    if ((uintptr_t)dy % xs || (uintptr_t)h % (kept ? 16 : xs) || (uintptr_t)dh % xs || (uintptr_t)dx % xs ||
        (vectors && ((uintptr_t)weight % ws || (uintptr_t)dweight % ws || (uintptr_t)dbias % ws)))
        return TS_ERR_ALIGNMENT;
    if (!in_place_ok(dx, dy, true, M, stride_dx, stride_dy) || !in_place_ok(dx, h, !kept, M, stride_dx, stride_h) ||
        !in_place_ok(dx, dh, true, M, stride_dx, stride_dh) || (dweight && dweight == dbias))
        return TS_ERR_INVALID_ARG;
    const bool long_rows = norm_shape(M, N, kGradMost).t == 0;
    const int64_t groups = M > 0 ? grad_groups(M, N) : 0;
    const int64_t part = (groups * 2 * N * 4 + 255) / 256 * 256;
    const int64_t need = M == 0 ? 0 : (sums || long_rows) ? part + (long_rows ? M * 16 : 0) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need || (uintptr_t)workspace % 256)) return TS_ERR_INVALID_ARG;
    st = have_device();
    if (st != TS_OK) return st;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    LayerGradArgs g = {dy, h, weight, dh, dx, sums ? static_cast<float*>(workspace) : nullptr,
                       long_rows ? reinterpret_cast<float*>(static_cast<char*>(workspace) + part) : nullptr,
                       (int)M, (int)N, w_dtype, stride_dy, stride_h, stride_dh, stride_dx, eps, 0};
    if (M > 0) {
        if (kept)
            st = dtype == TS_F16 ? run_grad<OutF16, true>(g, groups, hs)
                 : dtype == TS_BF16 ? run_grad<OutBF16, true>(g, groups, hs) : run_grad<OutF32, true>(g, groups, hs);
        else
            st = dtype == TS_F16 ? run_grad<OutF16, false>(g, groups, hs)
                 : dtype == TS_BF16 ? run_grad<OutBF16, false>(g, groups, hs) : run_grad<OutF32, false>(g, groups, hs);
        if (st != TS_OK) return st;
    }
    if (sums && !launch_reduce_columns(static_cast<float*>(workspace), (int)groups, (int)(2 * N), dweight, w_dtype, hs,
                                       (int)N, dbias))
        return TS_ERR_HIP;
    return TS_OK;
}

// Root-mean-square norm of rows with the residual's addition in front of it, 16-bit, 32-bit
// or e4m3 output with a scale per row, and its gradients.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w
//   dx = r (w dy) - h r^3 mean(w dy h) + dh,  dw = sum over rows of dy h r
//
// r^3 is never formed: from an rms of 4e12 on it is too small for fp32, below 1e-13 too large, far
// inside the range of h.  The second term is (h r) (r (r mean(w dy h))), whose every factor is of
// the size of h's own unit vector, dy or dx.
//
// Both are bound by memory: a row is read once into registers, where its sums, its largest
// |y| and its outputs are formed; nothing is read twice.  (Rows of 16385 to 32768 take more registers
// than a thread has for their gradients: 39, 63 and 159 are spilled in fp16, bf16 and fp32.)  Measured, bf16: 5000 x 8192 with residual to
// e4m3 54 us (287 MB, 5.3 TB/s); gradients of 8192 x 4096 with dh 47 us (268 MB) and 6.5 us for the sum of
// dw over 1024 workgroups; one row of 4096 4.9 us.
#include <hip/hip_runtime.h>

#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/tsgemm.h"
#include "plan.hpp"
#include "rows.hpp"

namespace ts {

struct NormArgs {
    const void *x, *residual, *weight;
    void *y, *h;
    float* scale;
    int M, N, w_type;
    long long ldx, ldr, ldy, ldh;
    float eps;
    long long first;   // workgroups before this launch's
};

constexpr float kE4M3Max = 448.0f;
constexpr float kMinScale = 0x1p-100f;   // keeps 1 / scale finite; rows of zeros take it

// Eight floats to e4m3 (round to nearest even; |v| <= 448 up to the rounding of the scale,
// which rounds back to 448).
__device__ __forceinline__ u32x2 pack8_e4m3(const float* v) {
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
    return u32x2{(uint32_t)lo, (uint32_t)hi};
}
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
__device__ __forceinline__ void store8_e4m3(uint8_t* p, int valid, const float* v) {
    const u32x2 w = pack8_e4m3(v);
    if (valid >= 8) {
        *reinterpret_cast<u32x2_a1*>(p) = w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) p[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
}
// Largest |v| as its bits, so that a NaN wins.
__device__ __forceinline__ uint32_t max8_bits(const float* v, uint32_t m) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v[e]) & 0x7fffffffu;
        m = b > m ? b : m;
    }
    return m;
}
__device__ __forceinline__ float row_scale(uint32_t max_bits) {
    const float s = __builtin_bit_cast(float, max_bits) / kE4M3Max;
    return s < kMinScale ? kMinScale : s;   // NaN stays NaN
}

// y / scale with one rounding: the product with the reciprocal, off by up to a step and a half of
// fp32, and one correction by its remainder.  (The product alone puts values next to the middle between
// two e4m3 numbers on the wrong side.)  An infinite scale has the reciprocal 0 and no remainder, so
// that finite values become 0.
struct Quotient {
    float inv, scale;
    __device__ __forceinline__ explicit Quotient(float s)
        : inv(1.0f / s), scale(s > 3.4028234e38f ? 0.0f : s) {}
    __device__ __forceinline__ float operator()(float v) const {
        const float q = v * inv;
        return __builtin_fmaf(__builtin_fmaf(-q, scale, v), inv, q);
    }
};

// T threads a row (T <= 256: 256 / T rows a workgroup), up to C groups of eight columns a
// thread, T * C * 8 >= N.
template <class TX, bool Q, int T, int C>
__global__ void __launch_bounds__(T < 256 ? 256 : T) rmsnorm_kernel(NormArgs g) {
    typedef typename Elt<TX>::T X;
    constexpr int RPW = T < 256 ? 256 / T : 1;
    __shared__ float lds[T > 64 ? T / 64 : 1];
    const long long m = (g.first + blockIdx.x) * RPW + threadIdx.x / T;
    const int t = threadIdx.x % T;
    if (m >= g.M) return;   // T <= 64 only: whole rows of lanes
    const X* x = static_cast<const X*>(g.x) + m * g.ldx;
    float v[C][8];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int n = (c * T + t) * 8, valid = g.N - n;
        load8<TX>(x + n, valid, v[c]);
        if (g.residual) {
            float r[8];
            load8<TX>(static_cast<const X*>(g.residual) + m * g.ldr + n, valid, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] += r[e];
            if (valid > 0) store8<TX>(static_cast<X*>(g.h) + m * g.ldh + n, valid, v[c]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(v[c][e], v[c][e], sum);
    }
    sum = row_sum<T>(sum, lds);
    const float r = 1.0f / __builtin_sqrtf(sum / (float)g.N + g.eps);
    uint32_t most = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int n = (c * T + t) * 8, valid = g.N - n;
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
        if (g.weight) load8_vec<TX>(g.weight, g.w_type, n, valid, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] = v[c][e] * r * w[e];
        if constexpr (Q) {
            if (valid < 8) {   // columns past N: a NaN row makes them NaN too, but they count for nothing
#pragma unroll
                for (int e = 0; e < 8; ++e) v[c][e] = e < valid ? v[c][e] : 0.0f;
            }
            most = max8_bits(v[c], most);
        } else if (valid > 0) {
            store8<TX>(static_cast<X*>(g.y) + m * g.ldy + n, valid, v[c]);
        }
    }
    if constexpr (Q) {
        const float s = row_scale(row_max<T>(most, lds));
        const Quotient by(s);
        if (t == 0) g.scale[m] = s;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = (c * T + t) * 8, valid = g.N - n;
            if (valid <= 0) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] = by(v[c][e]);
            store8_e4m3(static_cast<uint8_t*>(g.y) + m * g.ldy + n, valid, v[c]);
        }
    }
}

// Rows too long for the registers of a workgroup: the row is read again for each step.  h is
// written last, by the thread that reads its element, so it may take the place of x or the
// residual.
constexpr int kLongThreads = 1024;
template <class TX, bool Q>
__global__ void __launch_bounds__(kLongThreads) rmsnorm_long_kernel(NormArgs g) {
    typedef typename Elt<TX>::T X;
    __shared__ float lds[kLongThreads / 64];
    const long long m = g.first + blockIdx.x;
    const X* x = static_cast<const X*>(g.x) + m * g.ldx;
    auto load_h = [&](long long n, int valid, float* v) {
        load8<TX>(x + n, valid, v);
        if (g.residual) {
            float r[8];
            load8<TX>(static_cast<const X*>(g.residual) + m * g.ldr + n, valid, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += r[e];
        }
    };
    auto weights = [&](long long n, int valid, float* w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
        if (g.weight) load8_vec<TX>(g.weight, g.w_type, n, valid, w);
    };
    float sum = 0.0f;
    for (long long n = threadIdx.x * 8; n < g.N; n += kLongThreads * 8) {
        float v[8];
        load_h(n, (int)std::min<long long>(g.N - n, 8), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(v[e], v[e], sum);
    }
    sum = row_sum<kLongThreads>(sum, lds);
    const float r = 1.0f / __builtin_sqrtf(sum / (float)g.N + g.eps);
    Quotient by(1.0f);
    if constexpr (Q) {
        uint32_t most = 0;
        for (long long n = threadIdx.x * 8; n < g.N; n += kLongThreads * 8) {
            const int valid = (int)std::min<long long>(g.N - n, 8);
            float v[8], w[8];
            load_h(n, valid, v);
            weights(n, valid, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < valid ? v[e] * r * w[e] : 0.0f;
            most = max8_bits(v, most);
        }
        const float s = row_scale(row_max<kLongThreads>(most, lds));
        by = Quotient(s);
        if (threadIdx.x == 0) g.scale[m] = s;
    }
    for (long long n = threadIdx.x * 8; n < g.N; n += kLongThreads * 8) {
        const int valid = (int)std::min<long long>(g.N - n, 8);
        float v[8], w[8];
        load_h(n, valid, v);
        weights(n, valid, w);
        if (g.residual) store8<TX>(static_cast<X*>(g.h) + m * g.ldh + n, valid, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * r * w[e];
        if constexpr (Q) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = by(v[e]);
            store8_e4m3(static_cast<uint8_t*>(g.y) + m * g.ldy + n, valid, v);
        } else {
            store8<TX>(static_cast<X*>(g.y) + m * g.ldy + n, valid, v);
        }
    }
}

// ---- gradients ---------------------------------------------------------------------------

struct NormGradArgs {
    const void *dy, *h, *weight, *dh;
    void* dx;
    float* part;    // partial sums of dw, one row of N per workgroup, or null
    float* stats;   // long rows: r and r^2 mean(w dy h) of every row
    int M, N, w_type;
    long long ldy, ldh, lds, ldx;
    float eps;
    long long first;   // workgroups before this launch's (the launches of one workgroup a row)
};

// T threads a row, C groups of eight columns a thread, as above; a workgroup walks rows
// (its row groups: row, row + groups, ...), each thread holding the weights and the running
// sums of dw of its own columns in registers.
template <class TX, int T, int C>
__global__ void __launch_bounds__(T < 256 ? 256 : T) rmsnorm_grad_kernel(NormGradArgs g) {
    typedef typename Elt<TX>::T X;
    constexpr int RPW = T < 256 ? 256 / T : 1;
    __shared__ float lds1[T > 64 ? T / 64 : 1], lds2[T > 64 ? T / 64 : 1];
    const int groups = gridDim.x * RPW;
    const int group = blockIdx.x * RPW + threadIdx.x / T;
    const int t = threadIdx.x % T;
    float w[C][8], dw[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int n = (c * T + t) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[c][e] = 1.0f;
            dw[c][e] = 0.0f;
        }
        if (g.weight) load8_vec<TX>(g.weight, g.w_type, n, g.N - n, w[c]);
    }
    for (long long m = group; m < g.M; m += groups) {   // T > 64: one row a workgroup, so m is uniform
        float h[C][8], dy[C][8];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = (c * T + t) * 8, valid = g.N - n;
            load8<TX>(static_cast<const X*>(g.h) + m * g.ldh + n, valid, h[c]);
            load8<TX>(static_cast<const X*>(g.dy) + m * g.ldy + n, valid, dy[c]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s1 = __builtin_fmaf(h[c][e], h[c][e], s1);
                s2 = __builtin_fmaf(w[c][e] * dy[c][e], h[c][e], s2);
            }
        }
        s1 = row_sum<T>(s1, lds1);
        s2 = row_sum<T>(s2, lds2);
        const float r = 1.0f / __builtin_sqrtf(s1 / (float)g.N + g.eps);
        const float k = r * (r * (s2 / (float)g.N));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = (c * T + t) * 8, valid = g.N - n;
            if (valid <= 0) continue;
            float d[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float unit = h[c][e] * r;
                dw[c][e] = __builtin_fmaf(dy[c][e], unit, dw[c][e]);
                d[e] = __builtin_fmaf(r * w[c][e], dy[c][e], -(unit * k));
            }
            if (g.dh) {
                float a[8];
                load8<TX>(static_cast<const X*>(g.dh) + m * g.lds + n, valid, a);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] += a[e];
            }
            store8<TX>(static_cast<X*>(g.dx) + m * g.ldx + n, valid, d);
        }
    }
    if (!g.part) return;
    if constexpr (RPW == 1) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = (c * T + t) * 8, valid = g.N - n;
            if (valid > 0) store8<OutF32>(g.part + (long long)group * g.N + n, valid, dw[c]);
        }
    } else {   // the workgroup's row groups first, in order
        __shared__ float sums[256][9];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            __syncthreads();   // the last readers are done
#pragma unroll
            for (int e = 0; e < 8; ++e) sums[threadIdx.x][e] = dw[c][e];
            __syncthreads();
            for (int k = threadIdx.x; k < 8 * T; k += 256) {
                float s = 0.0f;
#pragma unroll
                for (int r = 0; r < RPW; ++r) s += sums[r * T + k / 8][k % 8];
                const int n = c * T * 8 + k;
                if (n < g.N) g.part[(long long)blockIdx.x * g.N + n] = s;
            }
        }
    }
}

// Long rows, in three steps: the two numbers of each row, the partial sums of dw by strips
// of columns, and dx element by element (last: dx may take the place of dy or dh).
template <class TX>
__global__ void __launch_bounds__(kLongThreads) rmsnorm_grad_stats_kernel(NormGradArgs g) {
    typedef typename Elt<TX>::T X;
    __shared__ float lds1[kLongThreads / 64], lds2[kLongThreads / 64];
    const long long m = g.first + blockIdx.x;
    float s1 = 0.0f, s2 = 0.0f;
    for (long long n = threadIdx.x * 8; n < g.N; n += kLongThreads * 8) {
        const int valid = (int)std::min<long long>(g.N - n, 8);
        float h[8], dy[8], w[8];
        load8<TX>(static_cast<const X*>(g.h) + m * g.ldh + n, valid, h);
        load8<TX>(static_cast<const X*>(g.dy) + m * g.ldy + n, valid, dy);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
        if (g.weight) load8_vec<TX>(g.weight, g.w_type, n, valid, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s1 = __builtin_fmaf(h[e], h[e], s1);
            s2 = __builtin_fmaf(w[e] * dy[e], h[e], s2);
        }
    }
    s1 = row_sum<kLongThreads>(s1, lds1);
    s2 = row_sum<kLongThreads>(s2, lds2);
    if (threadIdx.x == 0) {
        const float r = 1.0f / __builtin_sqrtf(s1 / (float)g.N + g.eps);
        g.stats[2 * m] = r;
        g.stats[2 * m + 1] = r * (r * (s2 / (float)g.N));
    }
}
// 256 threads: 64 strips of eight columns x 4 rows; blockIdx.y is the row group.
template <class TX>
__global__ void __launch_bounds__(256) rmsnorm_grad_dweight_kernel(NormGradArgs g) {
    typedef typename Elt<TX>::T X;
    __shared__ float sums[3][64][8];
    const long long n = ((long long)blockIdx.x * 64 + (threadIdx.x & 63)) * 8;
    const int rl = threadIdx.x >> 6;
    const int valid = (int)std::min<long long>(g.N - n, 8);
    float dw[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (valid > 0) {
        for (long long m = (long long)blockIdx.y * 4 + rl; m < g.M; m += (long long)gridDim.y * 4) {
            float h[8], dy[8];
            load8<TX>(static_cast<const X*>(g.h) + m * g.ldh + n, valid, h);
            load8<TX>(static_cast<const X*>(g.dy) + m * g.ldy + n, valid, dy);
            const float r = g.stats[2 * m];
#pragma unroll
            for (int e = 0; e < 8; ++e) dw[e] = __builtin_fmaf(dy[e], h[e] * r, dw[e]);
        }
    }
    if (rl > 0)
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[rl - 1][threadIdx.x & 63][e] = dw[e];
    __syncthreads();
    if (rl == 0 && valid > 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            dw[e] = ((dw[e] + sums[0][threadIdx.x][e]) + sums[1][threadIdx.x][e]) + sums[2][threadIdx.x][e];
        store8<OutF32>(g.part + (long long)blockIdx.y * g.N + n, valid, dw);
    }
}
template <class TX>
__global__ void __launch_bounds__(kLongThreads) rmsnorm_grad_dx_kernel(NormGradArgs g) {
    typedef typename Elt<TX>::T X;
    const long long m = g.first + blockIdx.x;
    const float r = g.stats[2 * m], k = g.stats[2 * m + 1];
    for (long long n = threadIdx.x * 8; n < g.N; n += kLongThreads * 8) {
        const int valid = (int)std::min<long long>(g.N - n, 8);
        float h[8], dy[8], w[8], a[8];
        load8<TX>(static_cast<const X*>(g.h) + m * g.ldh + n, valid, h);
        load8<TX>(static_cast<const X*>(g.dy) + m * g.ldy + n, valid, dy);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[e] = 1.0f;
            a[e] = 0.0f;
        }
        if (g.weight) load8_vec<TX>(g.weight, g.w_type, n, valid, w);
        if (g.dh) load8<TX>(static_cast<const X*>(g.dh) + m * g.lds + n, valid, a);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += __builtin_fmaf(r * w[e], dy[e], -(h[e] * r * k));
        store8<TX>(static_cast<X*>(g.dx) + m * g.ldx + n, valid, a);
    }
}

__global__ void __launch_bounds__(1024) reduce_columns_kernel(const float* part, int rows, int N, void* out, int type) {
    __shared__ float sums[16][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15;
    const int n = (int)blockIdx.x * 16 + c;
    float s = 0.0f;
    if (n < N) {
        const float* p = part + n;
#pragma unroll 4
        for (int r = threadIdx.x >> 4; r < rows; r += 64) s += p[(long long)r * N];
    }
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    if (lane < 16) sums[wave][c] = s;
    __syncthreads();
    if (threadIdx.x < 16 && n < N) {
#pragma unroll
        for (int w = 1; w < 16; ++w) s += sums[w][c];
        store_any(out, type, n, s);
    }
}
bool launch_reduce_columns(const float* part, int rows, int N, void* out, int type, hipStream_t stream) {
    void* args[] = {&part, &rows, &N, &out, &type};
    return enqueue(reinterpret_cast<const void*>(&reduce_columns_kernel), (N + 15LL) / 16, 1024, args, stream);
}

namespace {

// Shapes of the register kernels: threads a row and groups of eight columns a thread.
struct Shape {
    int t, c;
};

template <class TX, bool Q>
const void* norm_kernel(Shape s) {
#define TS_NORM(T, C) \
    if (s.t == T && s.c == C) return reinterpret_cast<const void*>(&rmsnorm_kernel<TX, Q, T, C>)
    TS_NORM(16, 1); TS_NORM(16, 2); TS_NORM(16, 4);
    TS_NORM(64, 1); TS_NORM(64, 2); TS_NORM(64, 4);
    TS_NORM(256, 1); TS_NORM(256, 2); TS_NORM(256, 4);
    TS_NORM(1024, 1); TS_NORM(1024, 2); TS_NORM(1024, 4); TS_NORM(1024, 8);
#undef TS_NORM
    return reinterpret_cast<const void*>(&rmsnorm_long_kernel<TX, Q>);
}
template <class TX>
const void* norm_grad_kernel(Shape s) {
#define TS_NORM(T, C) \
    if (s.t == T && s.c == C) return reinterpret_cast<const void*>(&rmsnorm_grad_kernel<TX, T, C>)
    TS_NORM(16, 1); TS_NORM(16, 2); TS_NORM(16, 4);
    TS_NORM(64, 1); TS_NORM(64, 2); TS_NORM(64, 4);
    TS_NORM(256, 1); TS_NORM(256, 2); TS_NORM(256, 4);
    TS_NORM(1024, 1); TS_NORM(1024, 2); TS_NORM(1024, 4);
#undef TS_NORM
    return nullptr;
}

// Fewest threads a row whose four groups cover it; with few rows (fewer than would give
// every CU a workgroup) one group a thread where the workgroup allows it.  {0, 0}: a long
// row.
Shape norm_shape(int64_t M, int64_t N, int most) {
    const int64_t groups = (N + 7) / 8;
    static const int kThreads[] = {16, 64, 256, 1024};
    for (int t : kThreads) {
        const int limit = t == 1024 ? most : 4;
        const int want = t < 1024 && M * t < 256 * 256 ? 1 : limit;
        if (groups > (int64_t)t * want) continue;
        int c = 1;
        while ((int64_t)t * c < groups) c *= 2;
        return Shape{t, c};
    }
    return Shape{0, 0};
}

int64_t norm_grad_groups(int64_t M, int64_t N) {
    const Shape s = norm_shape(M, N, 4);
    if (s.t == 0) return std::max<int64_t>(1, std::min<int64_t>((M + 63) / 64, 64));
    const int rpw = s.t < 256 ? 256 / s.t : 1;
    return std::min<int64_t>((M + rpw - 1) / rpw, 1024);
}

bool row_type(int32_t t) { return t == TS_F16 || t == TS_BF16 || t == TS_F32; }
int type_size(int32_t t) { return t == TS_F32 ? 4 : t == TS_E4M3 ? 1 : 2; }

ts_status norm_sizes(int64_t M, int64_t N) {
    if (M < 0 || N < 0) return TS_ERR_INVALID_ARG;
    if (M > INT_MAX / 2 || N >= 1 << 26) return TS_ERR_UNSUPPORTED;   // N: threads of the launches over columns
    return TS_OK;
}

ts_status have_device() {
    int dev;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return TS_ERR_NO_DEVICE;
    }
    return TS_OK;
}

ts_status launch(const void* fn, int64_t gx, int64_t gy, int threads, void* args, hipStream_t stream) {
    void* argv[] = {args};
    return enqueue(fn, gx, threads, argv, stream, gy) ? TS_OK : TS_ERR_HIP;
}

// One workgroup for every few rows: a launch holds fewer than 2^32 threads, so many rows take
// more than one.
template <class Args>
ts_status launch_rows(const void* fn, int64_t blocks, int threads, Args& g, hipStream_t stream) {
    const int64_t most = (1LL << 31) / threads;
    for (g.first = 0; g.first < blocks; g.first += most) {
        const ts_status st = launch(fn, std::min<int64_t>(blocks - g.first, most), 1, threads, &g, stream);
        if (st != TS_OK) return st;
    }
    return TS_OK;
}

template <class TX>
ts_status run_norm(NormArgs& g, bool q, hipStream_t stream) {
    const Shape s = norm_shape(g.M, g.N, 8);
    const void* fn = q ? norm_kernel<TX, true>(s) : norm_kernel<TX, false>(s);
    if (s.t == 0) return launch_rows(fn, g.M, kLongThreads, g, stream);
    const int rpw = s.t < 256 ? 256 / s.t : 1;
    return launch_rows(fn, ((int64_t)g.M + rpw - 1) / rpw, std::max(s.t, 256), g, stream);
}

template <class TX>
ts_status run_norm_grad(NormGradArgs& g, int64_t groups, hipStream_t stream) {
    const Shape s = norm_shape(g.M, g.N, 4);
    if (s.t != 0) {
        return launch(norm_grad_kernel<TX>(s), groups, 1, std::max(s.t, 256), &g, stream);
    }
    ts_status st = launch_rows(reinterpret_cast<const void*>(&rmsnorm_grad_stats_kernel<TX>), g.M, kLongThreads, g, stream);
    if (st == TS_OK && g.part)
        st = launch(reinterpret_cast<const void*>(&rmsnorm_grad_dweight_kernel<TX>), ((int64_t)g.N + 511) / 512, groups,
                    256, &g, stream);
    if (st == TS_OK)
        st = launch_rows(reinterpret_cast<const void*>(&rmsnorm_grad_dx_kernel<TX>), g.M, kLongThreads, g, stream);
    return st;
}

}  // namespace
}  // namespace ts

using namespace ts;

extern "C" ts_status ts_rmsnorm(const void* x, const void* residual, const void* weight, void* y, void* h,
                                float* scale, int64_t M, int64_t N, int64_t stride_x, int64_t stride_r,
                                int64_t stride_y, int64_t stride_h, int32_t x_dtype, int32_t w_dtype,
                                int32_t y_dtype, float eps, void* stream) {
    ts_status st = norm_sizes(M, N);
    if (st != TS_OK) return st;
    if (!row_type(x_dtype) || (weight && !row_type(w_dtype)) || !(row_type(y_dtype) || y_dtype == TS_E4M3) ||
        !(eps >= 0.0f) || eps > 3.4e38f)
        return TS_ERR_INVALID_ARG;
    const bool q = y_dtype == TS_E4M3;
    if ((!q && y_dtype != x_dtype) || (weight && w_dtype != x_dtype && w_dtype != TS_F32)) return TS_ERR_UNSUPPORTED;
    if (M == 0 || (N == 0 && !q)) return TS_OK;
    // rows without elements still have their scale, the least one: the kernel below reads and
    // writes nothing else of them
    if (q && !scale) return TS_ERR_INVALID_ARG;
    if (N > 0 && (!x || !y || (residual && !h) || (!residual && h))) return TS_ERR_INVALID_ARG;
    if (N > 0 && M > 1 && (stride_x < N || stride_y < N || (residual && (stride_r < N || stride_h < N)))) return TS_ERR_INVALID_ARG;
    const int xs = type_size(x_dtype);
    if ((uintptr_t)x % xs || (uintptr_t)residual % xs || (uintptr_t)h % xs || (uintptr_t)y % type_size(y_dtype) ||
        (weight && (uintptr_t)weight % type_size(w_dtype)) || (uintptr_t)scale % 4)
        return TS_ERR_ALIGNMENT;
    if (N > 0 && (y == h || !in_place_ok(h, x, true, M, stride_h, stride_x) ||
                  !in_place_ok(h, residual, true, M, stride_h, stride_r) ||
                  !in_place_ok(y, x, !q, M, stride_y, stride_x) || !in_place_ok(y, residual, !q, M, stride_y, stride_r)))
        return TS_ERR_INVALID_ARG;
    st = have_device();
    if (st != TS_OK) return st;
    NormArgs g = {x, residual, weight, y, h, scale, (int)M, (int)N, w_dtype, stride_x, stride_r, stride_y, stride_h, eps};
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    if (x_dtype == TS_F16) return run_norm<OutF16>(g, q, hs);
    if (x_dtype == TS_BF16) return run_norm<OutBF16>(g, q, hs);
    return run_norm<OutF32>(g, q, hs);
}

// Bytes: the partial sums of dw, then (long rows) two numbers per row.
extern "C" int64_t ts_rmsnorm_backward_workspace(int64_t M, int64_t N) {
    ts_status st = norm_sizes(M, N);
    if (st != TS_OK) return st;
    if (M == 0 || N == 0) return 0;
    const int64_t part = (norm_grad_groups(M, N) * N * 4 + 255) / 256 * 256;
    return part + (norm_shape(M, N, 4).t == 0 ? M * 8 : 0);
}

extern "C" ts_status ts_rmsnorm_backward(const void* dy, const void* h, const void* weight, const void* dh, void* dx,
                                         void* dweight, int64_t M, int64_t N, int64_t stride_dy, int64_t stride_h,
                                         int64_t stride_dh, int64_t stride_dx, int32_t dtype, int32_t w_dtype,
                                         float eps, void* stream, void* workspace, int64_t workspace_bytes) {
    ts_status st = norm_sizes(M, N);
    if (st != TS_OK) return st;
    if (!row_type(dtype) || ((weight || dweight) && !row_type(w_dtype)) || !(eps >= 0.0f) || eps > 3.4e38f)
        return TS_ERR_INVALID_ARG;
    if ((weight || dweight) && w_dtype != dtype && w_dtype != TS_F32) return TS_ERR_UNSUPPORTED;
    if (workspace_bytes < 0) return TS_ERR_INVALID_ARG;
    if (N == 0 || (M == 0 && !dweight)) return TS_OK;
    if (M > 0 && (!dy || !h || !dx)) return TS_ERR_INVALID_ARG;
    if (M > 1 && (stride_dy < N || stride_h < N || stride_dx < N || (dh && stride_dh < N))) return TS_ERR_INVALID_ARG;
    const int xs = type_size(dtype);
    if ((uintptr_t)dy % xs || (uintptr_t)h % xs || (uintptr_t)dh % xs || (uintptr_t)dx % xs ||
        ((weight || dweight) && ((uintptr_t)weight % type_size(w_dtype) || (uintptr_t)dweight % type_size(w_dtype))))
        return TS_ERR_ALIGNMENT;
    if (!in_place_ok(dx, dy, true, M, stride_dx, stride_dy) || !in_place_ok(dx, h, true, M, stride_dx, stride_h) ||
        !in_place_ok(dx, dh, true, M, stride_dx, stride_dh))
        return TS_ERR_INVALID_ARG;
    const bool long_rows = norm_shape(M, N, 4).t == 0;
    const int64_t groups = M > 0 ? norm_grad_groups(M, N) : 0;
    const int64_t part = (groups * N * 4 + 255) / 256 * 256;
    const int64_t need = M == 0 ? 0 : (dweight || long_rows) ? part + (long_rows ? M * 8 : 0) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need || (uintptr_t)workspace % 256)) return TS_ERR_INVALID_ARG;
    st = have_device();
    if (st != TS_OK) return st;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    NormGradArgs g = {dy, h, weight, dh, dx, dweight ? static_cast<float*>(workspace) : nullptr,
                      long_rows ? reinterpret_cast<float*>(static_cast<char*>(workspace) + part) : nullptr,
                      (int)M, (int)N, w_dtype, stride_dy, stride_h, stride_dh, stride_dx, eps};
    if (M > 0) {
        st = dtype == TS_F16 ? run_norm_grad<OutF16>(g, groups, hs)
             : dtype == TS_BF16 ? run_norm_grad<OutBF16>(g, groups, hs) : run_norm_grad<OutF32>(g, groups, hs);
        if (st != TS_OK) return st;
    }
    if (dweight && !launch_reduce_columns(static_cast<float*>(workspace), (int)groups, (int)N, dweight, w_dtype, hs))
        return TS_ERR_HIP;
    return TS_OK;
}

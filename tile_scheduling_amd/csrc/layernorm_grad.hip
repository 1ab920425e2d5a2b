// The gradients of layer norm (layernorm.hip):
//
//   g = w dy:  dx = r (g - mean(g)) - u (r mean(g u)) + dh,  dw = sum over rows of dy u,  db = of dy
//
// Bound by memory: a row is read once, and held as it lies there (half the registers of fp32 in 16 bits, a
// quarter for h kept in 8), beside the running sums of dw and db.  Measured: 8192 x 4096 bf16 with dh 51 us (268 MB,
// 5.2 TB/s) and 6.5 us for the sums of 512 workgroups; 1000 x 2048 fp16 with h in 8 bits 12 and 4 us (the partial sums of 500
// workgroups move 16 MB beside 10 MB of rows).
#include "layernorm.hpp"
#include "limits.hpp"

namespace ts {

struct LayerGradArgs {
    const void *dy, *h, *weight, *dh;
    void* dx;
    float* part;    // partial sums, one row of N of dw and one of db per workgroup, or null
    float* stats;   // long rows: mean, its correction and r of every row, and a place left over
    int M, N, w_type;
    long long ldy, ldh, lds, ldx;   // (h in 8 bits: ldh in bytes)
    float eps;
    long long first;   // workgroups before this launch's (the launches of one workgroup a row)
};

template <class TX, bool HK>
using HRow = typename std::conditional<HK, RawKept, Raw8<TX>>::type;

// T threads a row (T <= 256: 256 / T rows a workgroup), C groups of eight columns a thread,
// T * C * 8 >= N; a workgroup walks rows (its row groups: row, row + groups, ...), the next one on its way while this
// one is worked on, each thread holding the weights and the running sums of dw and db of its own columns in
// registers.  HK: h kept in 8 bits.
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
    constexpr bool AHEAD = T < 1024;   // (1024 threads have 128 registers each: 30 spilled, 84 -> 113 us)
    struct Row {
        HRow<TX, HK> h[C];
        Raw8<TX> dy[C], dh[C];
    };
    auto load = [&](Row& r, long long m) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = (c * T + t) * 8, valid = g.N - n;
            r.h[c].load(g.h, m, g.ldh, n, g.N, valid);
            r.dy[c].load(g.dy, m, g.ldy, n, g.N, valid);
            if (g.dh) r.dh[c].load(g.dh, m, g.lds, n, g.N, valid);
        }
    };
    Row next;
    if (AHEAD && group < g.M) load(next, group);
    for (long long m = group; m < g.M; m += groups) {   // T > 64: one row a workgroup, so m is uniform
        Row now;
        if constexpr (AHEAD) {
            now = next;
            if (m + groups < g.M) load(next, m + groups);
        } else {
            load(now, m);
        }
        HRow<TX, HK>* h = now.h;
        Raw8<TX>* dy = now.dy;
        float a[2] = {0.0f, 0.0f};   // sums of h and g
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
        float mean = a[0] * rn;
        asm("" : "+v"(mean));   // one number for all its uses, not a product joined to some of them
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
                const float unit = ((x[e] - mean) - off) * r;   // (mean + off rounds the correction away)
                dw[c][e] = __builtin_fmaf(y[e], unit, dw[c][e]);
                db[c][e] += y[e];
                d[e] = __builtin_fmaf(-unit, k2, __builtin_fmaf(r * w[c][e], y[e], -k1));
            }
            if (g.dh) {
                float f[8];
                now.dh[c].unpack(f, valid);
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

// Long rows, in three steps: mean and deviation of each row, the partial sums of dw and db by strips of columns,
// and dx by rows (last: dx may take the place of dy or dh), whose first pass sums g and g d.
template <class TX, bool HK>
__global__ void __launch_bounds__(kLongThreads) layernorm_grad_stats_kernel(LayerGradArgs g) {
    __shared__ float lds1[kLongThreads / 64][1], lds2[kLongThreads / 64][2];
    const long long m = g.first + blockIdx.x;
    const float rn = 1.0f / (float)g.N;
    auto each = [&](auto&& f) {
        for (long long n = threadIdx.x * 8; n < g.N; n += kLongThreads * 8) {
            const int valid = (int)std::min<long long>(g.N - n, 8);
            HRow<TX, HK> h;
            float x[8];
            h.load(g.h, m, g.ldh, n, g.N, valid);
            h.unpack(x, valid);
#pragma unroll
            for (int e = 0; e < 8; ++e) f(x[e], e < valid);
        }
    };
    float a[1] = {0.0f}, b[2] = {0.0f, 0.0f};
    each([&](float x, bool) { a[0] += x; });
    row_sums<kLongThreads, 1>(a, lds1);
    float mean = a[0] * rn;
    asm("" : "+v"(mean));   // the number that is stored
    each([&](float x, bool in) {
        const float d = in ? x - mean : 0.0f;
        b[0] += d;
        b[1] = __builtin_fmaf(d, d, b[1]);
    });
    row_sums<kLongThreads, 2>(b, lds2);
    if (threadIdx.x == 0) {
        g.stats[4 * m] = mean;
        g.stats[4 * m + 1] = b[0] * rn;
        g.stats[4 * m + 2] = inverse_deviation(b[0], b[1], (float)g.N, g.eps);
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
            const float mean = g.stats[4 * m], off = g.stats[4 * m + 1], r = g.stats[4 * m + 2];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[e] = __builtin_fmaf(y[e], ((x[e] - mean) - off) * r, s[e]);
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
    __shared__ float lds[kLongThreads / 64][2];
    const long long m = g.first + blockIdx.x;
    const float mean = g.stats[4 * m], off = g.stats[4 * m + 1], r = g.stats[4 * m + 2], rn = 1.0f / (float)g.N;
    float s[2] = {0.0f, 0.0f};   // sums of g and g d
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
        for (int e = 0; e < 8; ++e) {
            s[0] = __builtin_fmaf(w[e], y[e], s[0]);
            s[1] = __builtin_fmaf(w[e] * y[e], e < valid ? (x[e] - mean) - off : 0.0f, s[1]);
        }
    }
    row_sums<kLongThreads, 2>(s, lds);
    const float k1 = r * (s[0] * rn), k2 = r * (r * (s[1] * rn));
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
        for (int e = 0; e < 8; ++e) a[e] += __builtin_fmaf(-(((x[e] - mean) - off) * r), k2, __builtin_fmaf(r * w[e], y[e], -k1));
        store8<TX>(static_cast<X*>(g.dx) + m * g.ldx + n, valid, a);
    }
}

namespace {

// Threads a row and groups of columns a thread; {0, 0}: a long row.
Shape grad_shape(int64_t N) {
    const int64_t groups = (N + 7) / 8;
    static const Shape kShapes[] = {{16, 1}, {16, 2}, {64, 1}, {64, 2}, {256, 1}, {256, 2}, {512, 2}, {1024, 2}};
    static_assert(kLayerGradRow == 1024 * 2 * 8, "the last shape");
    for (const Shape& s : kShapes)
        if (groups <= (int64_t)s.t * s.c) return s;
    return Shape{0, 0};
}
// Workgroups: as many as a CU holds at two groups of columns a thread and 512 threads, or one group and 768.
// Each writes two rows of fp32 partial sums, which are read again, so that more of them cost more than
// they hide, and fewer leave the memory idle.  Measured, bf16, 256 / 512 / 768 / 1024 / 2048 workgroups: 8192 x 4096 with dh 79 / 59 /
// 68 / 76 / 89 us (without the next row's loads ahead 95 / 66 / 69 / 79 / 88), 16384 x 2048 110 / 67 / 62 / 64 / 73, 32768 x
// 1024 69 / 57 / 59 / 64 / 66, 65536 x 512 99 / 63 / 57 / 57 / 62; 512 threads 4096 x 8192 68 / 77 / 89 / 98 / 130.
int64_t grad_groups(int64_t M, int64_t N) {
    const Shape s = grad_shape(N);
    if (s.t == 0) return std::max<int64_t>(1, std::min<int64_t>((M + 63) / 64, 64));
    const int64_t need = s.t < 256 ? (M * s.t + 255) / 256 : M;
    const int64_t most = s.t > 256 ? 256 : s.c == 1 ? 768 : 512;
    const int64_t rounds = std::max<int64_t>(1, (need + most - 1) / most);   // rows a workgroup: as even as they get
    return (need + rounds - 1) / rounds;
}
template <class TX, bool HK>
const void* grad_kernel_of(Shape s) {
#define TS_NORM(T, C) \
    if (s.t == T && s.c == C) return reinterpret_cast<const void*>(&layernorm_grad_kernel<TX, HK, T, C>)
    TS_NORM(16, 1); TS_NORM(16, 2); TS_NORM(64, 1); TS_NORM(64, 2);
    TS_NORM(256, 1); TS_NORM(256, 2); TS_NORM(512, 2); TS_NORM(1024, 2);
#undef TS_NORM
    return nullptr;
}

template <class TX, bool HK>
ts_status run_grad(LayerGradArgs& g, int64_t groups, hipStream_t stream) {
    const Shape s = grad_shape(g.N);
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

}  // namespace
}  // namespace ts

using namespace ts;

// Bytes: the partial sums of dw and db, then (long rows) four fp32 per row.
extern "C" int64_t ts_layernorm_backward_workspace(int64_t M, int64_t N) {
    ts_status st = grad_sizes(M, N);
    if (st != TS_OK) return st;
    if (M == 0 || N == 0) return 0;
    const int64_t part = (grad_groups(M, N) * 2 * N * 4 + 255) / 256 * 256;
    return part + (grad_shape(N).t == 0 ? M * 16 : 0);
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
    const bool long_rows = grad_shape(N).t == 0;
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

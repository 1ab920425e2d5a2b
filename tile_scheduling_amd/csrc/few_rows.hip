// Product with a fused epilogue for up to 32 rows of A.  A row of C costs a dot product with
// every column of B, so the time is that of reading B once; what matters is how many bytes of
// it are in flight.  Each workgroup owns a few columns and all of K, its waves take K steps
// in turn and keep several steps' loads in flight in registers (nothing of B is shared, so
// nothing is staged), and the partial sums meet in LDS in wave order: one launch, no
// workspace, the same bits on every run.  The 16 x 16 matrix instructions do the products
// with the rows of A padded to 16: rows past M (and columns past N) repeat the last one and
// are not stored.  Every load takes any element alignment, so nothing is packed.  Measured, bf16, B [N][K]:
// 1 x 4096 x 4096 7.7 us (4.4 TB/s), 1 x 28672 x 4096 46 us (5.1 TB/s); e4m3 4 x 8192 x 8192 12.8 us (5.3 TB/s);
// B [K][N] 13 x 12290 x 1000 8.9 us (2.8 TB/s), 1 x 28672 x 4096 52 us (4.6 TB/s).
//
//   B [N][K] (few_nt): a wave reads 128 bytes of 16 rows of B a step, lane group g bytes
//     32 g .. 32 g + 31 of each, which are its k of two 16-bit products or one 8-bit one
//     (which k a lane holds does not matter as long as A's lanes hold the same).
//   B [K][N] (few_nn): a wave reads 32 rows of B a step, V columns of 8 rows a lane, and
//     turns them in registers into V operands of 16 columns (one every V) x 32 k.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "few_rows.hpp"
#include "plan.hpp"
#include "schedule.hpp"

namespace ts {

typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));

template <class TI>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (std::is_same<TI, InF16>::value)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// The product of 32 bytes of each operand a lane; WIDE8 as in Engine.
template <class TI, bool WIDE8>
__device__ __forceinline__ f32x4 mfma_pair16(const u32x4* a, const u32x4* b, f32x4 c) {
    if constexpr (!std::is_same<TI, InE4M3>::value) {
        c = mfma16<TI>(a[0], b[0], c);
        return mfma16<TI>(a[1], b[1], c);
    } else if constexpr (WIDE8) {
        const i32x8 x = {(int)a[0][0], (int)a[0][1], (int)a[0][2], (int)a[0][3], (int)a[1][0], (int)a[1][1], (int)a[1][2], (int)a[1][3]};
        const i32x8 y = {(int)b[0][0], (int)b[0][1], (int)b[0][2], (int)b[0][3], (int)b[1][0], (int)b[1][1], (int)b[1][2], (int)b[1][3]};
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 0, 0, 0, 0, 0, 0);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            c = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen_e4m3(a[h][0], a[h][1]), widen_e4m3(b[h][0], b[h][1]), c, 0, 0, 0);
            c = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen_e4m3(a[h][2], a[h][3]), widen_e4m3(b[h][2], b[h][3]), c, 0, 0, 0);
        }
        return c;
    }
}

// 16 bytes at p, those at or past `left` zero; `room`: bytes of the row before p.  Where the row
// has 16 bytes, its last 16 are loaded and shifted: byte loads behind branches wait one for another.
__device__ __forceinline__ u32x4 load16_left(const uint8_t* p, long long left, long long room) {
    u32x4 v = {0, 0, 0, 0};
    if (left <= 0) return v;
    const int cut = left < 16 ? 16 - (int)left : 0;
    if (room >= cut) {
        v = *reinterpret_cast<const u32x4_a1*>(p - cut);
        uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
        if (cut >= 8) {
            lo = hi;
            hi = 0;
        }
        const int sh = 8 * (cut & 7);
        lo = sh ? lo >> sh | hi << (64 - sh) : lo;
        hi >>= sh;
        return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
#pragma unroll
    for (int e = 0; e < 15; ++e)
        if (e < left) v[e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
    return v;
}

// One element of C from its fp32 sum.
template <class TO>
__device__ __forceinline__ void finish_element(const FewArgs& g, float v, int m, long long n) {
    typedef typename Elt<TO>::T T;
    if (g.scale_a) v *= g.scale_a[m];
    if (g.scale_b) v *= g.scale_b[n];
    if (g.bias) v += load_any(g.bias, g.bias_type, n);
    const float in = g.aux_in ? (float)static_cast<const T*>(g.aux_in)[m * g.ld_in + n] : 0.0f;
    if (g.grad) {
        act_slopes<1>(g.act, &v, &in);
    } else {
        if (g.aux_out) static_cast<T*>(g.aux_out)[m * g.ld_out + n] = (T)v;
        act_values<1>(g.act, &v);
        v += in;
    }
    static_cast<T*>(g.C)[m * g.ldc + n] = (T)v;
}

// Partial sums of the waves, added in wave order, to C.  acc[x][y]: products of column group x
// with row group y; lane l holds column position 4 (l / 16) + r, row l mod 16; column position
// p of group x is column p * STRIDE + x * STEP of the workgroup's.
template <class TO, int WAVES, int NX, int MT, int STRIDE, int STEP>
__device__ __forceinline__ void meet_and_finish(const FewArgs& g, const f32x4 (*acc)[MT], float* red, long long n0) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    constexpr int TILES = NX * MT;
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
        for (int y = 0; y < MT; ++y)
            *reinterpret_cast<f32x4*>(red + ((wave * TILES + x * MT + y) * 64 + lane) * 4) = acc[x][y];
    __syncthreads();
    // outputs row by row, columns next to each other on neighbouring threads
    constexpr int COLS = 16 * NX;
    for (int o = threadIdx.x; o < COLS * 16 * MT; o += WAVES * 64) {
        const int m = o / COLS, c = o % COLS;
        const int x = STEP == 1 ? c % NX : c / 16, p = STEP == 1 ? c / NX : c % 16;
        const long long n = n0 + p * STRIDE + x * STEP;
        if (m >= g.M || n >= g.N) continue;
        const float* r = red + ((x * MT + m / 16) * 64 + (p >> 2) * 16 + m % 16) * 4 + (p & 3);
        float v = r[0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += r[w * TILES * 256];
        finish_element<TO>(g, v, m, n);
    }
}

constexpr int kNtWaves = 8;
// NX groups of 16 columns, MT groups of 16 rows, U steps in flight.
template <class TI, class TO, int NX, int MT, int U>
__global__ void __launch_bounds__(kNtWaves * 64) few_nt_kernel(FewArgs g) {
    constexpr int ES = std::is_same<TI, InE4M3>::value ? 1 : 2;
    constexpr bool WIDE8 = !std::is_same<TO, OutF32>::value;
    __shared__ __attribute__((aligned(16))) float red[kNtWaves * NX * MT * 256];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const long long n0 = (long long)xcd_remap(blockIdx.x, g.tiles, g.xcds) * (16 * NX);
    const long long kb = (long long)g.K * ES;   // bytes of a row
    const uint8_t *b[NX], *a[MT];
    const int r16 = lane & 15, at = (lane >> 4) * 32;
#pragma unroll
    for (int x = 0; x < NX; ++x) {
        const long long n = n0 + 16 * x + r16;
        b[x] = static_cast<const uint8_t*>(g.B) + (n < g.N ? n : g.N - 1) * g.ldb * ES + at;
    }
#pragma unroll
    for (int y = 0; y < MT; ++y) {
        const int m = 16 * y + r16;
        a[y] = static_cast<const uint8_t*>(g.A) + (m < g.M ? m : g.M - 1) * g.lda * ES + at;
    }
    f32x4 acc[NX][MT];
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
        for (int y = 0; y < MT; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
    const int full = (int)(kb / 128);   // whole steps
    auto steps = [&](int s, auto count) {
        constexpr int CNT = decltype(count)::value;
        u32x4 fb[CNT][NX][2], fa[CNT][MT][2];
#pragma unroll
        for (int u = 0; u < CNT; ++u) {
            const long long off = (long long)(s + u * kNtWaves) * 128;
#pragma unroll
            for (int x = 0; x < NX; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) fb[u][x][h] = *reinterpret_cast<const u32x4_a1*>(b[x] + off + 16 * h);
#pragma unroll
            for (int y = 0; y < MT; ++y)
#pragma unroll
                for (int h = 0; h < 2; ++h) fa[u][y][h] = *reinterpret_cast<const u32x4_a1*>(a[y] + off + 16 * h);
        }
        __builtin_amdgcn_sched_barrier(0);   // every load is issued before the first product
#pragma unroll
        for (int u = 0; u < CNT; ++u)
#pragma unroll
            for (int x = 0; x < NX; ++x)
#pragma unroll
                for (int y = 0; y < MT; ++y) acc[x][y] = mfma_pair16<TI, WIDE8>(fb[u][x], fa[u][y], acc[x][y]);
    };
    int s = wave;
    for (; s + (U - 1) * kNtWaves < full; s += U * kNtWaves) steps(s, std::integral_constant<int, U>{});
    if constexpr (U > 4) {   // what is left, as few waits as it takes
        if (s + 3 * kNtWaves < full) {
            steps(s, std::integral_constant<int, 4>{});
            s += 4 * kNtWaves;
        }
    }
    if (s + kNtWaves < full) {
        steps(s, std::integral_constant<int, 2>{});
        s += 2 * kNtWaves;
    }
    for (; s < full; s += kNtWaves) steps(s, std::integral_constant<int, 1>{});
    if (kb % 128 && wave == full % kNtWaves) {   // the last, partial step: both operands zero past K
        const long long off = (long long)full * 128;
        u32x4 fb[NX][2], fa[MT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long left = kb - off - at - 16 * h;
#pragma unroll
            for (int x = 0; x < NX; ++x) fb[x][h] = load16_left(b[x] + off + 16 * h, left, kb - left);
#pragma unroll
            for (int y = 0; y < MT; ++y) fa[y][h] = load16_left(a[y] + off + 16 * h, left, kb - left);
        }
#pragma unroll
        for (int x = 0; x < NX; ++x)
#pragma unroll
            for (int y = 0; y < MT; ++y) acc[x][y] = mfma_pair16<TI, WIDE8>(fb[x], fa[y], acc[x][y]);
    }
    meet_and_finish<TO, kNtWaves, NX, MT, 1, 16>(g, acc, red, n0);
}

constexpr int kNnWaves = 16;
// V columns a lane (16 V a workgroup), U steps of 32 rows of B in flight.
template <class TI, class TO, int V, int MT, int U>
__global__ void __launch_bounds__(kNnWaves * 64) few_nn_kernel(FewArgs g) {
    typedef typename std::conditional<V == 4, u32x2_a2, u32_a2>::type Vec;
    constexpr int W = V / 2;   // dwords of a lane's piece of a row
    __shared__ __attribute__((aligned(16))) float red[kNnWaves * V * MT * 256];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const long long n0 = (long long)xcd_remap(blockIdx.x, g.tiles, g.xcds) * (16 * V);
    const int r16 = lane & 15, kg = (lane >> 4) * 8;
    const long long n = n0 + r16 * V;
    const int cols = (int)(g.N - n < V ? (g.N - n > 0 ? g.N - n : 0) : V);   // of this lane's, inside B
    const uint16_t* b = static_cast<const uint16_t*>(g.B) + (cols > 0 ? n : 0) + kg * g.ldb;
    const uint16_t* a[MT];
#pragma unroll
    for (int y = 0; y < MT; ++y) {
        const int m = 16 * y + r16;
        a[y] = static_cast<const uint16_t*>(g.A) + (m < g.M ? m : g.M - 1) * g.lda + kg;
    }
    f32x4 acc[V][MT];
#pragma unroll
    for (int x = 0; x < V; ++x)
#pragma unroll
        for (int y = 0; y < MT; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
    // row j of a lane's 8 x V piece at p
    auto row_of = [&](const uint16_t* p, uint32_t* w) {
        if (cols == V) {
            const Vec v = *reinterpret_cast<const Vec*>(p);
            __builtin_memcpy(w, &v, sizeof v);
        } else {
#pragma unroll
            for (int d = 0; d < W; ++d)
                w[d] = (2 * d < cols ? (uint32_t)p[2 * d] : 0u) | (2 * d + 1 < cols ? (uint32_t)p[2 * d + 1] << 16 : 0u);
        }
    };
    auto multiply = [&](const uint32_t (*w)[W], const u32x4* fa) {
#pragma unroll
        for (int x = 0; x < V; ++x) {
            u32x4 f;
#pragma unroll
            for (int d = 0; d < 4; ++d)
                f[d] = __builtin_amdgcn_perm(w[2 * d + 1][x / 2], w[2 * d][x / 2], x % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
            for (int y = 0; y < MT; ++y) acc[x][y] = mfma16<TI>(f, fa[y], acc[x][y]);
        }
    };
    const int full = g.K / 32;
    auto steps = [&](int s, auto count) {
        constexpr int CNT = decltype(count)::value;
        uint32_t w[CNT][8][W];
        u32x4 fa[CNT][MT];
#pragma unroll
        for (int u = 0; u < CNT; ++u) {
            const long long k = (long long)(s + u * kNnWaves) * 32;
#pragma unroll
            for (int j = 0; j < 8; ++j) row_of(b + (k + j) * g.ldb, w[u][j]);
#pragma unroll
            for (int y = 0; y < MT; ++y) fa[u][y] = *reinterpret_cast<const u32x4_a2*>(a[y] + k);
        }
        __builtin_amdgcn_sched_barrier(0);   // every load is issued before the first product
#pragma unroll
        for (int u = 0; u < CNT; ++u) multiply(w[u], fa[u]);
    };
    int s = wave;
    for (; s + (U - 1) * kNnWaves < full; s += U * kNnWaves) steps(s, std::integral_constant<int, U>{});
    for (; s < full; s += kNnWaves) steps(s, std::integral_constant<int, 1>{});
    if (g.K % 32 && wave == full % kNnWaves) {   // the last, partial step
        const long long k = (long long)full * 32;
        const int left = g.K - (int)k - kg;      // rows of this lane's eight inside B
        uint32_t w[8][W];
        u32x4 fa[MT];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int d = 0; d < W; ++d) w[j][d] = 0;
            if (j < left) row_of(b + (k + j) * g.ldb, w[j]);
        }
#pragma unroll
        for (int y = 0; y < MT; ++y) fa[y] = load16_left(reinterpret_cast<const uint8_t*>(a[y] + k), 2 * left, 2LL * (k + kg));
        multiply(w, fa);
    }
    meet_and_finish<TO, kNnWaves, V, MT, V, 1>(g, acc, red, n0);
}

namespace {

// Column groups a workgroup of few_nt: as few as leave one workgroup on each of 256 CUs, up to two,
// with more than 16 rows four: the rows of A are read for each group of columns by every
// workgroup, which for 32 rows is 2 / NX times the bytes of B.  Measured, K = 4096, bf16, one / two / four groups: 1 row
// N = 4096 7.8 / 10.8 / 18.7 us, 8192 16.6 / 15.2 / 20.7, 28672 47.5 / 46.9 / 47.8; 16 rows 8192 20.7 / 15.9 / 23.9,
// 28672 64.8 / 50.8 / 50.9; 32 rows 4096 14.1 / 18.6 / 26.8, 8192 27.4 / 20.4 / 28.5, 12290 50.0 / 36.9 / 30.3, 28672
// 89.9 / 72.6 / 58.4; e4m3, 32 rows, 28672 52.6 / 42.6 / 38.4.
// Columns a lane of few_nn: two, or four where two make more than 256 workgroups (of 16 waves, one on a
// CU): 16 rows 8192 x 8192 41.8 / 46.3 us, 12290 x 4096 39.6 / 35.3, 28672 x 4096 77.3 / 59.7.
constexpr int kGroups = 256;
template <class TI, class TO, int MT>
const void* nt_kernel(int nx) {
    if (nx == 4) return reinterpret_cast<const void*>(&few_nt_kernel<TI, TO, 4, MT, (MT == 1 ? 3 : 2)>);
    if (nx == 2) return reinterpret_cast<const void*>(&few_nt_kernel<TI, TO, 2, MT, 4>);
    return reinterpret_cast<const void*>(&few_nt_kernel<TI, TO, 1, MT, (MT == 1 ? 8 : 4)>);
}
template <class TI, class TO, int MT>
const void* nn_kernel(int v) {
    if (v == 4) return reinterpret_cast<const void*>(&few_nn_kernel<TI, TO, 4, MT, 2>);
    return reinterpret_cast<const void*>(&few_nn_kernel<TI, TO, 2, MT, (MT == 1 ? 3 : 2)>);
}
template <class TI, class TO>
const void* few_kernel(bool b_kmaj, int mt, int width) {
    if constexpr (std::is_same<TI, InE4M3>::value) {
        return mt == 1 ? nt_kernel<TI, TO, 1>(width) : nt_kernel<TI, TO, 2>(width);
    } else {
        if (b_kmaj) return mt == 1 ? nt_kernel<TI, TO, 1>(width) : nt_kernel<TI, TO, 2>(width);
        return mt == 1 ? nn_kernel<TI, TO, 1>(width) : nn_kernel<TI, TO, 2>(width);
    }
}

}  // namespace

bool launch_few_rows(FewArgs& g, int ab, int c, bool b_kmaj, hipStream_t stream) {
    const int mt = g.M > 16 ? 2 : 1;
    int width, cols;
    if (b_kmaj) {
        width = g.N <= 16 * kGroups ? 1 : mt == 1 || g.N <= 32 * kGroups ? 2 : 4;
        cols = 16 * width;
    } else {
        width = g.N <= 32 * kGroups ? 2 : 4;
        cols = 16 * width;
    }
    g.tiles = (int)(((int64_t)g.N + cols - 1) / cols);
    const void* fn;
    if (ab == ELT_F16) fn = c == ELT_F32 ? few_kernel<InF16, OutF32>(b_kmaj, mt, width) : few_kernel<InF16, OutF16>(b_kmaj, mt, width);
    else if (ab == ELT_BF16) fn = c == ELT_F32 ? few_kernel<InBF16, OutF32>(b_kmaj, mt, width) : few_kernel<InBF16, OutBF16>(b_kmaj, mt, width);
    else fn = c == ELT_F32 ? few_kernel<InE4M3, OutF32>(true, mt, width)
              : c == ELT_F16 ? few_kernel<InE4M3, OutF16>(true, mt, width) : few_kernel<InE4M3, OutBF16>(true, mt, width);
    void* args[] = {&g};
    return enqueue(fn, g.tiles, (b_kmaj ? kNtWaves : kNnWaves) * 64, args, stream);
}

}  // namespace ts

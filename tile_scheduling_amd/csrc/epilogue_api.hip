// C-ABI of the product with a fused epilogue (ts_gemm_epilogue): argument checks, operand
// packing, launch planning and dispatch.  See include/tsgemm.h for the contract.
#include <hip/hip_runtime.h>

#include <limits.h>
#include <stdint.h>
#include <string.h>

#include <map>
#include <mutex>
#include <tuple>

#include "../../include/tsgemm.h"
#include "epilogue.hpp"
#include "few_rows.hpp"
#include "split.hpp"
#include "plan.hpp"
#include "rows.hpp"

namespace ts {

// Copies rows of row_bytes bytes (any alignment, `pitch` apart) to rows of `chunks` 16-byte
// chunks, zero behind the data.  Runs in front of a product whose operand the direct-to-LDS
// loads cannot take as it is (its rows not 16-byte aligned, or K not a multiple of 16 bytes,
// so that a 16-byte chunk would mix the end of a row with the next one); both operands of a
// product in one launch.  A workgroup takes 1024 consecutive chunks, four a thread in flight:
// 12290 + 5000 rows of 1000 bytes 9.5 us (3.6 TB/s; with one chunk a thread and byte loads at the ends 16).
struct PackArgs {
    struct Matrix {
        const uint8_t* src;
        uint8_t* dst;
        long long pitch, row_bytes, chunks, blocks;   // blocks: workgroups, 0 = nothing to do
        long long rows;
    } m[2];
};
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
constexpr int kPackChunks = 1024;
__global__ void __launch_bounds__(256) pack_rows_kernel(PackArgs g) {
    const bool second = blockIdx.x >= g.m[0].blocks;
    const PackArgs::Matrix& p = g.m[second];
    const long long first = (long long)(blockIdx.x - (second ? g.m[0].blocks : 0)) * kPackChunks;
    const long long r0 = first / p.chunks, left = p.chunks * p.rows - first;
    const uint32_t c0 = (uint32_t)(first - r0 * p.chunks), chunks = (uint32_t)p.chunks;
    u32x4 v[4];
    if (p.row_bytes >= 16) {
        // the last chunk of a row is the row's last 16 bytes, shifted: no loads behind a branch
        uint32_t cut[4];   // bytes that the load begins before the chunk
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = threadIdx.x + 256 * i < left ? threadIdx.x + 256 * i : 0;
            const uint32_t r = (c0 + c) / chunks;
            const long long b = (long long)(c0 + c - r * chunks) * 16, last = p.row_bytes - 16;
            cut[i] = b > last ? (uint32_t)(b - last) : 0;
            v[i] = *reinterpret_cast<const u32x4_a1*>(p.src + (r0 + r) * p.pitch + (b - cut[i]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint64_t lo = v[i][0] | (uint64_t)v[i][1] << 32, hi = v[i][2] | (uint64_t)v[i][3] << 32;
            if (cut[i] >= 8) {
                lo = hi;
                hi = 0;
            }
            const uint32_t sh = 8 * (cut[i] & 7);
            lo = sh ? lo >> sh | hi << (64 - sh) : lo;
            hi >>= sh;
            v[i] = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = threadIdx.x + 256 * i;
            u32x4 w = {0, 0, 0, 0};
            if (c < left) {   // one chunk a row
                const uint8_t* s = p.src + (first + c) * p.pitch;
#pragma unroll
                for (int e = 0; e < 15; ++e)
                    if (e < p.row_bytes) w[e >> 2] |= (uint32_t)s[e] << (8 * (e & 3));
            }
            v[0] = i == 0 ? w : v[0];
            v[1] = i == 1 ? w : v[1];
            v[2] = i == 2 ? w : v[2];
            v[3] = i == 3 ? w : v[3];
        }
    }
    u32x4* d = reinterpret_cast<u32x4*>(p.dst) + first + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (threadIdx.x + 256 * i < left) d[256 * i] = v[i];
}

__global__ void clear_flags_kernel(int* p, int n) {
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) p[i] = 0;
}

namespace {

constexpr int64_t kOffsetLimit = 1LL << 30;   // in-tile byte offsets of the direct-to-LDS loads
constexpr int64_t kMaxExtent = INT_MAX - 1024;    // rows and columns of the last tile stay ints
constexpr int64_t kMaxStride = (1LL << 26) - 1;   // 32-bit lane offsets of the epilogue (16 rows of 4 bytes)
// K split (splits_of): programs at most, K steps each at least.  256, here, in the choice of the tile
// and in few_rows.hip: the CUs of a whole MI355X; a workspace's size then needs no device.
constexpr int64_t kSplitPrograms = 256, kSplitSteps = 8;
constexpr int kSpin = 1 << 24;                // sleeps before a stream-K wait gives up (about a second)

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// One operand as the kernel reads it: rows of `ld` elements, either along K (kmaj) or
// along M / N.
struct Operand {
    bool kmaj;
    int64_t ld;            // elements between stored rows, as given
    int64_t rows, cols;    // stored rows and their elements
    bool pack;             // copied to aligned rows first
    int64_t packed_bytes;
};

struct EpiPlan {
    Plan p;
    int path, kind, out;
    int special = 0;       // special form of the epilogue (EPI_SPECIAL + ...), 0: the general one
    int es;                // operand element size in bytes
    Operand a, b;
    bool few;              // few_rows.hip runs it: none of the rest is filled
    int64_t kp;            // K as the kernel sees it, elements (a multiple of 16 bytes if an operand is kmaj)
    WorkspaceLayout sk;
    int splits;            // EPI_SPLIT: programs that share a tile's K
    int64_t sums_bytes;    // and their fp32 sums, at the workspace's start
    int64_t off_a, off_b, total;   // workspace offsets of the packed operands, and its size
};

bool known_type(int32_t t) { return t == TS_F16 || t == TS_BF16 || t == TS_F32 || t == TS_E4M3; }

// Layout of an operand with `rows` x K (A) or K x `rows` (B) logical elements: s_r and
// s_k are the strides along its rows (M or N) and along K.
ts_status operand_layout(int64_t rows, int64_t K, int64_t s_r, int64_t s_k, bool kmaj_only, Operand* o) {
    if (s_r < 0 || s_k < 0) return TS_ERR_INVALID_ARG;
    const bool k_ok = K <= 1 || s_k == 1;
    const bool r_ok = rows <= 1 || s_r == 1;
    if (!k_ok && !r_ok) return TS_ERR_UNSUPPORTED;
    // a single row along M or N, or a single k: whichever reading its unit stride allows
    o->kmaj = kmaj_only ? true : (k_ok && r_ok) ? (rows <= 1 ? s_k == 1 : s_r != 1) : k_ok;
    if (kmaj_only && !k_ok) return TS_ERR_UNSUPPORTED;
    o->rows = o->kmaj ? rows : K;
    o->cols = o->kmaj ? K : rows;
    o->ld = o->kmaj ? s_r : s_k;
    if (o->rows <= 1) o->ld = o->cols;
    if (o->ld < o->cols) return TS_ERR_INVALID_ARG;
    if (o->ld > INT_MAX) return TS_ERR_UNSUPPORTED;
    o->pack = false;
    o->packed_bytes = 0;
    return TS_OK;
}

// Whether the loads take the operand as it lies; else it is packed.  `tile` is its extent
// of a tile along the stored rows (rows of M / N, or of K).
ts_status operand_pack(Operand* o, uintptr_t base, int es, int tile) {
    if (o->kmaj) {
        o->pack = base % 16 != 0 || (o->ld * es) % 16 != 0 || (o->cols * es) % 16 != 0 ||
                  tile * o->ld * es >= kOffsetLimit;
    } else {
        o->pack = base % 4 != 0 || o->ld % 2 != 0 || o->cols % 2 != 0 || tile * o->ld * es >= kOffsetLimit;
    }
    if (o->pack) {
        const int64_t pitch = round_up(o->cols * es, 16);
        if (tile * pitch >= kOffsetLimit) return TS_ERR_UNSUPPORTED;
        o->packed_bytes = round_up(pitch * o->rows, 256);
    }
    return TS_OK;
}

// Sleeps (320 clocks, FusedStore::start) between the starts of the eight groups of programs.
// With fp32 C a 256 tile moves 256 KiB after its K loop, 512 KiB with a matrix read beside it, as
// long as 9 or 18 K steps at the copy rate while all CUs do it at once; spread over a part of a
// tile's time, the groups' traffic overlaps the others' products.  Measured with 4 tiles a program
// (4096 x 16384), together / spread: with residual K = 512 131 / 121 us, 1024 177 / 166, 2048 274 / 261,
// 4096 488 / 473; without 512 95 / 86, 1024 137 / 135, and no gain from 2048 on.  With 16-bit C 0 to 10 %
// slower at every K.  Spread by XCD instead (its programs share operands): residual 512 136, 1024 182.
int stagger_sleeps(const EpiPlan& e, bool reads) {
    const SchedArgs& s = e.p.s;
    if (e.kind != EPI_XTILE || e.p.cfg != CFG_256W8 || e.out != TS_F32 || s.num_tiles < 3 * (int64_t)s.grid) return 0;
    return reads ? std::min(s.ks, 64) / 4 + 4 : s.ks <= 16 ? s.ks / 4 : 0;
}

// The special form of an epilogue, 0 if it has none.  They exist where the 256 tile runs (see
// SpecialStore): one use of aux_in or aux_out at most, 16-bit operands, A stored [M][K].
int special_kind(const ts_epilogue& x, const void* C, int64_t stride_cm, int32_t c) {
    const int fam = x.activation == TS_ACT_NONE ? FAM_NONE : x.activation == TS_ACT_RELU ? FAM_RELU
                    : x.activation == TS_ACT_GELU ? FAM_ERF : FAM_SIGMOID;
    if (!x.grad && x.residual && x.preact) return 0;
    int aux = x.grad ? AUX_GRAD : x.residual ? AUX_RESIDUAL : x.preact ? AUX_PREACT : AUX_NONE;
    if (aux == AUX_PREACT && c != TS_F32 && (fam == FAM_ERF || fam == FAM_SIGMOID) && (uintptr_t)C % 128 == 0 &&
        (uintptr_t)x.preact % 128 == 0 && stride_cm * 2 % 128 == 0 && x.stride_pm * 2 % 128 == 0)
        aux = AUX_LINES;
    return EPI_SPECIAL + 4 * aux + fam;
}

const void* epi_kernel_of(const EpiPlan& e, int32_t ab) {
    const int f32 = e.out == TS_F32;
    if (e.special && e.kind == EPI_XTILE && e.p.cfg == CFG_256W8) {
        const void* fn = nullptr;
        if (e.path == PATH_EDGE_NN)
            fn = ab == TS_F16 ? epi_special_f16_nn(f32, e.special) : ab == TS_BF16 ? epi_special_bf16_nn(f32, e.special) : nullptr;
        if (e.path == PATH_EDGE_BT)
            fn = ab == TS_F16 ? epi_special_f16_nt(f32, e.special) : ab == TS_BF16 ? epi_special_bf16_nt(f32, e.special) : nullptr;
        if (e.path == PATH_EDGE_AT)
            fn = ab == TS_F16 ? epi_special_f16_tn(f32, e.special) : ab == TS_BF16 ? epi_special_bf16_tn(f32, e.special) : nullptr;
        if (fn) return fn;
    }
    if (e.p.cfg == CFG_128) {
        if (ab == TS_F16) return epi_kernels_cfg128_f16(f32, e.path, e.kind);
        if (ab == TS_BF16) return epi_kernels_cfg128_bf16(f32, e.path, e.kind);
        return epi_kernels_cfg128_e4m3(e.out, e.path, e.kind);
    }
    if (ab == TS_F16) return epi_kernels_cfg256w8_f16(f32, e.path, e.kind);
    if (ab == TS_BF16) return epi_kernels_cfg256w8_bf16(f32, e.path, e.kind);
    return epi_kernels_cfg256w8_e4m3(e.out, e.path, e.kind);
}

// What planning asks the runtime or computes at length, kept per kernel and per tile grid:
// workgroups a CU holds, and the order the locality model chooses.
std::mutex g_cache_mutex;
std::map<std::pair<int, const void*>, int> g_occupancy;
struct OrderChoice {
    int order, group_m, remap, reuse;
};
std::map<std::tuple<int, int, int, int, int>, OrderChoice> g_orders;
constexpr size_t kMaxOrders = 4096;

int occupancy_of(int dev, const void* fn, int threads) {
    std::lock_guard<std::mutex> lock(g_cache_mutex);
    auto it = g_occupancy.find({dev, fn});
    if (it != g_occupancy.end()) return it->second;
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, 0) != hipSuccess || n < 1) {
        (void)hipGetLastError();
        n = 1;
    }
    g_occupancy[{dev, fn}] = n;
    return n;
}

// resolve_grid with the chosen order kept by what it depends on: the tile grid, the programs (in
// stream-K mode at most one per K step, so the number of K steps counts) and how many of them run
// together.
ts_status resolve(Plan* p, int cu_count, int ppc, int xcds) {
    if (!p->auto_order || p->s.num_tiles == 0) return resolve_grid(p, cu_count, ppc, xcds);
    const int64_t cap = p->mode == TS_MODE_STREAMK ? (int64_t)p->s.num_tiles * std::max(p->s.ks, 1) : p->s.num_tiles;
    const int64_t want = p->mode == TS_MODE_TILED ? p->s.num_tiles
                                                  : (p->requested_programs ? p->requested_programs : cu_count * ppc);
    const auto key = std::make_tuple(p->s.nm, p->s.nn, (int)std::min(want, cap), cu_count * ppc, xcds * 8 + p->mode);
    OrderChoice c;
    bool found = false;
    {
        std::lock_guard<std::mutex> lock(g_cache_mutex);
        auto it = g_orders.find(key);
        if (it != g_orders.end()) {
            c = it->second;
            found = true;
        }
    }
    if (!found) {
        ts_status st = resolve_grid(p, cu_count, ppc, xcds);
        if (st != TS_OK) return st;
        c = OrderChoice{p->s.order, p->s.group_m, p->s.remap, p->l2_reuse_pm};
        std::lock_guard<std::mutex> lock(g_cache_mutex);
        if (g_orders.size() >= kMaxOrders) g_orders.clear();
        g_orders[key] = c;
        return TS_OK;
    }
    p->auto_order = false;
    p->s.order = c.order;
    p->s.group_m = c.group_m;
    p->s.remap = c.remap;
    return resolve_grid(p, cu_count, ppc, xcds);
}

// Programs that share the K of each of `tiles` 128 tiles of `ks` K steps; 1: none does.  A tile
// alone waits for memory in every step (0.6 us), so K is split until a program is on each of 256
// CUs, in parts of 8 steps at least, if the steps saved outweigh the second launch and the sums'
// way through memory (6 steps and one for 16 programs).  Measured, whole / split, bf16: 64 x 4096 x 4096
// 41.4 / 17.8 us, 256 x 4096 x 4096 41.2 / 22.7, 512 x 4096 x 4096 42.0 / 32.2, 1000 x 512 x 2048 23.4 / 16.1,
// 200 x 512 x 16384 144 / 20.7; e4m3 128 x 8192 x 8192 60.0 / 27.9.  With parts of 4 steps 1000 x 512
// x 2048 took 19.4 and 256 x 256 x 16384 24.9 against 18.7; with 512 programs 256 x 4096 x 4096 23.6, 64 x
// 16384 x 4096 36.6 against 45.2 but [K][N] 41.4 against 39.4.  Not worth it: 1024 x 1024 x 1024 15.2 /
// 15.9, 512 x 2048 x 1000 14.8 / 16.1.
int splits_of(int64_t tiles, int64_t ks) {
    const int64_t s = std::min<int64_t>(kSplitPrograms / std::max<int64_t>(tiles, 1), ks / kSplitSteps);
    return s > 1 && ks - cdiv64(ks, s) > 6 + tiles * s / 16 ? (int)s : 1;
}

// Everything but the device: types, layouts, tile, schedule, packing.
ts_status epi_plan(const void* A, const void* B, int64_t M, int64_t N, int64_t K, int64_t sam, int64_t sak,
                   int64_t sbk, int64_t sbn, int32_t ab, int32_t c, const ts_schedule* sp, EpiPlan* e) {
    if (M < 0 || N < 0 || K < 0) return TS_ERR_INVALID_ARG;
    if (M > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return TS_ERR_UNSUPPORTED;
    if (!known_type(ab) || !known_type(c)) return TS_ERR_INVALID_ARG;
    if (ab == TS_F32 || c == TS_E4M3 || (ab == TS_F16 && c == TS_BF16) || (ab == TS_BF16 && c == TS_F16))
        return TS_ERR_UNSUPPORTED;
    ts_schedule s = {TS_ORDER_AUTO, 1, TS_MODE_AUTO, 0, 0, TS_TILE_AUTO, TS_INDEX_DIVIDE};
    if (sp) s = *sp;
    if (s.order != TS_ORDER_ROW_MAJOR && s.order != TS_ORDER_GROUPED && s.order != TS_ORDER_AUTO)
        return TS_ERR_INVALID_ARG;
    if (s.order == TS_ORDER_GROUPED && s.group_m < 1) return TS_ERR_INVALID_ARG;
    if (s.mode != TS_MODE_TILED && s.mode != TS_MODE_PERSISTENT && s.mode != TS_MODE_CROSSTILE &&
        s.mode != TS_MODE_STREAMK && s.mode != TS_MODE_AUTO)
        return TS_ERR_INVALID_ARG;
    if (s.index_math != TS_INDEX_DIVIDE && s.index_math != TS_INDEX_MULSHIFT) return TS_ERR_INVALID_ARG;
    if (s.num_programs < 0 || (s.xcd_remap != 0 && s.xcd_remap != 1)) return TS_ERR_INVALID_ARG;
    if (s.tile_config < TS_TILE_AUTO || s.tile_config > TS_TILE_256x256x64_PP) return TS_ERR_INVALID_ARG;
    if (s.tile_config != TS_TILE_AUTO && s.tile_config != TS_TILE_128x128x64 && s.tile_config != TS_TILE_256x256x64_W8)
        return TS_ERR_UNSUPPORTED;

    e->es = ab == TS_E4M3 ? 1 : 2;
    e->out = c;
    ts_status st = operand_layout(M, K, sam, sak, ab == TS_E4M3, &e->a);
    if (st != TS_OK) return st;
    st = operand_layout(N, K, sbn, sbk, ab == TS_E4M3, &e->b);
    if (st != TS_OK) return st;
    e->path = e->a.kmaj ? (e->b.kmaj ? PATH_EDGE_BT : PATH_EDGE_NN) : (e->b.kmaj ? PATH_EDGE_ATBT : PATH_EDGE_AT);

    // few rows and a schedule that leaves everything to the library: one pass over B
    const bool open = s.order == TS_ORDER_AUTO && s.mode == TS_MODE_AUTO && s.tile_config == TS_TILE_AUTO && s.num_programs == 0;
    // (B stored [K][N]: up to the K where the split tiles win, us few / tiles: 16 rows 4096 x 4096 14.9 / 17.6, 8192 x
    // 8192 41.8 / 39.1, 4096 x 14336 66.5 / 37.4; 32 rows 12290 x 1000 12.5 / 16.8, 4096 x 4096 18.5 / 17.6, 28672 x 4096
    // 71.1 / 62.3)
    e->few = open && M > 0 && M <= kFewRows && N < 1 << 26 && e->a.kmaj &&   // N: threads of a launch
             (e->b.kmaj || K < (M > 16 ? 4096 : 8192));
    e->splits = 1;
    e->sums_bytes = 0;
    if (e->few) {
        e->kind = 0;
        return TS_OK;
    }

    Plan& p = e->p;
    // Up to 128 tiles of 256 leave half the CUs idle or more, while their four times as many 128
    // tiles run all at once, two on a CU.  K = 4096, 128 tile / 256 tile: bf16 with 128 tiles of 256 66.3 /
    // 76.1 us, with 136 98.2 / 76.3; fp32 C with residual 71.1 / 86.0, 107 / 89.2; e4m3 36.1 / 45.4, 53.9 / 45.4.
    p.cfg = s.tile_config != TS_TILE_AUTO ? s.tile_config
            : cdiv64(M, 256) * cdiv64(N, 256) > 128 ? CFG_256W8 : CFG_128;
    p.bm = p.bn = p.cfg == CFG_128 ? 128 : 256;
    p.bk = 128 / e->es;   // one slice row is 128 bytes
    st = operand_pack(&e->a, (uintptr_t)A, e->es, e->a.kmaj ? p.bm : p.bk);
    if (st != TS_OK) return st;
    st = operand_pack(&e->b, (uintptr_t)B, e->es, e->b.kmaj ? p.bn : p.bk);
    if (st != TS_OK) return st;
    e->kp = e->a.kmaj || e->b.kmaj ? round_up(K, 16 / e->es) : K;
    // the kernels run at least two K steps a tile; slices past K read as zero
    const int64_t nm = cdiv64(M, p.bm), nn = cdiv64(N, p.bn), ks = std::max<int64_t>(2, cdiv64(e->kp, p.bk));
    if (nm * nn > INT_MAX / 2) return TS_ERR_UNSUPPORTED;
    if (s.mode == TS_MODE_AUTO) s.mode = TS_MODE_CROSSTILE;
    p.mode = s.mode;
    p.io = 0;
    p.masked = true;
    p.path = e->path;
    p.vec_a = p.vec_b = p.vec_c = 0;
    p.requested_programs = s.num_programs;
    p.s.nm = (int)nm;
    p.s.nn = (int)nn;
    p.s.ks = (int)ks;
    p.s.num_tiles = (int)(nm * nn);
    p.auto_order = s.order == TS_ORDER_AUTO;
    p.l2_reuse_pm = -1;
    p.s.order = p.auto_order ? TS_ORDER_ROW_MAJOR : s.order;
    p.s.group_m = s.order == TS_ORDER_GROUPED ? (int)std::min<int64_t>(s.group_m, std::max<int64_t>(nm, 1)) : 1;
    p.s.remap = p.auto_order ? 0 : s.xcd_remap;
    p.s.xcds = 8;
    p.s.grid = 0;
    p.s.fastdiv = s.index_math == TS_INDEX_MULSHIFT;
    p.max_items = 0;
    e->kind = p.mode == TS_MODE_STREAMK ? EPI_STREAMK : EPI_XTILE;
    if (open && p.cfg == CFG_128) {
        e->splits = splits_of(nm * nn, ks);
        if (e->splits > 1) {
            e->kind = EPI_SPLIT;
            e->sums_bytes = e->splits * nm * nn * (int64_t)p.bm * p.bn * 4;
        }
    }
    return TS_OK;
}

// The grid and the workspace; needs the device where the grid does.
ts_status epi_resolve(EpiPlan* e, int32_t ab, int dev, const DeviceInfo* di) {
    Plan& p = e->p;
    if (e->kind == EPI_SPLIT) {
        p.s.grid = p.s.num_tiles * e->splits;
        p.s.xcds = di ? di->xcds : 8;
        e->sk = WorkspaceLayout{0, 0, 0};
        e->off_a = e->sums_bytes;
        e->off_b = e->off_a + e->a.packed_bytes;
        e->total = e->off_b + e->b.packed_bytes;
        return TS_OK;
    }
    int ppc = 0;
    if (di) ppc = occupancy_of(dev, epi_kernel_of(*e, ab), p.cfg == CFG_128 ? Cfg128::NT : Cfg256w8::NT);
    ts_status st = di ? resolve(&p, di->cu_count, ppc, di->xcds) : resolve_grid(&p, 0, 0, 8);
    if (st != TS_OK) return st;
    e->sk = workspace_layout(p);
    e->off_a = round_up(e->sk.total, 256);
    e->off_b = e->off_a + e->a.packed_bytes;
    e->total = e->off_b + e->b.packed_bytes;
    return TS_OK;
}

bool grid_needs_device(const EpiPlan& e) { return e.p.mode != TS_MODE_TILED && e.p.requested_programs == 0; }

ts_status check_epilogue(const ts_epilogue* x, const void* C, int64_t M, int64_t N, int32_t ab, int32_t c) {
    if (!x) return TS_OK;
    const int ce = c == TS_F32 ? 4 : 2;
    if (x->activation < TS_ACT_NONE || x->activation > TS_ACT_SILU || (x->grad != 0 && x->grad != 1))
        return TS_ERR_INVALID_ARG;
    if (x->bias && x->bias_dtype != TS_F16 && x->bias_dtype != TS_BF16 && x->bias_dtype != TS_F32)
        return TS_ERR_INVALID_ARG;
    if (x->grad && (!x->preact || x->bias || x->residual)) return TS_ERR_INVALID_ARG;
    if (!x->grad && x->preact && (x->preact == C || x->preact == x->residual)) return TS_ERR_INVALID_ARG;
    if ((x->scale_a || x->scale_b) && ab != TS_E4M3) return TS_ERR_INVALID_ARG;
    if (x->residual && M > 1 && x->stride_rm < N) return TS_ERR_INVALID_ARG;
    if (x->preact && M > 1 && x->stride_pm < N) return TS_ERR_INVALID_ARG;
    if ((uintptr_t)x->bias % (x->bias_dtype == TS_F32 ? 4 : 2) || (uintptr_t)x->residual % ce ||
        (uintptr_t)x->preact % ce || (uintptr_t)x->scale_a % 4 || (uintptr_t)x->scale_b % 4)
        return TS_ERR_ALIGNMENT;
    return TS_OK;
}

PackArgs::Matrix pack_of(const Operand& o, const void* src, int es, char* dst) {
    const int64_t chunks = round_up(o.cols * es, 16) / 16;
    const int64_t blocks = o.pack ? cdiv64(chunks * o.rows, kPackChunks) : 0;
    return PackArgs::Matrix{static_cast<const uint8_t*>(src), reinterpret_cast<uint8_t*>(dst), o.ld * es, o.cols * es,
                            std::max<int64_t>(chunks, 1), blocks, o.rows};
}

}  // namespace
}  // namespace ts

using namespace ts;

extern "C" int64_t ts_gemm_epilogue_workspace(const void* A, const void* B, int64_t M, int64_t N, int64_t K,
                                              int64_t stride_am, int64_t stride_ak, int64_t stride_bk,
                                              int64_t stride_bn, int32_t ab_dtype, int32_t c_dtype,
                                              const ts_schedule* sched) {
    EpiPlan e;
    ts_status st = epi_plan(A, B, M, N, K, stride_am, stride_ak, stride_bk, stride_bn, ab_dtype, c_dtype, sched, &e);
    if (st != TS_OK) return st;
    if (M == 0 || N == 0 || e.few) return 0;
    if (e.kind != EPI_STREAMK) return e.sums_bytes + e.a.packed_bytes + e.b.packed_bytes;
    int dev = 0;
    DeviceInfo di;
    const bool need = grid_needs_device(e);
    if (need) {
        st = current_device(&dev, &di);
        if (st != TS_OK) return st;
    }
    st = epi_resolve(&e, ab_dtype, dev, need ? &di : nullptr);
    return st != TS_OK ? st : e.total;
}

extern "C" ts_status ts_gemm_epilogue(const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K,
                                      int64_t stride_am, int64_t stride_ak, int64_t stride_bk, int64_t stride_bn,
                                      int64_t stride_cm, int64_t stride_cn, int32_t ab_dtype, int32_t c_dtype,
                                      const ts_epilogue* epi, const ts_schedule* sched, void* stream,
                                      void* workspace, int64_t workspace_bytes) {
    EpiPlan e;
    ts_status st = epi_plan(A, B, M, N, K, stride_am, stride_ak, stride_bk, stride_bn, ab_dtype, c_dtype, sched, &e);
    if (st != TS_OK) return st;
    st = check_epilogue(epi, C, M, N, ab_dtype, c_dtype);
    if (st != TS_OK) return st;
    if (workspace_bytes < 0) return TS_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return TS_OK;
    if (!C || (K > 0 && (!A || !B))) return TS_ERR_INVALID_ARG;
    if (N > 1 && stride_cn != 1) return TS_ERR_UNSUPPORTED;
    if (M <= 1) stride_cm = N;
    if (stride_cm < N) return TS_ERR_INVALID_ARG;
    if (M > 1 && (stride_cm > kMaxStride || (epi && ((epi->residual && epi->stride_rm > kMaxStride) ||
                                                     (epi->preact && epi->stride_pm > kMaxStride)))))
        return TS_ERR_UNSUPPORTED;
    const int ce = c_dtype == TS_F32 ? 4 : 2;
    if ((uintptr_t)A % e.es || (uintptr_t)B % e.es || (uintptr_t)C % ce) return TS_ERR_ALIGNMENT;
    if (epi && (!in_place_ok(C, epi->residual, true, M, stride_cm, epi->stride_rm) ||
                !in_place_ok(C, epi->preact, true, M, stride_cm, epi->stride_pm)))
        return TS_ERR_INVALID_ARG;

    const ts_epilogue plain = {};
    e.special = special_kind(epi ? *epi : plain, C, stride_cm, c_dtype);

    if (e.few) {
        int dev;
        DeviceInfo di;
        st = current_device(&dev, &di);
        if (st != TS_OK) return st;
        FewArgs f;
        memset(&f, 0, sizeof f);
        f.A = A;
        f.B = B;
        f.C = C;
        f.M = (int)M;
        f.N = (int)N;
        f.K = (int)K;
        f.lda = e.a.ld;
        f.ldb = e.b.ld;
        f.ldc = stride_cm;
        f.xcds = di.xcds;
        if (epi) {
            f.act = epi->activation;
            f.grad = epi->grad;
            f.bias = epi->bias;
            f.bias_type = epi->bias_dtype;
            f.aux_in = epi->grad ? epi->preact : epi->residual;
            f.ld_in = M > 1 ? (epi->grad ? epi->stride_pm : epi->stride_rm) : N;
            f.aux_out = epi->grad ? nullptr : epi->preact;
            f.ld_out = M > 1 ? epi->stride_pm : N;
            f.scale_a = epi->scale_a;
            f.scale_b = epi->scale_b;
        }
        return launch_few_rows(f, ab_dtype, c_dtype, e.b.kmaj, static_cast<hipStream_t>(stream)) ? TS_OK : TS_ERR_HIP;
    }

    auto workspace_ok = [&](int64_t need) {
        return need == 0 || (workspace && workspace_bytes >= need && (uintptr_t)workspace % 256 == 0);
    };
    if (e.kind != EPI_STREAMK && !workspace_ok(e.sums_bytes + e.a.packed_bytes + e.b.packed_bytes))
        return TS_ERR_INVALID_ARG;
    if (e.kind == EPI_STREAMK && !grid_needs_device(e)) {
        EpiPlan q = e;
        st = epi_resolve(&q, ab_dtype, 0, nullptr);
        if (st != TS_OK) return st;
        if (!workspace_ok(q.total)) return TS_ERR_INVALID_ARG;
    }
    int dev;
    DeviceInfo di;
    st = current_device(&dev, &di);
    if (st != TS_OK) return st;
    st = epi_resolve(&e, ab_dtype, dev, &di);
    if (st != TS_OK) return st;
    if (!workspace_ok(e.total)) return TS_ERR_INVALID_ARG;

    const hipStream_t hs = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    if (e.sk.total > 0) {
        int* flags = reinterpret_cast<int*>(ws);
        int words = (int)(e.sk.header / 4);
        void* argv[] = {&flags, &words};
        if (!enqueue(reinterpret_cast<const void*>(&clear_flags_kernel), (words + 255) / 256, 256, argv, hs)) return TS_ERR_HIP;
    }
    PackArgs pk = {{pack_of(e.a, A, e.es, ws + e.off_a), pack_of(e.b, B, e.es, ws + e.off_b)}};
    const int64_t pack_blocks = pk.m[0].blocks + pk.m[1].blocks;
    if (pack_blocks > 0) {
        void* argv[] = {&pk};
        if (!enqueue(reinterpret_cast<const void*>(&pack_rows_kernel), pack_blocks, 256, argv, hs)) return TS_ERR_HIP;
    }

    // Sizes along K count 16-bit units (pairs of 8-bit elements).
    const int unit = 2 / e.es;
    const int64_t kk = e.kp / unit;
    SplitArgs g;
    memset(&g, 0, sizeof g);
    auto pitch = [&](const Operand& o) {
        return (o.pack ? round_up(o.cols * e.es, 16) / e.es : o.ld) / unit;
    };
    g.A = reinterpret_cast<const uint16_t*>(e.a.pack ? ws + e.off_a : A);
    g.B = reinterpret_cast<const uint16_t*>(e.b.pack ? ws + e.off_b : B);
    g.C = C;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)kk;
    // a single row needs no pitch, but the loads of a tile's other rows (past the end,
    // reading zero) form their offsets with it
    g.lda = e.a.kmaj && e.a.rows <= 1 ? kk : pitch(e.a);
    g.ldb = e.b.kmaj && e.b.rows <= 1 ? kk : pitch(e.b);
    g.ldc = stride_cm;
    // bytes to the end of the last row, its padding included where it was packed (an odd row
    // length would cut the last element's dword)
    auto extent = [&](const Operand& o, int64_t ld) {
        const int64_t cols = (o.pack ? round_up(o.cols * e.es, 16) / e.es : o.cols) / unit;
        return K == 0 ? 0 : ((o.rows - 1) * ld + cols) * 2;
    };
    g.a_bytes = extent(e.a, g.lda);
    g.b_bytes = extent(e.b, g.ldb);
    g.s = e.p.s;
    if (e.sk.total > 0) {
        g.sk_flags = reinterpret_cast<int*>(ws);
        g.sk_err = reinterpret_cast<int*>(ws) + e.p.s.grid;
        g.sk_part = reinterpret_cast<float*>(ws + e.sk.header);
    }
    g.sk_spin = kSpin;
    if (epi) {
        g.act = epi->activation;
        g.grad = epi->grad;
        g.bias = epi->bias;
        g.bias_type = epi->bias_dtype;
        g.aux_in = epi->grad ? epi->preact : epi->residual;
        g.ld_in = M > 1 ? (epi->grad ? epi->stride_pm : epi->stride_rm) : N;
        g.aux_out = epi->grad ? nullptr : epi->preact;
        g.ld_out = M > 1 ? epi->stride_pm : N;
        g.scale_a = epi->scale_a;
        g.scale_b = epi->scale_b;
    }
    g.stagger = stagger_sleeps(e, g.aux_in != nullptr);
    const int threads = e.p.cfg == CFG_128 ? Cfg128::NT : Cfg256w8::NT;
    void* args[] = {&g};
    if (e.kind == EPI_SPLIT) {
        g.sums = reinterpret_cast<float*>(ws);
        g.ld_sums = (int64_t)e.p.s.nn * e.p.bn;
        g.split_stride = (int64_t)e.p.s.nm * e.p.bm * g.ld_sums;
        g.splits = e.splits;
    }
    if (!enqueue(epi_kernel_of(e, ab_dtype), e.p.s.grid, threads, args, hs) ||
        (e.kind == EPI_SPLIT && !launch_split_finish(g, c_dtype, hs)))
        return TS_ERR_HIP;
    return TS_OK;
}

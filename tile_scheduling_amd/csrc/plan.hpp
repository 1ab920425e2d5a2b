// Launch planning shared by the entry points of the tiled product: device properties,
// the order chosen from the locality model, the grid and the stream-K workspace.
#pragma once

#include <hip/hip_runtime.h>

#include <limits.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>
#include <vector>

#include "../../include/tsgemm.h"
#include "internal.hpp"

namespace ts {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
    int cu_count = 0;
    int xcds = 8;
};

inline std::once_flag g_dev_once[kMaxDevices];
inline DeviceInfo g_dev[kMaxDevices];

// Properties of the current device, queried once per device.
inline ts_status current_device(int* dev_out, DeviceInfo* info) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)hipGetLastError();
        return TS_ERR_NO_DEVICE;
    }
    std::call_once(g_dev_once[dev], [dev]() {
        int cus = 0, x = 0;
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) cus = 0;
        if (hipDeviceGetAttribute(&x, hipDeviceAttributeNumberOfXccs, dev) != hipSuccess || x < 1 || x > 64) x = 8;
        (void)hipGetLastError();
        g_dev[dev].cu_count = cus;
        g_dev[dev].xcds = x;
    });
    if (g_dev[dev].cu_count <= 0) return TS_ERR_NO_DEVICE;
    *dev_out = dev;
    *info = g_dev[dev];
    return TS_OK;
}

// Enqueues a kernel; false if that failed.  Judged by this launch alone: the runtime's last error may
// be one that another call of the program left.
inline bool enqueue(const void* fn, int64_t grid_x, int threads, void** args, hipStream_t stream, int64_t grid_y = 1) {
    if (hipLaunchKernel(fn, dim3((unsigned)grid_x, (unsigned)grid_y), dim3((unsigned)threads), args, 0, stream) == hipSuccess)
        return true;
    (void)hipGetLastError();   // reported by the caller's status
    return false;
}

struct Plan {
    bool auto_order;        // TS_ORDER_AUTO: order, G and remap chosen in resolve_grid
    int l2_reuse_pm;        // the locality model's reuse of the resolved order (1/1000)
    int cfg;                // CFG_*
    int bm, bn, bk;
    int io;                 // IO_*
    int mode;
    bool masked;            // the tiles do not cover M x N x K exactly, or rows defeat 16-byte access
    int path;               // PATH_*: which kernel runs a masked plan
    int vec_a, vec_b, vec_c;
    SchedArgs s;            // grid filled once the device is known (persistent auto)
    int requested_programs; // 0 = auto
    int64_t max_items;
};

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Locality model of a schedule: the first `concurrent` workgroups of the launch
// (the ones resident together; workgroup w runs on XCD w mod X) and the tiles they
// start on.  Each XCD's L2 serves the A row panels and B column panels its tiles
// share, so the cost is the number of distinct (XCD, tile row) plus (XCD, tile
// column) pairs; the reuse fraction is 1 - cost / (2 x tiles).
inline void locality_cost(const SchedArgs& s0, int concurrent, int64_t* cost, int64_t* tiles) {
    SchedArgs s = s0;
    s.fastdiv = 0;
    std::vector<int64_t> rows, cols;
    const int n = concurrent < s.grid ? concurrent : s.grid;
    for (int w = 0; w < n; ++w) {
        const int start = s.remap ? xcd_remap(w, s.grid, s.xcds) : w;
        if (start >= s.num_tiles) continue;
        int tm, tn;
        tile_coords(s, start, tm, tn);
        const int64_t x = w % s.xcds;
        rows.push_back((x << 32) | tm);
        cols.push_back((x << 32) | tn);
    }
    std::sort(rows.begin(), rows.end());
    std::sort(cols.begin(), cols.end());
    *tiles = (int64_t)rows.size();
    *cost = (int64_t)(std::unique(rows.begin(), rows.end()) - rows.begin()) +
            (int64_t)(std::unique(cols.begin(), cols.end()) - cols.begin());
}

// TS_ORDER_AUTO: the candidate of least locality cost, ties to the earlier one.
inline void choose_order(SchedArgs* s, int concurrent, int* reuse_pm) {
    struct Cand { int order, G, remap; };
    static const Cand kCands[] = {{ORDER_GROUPED, 8, 1},  {ORDER_GROUPED, 4, 1},  {ORDER_GROUPED, 16, 1},
                                  {ORDER_ROW_MAJOR, 1, 0}, {ORDER_ROW_MAJOR, 1, 1}, {ORDER_GROUPED, 8, 0},
                                  {ORDER_GROUPED, 4, 0},  {ORDER_GROUPED, 16, 0}, {ORDER_GROUPED, 2, 1},
                                  {ORDER_GROUPED, 32, 1}, {ORDER_GROUPED, 2, 0},  {ORDER_GROUPED, 32, 0}};
    int64_t best_cost = -1, best_tiles = 0;
    SchedArgs best = *s;
    for (const Cand& c : kCands) {
        if (c.order == ORDER_GROUPED && c.G > s->nm) continue;   // the same map as a smaller G
        SchedArgs t = *s;
        t.order = c.order;
        t.group_m = c.G;
        t.remap = c.remap;
        int64_t cost, tiles;
        locality_cost(t, concurrent, &cost, &tiles);
        if (best_cost < 0 || cost < best_cost) {
            best_cost = cost;
            best_tiles = tiles;
            best = t;
        }
    }
    *s = best;
    *reuse_pm = best_tiles > 0 ? (int)(1000 - (1000 * best_cost) / (2 * best_tiles)) : 0;
}

// Resolve the grid; cu/ppc of 0 mean "unknown" (host-only callers must pass
// num_programs explicitly in persistent modes).
inline ts_status resolve_grid(Plan* p, int cu_count, int ppc, int xcds) {
    p->s.xcds = xcds > 0 ? xcds : 8;
    if (p->s.num_tiles == 0) {
        p->s.grid = 0;
        p->max_items = 0;
        return TS_OK;
    }
    const int64_t ksp = p->s.ks > 0 ? p->s.ks : 1;
    if (p->mode == TS_MODE_TILED) {
        p->s.grid = p->s.num_tiles;
    } else {
        int64_t P = p->requested_programs;
        if (P == 0) {
            if (cu_count <= 0 || ppc <= 0) return TS_ERR_NO_DEVICE;
            P = (int64_t)cu_count * ppc;
        }
        // persistent: at most one program per tile; stream-K: per (tile, K step) item
        const int64_t cap = p->mode == TS_MODE_STREAMK ? (int64_t)p->s.num_tiles * ksp : p->s.num_tiles;
        p->s.grid = (int)(P < cap ? P : cap);
    }
    if (p->mode == TS_MODE_STREAMK) {
        const StreamK sk(p->s);
        p->max_items = cdiv64(sk.dp_tiles, p->s.grid) * ksp + sk.q + (sk.rem > 0 ? 1 : 0);
    } else {
        p->max_items = cdiv64(p->s.num_tiles, p->s.grid) * ksp;
    }
    // workgroups resident together: the device's CUs x workgroups per CU (256 CUs
    // and the plan's own grid when no device is known)
    const int64_t resident = (cu_count > 0 && ppc > 0) ? (int64_t)cu_count * ppc : 256;
    const int concurrent = (int)(resident < p->s.grid ? resident : p->s.grid);
    if (p->auto_order) {
        choose_order(&p->s, concurrent, &p->l2_reuse_pm);
    } else {
        int64_t cost, tiles;
        locality_cost(p->s, concurrent, &cost, &tiles);
        p->l2_reuse_pm = tiles > 0 ? (int)(1000 - (1000 * cost) / (2 * tiles)) : 0;
    }
    if (p->s.fastdiv) set_fastdiv(p->s);
    return TS_OK;
}

// Stream-K workspace of a resolved plan: a header of one flag per range plus an
// error counter (rounded up to 256 bytes), then one fp32 partial tile per range.
// Zero when the launch splits no tile.
struct WorkspaceLayout {
    int64_t header, part_bytes, total;
};
inline WorkspaceLayout workspace_layout(const Plan& p) {
    WorkspaceLayout w{0, 0, 0};
    if (p.mode != TS_MODE_STREAMK || p.s.grid == 0 || StreamK(p.s).sk_items == 0) return w;
    w.header = ((int64_t)(p.s.grid + 1) * 4 + 255) / 256 * 256;
    w.part_bytes = (int64_t)p.bm * p.bn * 4;
    w.total = w.header + (int64_t)p.s.grid * w.part_bytes;
    return w;
}

}  // namespace ts

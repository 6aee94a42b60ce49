// kv8_few_window.cu -- attention through a window of few query rows over the int8 cache.
#include "kv8_attend.cuh"
#include "kv8_more.h"

namespace bsg {

cudaError_t launch_few_window(const KvCall &a, const KvPlan &p, cudaStream_t st) {
    const int parts = a.dtype == BSG_F32 ? 2 : 1;
    const AttendPlan plan{parts, p.nt, (int)a.rows, p.row_tiles, p.width, p.splits};
    const AttendArgs args{a.c, a.table, a.table_ld, a.lens, a.q, a.out, a.dtype, a.tokens, a.heads, (int)a.rows,
                          p.row_tiles, p.width, p.splits, a.scale, a.lse, a.part_o, a.part_ml, a.dstatus, a.counts,
                          a.window, a.sinks, a.later};
    switch (a.c.dim) {
        case 32: return launch_attend_nt<32, kWindow>(args, plan, a.B, st);
        case 64: return launch_attend_nt<64, kWindow>(args, plan, a.B, st);
        case 96: return launch_attend_nt<96, kWindow>(args, plan, a.B, st);
        case 128: return launch_attend_nt<128, kWindow>(args, plan, a.B, st);
        default: return launch_attend_nt<256, kWindow>(args, plan, a.B, st);
    }
}

KvPlan kv_plan(const bsg_kv8_cache &c, bool few, int dtype, int64_t rows, int64_t B, int64_t positions, int64_t of_block,
               bool later) {
    KvPlan p = {};
    const int64_t groups = B * c.heads;
    if (few) {
        const AttendPlan a = attend_plan_of(c, (positions + 15) / 16, B, rows, dtype == BSG_F32 ? 2 : 1);
        p.splits = a.splits, p.nt = a.nt, p.row_tiles = a.row_tiles, p.width = a.width;
        // Where chunks fill the card, 256 positions at least to each, four tiles to each of its warps:
        // smaller ones leave little but their start and their part of the join (64 sequences of up to
        // 511 own tokens behind a prefix: 66 -> 60 us for all).
        const int64_t fill = (5 * (int64_t)device_sm_count() + groups - 1) / groups, most = (positions + 255) / 256;
        const int64_t cap = fill > most ? fill : most;
        if (p.splits > cap) p.splits = (int)cap;
    } else {
        // as many chunks as fill the card once, of two tiles at least
        const int64_t block = c.dim == 256 ? 128 : 256, tile = c.dim == 256 ? 64 : 128;
        p.row_blocks = (int)((rows + block - 1) / block);
        int64_t splits = device_sm_count() / (p.row_blocks * groups);
        if (splits > (positions + tile - 1) / tile / 2) splits = (positions + tile - 1) / tile / 2;
        p.splits = (int)(splits < 1 ? 1 : splits);
        p.tiles = (int)((of_block + tile * p.splits - 1) / (tile * p.splits));
    }
    p.parts = p.splits > 1 || later ? (size_t)groups * rows * p.splits : 0;
    return p;
}

}  // namespace bsg

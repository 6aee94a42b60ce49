// kv8_few_prefix.cu -- attention over a shared prefix of few query rows over the int8 cache.
#include "kv8_attend.cuh"
#include "kv8_more.h"

namespace bsg {

cudaError_t launch_few_prefix(const KvCall &a, const KvPlan &p, cudaStream_t st) {
    const int parts = a.dtype == BSG_F32 ? 2 : 1;
    const AttendPlan plan{parts, p.nt, (int)a.rows, p.row_tiles, p.width, p.splits};
    const AttendArgs args{a.c, a.table, a.table_ld, a.lens, a.q, a.out, a.dtype, a.tokens, a.heads, (int)a.rows,
                          p.row_tiles, p.width, p.splits, a.scale, a.lse, a.part_o, a.part_ml, a.dstatus, a.counts,
                          a.window, a.sinks, a.later};
    switch (a.c.dim) {
        case 32: return launch_attend_nt<32, kPrefix>(args, plan, a.B, st);
        case 64: return launch_attend_nt<64, kPrefix>(args, plan, a.B, st);
        case 96: return launch_attend_nt<96, kPrefix>(args, plan, a.B, st);
        case 128: return launch_attend_nt<128, kPrefix>(args, plan, a.B, st);
        default: return launch_attend_nt<256, kPrefix>(args, plan, a.B, st);
    }
}

}  // namespace bsg

// kv8_more.h -- what the translation units of windowed and shared-prefix attention share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bsg_internal.h"

namespace bsg {

// One launch of attention: of the sequences' own positions, or (B = 1, rows of all
// sequences) of the prefix's.
struct KvCall {
    const bsg_kv8_cache &c;
    const int32_t *table;
    int64_t table_ld;
    const int32_t *lens, *counts;
    const bsg_tokens &q, &out;
    int dtype, tokens, heads, window, sinks;
    int64_t B, rows;  // rows: of a key/value head and sequence
    float scale;
    float *lse;
    int later;        // what is found is joined with another launch's
    float *part_o;    // [sequence][head][row][chunk][dim]: outputs before the division by the sum,
    float2 *part_ml;  // and the reference (log 2) and sum (0: nothing seen)
    int32_t *dstatus;
};

// How it is cut: chunks of a row's positions, and the partial outputs that they leave.
struct KvPlan {
    int splits;
    size_t parts;
    int row_blocks, tiles;     // of the tiles' kernel (TileArgs), and the tiles of a chunk at most
    int nt, row_tiles, width;  // of the kernel of few rows
};
// positions: that the rows of a head and sequence see at most; of_block: those that some rows of one CTA see.
KvPlan kv_plan(const bsg_kv8_cache &c, bool few, int dtype, int64_t rows, int64_t B, int64_t positions, int64_t of_block,
               bool later);

cudaError_t launch_few_window(const KvCall &a, const KvPlan &p, cudaStream_t st);
cudaError_t launch_few_prefix(const KvCall &a, const KvPlan &p, cudaStream_t st);
cudaError_t launch_tiles_window(const KvCall &a, const KvPlan &p, cudaStream_t st);
cudaError_t launch_tiles_prefix(const KvCall &a, const KvPlan &p, cudaStream_t st);

}  // namespace bsg

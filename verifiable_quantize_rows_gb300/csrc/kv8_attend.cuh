// kv8_attend.cuh -- attention of few query rows over the int8 cache: the kernel of
// kv8.cu's calls, of windows (kv8_few_window.cu) and of shared prefixes (kv8_few_prefix.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bsg_internal.h"
#include "bsg_ptx.cuh"
#include "kv8_seen.cuh"
#include "serve.cuh"

namespace bsg {
namespace {

// ---- attention ----------------------------------------------------------------
//
// out = sum_j p_j v_j over one sequence and key/value head, for the rows (query
// tokens x query heads) that share it.  The work is reading 2 len dim bytes of
// codes once; a CTA takes a chunk of the positions, its warps every kWarps-th
// tile of 16 positions each, and all is joined at the end.  Per tile and warp:
//
//   S^T (16 positions x 8 slots) = K (16 x dim) . Q^T      mma m16n8k16, f32 sums
//   p' = 2^(S' - ref),  S' = S * key scale * softmax scale * log2 e + log2(value scale)
//   O^T (dim x 8 slots) += V^T (dim x 16) . P'^T (16 x 8 slots),  l += p' / value scale
//
// The value scale rides in the exponent, so the second product adds up in the
// tensor cores' own accumulators; `ref` is then 2^-11 of a maximum of p v's size.  Value
// scales below 1e-30 count as 1e-30.
//
// Each warp copies its own tiles ahead into a ring of shared memory (cp.async,
// kStages tiles of 32 dim bytes) and takes them from there to the tensor cores
// as they lie: a lane's 16 bytes of a row serve as the A operand's rows and
// columns in whatever order they come, because the order of the summed index
// and of dim are free as long as Q and the output follow it.
// An int8 code q becomes the f16 q exactly: the byte q + 128 placed under the
// exponent of 1024, less 1152.  m16n8k16 and not tcgen05: up to 16 rows are
// 64 operations to a byte at most, and what bounds the kernel is HBM.
//
// A slot is one column of the 8: a row, or (kParts = 2, f32) one of a row's two
// f16 parts hi + 2^-11 lo.  Queries are taken relative to their largest |q|
// (a power of two), so two parts keep 2^-22 of it.  16-bit types have one part: their
// queries are exact in it, down to 2^-38 of the row's largest.
//
// A p' goes to the second product as two f16 parts for every type, f32's as a slot
// each, 16-bit types' as p' = hi + lo in one accumulator, by a second multiplication with
// the same codes.  hi + lo leaves out 2^-24 of p' at most, or 2^-25 where that is more (the
// least f16 step is 2^-24), 2^-36 of the largest.  (By hi alone, as an output in 16 bits
// might seem to allow, a sum of many positions that cancel is off by more than its own
// rounding: f16 outputs 2.9e-4 off 64 bits in place of 2.1e-4; and below 2^-14 of the
// largest p' a position lost bit after bit.)
//
// The running reference `ref` is 2^-11 of a row's maximum, and follows it only when that
// is more than 2^4 above: a p' stays below 2^15, which f16 holds, the largest is at
// least 2^11, and the outputs are rescaled a few times per row instead of at every tile.

// The tensor cores cut off what they add to an f32 sum, always towards 0 (some 2^-24 of it with each
// product), and a plain sum of many equal terms rounds the same way each time.  So a warp's outputs
// and sums are added, rounded, to a second set every kAnew tiles of its chunk and begun anew.  That
// set lies in local memory, beside a pass over the outputs that a moved reference takes as well.
// Off 64 bits with equal scores and values of one sign, 512 sequences of 131072 positions, one chunk
// each: f32 2.0e-4 (mean) without, 7e-7 with, 2.6e-6 every 64 tiles, 3.5e-7 every 16; f16, 2^20
// positions, 9.0e-4 and 2e-5 (128 tiles).  It takes a kernel of its own, for chunks that may have more
// tiles to a warp: 512 sequences of 8192, 8 heads of 128, f32 1272 us without, 1400 with (1335 every
// 64 tiles); 256 of 32768 and 64 dims, bf16 1286 and 1410.
// (More chunks instead of it cost less where tables are full, but where they have room for 131072 and
// hold 4096 a call of 256 sequences took 675 us; 341 without either, 361 with this.)

// The positions are cut into chunks, a CTA each, several for each place on the
// card, so that the hardware's own scheduling evens out what SMs and lengths
// differ by.  (Equal shares of all tiles for just the resident CTAs were slower,
// 143 against 135 us at two sequences of 131071 and 262143 and 113 against 93 at
// 64 ragged ones: SMs do not read at the same rate.  Chunks of one size were too,
// by up to 10 % where their waves came out badly.)
// A chunk that is its whole sequence is finished in place; otherwise a second launch
// joins the chunks.  (As a cluster that joins its chunks itself, one launch: 7.1 against
// 6.2 us at 12 heads and 1021 positions, 13.4 against 10.2 at 8 heads and 4000.)
//
// Measured: 64 ragged sequences of up to 8190, 8 heads of 128 (538 MB) 94 us, 0.84 of the
// floor's rate; two of up to 262143 with 4 query tokens 164 us, 0.73; 1001 positions of
// 12 heads of 64 6.4 us.  What bounds it: HBM with few rows; with 16 and more the tensor
// cores beside the unpacking (probabilities in one part, whose outputs were not good to
// their last bit: 146 us, and 92 with one query token); the short ones their two launches.
// Through windows of 4096, 64 sequences of one token (407 MB) 96 us, 0.80.

constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kMaxSplits = 1024;
constexpr float kRefNone = -3.0e38f;  // the reference of a row that has seen nothing
// Tiles of a warp to one sum.  f32: 32 products, 2^-20 or so; 16 bits: 256, 2^-16, where f16's own rounding is 2^-11.
template <int kParts>
constexpr int kAnew = kParts == 2 ? 32 : 128;
constexpr float kTop = 11.0f, kMost = 15.0f;  // exponents of a new reference's largest p', and of any

// 16 bytes from global to shared memory, asynchronously, past L1.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the newest N groups are done
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D += A B, A 16 x 16 f16 (row), B 16 x 8 f16 (column), D f32.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 f16 matrix held two elements to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) { return bits(__floats2half2_rn(lo, hi)); }

// Two codes, already + 128 (unsigned bytes `sel` picks of x), as f16.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_half2(uint32_t x) {
    const uint32_t m = __byte_perm(x, 0x64646464u, SEL);
    const uint32_t bias = 0x64806480u;  // 1152, 1152
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&m),
                              *reinterpret_cast<const __half2 *>(&bias));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Which dim the lane's word `w` of a value row starts at (g = lane / 4): 16-byte pieces of 128
// bytes, then smaller ones.  (A key row's, t = lane % 4: of 64 bytes, load_key_row's.)
template <int D>
__host__ __device__ constexpr int value_dim(int w, int g) {
    return D >= 128  ? w / 4 * 128 + 16 * g + w % 4 * 4
           : D == 96 ? (w < 2 ? 8 * g + 4 * w : 64 + 4 * g)
                     : (D / 8) * g + 4 * w;
}

// Where byte `col` (the start of a lane's piece) of row `r` of a tile lies in
// shared memory.  Rows of 128 bytes or more would put the rows that one
// instruction reads on the same banks; their 16-byte pieces are permuted by
// the row so that both products read without conflicts.
template <int D>
__device__ __forceinline__ int tile_at(int r, int col) {
    if (D < 128) return r * D + col;
    return r * D + (col ^ ((((r >> 1 & 3) << 1) ^ ((r & 1) << 2)) << 4));
}

template <int D>
__device__ __forceinline__ void load_key_row(uint32_t (&w)[D / 16], const uint8_t *tile, int r,
                                             int t) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        const uint4 v = *reinterpret_cast<const uint4 *>(tile + tile_at<D>(r, 64 * c + 16 * t));
        w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
    }
    if (D % 64) {
        const uint2 v =
            *reinterpret_cast<const uint2 *>(tile + tile_at<D>(r, D / 64 * 64 + 8 * t));
        w[D / 16 - 2] = v.x, w[D / 16 - 1] = v.y;
    }
}

template <int D>
__device__ __forceinline__ void load_value_row(uint32_t (&w)[D / 32], const uint8_t *tile, int r,
                                               int g) {
    if constexpr (D >= 128) {
#pragma unroll
        for (int c = 0; c < D / 128; ++c) {
            const uint4 v =
                *reinterpret_cast<const uint4 *>(tile + tile_at<D>(r, 128 * c + 16 * g));
            w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
        }
    } else if constexpr (D >= 64) {
        const uint2 v = *reinterpret_cast<const uint2 *>(tile + tile_at<D>(r, 8 * g));
        w[0] = v.x, w[1] = v.y;
        if constexpr (D == 96)
            w[2] = *reinterpret_cast<const uint32_t *>(tile + tile_at<D>(r, 64 + 4 * g));
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(tile + tile_at<D>(r, 4 * g));
    }
}

struct AttendArgs {
    bsg_kv8_cache c;
    const int32_t *table;
    int64_t table_ld;
    const int32_t *lens;
    bsg_tokens q, out;
    int dtype, tokens, heads, rows, row_tiles;
    int width, splits;  // tiles of a table's width, and the chunks it is cut into
    float scale;
    float *lse;
    float *part_o;    // [sequence][head][row][split][D]: the chunks' outputs
    float2 *part_ml;  // their reference and sum
    int32_t *dstatus;
    const int32_t *counts;  // kWindow
    int window, sinks, later;  // later: kWindow leaves partial outputs, one chunk or not
};

// What the rows see.  kWhole: their sequence up to their own position, finished where it is one
// chunk.  kWindow: a window with sinks; the chunks cut the tiles that some row of the CTA sees.
// kPrefix: the rows of all sequences (as one), which see the positions below *lens.  But for
// kWhole, what a CTA finds is joined later where there are chunks, or always (kPrefix, later); a
// chunk that saw nothing leaves a sum of 0.
enum AttendMode : int { kWhole = 0, kWindow = 1, kPrefix = 2 };

__device__ __forceinline__ void store_any(void *p, int64_t i, int dtype, float x) {
    if (dtype == BSG_F32)
        static_cast<float *>(p)[i] = x;
    else if (dtype == BSG_F16)
        static_cast<__half *>(p)[i] = __float2half_rn(x);
    else
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}

// Row r of a key/value head's rows: its query token and query head.
struct RowAt {
    int token, head;
};
__device__ __forceinline__ RowAt row_at(const AttendArgs &a, int hk, int r) {
    const int share = a.heads / a.c.heads;
    return {r / share, hk * share + r % share};
}

// The cached length of sequence b, cut to the table's.
__device__ __forceinline__ int length_of(const AttendArgs &a, int b, bool report) {
    const int len = __ldg(a.lens + b);
    const int64_t most = a.table_ld * a.c.page_tokens;
    if (len >= 0 && len <= most) return len;
    if (report) set_status(a.dstatus, BSG_DSTATUS_RANGE);
    return len < 0 ? 0 : (int)most;
}

// One row's result: o = sum / l (0 where nothing was seen) and lse.
__device__ __forceinline__ void store_row(const AttendArgs &a, int b, int hk, int r, int d, float o,
                                          float m, float l) {
    const RowAt at = row_at(a, hk, r);
    store_any(a.out.data,
              b * a.out.stride_batch + at.token * a.out.stride_token +
                  at.head * a.out.stride_head + d,
              a.dtype, l > 0.0f || l != l ? o / l : 0.0f);
    if (d == 0 && a.lse)
        a.lse[((int64_t)b * a.tokens + at.token) * a.heads + at.head] =
            l > 0.0f || l != l ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// Floats of a row of partial outputs: its dims, then its sum.
template <int D>
__host__ __device__ constexpr int pitch() { return D + 4; }

// Shared memory: the queries, then the warps' rings, whose place the warps'
// outputs take at the end.
template <int D, int NT, int kParts>
constexpr int attend_smem() {
    constexpr int rings = kWarps * kStages * 32 * D;
    constexpr int join = kWarps * (8 * NT / kParts) * pitch<D>() * 4;
    return NT * (D / 16) * 32 * 8 + (rings > join ? rings : join);
}

// CTAs on an SM: what registers and shared memory allow.
template <int D, int NT>
constexpr int attend_per_sm() {
    return D == 32    ? (NT == 1 ? 7 : NT == 2 ? 5 : 3)
           : D == 64  ? (NT == 1 ? 5 : NT == 2 ? 4 : 3)
           : D == 96  ? (NT == 1 ? 5 : NT == 2 ? 4 : 2)
           : D == 128 ? (NT == 1 ? 4 : NT == 2 ? 3 : 2)
                      : 2;
}

// Where chunk i begins: chunks shrink from 1.6 to 0.4 of their mean, so that
// those that start together do not end together, and the last are small.
__device__ __forceinline__ int chunk_begin(const AttendArgs &a, int i) {
    const int64_t n = a.splits, part = (16 * n - 6 * i) * i;  // of 10 n^2
    return i >= n ? a.width : (int)(part * (a.width / kWarps) / (10 * n * n)) * kWarps;
}

// grid (heads x row tiles, B, splits): the first chunks of all first
template <int D, int NT, int kParts, int kMode, bool kLong>
__global__ void __launch_bounds__(kWarps * 32, attend_per_sm<D, NT>())
    kv8_attend_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int kRows = 8 * NT / kParts;  // rows of a group
    constexpr int kPitch = pitch<D>();
    constexpr int kStep = D / 16;           // k16 steps of q.k, m16 tiles of the output
    extern __shared__ __align__(16) uint8_t smem[];
    uint2 *q_s = reinterpret_cast<uint2 *>(smem);                   // [NT][kStep][32 lanes]
    uint8_t *ring_s = smem + NT * kStep * 32 * 8;                   // [warp][stage][K, V tile]
    float *o_s = reinterpret_cast<float *>(ring_s);                 // [warp][row][kPitch]: l at D
    __shared__ float4 scales_s[kWarps][kStages];                    // of a stage's tile; w: 1 if there
    __shared__ float mul_s[kRows];                                  // score multiplier of each row
    __shared__ float max_s[kRows][kWarps];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
    const int P = a.c.page_tokens;
    const int b = blockIdx.y, hk = blockIdx.x / a.row_tiles, r0 = blockIdx.x % a.row_tiles * kRows;
    const int split = blockIdx.z;
    int rows = min(kRows, a.rows - r0);
    griddep_launch_dependents();

    // Tiles [tile0, tiles) of what the rows see; kWhole: the pages of the warp's first 32 of
    // them are looked up, one to a lane, before the length is known.
    const int32_t *table = a.table + b * a.table_ld;
    const int tile0 = chunk_begin(a, split), tile1 = chunk_begin(a, split + 1);
    int next = tile0 + warp, in_batch = 0;
    int64_t slot = (int64_t)(next + lane * kWarps) * 16 / P;
    int my_page = kMode == kWhole && slot < a.table_ld ? __ldg(table + slot) : -1;
    const int len = length_of(a, b, blockIdx.x == 0 && split == 0 && tid == 0);
    const int share = a.heads / a.c.heads;
    int count = a.tokens, pos0 = len - a.tokens;  // of the sequence's tokens; token 0's position
    Seen seen = {};
    if constexpr (kMode == kWindow) {
        if (a.counts) {
            count = __ldg(a.counts + b);
            if (count < 0 || count > a.tokens) {
                if (blockIdx.x == 0 && split == 0 && tid == 0) set_status(a.dstatus, BSG_DSTATUS_RANGE);
                count = 0;
            }
            rows = min(rows, count * share - r0);
            if (rows <= 0) return;
            pos0 = len - count;
        }
        seen = seen_by<16>(pos0 + r0 / share, pos0 + (r0 + rows - 1) / share, a.window, a.sinks);
    }
    const int all = kMode == kWindow ? seen.tiles : (len + 15) / 16;
    const int tiles = min(all, tile1);
    auto real = [&](int tile) { return kMode == kWindow ? seen.tile(tile) : tile; };  // where it lies in the sequence
    auto part_at = [&](int r) { return (((int64_t)b * a.c.heads + hk) * a.rows + r0 + r) * a.splits + split; };
    if (tile0 >= all && (kMode != kWhole || split > 0)) {  // kWhole: the join knows that it has no part
        if (kMode == kPrefix || (kMode == kWindow && (a.splits > 1 || a.later))) {
            if (tid < rows) a.part_ml[part_at(tid)] = make_float2(0.0f, 0.0f);
            return;
        }
        if (split > 0) return;
    }
    if (kMode != kWhole && next + lane * kWarps < tiles) my_page = __ldg(table + (int64_t)real(next + lane * kWarps) * 16 / P);

    // The queries' loads go first, all of them together.
    constexpr int kMine = (kRows + kWarps - 1) / kWarps;  // rows of a warp
    float q[kMine][D / 32];
    auto load_queries = [&](auto type) {
        using T = decltype(type);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int r = warp + i * kWarps;
            const RowAt at = row_at(a, hk, r0 + r);
            const int64_t of = kMode == kPrefix ? at.token / a.tokens * a.q.stride_batch + at.token % a.tokens * a.q.stride_token
                                                : b * a.q.stride_batch + at.token * a.q.stride_token;
            const T *row = static_cast<const T *>(a.q.data) + of + at.head * a.q.stride_head + lane;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) q[i][j] = r < rows ? to_f32(row[32 * j]) : 0.0f;
        }
    };
    if (kParts == 2)
        load_queries(float{});
    else if (a.dtype == BSG_F16)
        load_queries(__half{});
    else
        load_queries(__nv_bfloat16{});

    // The warp's tiles are fetched kStages ahead: where its next 32 lie in the
    // pool (in tiles; -1: nowhere) and their scales, one to a lane.
    uint8_t *ring = ring_s + warp * kStages * 32 * D;
    const int8_t *k_lane = a.c.k + lane * 16, *v_lane = a.c.v + lane * 16;
    int my_at;
    float4 my_scales;
    auto look_up = [&]() {
        const int tile = next + lane * kWarps;
        my_at = -1;
        my_scales = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (tile >= tiles) return;
        if (my_page < 0 || my_page >= a.c.pages) {
            set_status(a.dstatus, BSG_DSTATUS_RANGE);
            return;
        }
        const int64_t ph = (int64_t)my_page * a.c.heads + hk;
        my_at = (int)(ph * (P / 16) + real(tile) % (P / 16));
        const float vs = fmaxf(a.c.v_scale[ph], 1e-30f);
        my_scales = make_float4(a.c.k_scale[ph], log2f(vs), __frcp_rn(vs), 1.0f);
    };
    look_up();
    // A group of copies each time, so that they count; no copies past the last
    // tile, or where its page is none.
    auto fetch = [&](int stage) {
        if (in_batch == 32) {
            in_batch = 0;
            const int tile = next + lane * kWarps;
            if (tile < tiles) my_page = __ldg(table + (int64_t)real(tile) * 16 / P);
            look_up();
        }
        const int at = __shfl_sync(0xffffffffu, my_at, in_batch);
        if (lane == in_batch) scales_s[warp][stage] = my_scales;
        if (at >= 0) {
            const int8_t *k = k_lane + (int64_t)at * (16 * D), *v = v_lane + (int64_t)at * (16 * D);
            const uint32_t dst = smem_u32(ring + stage * 32 * D);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int e = (i * 32 + lane) * 16;
                copy16(dst + tile_at<D>(e / D, e % D), k + i * 512);
                copy16(dst + 16 * D + tile_at<D>(e / D, e % D), v + i * 512);
            }
        }
        copies_commit();
        ++in_batch;
        next += kWarps;
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(i);
    int stage = 0;

    // Queries: each row relative to a power of two near its largest |q|, in
    // f16 parts, laid out as the B operand.
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int r = warp + i * kWarps;
        if (r >= kRows) break;
        float m = 0.0f;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            bad |= !isfinite(q[i][j]);
            m = fmaxf(m, fabsf(q[i][j]));
        }
        if (bad) set_status(a.dstatus, BSG_DSTATUS_NONFINITE);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        // 2^e with m 2^e in [2^13, 2^14); e <= 126 leaves subnormal rows their small error
        const int e = min(126, 13 + 127 - (int)(__float_as_uint(m) >> 23));
        const float up = __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
        if (lane == 0)
            mul_s[r] = a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 - max(e, -126)) << 23);
        __half *qh = reinterpret_cast<__half *>(q_s);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const int d = lane + 32 * j;
            // the step and lane whose word covers dim d
            int w, tt;
            if (d < D / 64 * 64)
                w = d / 64 * 4 + d % 16 / 4, tt = d % 64 / 16;
            else
                w = D / 64 * 4 + d % 8 / 4, tt = d % 32 / 8;
            const float y = q[i][j] * up;
            const __half hi = __float2half_rn(y);
            const int slot = r * kParts;
            const int word = ((slot / 8 * kStep + w) * 32 + slot % 8 * 4 + tt) * 4 + d % 4;
            qh[word] = hi;
            if (kParts == 2) qh[word + 16] = __float2half_rn((y - __half2float(hi)) * 2048.0f);
        }
    }
    __syncthreads();

    // The lane's columns: slots 2t, 2t + 1 of each 8.
    float mul[NT][2], ref[NT][2], sum[NT][2];
    int see[NT][2], low[NT][2];
    float acc[NT][kStep][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = (8 * n + 2 * t + u) / kParts;
            mul[n][u] = mul_s[r];
            ref[n][u] = 0.0f;
            sum[n][u] = 0.0f;
            see[n][u] = r >= rows ? 0 : kMode == kPrefix ? len : pos0 + row_at(a, hk, r0 + r).token + 1;
            low[n][u] = kMode == kWindow && a.window && see[n][u] > a.window ? see[n][u] - a.window : 0;
        }
#pragma unroll
        for (int i = 0; i < kStep; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[n][i][u] = 0.0f;
    }

    // kWindow: what every row of the CTA sees.
    const int all_see = pos0 + r0 / share + 1, last_pos = pos0 + (r0 + rows - 1) / share;
    const int all_low = a.window && last_pos >= a.window ? last_pos - a.window + 1 : 0;

    // Rows that have seen nothing yet (bit 2n + u; their ref is 0): only before
    // the warp's first tile, or where that is one some row may not see (kWindow: or some tiles on).
    uint32_t none = 0xffffffffu, live = 0;  // live: rows that see something at all
    if (kMode == kWindow)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int u = 0; u < 2; u += kParts) live |= see[n][u] > 0 ? 1u << (2 * n + u) : 0u;
    bool fresh = true;
    int due = kAnew<kParts>;  // the warp's tile before which its sums are begun anew (or the next that is there)
    // kLong: what was added up before the sums were begun anew, relative to the references then (a
    // row that had seen nothing: -inf, no part of it).
    alignas(16) float kept[NT][kStep][4];
    volatile float kept_sum[NT][2], kept_ref[NT][2];
    auto with_kept = [&](bool some, bool keep) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f[2];
#pragma unroll
            for (int u = 0; u < 2; u += kParts) {
                f[u] = some ? exp2_fast(kept_ref[n][u] - ref[n][u]) : 0.0f;
                if (some) sum[n][u] = fmaf(kept_sum[n][u], f[u], sum[n][u]);
                if (keep) {
                    kept_sum[n][u] = sum[n][u];
                    sum[n][u] = 0.0f;
                    kept_ref[n][u] = none & (1u << (2 * n + u)) ? -INFINITY : ref[n][u];
                }
            }
            if (kParts == 2) f[1] = f[0];
            constexpr int kBatch = kStep % 4 ? 2 : 4;  // loads sent together
#pragma unroll
            for (int i0 = 0; i0 < kStep; i0 += kBatch) {
                float before[kBatch][4];
                if (some)
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        asm volatile("ld.local.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(before[i][0]), "=f"(before[i][1]), "=f"(before[i][2]), "=f"(before[i][3])
                                     : "l"(__cvta_generic_to_local(kept[n][i0 + i])) : "memory");
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    float(&o)[4] = acc[n][i0 + i];
                    if (some)
#pragma unroll
                        for (int u = 0; u < 4; ++u) o[u] = fmaf(before[i][u], f[u % 2], o[u]);
                    if (keep) {
                        asm volatile("st.local.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(__cvta_generic_to_local(kept[n][i0 + i])),
                                     "f"(o[0]), "f"(o[1]), "f"(o[2]), "f"(o[3]) : "memory");
#pragma unroll
                        for (int u = 0; u < 4; ++u) o[u] = 0.0f;
                    }
                }
            }
        }
    };
    for (int tile = tile0 + warp; tile < tiles; tile += kWarps) {
        copies_wait<kStages - 1>();
        __syncwarp();
        const uint8_t *kt = ring + stage * 32 * D, *vt = kt + 16 * D;
        const float4 of_tile = scales_s[warp][stage];
        if (of_tile.w == 0.0f) {
            __syncwarp();
            fetch(stage);
            stage = stage + 1 == kStages ? 0 : stage + 1;
            continue;
        }
        uint32_t kr[2][D / 16];
        load_key_row<D>(kr[0], kt, g, t);
        load_key_row<D>(kr[1], kt, g + 8, t);
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int u = 0; u < 4; ++u) s[n][u] = 0.0f;
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            const uint32_t x0 = kr[0][i] ^ 0x80808080u, x1 = kr[1][i] ^ 0x80808080u;
            const uint32_t a0 = codes_half2<0x4140>(x0), a1 = codes_half2<0x4140>(x1);
            const uint32_t a2 = codes_half2<0x4342>(x0), a3 = codes_half2<0x4342>(x1);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint2 q = q_s[(n * kStep + i) * 32 + lane];
                mma_16816(s[n], a0, a1, a2, a3, q.x, q.y);
            }
        }

        // Exponents relative to the reference; kParts = 2: one row's in x[n][0]
        // and x[n][2].
        float x[NT][4], most = -INFINITY;
        const int at = real(tile) * 16;
        // some row may not see all of it
        const bool edge = kMode == kPrefix   ? at + 16 > len
                          : kMode == kWindow ? at + 16 > all_see || (at < all_low && at + 16 > a.sinks)
                                             : at + 16 > len - a.tokens;
        auto exponents = [&]() {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int u = 0; u < 4; u += kParts) {
                    const float score = kParts == 2 ? fmaf(s[n][u + 1], 0x1p-11f, s[n][u]) : s[n][u];
                    x[n][u] = fmaf(score, of_tile.x * mul[n][u % 2], of_tile.y - ref[n][u % 2]);
                    const int j = at + g + u / 2 * 8;
                    if (edge && (j >= see[n][u % 2] || (kMode == kWindow && j < low[n][u % 2] && j >= a.sinks)))
                        x[n][u] = -INFINITY;
                    most = fmaxf(most, x[n][u]);
                }
        };
        exponents();
        const bool anew = kLong && (tile - tile0) / kWarps >= due;
        if (__any_sync(0xffffffffu, most > kMost || fresh || edge || anew)) {
            if (kMode != kWindow) fresh = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float keep[2];
#pragma unroll
                for (int u = 0; u < 2; u += kParts) {
                    float m = fmaxf(x[n][u], x[n][u + 2]);
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    keep[u] = 1.0f;
                    // each row by itself: no other row's values move its reference
                    const uint32_t bit = 1u << (2 * n + u);
                    if (none & bit ? m > -INFINITY : m > kMost) {
                        ref[n][u] += m - kTop;
                        keep[u] = none & bit ? 0.0f : exp2_fast(kTop - m);
                        sum[n][u] *= keep[u];
                        none &= ~bit;
                    }
                }
                if (kParts == 2) keep[1] = keep[0];
#pragma unroll
                for (int i = 0; i < kStep; ++i)
#pragma unroll
                    for (int u = 0; u < 4; ++u) acc[n][i][u] *= keep[u % 2];
            }
            if constexpr (kLong)
                if (anew) {
                    with_kept(due > kAnew<kParts>, true);
                    due = (tile - tile0) / kWarps + kAnew<kParts>;
                }
            // a row whose window begins after this tile sees its first one later
            if (kMode == kWindow) fresh = __any_sync(0xffffffffu, (none & live) != 0);
            exponents();
        }
        // Probabilities, as the B operand of the second product.
        uint32_t p01[NT], p89[NT], lo01[NT], lo89[NT];  // lo: of 16-bit types
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (kParts == 2) {
                const float pa = exp2_fast(x[n][0]), pb = exp2_fast(x[n][2]);
                sum[n][0] = fmaf(pa + pb, of_tile.z, sum[n][0]);
                const float ha = __half2float(__float2half_rn(pa));
                const float hb = __half2float(__float2half_rn(pb));
                p01[n] = transpose8(pack_half2(ha, (pa - ha) * 2048.0f));
                p89[n] = transpose8(pack_half2(hb, (pb - hb) * 2048.0f));
            } else {
                float p[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) p[u] = exp2_fast(x[n][u]);
                sum[n][0] = fmaf(p[0] + p[2], of_tile.z, sum[n][0]);
                sum[n][1] = fmaf(p[1] + p[3], of_tile.z, sum[n][1]);
                const __half2 h01 = __floats2half2_rn(p[0], p[1]), h89 = __floats2half2_rn(p[2], p[3]);
                const float2 f01 = __half22float2(h01), f89 = __half22float2(h89);
                p01[n] = transpose8(bits(h01));
                p89[n] = transpose8(bits(h89));
                lo01[n] = transpose8(pack_half2(p[0] - f01.x, p[1] - f01.y));
                lo89[n] = transpose8(pack_half2(p[2] - f89.x, p[3] - f89.y));
            }
        }
        uint32_t vr[4][D / 32];
        load_value_row<D>(vr[0], vt, 2 * t, g);
        load_value_row<D>(vr[1], vt, 2 * t + 1, g);
        load_value_row<D>(vr[2], vt, 2 * t + 8, g);
        load_value_row<D>(vr[3], vt, 2 * t + 9, g);
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            const uint32_t x0 = vr[0][w] ^ 0x80808080u, x1 = vr[1][w] ^ 0x80808080u;
            const uint32_t x2 = vr[2][w] ^ 0x80808080u, x3 = vr[3][w] ^ 0x80808080u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // two dims of positions 2t, 2t + 1, and of 2t + 8, 2t + 9
                const uint32_t lo = __byte_perm(x0, x1, h ? 0x7362 : 0x5140);
                const uint32_t hi = __byte_perm(x2, x3, h ? 0x7362 : 0x5140);
                const uint32_t a0 = codes_half2<0x4140>(lo), a1 = codes_half2<0x4342>(lo);
                const uint32_t a2 = codes_half2<0x4140>(hi), a3 = codes_half2<0x4342>(hi);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma_16816(acc[n][2 * w + h], a0, a1, a2, a3, p01[n], p89[n]);
                if (kParts == 1)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_16816(acc[n][2 * w + h], a0, a1, a2, a3, lo01[n], lo89[n]);
            }
        }
        __syncwarp();  // every lane has read the stage
        fetch(stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    if constexpr (kLong)
        if (due > kAnew<kParts>) with_kept(true, false);
    copies_wait<0>();
    __syncthreads();  // the rings are free

    // Join the warps: sums over the lanes of a column, then over the warps,
    // each relative to the largest reference.
    float *mine = o_s + warp * kRows * kPitch;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int u = 0; u < 2; u += kParts) {
            float l = sum[n][u];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int r = (8 * n + 2 * t + u) / kParts;
            if (g == 0) {
                mine[r * kPitch + D] = l;
                max_s[r][warp] = none & (1u << (2 * n + u)) ? kRefNone : ref[n][u];
            }
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                const int d = value_dim<D>(i / 2, g) + i % 2 * 2;
                float2 o;
                if (kParts == 2)
                    o = make_float2(fmaf(acc[n][i][1], 0x1p-11f, acc[n][i][0]),
                                    fmaf(acc[n][i][3], 0x1p-11f, acc[n][i][2]));
                else
                    o = make_float2(acc[n][i][u], acc[n][i][u + 2]);
                *reinterpret_cast<float2 *>(mine + r * kPitch + d) = o;
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < rows * (D / 4); e += kWarps * 32) {
        const int r = e / (D / 4), d = e % (D / 4) * 4;
        float m = max_s[r][0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = fmaxf(m, max_s[r][w]);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float l = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2_fast(max_s[r][w] - m);
            const float *p = o_s + (w * kRows + r) * kPitch;
            const float4 v = *reinterpret_cast<const float4 *>(p + d);
            o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y);
            o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
            l = fmaf(p[D], f, l);
        }
        if (kMode == kWhole ? split == 0 && all <= tile1 : kMode == kWindow && a.splits == 1 && !a.later) {
            store_row(a, b, hk, r0 + r, d, o.x, m, l);
            store_row(a, b, hk, r0 + r, d + 1, o.y, m, l);
            store_row(a, b, hk, r0 + r, d + 2, o.z, m, l);
            store_row(a, b, hk, r0 + r, d + 3, o.w, m, l);
        } else {
            const int64_t part = part_at(r);
            *reinterpret_cast<float4 *>(a.part_o + part * D + d) = o;
            if (d == 0) a.part_ml[part] = make_float2(m, l);
        }
    }
}

// How a call is laid out: the slots of 8 that a CTA holds, and the chunks.
// Chunks follow the table's width alone (lengths are in device memory).
struct AttendPlan {
    int parts, nt, rows, row_tiles, width, splits;
};

template <int D>
int attend_places(int nt) {
    return nt == 1 ? attend_per_sm<D, 1>() : nt == 2 ? attend_per_sm<D, 2>() : attend_per_sm<D, 4>();
}

// rows: of a key/value head and sequence; most: tiles of positions that a sequence may have.
inline AttendPlan attend_plan_of(const bsg_kv8_cache &c, int64_t most, int64_t B, int64_t rows, int parts) {
    AttendPlan p;
    p.parts = parts;
    p.rows = (int)rows;
    const int slots = p.rows * parts;
    p.nt = slots <= 8 ? 1 : slots <= 16 || c.dim == 256 ? 2 : 4;
    p.row_tiles = (slots + 8 * p.nt - 1) / (8 * p.nt);
    const int n = c.dim == 32    ? attend_places<32>(p.nt)
                  : c.dim == 64  ? attend_places<64>(p.nt)
                  : c.dim == 96  ? attend_places<96>(p.nt)
                  : c.dim == 128 ? attend_places<128>(p.nt)
                                 : attend_places<256>(p.nt);
    const int64_t places = (int64_t)device_sm_count() * n, groups = B * c.heads * p.row_tiles;
    // 3 and 6 chunks a place: 99 and 96 us against 94 (64 ragged sequences), 145 and 154 against 146 (two long
    // ones; then with probabilities in one part)
    constexpr int kPerPlace = 4;
    int64_t splits = (kPerPlace * places + groups - 1) / groups;
    if (splits > kMaxSplits) splits = kMaxSplits;
    if (splits > (most + kWarps - 1) / kWarps) splits = (most + kWarps - 1) / kWarps;
    p.splits = (int)splits;
    p.width = (int)((most + kWarps - 1) / kWarps * kWarps);
    return p;
}

inline AttendPlan attend_plan(const bsg_kv8_cache &c, int64_t table_ld, int64_t B, int64_t T, int heads, int parts) {
    return attend_plan_of(c, table_ld * (c.page_tokens / 16), B, T * (heads / c.heads), parts);
}

template <int D, int NT, int kParts, int kMode, bool kLong>
cudaError_t launch_attend_as(const AttendArgs &a, const AttendPlan &p, int64_t B, cudaStream_t st) {
    constexpr int smem = attend_smem<D, NT, kParts>();
    static bool set[64] = {false};  // this kernel's shared memory, on each device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (smem > 48 * 1024 && (dev >= 64 || !set[dev])) {
        e = cudaFuncSetAttribute(kv8_attend_kernel<D, NT, kParts, kMode, kLong>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) set[dev] = true;
    }
    const dim3 grid((unsigned)(a.c.heads * p.row_tiles), (unsigned)B, (unsigned)p.splits);
    kv8_attend_kernel<D, NT, kParts, kMode, kLong><<<grid, kWarps * 32, smem, st>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

// The kernel that begins sums anew where a warp may have more tiles than one sum takes: the first
// chunk is the longest.
template <int D, int NT, int kParts, int kMode>
cudaError_t launch_attend(const AttendArgs &a, const AttendPlan &p, int64_t B, cudaStream_t st) {
    const int64_t n = p.splits, most = n == 1 ? p.width / kWarps : (16 * n - 6) * (p.width / kWarps) / (10 * n * n) + 1;
    return most > kAnew<kParts> ? launch_attend_as<D, NT, kParts, kMode, true>(a, p, B, st)
                                : launch_attend_as<D, NT, kParts, kMode, false>(a, p, B, st);
}

template <int D, int kMode>
cudaError_t launch_attend_nt(const AttendArgs &a, const AttendPlan &p, int64_t B, cudaStream_t st) {
    cudaError_t e = cudaErrorInvalidValue;
    if (p.parts == 1) {
        if (p.nt == 1) e = launch_attend<D, 1, 1, kMode>(a, p, B, st);
        if (p.nt == 2) e = launch_attend<D, 2, 1, kMode>(a, p, B, st);
        if constexpr (D < 256)
            if (p.nt == 4) e = launch_attend<D, 4, 1, kMode>(a, p, B, st);
    } else {
        if (p.nt == 1) e = launch_attend<D, 1, 2, kMode>(a, p, B, st);
        if (p.nt == 2) e = launch_attend<D, 2, 2, kMode>(a, p, B, st);
        if constexpr (D < 256)
            if (p.nt == 4) e = launch_attend<D, 4, 2, kMode>(a, p, B, st);
    }
    return e;
}

}  // namespace
}  // namespace bsg

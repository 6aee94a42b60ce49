// wgroups.cu -- int4 weights with one scale per group of rows and column: the
// storage, and products of a few rows with it.
//
// The storage is wquant.cu's scheme ("Precision" manual, section "Integer
// weights") on blocks of `group` rows: s = absmax / 7 rounded to f32, codes
// the integer nearest w / s, ties to even, all-zero blocks s = 0.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "bsg_internal.h"
#include "bsg_ptx.cuh"
#include "serve.cuh"
#include "wq_round.cuh"

namespace cg = cooperative_groups;

namespace bsg {
namespace {

// ---- storage ------------------------------------------------------------------
//
// One read of W and one write of the codes: HBM bounds it.  A CTA takes 128 columns
// of a group, a warp every 8th row of it, a lane 4 columns; a lane's rows stay in
// registers between the maximum and the codes (kKept of them: groups up to 8 kKept
// rows are read once).  Longer groups go to a cluster of up to 8 CTAs, what does not
// fit the registers is read twice.
//
// A code is RN(w RN(1/s)) where that lies more than 2^-14 from a half-integer, as
// wq_round.cuh shows, and the exact quotient's otherwise; a magic number rounds
// it, and the sum's low bits are the code.  |w RN(1/s)| <= 7 (1 + 2^-22), so there is
// nothing to clamp, but for scales near or below the least normal number: those
// columns take the exact path throughout.
//
// Measured: 16384 x 16384 in groups of 64 343 us (0.52 of the floor's rate; a thread
// to two columns that read them twice 519), of 128 364 (643), the whole column 828
// (12009); 8191 x 12289 (unaligned rows) in groups of 32 140 (171; 213 with the same 8
// warps, which have half as many rows to hold), 768 x 50304 57 (94).  What bounds it:
// a CTA's loads, barrier and stores follow one another, and 24 warps an SM overlap
// them by half; at 32 warps the rows spill (365 us).
constexpr int kStoreCols = 128;

struct StoreArgs {
    const float *W;
    uint8_t *Q;
    float *scale;
    int32_t *dstatus;
    int64_t K, N, ldw, group, ldq, lds;
    int ranks;
    bool vec, pairs;  // rows of W on 16 bytes, of Q on 2
};

__device__ __noinline__ uint32_t exact_code(float w, float s) { return (uint32_t)wq_round_quotient_exact(w, s, 7); }

template <int kWarps, int kKept>
__global__ void __launch_bounds__(kWarps * 32, kKept == 8 ? 24 / kWarps : 2)
    wquant_groups_kernel(const __grid_constant__ StoreArgs a) {
    __shared__ uint32_t max_s[kWarps][kStoreCols], top_s[kStoreCols];
    __shared__ float scale_s[kStoreCols];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = a.ranks;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t tile0 = (int64_t)(blockIdx.x / ranks) * kStoreCols, col = tile0 + lane * 4;
    const int64_t groups = (a.K + a.group - 1) / a.group;
    auto load = [&](int64_t k) {
        const float *p = a.W + k * a.ldw + col;
        if (a.vec && col + 4 <= a.N) return __ldg(reinterpret_cast<const float4 *>(p));
        return make_float4(col < a.N ? p[0] : 0.0f, col + 1 < a.N ? p[1] : 0.0f, col + 2 < a.N ? p[2] : 0.0f,
                           col + 3 < a.N ? p[3] : 0.0f);
    };
    for (int64_t g = blockIdx.y; g < groups; g += gridDim.y) {
        const int64_t g0 = g * a.group, rows = (a.K - g0 < a.group ? a.K - g0 : a.group);
        const int64_t first = g0 + rows * rank / ranks + warp, end = g0 + rows * (rank + 1) / ranks;
        const int64_t rest = first + kKept * kWarps;
        float4 v[kKept];
#pragma unroll
        for (int i = 0; i < kKept; ++i)
            v[i] = first + i * kWarps < end ? load(first + i * kWarps) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        uint32_t top[4] = {0, 0, 0, 0};
        auto raise = [&](const float4 &x) {
            top[0] = max(top[0], __float_as_uint(x.x) & 0x7fffffffu);
            top[1] = max(top[1], __float_as_uint(x.y) & 0x7fffffffu);
            top[2] = max(top[2], __float_as_uint(x.z) & 0x7fffffffu);
            top[3] = max(top[3], __float_as_uint(x.w) & 0x7fffffffu);
        };
#pragma unroll
        for (int i = 0; i < kKept; ++i) raise(v[i]);
#pragma unroll 4
        for (int64_t k = rest; k < end; k += kWarps) raise(load(k));
        *reinterpret_cast<uint4 *>(&max_s[warp][lane * 4]) = make_uint4(top[0], top[1], top[2], top[3]);
        __syncthreads();
        uint32_t m = 0;
        if (tid < kStoreCols) {
#pragma unroll
            for (int i = 0; i < kWarps; ++i) m = max(m, max_s[i][tid]);
            top_s[tid] = m;
        }
        if (ranks > 1) {
            cluster.sync();
            if (tid < kStoreCols)
                for (int i = 0; i < ranks; ++i) m = max(m, *cluster.map_shared_rank(&top_s[tid], i));
        }
        if (tid < kStoreCols) {
            if (m >= 0x7f800000u) set_status(a.dstatus, BSG_DSTATUS_NONFINITE);
            const float s = __fdiv_rn(__uint_as_float(m), 7.0f);
            scale_s[tid] = s;
            if (rank == 0 && tile0 + tid < a.N) a.scale[g * a.lds + tile0 + tid] = s;
        }
        __syncthreads();
        float s[4], r[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            s[c] = scale_s[lane * 4 + c];
            r[c] = s[c] == 0.0f || !isfinite(s[c]) ? 0.0f : s[c] < 0x1p-120f ? NAN : __frcp_rn(s[c]);
        }
        auto code = [&](float w, int c) -> uint32_t {
            const float x = __fmul_rn(w, r[c]), y = __fadd_rn(x, 12582912.0f);  // 1.5 2^23
            const float off = fabsf(__fsub_rn(x, __fsub_rn(y, 12582912.0f)));
            return off <= 0.5f - 0x1p-14f ? __float_as_uint(y) : exact_code(w, s[c]);
        };
        auto put = [&](int64_t k, const float4 &x) {
            const uint32_t even = __byte_perm(code(x.x, 0), code(x.z, 2), 0x0040);
            const uint32_t odd = __byte_perm(code(x.y, 1), code(x.w, 3), 0x0040);
            const uint32_t w = (even & 0x0f0fu) | (odd << 4 & 0xf0f0u);
            uint8_t *q = a.Q + k * a.ldq + col / 2;
            if (a.pairs && col + 2 < a.N) {
                *reinterpret_cast<uint16_t *>(q) = (uint16_t)w;
            } else {
                if (col < a.N) q[0] = (uint8_t)w;
                if (col + 2 < a.N) q[1] = (uint8_t)(w >> 8);
            }
        };
#pragma unroll
        for (int i = 0; i < kKept; ++i)
            if (first + i * kWarps < end) put(first + i * kWarps, v[i]);
#pragma unroll 4
        for (int64_t k = rest; k < end; k += kWarps) put(k, load(k));
        // nobody writes the maxima again, or leaves, while another reads them
        if (ranks > 1)
            cluster.sync();
        else
            __syncthreads();
    }
}

// ---- products ---------------------------------------------------------------
//
// Y[m][n] = sum_g s[g][n] sum_{k in g} X[m][k] q[k][n] for up to 16 rows.  What
// has to be read is half a byte per weight, and at most 16 rows are 64
// operations to a byte: HBM bounds it, provided a weight costs the SM less than
// 2.7 instructions per lane.  So the products run on the tensor cores
// (m16n8k16, the weights as the 16-row operand, X's rows as the 8 columns), and
// a weight is unpacked with one and an eighth:
//
//   Two rows' 16-bit pieces of 4 codes side by side (a byte permute), masked to one
//   nibble each with its top bit flipped (u = q + 8; one LOP3), are two f16
//   subnormals, u 2^-24 (low nibble of a byte) or u 2^-20 (high); one f16
//   multiply-add makes them q 2^-10.
//   (Left subnormal, with 8 sum_k x taken off the sums, they cost a third less
//   and lost ten bits: the tensor cores align products by the exponent field.)
//
// f32 rows are two f16 parts, hi + 2^-11 lo (two columns), 16-bit rows one, all
// relative to a power of two near the largest |x| of kChunk consecutive k of
// the row, so that f16's range holds them.  What they add up to is brought to 2^-10 of
// its true size before it is scaled and added (f32 holds that of any 64 finite x, below
// 2^128 2^3 2^6 2^-10), so that chunks of any sizes, zeros among them, meet in one sum as
// they would in plain f32.  (Sums kept at their chunks' sizes and moved from one to the next
// ran over where chunks of zeros followed large ones, and took 52 against 50 us at 8 f32 rows
// of 16384 x 16384.)  A first, small launch lays the parts out
// as the B operand; it runs beside the start of the second, whose weights are
// on their way meanwhile.  (With each CTA making its own parts in shared memory
// its warps met at a barrier every kChunk: 62 against 53 us at 16384^2, 8 rows.)
//
// A CTA takes 512 columns in units of 64 rows, a warp 64 of them.  Units are
// copied ahead by TMA, their codes, their scales and X's parts, each stage sent for
// by the last warp to read what it held; groups' sums are
// scaled once a unit, or once each 32 rows where a group may end there (kFolds).
// 64 columns to a warp: at 128 their sums left room for 8 warps on an SM, and it
// issued on 0.35 of the cycles.  K is split over CTAs, whose sums a third launch
// adds up in the order of k.  (Joined by clusters through distributed shared
// memory, a fifth of the places stayed empty; by the last warp to arrive, its
// loads alone took up to 13 us.)
//
// Measured on the device: 16384 x 16384, 8 f32 rows 50 us (0.45 of the floor's rate), 1
// row 38, 8 bf16 rows 40 (0.56); 8191 x 12289, 5 bf16 rows 21.0 (0.38); 8192 x 8192, 8 f16
// rows 15.5, 16 bf16 rows 20; 4096 x 4096, 8 f16 rows 8.8.  What bounds it is no one thing: at
// 8 f32 rows of 16384 x 16384 the tensor pipe is busy for 33 % of the cycles, ALU 31, FMA
// 26, and an instruction issues in 0.47 of them.  The copies without the products took
// 38 of 55 us when that was measured, the products without the copies 42: each well over the
// floor, and overlapping in part.  What counts of the products: the ALU takes an
// instruction every other cycle, and 6 of them for 256 weights are 12 cycles (8 more,
// the flip by itself, cost 6 us of 42); m16n8k16 takes 8 more for each 8 slots (measured: 16
// together with 4 f16 multiply-adds).  Weights that lie in L2 are no faster.  The parts'
// launch and the join are 1 to 2 us each.  Below some 4096 x 4096 it is the three launches and
// the first copies, about 5 us.  (The shift of a 16-bit piece as a product on the FMA
// pipe: 44 us.)

constexpr int kWarps = 8, kWarpCols = 64, kCtaCols = kWarps * kWarpCols;
constexpr int kUnit = 64;
constexpr int kChunk = 256;                   // k that share a power of two
constexpr int kSteps = kUnit / 16;
constexpr int kBoxCols = 256;                 // columns of one TMA copy: rows of 128 bytes
constexpr int kBox = kUnit * kBoxCols / 2;    // bytes of its codes
constexpr int kCodes = kCtaCols / kBoxCols * kBox;

// CTAs on an SM: two; one of four slot tiles; three (80 registers a thread, fewer units
// each) of one slot tile where a group ends once a unit; with the scales of 32-row
// groups they would spill.  Three against two: 16384 x 16384, 1 row 42.6 and 46.0 us, 8 bf16
// rows 44.2 and 49.3 (before the join was quicker); 8 x 4096 x 4096 9.3 and 9.4; 8 x
// 8192 x 8192 16.4 and 15.9.
constexpr int matvec_per_sm(int nt, int folds) { return nt == 4 ? 1 : nt == 1 && folds == 1 ? 3 : 2; }
// Units on their way or in use: 180 to 212 KB of shared memory for the CTAs of an SM.
__host__ __device__ constexpr int stages(int folds, int per_sm) {
    return (per_sm == 1 ? 8 : per_sm == 2 ? 5 : 3) - (folds == 2 ? 1 : 0);
}
// Bytes of a unit's parts of X, and of a stage: codes, scales, parts.
template <int NT>
__host__ __device__ constexpr int part_bytes() { return kSteps * NT * 256; }
template <int NT, int kFolds>
__host__ __device__ constexpr int stage_bytes() { return kCodes + kFolds * kCtaCols * 4 + part_bytes<NT>(); }
template <int NT, int kFolds, int kPerSm>
constexpr int matvec_smem() { return stages(kFolds, kPerSm) * stage_bytes<NT, kFolds>() + 1024; }

// The workspace: the parts of X, [step of 16 k][NT][lane] pairs of registers; the
// exponents that chunks are raised by, [chunk][16]; the splits' sums,
// [split][row][column].
inline int64_t part_chunks(int64_t K) { return (K + kChunk - 1) / kChunk; }

struct MatvecArgs {
    CUtensorMap q_map, s_map;  // where tma_q, tma_s
    const uint2 *parts;
    const int *up;
    float *sums;
    int cols;  // of a row of sums
    int splits;  // of K
    const uint8_t *Q;
    int64_t ldq;
    const float *scale;
    int64_t lds;
    void *Y;
    int64_t ldy;
    int32_t *dstatus;
    int group, M, N, K, relu;
    int tma_q, tma_s;  // Q's (the scales') rows start on 16 bytes
};

__device__ __forceinline__ void copy_async4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

// D = A B + C with A 16 x 16 and B 16 x 8 f16, C and D f32.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint2 b, float c0, float c1, float c2,
                                        float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y), "f"(c0), "f"(c1), "f"(c2),
          "f"(c3));
}

// v & mask ^ flip, in one instruction
__device__ __forceinline__ uint32_t masked_flip(uint32_t v, uint32_t mask, uint32_t flip) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(v), "r"(mask), "r"(flip));
    return r;
}

// The codes in the low (high) nibbles of bytes 0 and 2 as f16 q 2^-10.
__device__ __forceinline__ uint32_t codes_f16(uint32_t u, uint32_t up) {
    const uint32_t minus8 = 0xa000a000u;  // -8 2^-10
    const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&u), *reinterpret_cast<const __half2 *>(&up),
                              *reinterpret_cast<const __half2 *>(&minus8));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t low_codes(uint32_t v) {
    return codes_f16(masked_flip(v, 0x000f000fu, 0x00080008u), 0x74007400u);  // u 2^-24 times 2^14
}
__device__ __forceinline__ uint32_t high_codes(uint32_t v) {
    return codes_f16(masked_flip(v, 0x00f000f0u, 0x00800080u), 0x64006400u);  // u 2^-20 times 2^10
}

// 16 bytes at any address, of which the first `bytes` are wanted; whole words
// where they lie inside [lo, hi), bytes at its ends.
__device__ __forceinline__ uint4 load_unaligned16(const uint8_t *p, int bytes, const uint8_t *lo,
                                                  const uint8_t *hi) {
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 3);
    const uint8_t *q = p - off;
    uint32_t w[4];
    if (q >= lo && q + 20 <= hi) {
        uint32_t x[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) x[i] = __ldg(reinterpret_cast<const uint32_t *>(q) + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(x[i], x[i + 1], 8 * off);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = 0;
            for (int j = 0; j < 4; ++j)
                if (4 * i + j < bytes) w[i] |= (uint32_t)p[4 * i + j] << (8 * j);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// X's parts: one CTA to a chunk, a row to a warp.  Lane 4s + t of a step holds, of
// slot s, rows 2t + {0, 1, 8, 9}.
template <typename T, int NT>
__global__ void __launch_bounds__(256)
    wgroups_parts_kernel(const T *__restrict__ X, int64_t ldx, int M, int K, uint2 *__restrict__ parts,
                         int *__restrict__ up, int32_t *__restrict__ dstatus) {
    constexpr int kParts = sizeof(T) == 4 ? 2 : 1;
    __shared__ uint2 x_s[kChunk / 16 * NT * 32];
    __half *xh = reinterpret_cast<__half *>(x_s);
    const int k0 = blockIdx.x * kChunk, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    griddep_launch_dependents();
    for (int r = warp; r < 8 * NT / kParts; r += 8) {
        float x[kChunk / 32];
        uint32_t top = 0;
        const T *row = X + (int64_t)min(r, M - 1) * ldx + k0 + lane;
        const int left = r < M ? K - k0 - lane : 0;
#pragma unroll
        for (int j = 0; j < kChunk / 32; ++j) x[j] = 32 * j < left ? to_f32(row[32 * j]) : 0.0f;
#pragma unroll
        for (int j = 0; j < kChunk / 32; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        // 2^e with the largest |x| 2^e in [2^13, 2^14)
        const int e = max(-126, min(126, 13 + 127 - (int)(top >> 23)));
        const float by = __uint_as_float((uint32_t)(e + 127) << 23);
        if (lane == 0) {
            if (top >= 0x7f800000u) set_status(dstatus, BSG_DSTATUS_NONFINITE);
            up[blockIdx.x * 16 + r] = e;
        }
        const int slot = r * kParts, kk = lane % 16;  // of step 2j + lane / 16
        const int t = kk / 2 % 4, i = kk % 2 + kk / 8 * 2;
        const int at = ((lane / 16 * NT + slot / 8) * 32 + slot % 8 * 4 + t) * 4 + i;
#pragma unroll
        for (int j = 0; j < kChunk / 32; ++j) {
            const float y = x[j] * by;
            const __half hi = __float2half_rn(y);
            xh[at + j * 2 * NT * 128] = hi;
            if (kParts == 2) xh[at + j * 2 * NT * 128 + 16] = __float2half_rn((y - __half2float(hi)) * 2048.0f);
        }
    }
    __syncthreads();
    const uint4 *from = reinterpret_cast<const uint4 *>(x_s);
    uint4 *to = reinterpret_cast<uint4 *>(parts) + (int64_t)blockIdx.x * (kChunk / 16 * NT * 16);
    for (int i = threadIdx.x; i < kChunk / 16 * NT * 16; i += 256) to[i] = from[i];
}

template <typename T>
__device__ __forceinline__ void store_pair(const MatvecArgs &a, int r, int c, float2 v) {
    T *y = static_cast<T *>(a.Y) + r * a.ldy + c;
    if (c < a.N) y[0] = from_f32<T>(a.relu && !(v.x > 0.0f) ? 0.0f : v.x);
    if (c + 1 < a.N) y[1] = from_f32<T>(a.relu && !(v.y > 0.0f) ? 0.0f : v.y);
}

// grid: splits of K x column tiles, the splits of a tile side by side (in one dimension:
// 2^25 columns are one tile more than a grid's others hold)
template <typename T, int NT, int kFolds, int kPerSm>
__global__ void __launch_bounds__(kWarps * 32, kPerSm)
    wgroups_matvec_kernel(const __grid_constant__ MatvecArgs a) {
    constexpr int kParts = sizeof(T) == 4 ? 2 : 1;
    constexpr int kFoldSteps = kSteps / kFolds, kStages = stages(kFolds, kPerSm);
    constexpr int kStage = stage_bytes<NT, kFolds>(), kScalesAt = kCodes, kPartsAt = kCodes + kFolds * kCtaCols * 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023);  // the swizzle's period
    __shared__ uint64_t full[kStages];
    __shared__ int readers[kStages];  // warps that have yet to read a stage
    __shared__ volatile int gave_up, never;
    const int ranks = a.splits, rank = blockIdx.x % ranks;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
    const int units = (a.K + kUnit - 1) / kUnit;
    const int u0 = (int)((int64_t)units * rank / ranks), u1 = (int)((int64_t)units * (rank + 1) / ranks);
    const int tile0 = (int)(blockIdx.x / ranks) * kCtaCols, col0 = tile0 + warp * kWarpCols;  // the warp's first column
    const bool busy = col0 < a.N;
    const int boxes = a.N - tile0 > kBoxCols ? 2 : 1;
    const int busy_warps = min(kWarps, (a.N - tile0 + kWarpCols - 1) / kWarpCols);
    if (tid < kStages) {
        mbar_init(&full[tid], 1);
        readers[tid] = busy_warps;
    }
    if (tid == 0) gave_up = never = 0;
    fence_mbar_init();
    __syncthreads();

    // One thread's copies of a unit: codes and scales (weights: there from the
    // start), then X's parts.
    const int copied = part_bytes<NT>() + (a.tma_q ? boxes * kBox : 0) + (a.tma_s ? boxes * kFolds * kBoxCols * 4 : 0);
    auto copy_weights = [&](int unit, int stage) {
        uint8_t *to = smem + stage * kStage;
        mbar_arrive_expect_tx(&full[stage], copied);
        for (int i = 0; i < boxes; ++i) {
            if (a.tma_q)
                tma_load_2d(&a.q_map, &full[stage], to + i * kBox, (tile0 + i * kBoxCols) / 2, unit * kUnit);
            if (a.tma_s)
#pragma unroll
                for (int f = 0; f < kFolds; ++f)
                    tma_load_2d(&a.s_map, &full[stage], to + kScalesAt + (f * kCtaCols + i * kBoxCols) * 4,
                                tile0 + i * kBoxCols, (unit * kUnit + 32 * f) / a.group);
        }
    };
    auto copy_parts = [&](int unit, int stage) {
        bulk_load(smem + stage * kStage + kPartsAt, a.parts + (int64_t)unit * (part_bytes<NT>() / 8), part_bytes<NT>(),
                  &full[stage]);
    };
    // Rows that TMA does not take: each warp copies its own columns, in the
    // places that TMA's 128-byte swizzle would give them.
    int f_unit = u0;
    auto copy_unaligned = [&](int stage) {
        uint8_t *to = smem + stage * kStage;
        if (busy && f_unit < u1) {
            const int k0 = f_unit * kUnit;
            if (!a.tma_q) {
                const int half = (a.N + 1) / 2, c = lane % 2;
                const int bytes = min(16, half - col0 / 2 - 16 * c), piece = warp % 4 * 2 + c;
                const uint8_t *q_end = a.Q + (int64_t)(a.K - 1) * a.ldq + half;
                const uint8_t *p = a.Q + (int64_t)(k0 + lane / 2) * a.ldq + col0 / 2 + 16 * c;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 16 + lane / 2;
                    if (bytes > 0 && k0 + r < a.K)
                        *reinterpret_cast<uint4 *>(to + warp / 4 * kBox + r * 128 + ((piece ^ (r & 7)) << 4)) =
                            load_unaligned16(p + i * 16 * a.ldq, bytes, a.Q, q_end);
                }
            }
            if (!a.tma_s) {
#pragma unroll
                for (int f = 0; f < kFolds; ++f) {
                    const float *s = a.scale + (int64_t)(min(k0 + 32 * f, a.K - 1) / a.group) * a.lds + col0;
                    const uint32_t at = smem_u32(to + kScalesAt + (f * kCtaCols + warp * kWarpCols) * 4);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bool in = col0 + i * 32 + lane < a.N;
                        copy_async4(at + (i * 32 + lane) * 4, in ? s + i * 32 + lane : s, in ? 4 : 0);
                    }
                }
            }
        }
        ++f_unit;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const bool all_tma = a.tma_q && a.tma_s;
    const int mine = warp < kStages && lane == 0 && u0 + warp < u1 ? warp : -1;  // the stage that this thread fills
    if (mine >= 0) copy_weights(u0 + mine, mine);
    if (!all_tma)
        for (int i = 0; i < kStages; ++i) copy_unaligned(i);
    griddep_wait();  // X's parts are there
    griddep_launch_dependents();
    if (mine >= 0) copy_parts(u0 + mine, mine);

    // The lane's 8 columns 8g .. 8g + 7, its slots 2t and 2t + 1 of each 8: sums of 2^-10
    // of their true size, of the rows in those slots.
    constexpr int kRows = 2 / kParts;  // rows of two slots
    float acc[4][NT][2 * kRows];
    float by[NT][kRows];       // the parts' sums, 2^e too large, times this
    int up_next[NT][kRows];    // e of the coming chunk
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2 * kRows; ++i) acc[m][n][i] = 0.0f;

    // Where the lane finds its columns' codes of rows 2t and 2t + 1 (+ 8): the
    // swizzle puts the rows of four lanes on banks of their own.
    const int piece = warp % 4 * 2 + (g >> 2), even_at = 2 * t * 128 + ((piece ^ 2 * t) << 4) + (g & 3) * 4;
    const int odd_at = (2 * t + 1) * 128 + ((piece ^ (2 * t + 1)) << 4) + (g & 3) * 4;
    uint32_t parity = 0;
    int stage = 0;
    constexpr int kChunkUnits = kChunk / kUnit;
    auto load_up = [&](int chunk) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < kRows; ++i) up_next[n][i] = __ldg(a.up + chunk * 16 + (8 * n + 2 * t) / kParts + i);
    };
    if (u0 < u1) load_up(u0 / kChunkUnits);
    if (busy)
        for (int u = u0; u < u1; ++u) {
            if (u == u0 || u % kChunkUnits == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
                        by[n][i] = __uint_as_float((uint32_t)(127 - up_next[n][i]) << 23);  // |e| <= 126
                if ((u / kChunkUnits + 1) * kChunkUnits < u1) load_up(u / kChunkUnits + 1);
            }
            if (!mbar_wait(&full[stage], parity, &gave_up)) {
                gave_up = 1;
                set_status(a.dstatus, BSG_DSTATUS_TIMEOUT);
                break;
            }
            if (!all_tma) asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();
            const uint8_t *at = smem + stage * kStage;
#pragma unroll
            for (int f = 0; f < kFolds; ++f) {
                const float4 *scales =
                    reinterpret_cast<const float4 *>(at + kScalesAt + (f * kCtaCols + warp * kWarpCols) * 4) + 2 * g;
                const uint8_t *codes = at + warp / 4 * kBox + f * kFoldSteps * 2048;
                const uint2 *xb = reinterpret_cast<const uint2 *>(at + kPartsAt) + f * kFoldSteps * NT * 32 + lane;
                float d[4][NT][4];  // this fold's sums
#pragma unroll
                for (int s = 0; s < kFoldSteps; ++s) {
                    uint2 x[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) x[n] = xb[(s * NT + n) * 32];
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = *reinterpret_cast<const uint32_t *>(codes + (i % 2 ? odd_at : even_at) + s * 2048 +
                                                                   i / 2 * 1024);
#pragma unroll
                    for (int quad = 0; quad < 2; ++quad) {  // 4 columns: a 16-bit piece of a row
                        const uint32_t sel = quad ? 0x7632 : 0x5410;
                        const uint32_t p0 = __byte_perm(w[0], w[1], sel), p1 = __byte_perm(w[2], w[3], sel);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t v0 = p0 >> (8 * h), v1 = p1 >> (8 * h);
                            const uint32_t a0 = low_codes(v0), a1 = high_codes(v0);
                            const uint32_t a2 = low_codes(v1), a3 = high_codes(v1);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                float(&y)[4] = d[2 * quad + h][n];
                                if (s == 0)
                                    mma_f16(y, a0, a1, a2, a3, x[n], 0.0f, 0.0f, 0.0f, 0.0f);
                                else
                                    mma_f16(y, a0, a1, a2, a3, x[n], y[0], y[1], y[2], y[3]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int quad = 0; quad < 2; ++quad) {
                    const float4 sc = scales[quad];
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const float(&y)[4] = d[2 * quad + half][n];
                            float(&to)[2 * kRows] = acc[2 * quad + half][n];
                            const float s0 = half ? sc.z : sc.x, s1 = half ? sc.w : sc.y;
                            if constexpr (kParts == 2) {
                                const float low = by[n][0] * 0x1p-11f;
                                to[0] = fmaf(fmaf(y[1], low, y[0] * by[n][0]), s0, to[0]);
                                to[1] = fmaf(fmaf(y[3], low, y[2] * by[n][0]), s1, to[1]);
                            } else {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    to[i] = fmaf(y[i] * by[n][i % 2], i < 2 ? s0 : s1, to[i]);
                            }
                        }
                }
            }
            __syncwarp();  // every lane has read the stage
            if (!all_tma) copy_unaligned(stage);
            if (lane == 0) {  // the last warp to read a stage sends for its next unit
                __threadfence_block();
                if (atomicSub(&readers[stage], 1) == 1 && u + kStages < u1) {
                    readers[stage] = busy_warps;
                    __threadfence_block();
                    copy_weights(u + kStages, stage);
                    copy_parts(u + kStages, stage);
                }
            }
            if (++stage == kStages) stage = 0, parity ^= 1;
        }
    if (gave_up)  // the copies in flight, with the same limit: a stage's last phase, if it has begun
        for (int i = 0; i < kStages; ++i) mbar_wait(&full[i], parity ^ (i < stage ? 1u : 0u), &never);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!busy) return;

    // The warp's sums at their true size, to Y or to the workspace.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = (8 * n + 2 * t) / kParts + i;
            if (r >= a.M) continue;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float2 v = make_float2(acc[m][n][i] * 1024.0f, acc[m][n][i + kRows] * 1024.0f);
                const int c = col0 + 8 * g + 2 * m;
                if (ranks > 1)
                    *reinterpret_cast<float2 *>(a.sums + ((int64_t)rank * a.M + r) * a.cols + c) = v;
                else
                    store_pair<T>(a, r, c, v);
            }
        }
}

constexpr int kMaxMatvecSplits = 32, kJoinSides = 8, kJoinCols = 64;

// Adds the splits' sums: grid (column tiles, rows), kJoinSides warps with a share of the
// splits each, whose loads are all on their way at once.  (A thread to all splits of
// four columns: 12.5 against 9.4 us for 8 x 4096 x 4096 in all, 54.6 against 52.2 for
// 8 x 16384 x 16384.)
template <typename T>
__global__ void __launch_bounds__(kJoinSides * 32) wgroups_join_kernel(const __grid_constant__ MatvecArgs a, int splits) {
    constexpr int kEach = kMaxMatvecSplits / kJoinSides;
    __shared__ float2 part_s[kJoinSides][32];
    const int side = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int c = blockIdx.x * kJoinCols + lane * 2, r = blockIdx.y;
    const int each = (splits + kJoinSides - 1) / kJoinSides, k0 = side * each, k1 = min(splits, k0 + each);
    const int64_t step = (int64_t)a.M * a.cols;
    griddep_wait();
    const float *from = a.sums + (int64_t)r * a.cols + c;
    float2 y = make_float2(0.0f, 0.0f), v[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        v[k] = make_float2(0.0f, 0.0f);
        if (k0 + k < k1 && c < a.N) v[k] = __ldcg(reinterpret_cast<const float2 *>(from + (k0 + k) * step));
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) y.x += v[k].x, y.y += v[k].y;
    part_s[side][lane] = y;
    __syncthreads();
    if (side || c >= a.N) return;
#pragma unroll
    for (int i = 1; i < kJoinSides; ++i) y.x += part_s[i][lane].x, y.y += part_s[i][lane].y;
    store_pair<T>(a, r, c, y);
}

// ---- small products ---------------------------------------------------------
//
// Where the weights are few, the three launches above cost more than the products.
// This is one launch on the CUDA cores, without a workspace: 8 lanes take 64
// columns (a word of 8 codes each), the 32 such parts of a CTA and the CTAs of a
// cluster split K evenly, so that a lane has a few rows, loaded at once; their sums
// meet by shuffles and in (distributed) shared memory, always in one order.  A code
// becomes a float by the magic number 2^23, exactly, and X is used in f32, as 2^-10 of what
// it is, so that a group's sum before its scale does not run over where Y would not.
//
// What bounds it: the launch, one round of loads and the cluster's two barriers at
// the small end; 4 + M instructions per weight beyond.  Measured on the device, this
// against the three launches: 768 x 2304 f32, 1 row 4.1 and 4.5 us, 2 rows 4.4 and 4.6, 4
// rows 5.0 and 4.9; 768 x 768, 1 row 3.9 and 4.2, 4 rows 4.8 and 4.6; 2048 x 2048 bf16, 1
// row 5.0 and 4.6, 2 rows 4.8 (both the three launches); 3000 x 768, 1 row 5.6 and 4.7.  The
// host's part is 3 us against 7.5.  So it is taken up to 2^22 products, rows counted as 1, 2
// or 4: what it loses on the device at the upper end, which is all that a graph sees, is
// less than what a call by itself saves.
// (12 rows' instructions in a line, most of them run once: 4.7 us at 768 x 2304, 7.0
// against 5.7 at 3072 x 768, waiting for instructions.  256 columns to a CTA, a quarter of
// the lanes on K: 6.5 and 17.1.)
constexpr int kSmallWarps = 8, kSmallCols = 64, kSmallX = 8192;  // floats of X that a CTA stages

struct SmallArgs {
    const void *X;
    int64_t ldx;
    const uint8_t *Q;
    int64_t ldq;
    const float *scale;
    int64_t lds;
    void *Y;
    int64_t ldy;
    int32_t *dstatus;
    int group, M, N, K, relu, ranks;
    bool words;  // Q's rows start on words
};

// A word of codes, of which the first `bytes` are wanted.
__device__ __forceinline__ uint32_t load_codes(const uint8_t *p, int bytes, bool words) {
    if (words && bytes >= 4) return __ldg(reinterpret_cast<const uint32_t *>(p));
    uint32_t w = 0;
    for (int i = 0; i < min(bytes, 4); ++i) w |= (uint32_t)p[i] << (8 * i);
    return w;
}

// grid: column tiles x CTAs of a cluster; MT >= M rows
template <typename T, int MT>
__global__ void __launch_bounds__(kSmallWarps * 32) wgroups_small_kernel(const __grid_constant__ SmallArgs a) {
    __shared__ float x_s[kSmallX];
    __shared__ float sum_s[kSmallWarps][MT][kSmallCols];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = a.ranks;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int k0 = (int)((int64_t)a.K * rank / ranks), k1 = (int)((int64_t)a.K * (rank + 1) / ranks), n = k1 - k0;
    const int tile0 = (int)(blockIdx.x / ranks) * kSmallCols, col = tile0 + lane % 8 * 8;  // the lane's first column
    const int part = tid / 8;                                               // its rows
    constexpr int kParts = kSmallWarps * 4;
    const int ks = k0 + n * part / kParts, ke = k0 + n * (part + 1) / kParts;
    const int bytes = (a.N + 1) / 2 - col / 2;  // of its columns and those after them
    const uint8_t *q = a.Q + (int64_t)ks * a.ldq + col / 2;
    constexpr int kAhead = 8;
    uint32_t w[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        w[i] = ks + i < ke && bytes > 0 ? load_codes(q + i * a.ldq, bytes, a.words) : 0x88888888u;
    int g = ks / a.group;
    int64_t g_end = (int64_t)(g + 1) * a.group;
    float sc[8];
    auto load_scales = [&]() {
#pragma unroll
        for (int i = 0; i < 8; ++i) sc[i] = col + i < a.N ? __ldg(a.scale + g * a.lds + col + i) : 0.0f;
    };
    load_scales();
    bool bad = false;
    for (int e = tid; e < MT * n; e += kSmallWarps * 32) {
        const int m = e / n, k = e % n;
        const float x = m < a.M ? to_f32(static_cast<const T *>(a.X)[m * a.ldx + k0 + k]) : 0.0f;
        bad |= !isfinite(x);
        x_s[e] = x * 0x1p-10f;
    }
    if (bad) set_status(a.dstatus, BSG_DSTATUS_NONFINITE);
    __syncthreads();

    float acc[MT][8], sum[MT][8];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[m][i] = sum[m][i] = 0.0f;
    // a row at a time: the words move up, so that one row's instructions serve all
#pragma unroll 1
    for (int k = ks; k < ke; ++k) {
        if (k >= g_end) {  // a group ends: its sums at its scales
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int c = 0; c < 8; ++c) sum[m][c] = fmaf(acc[m][c], sc[c], sum[m][c]), acc[m][c] = 0.0f;
            ++g;
            g_end += a.group;
            load_scales();
        }
        const uint32_t u = w[0] ^ 0x88888888u;
#pragma unroll
        for (int i = 0; i + 1 < kAhead; ++i) w[i] = w[i + 1];
        if (k + kAhead < ke && bytes > 0)
            w[kAhead - 1] = load_codes(q + (int64_t)(k + kAhead - ks) * a.ldq, bytes, a.words);
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // 2^23 + code + 8, less 2^23 + 8
            const float v = __fadd_rn(__uint_as_float((u >> (4 * c) & 15u) | 0x4b000000u), -8388616.0f);
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[m][c] = fmaf(x_s[m * n + k - k0], v, acc[m][c]);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            float y = fmaf(acc[m][c], sc[c], sum[m][c]);
            y += __shfl_xor_sync(0xffffffffu, y, 8);
            y += __shfl_xor_sync(0xffffffffu, y, 16);
            if (lane < 8) sum_s[warp][m][lane * 8 + c] = y;
        }
    __syncthreads();
    auto store = [&](int m, int c, float y) {
        y *= 1024.0f;
        if (m < a.M && tile0 + c < a.N)
            static_cast<T *>(a.Y)[m * a.ldy + tile0 + c] = from_f32<T>(a.relu && !(y > 0.0f) ? 0.0f : y);
    };
    for (int e = tid; e < MT * kSmallCols; e += kSmallWarps * 32) {  // a thread's own element: written after it is read
        const int m = e / kSmallCols, c = e % kSmallCols;
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < kSmallWarps; ++i) y += sum_s[i][m][c];
        if (ranks == 1)
            store(m, c, y);
        else
            sum_s[0][m][c] = y;
    }
    if (ranks == 1) return;
    cluster.sync();
    const int c0 = kSmallCols * rank / ranks, cols = kSmallCols * (rank + 1) / ranks - c0;
    for (int e = tid; e < MT * cols; e += kSmallWarps * 32) {
        const int m = e / cols, c = c0 + e % cols;
        float of[8], y = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) of[i] = i < ranks ? *cluster.map_shared_rank(&sum_s[0][m][c], i) : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) y += of[i];
        store(m, c, y);
    }
    cluster.sync();  // no CTA leaves while another reads its sums
}

inline int small_rows(int64_t M) { return M <= 2 ? (int)M : 4; }

// CTAs that split K in the small form: up to 8, until two CTAs to an SM are there or
// a lane has two rows left; 0 where the products are not small.
inline int small_ranks(int64_t M, int64_t N, int64_t K) {
    if (M > 4 || small_rows(M) * N * K > (1 << 22)) return 0;
    const int64_t tiles = (N + kSmallCols - 1) / kSmallCols, xs = small_rows(M) * K;
    int ranks = 1;
    while (ranks < 8 && (tiles * ranks < 2 * device_sm_count() || xs > ranks * kSmallX) &&
           K >= ranks * kSmallWarps * 16)
        ranks *= 2;
    return small_rows(M) * ((K + ranks - 1) / ranks) > kSmallX ? 0 : ranks;
}

template <typename T, int MT>
cudaError_t launch_small(const SmallArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.N + kSmallCols - 1) / kSmallCols * a.ranks));
    cfg.blockDim = dim3(kSmallWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, wgroups_small_kernel<T, MT>, a);
}

// The split of K that ends first, by what was measured: what a CTA takes to start
// and for a unit, alone on its SM or with one or two others; a split's sums are
// written and read once through L2.
inline int matvec_splits(int64_t M, int64_t N, int64_t K, int nt, int per_sm) {
    const int64_t tiles = (N + kCtaCols - 1) / kCtaCols, units = (K + kUnit - 1) / kUnit;
    const int64_t sms = device_sm_count(), places = per_sm * sms;
    const double unit_us[3] = {per_sm == 1 ? 1.9 : nt == 2 ? 0.95 : per_sm == 3 ? 0.85 : 0.75,
                               nt == 2 ? 1.4 : per_sm == 3 ? 1.2 : 1.0, 1.45};
    int splits = 1;
    double best = 1e30;
    for (int r = 1; r <= kMaxMatvecSplits && r <= units; ++r) {
        const int with = tiles * r <= sms ? 0 : tiles * r <= 2 * sms ? 1 : 2, among = std::min(with, per_sm - 1);
        const double us = (double)((tiles * r + places - 1) / places) *
                              ((among == 2 ? 3.5 : 3.0) + unit_us[among] * (double)((units + r - 1) / r)) +
                          (r > 1 ? 2.0 + 8e-6 / 6.0 * (double)(r * M * N) : 0.0);
        if (us < best) best = us, splits = r;
    }
    return splits;
}

template <typename T, int NT, int kFolds, int kPerSm>
cudaError_t launch_matvec(MatvecArgs &a, cudaStream_t st) {
    constexpr int smem = matvec_smem<NT, kFolds, kPerSm>();
    auto *kernel = wgroups_matvec_kernel<T, NT, kFolds, kPerSm>;
    static bool set[64] = {false};  // this kernel's attribute, on each device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    const int splits = a.splits = matvec_splits(a.M, a.N, a.K, NT, kPerSm);
    cfg.gridDim = dim3((unsigned)(a.cols / kCtaCols * splits));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];  // each launch beside the end of the one before it
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess || splits == 1) return e;
    cfg.gridDim = dim3((unsigned)((a.N + kJoinCols - 1) / kJoinCols), (unsigned)a.M);
    cfg.blockDim = dim3(kJoinSides * 32);
    cfg.dynamicSmemBytes = 0;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, wgroups_join_kernel<T>, a, splits);
}

template <typename T, int NT>
cudaError_t launch_matvec(MatvecArgs &a, const T *X, int64_t ldx, void *ws, cudaStream_t st) {
    const int64_t chunks = part_chunks(a.K);
    uint2 *parts = static_cast<uint2 *>(ws);
    int *up = reinterpret_cast<int *>(parts + chunks * (kChunk / 16 * NT * 32));
    a.parts = parts;
    a.up = up;
    a.cols = (int)round_up(a.N, kCtaCols);
    a.sums = reinterpret_cast<float *>(up + chunks * 16);
    wgroups_parts_kernel<T, NT><<<(unsigned)chunks, 256, 0, st>>>(X, ldx, a.M, a.K, parts, up, a.dstatus);
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return a.group % kUnit ? launch_matvec<T, NT, 2, matvec_per_sm(NT, 2)>(a, st)
                           : launch_matvec<T, NT, 1, matvec_per_sm(NT, 1)>(a, st);
}

}  // namespace

cudaError_t launch_wquant_groups(const float *W, int64_t K, int64_t N, int64_t ldw, int64_t group,
                                 uint8_t *Q, int64_t ldq, float *scale, int64_t lds,
                                 int32_t *dstatus, cudaStream_t st) {
    group = std::min(group, K);
    const int64_t groups = (K + group - 1) / group, tiles = (N + kStoreCols - 1) / kStoreCols;
    int ranks = 1;
    while (ranks < 8 && group > ranks * 128) ranks *= 2;
    const StoreArgs a{W, Q, scale, dstatus, K, N, ldw, group, ldq, lds, ranks,
                      reinterpret_cast<uintptr_t>(W) % 16 == 0 && ldw % 4 == 0,
                      (reinterpret_cast<uintptr_t>(Q) | (uintptr_t)ldq) % 2 == 0};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * ranks), (unsigned)std::min<int64_t>(groups, 65535));
    cfg.blockDim = dim3(group <= 32 ? 128 : 256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, group <= 32   ? wquant_groups_kernel<4, 8>
                                    : group <= 64 ? wquant_groups_kernel<8, 8>
                                                  : wquant_groups_kernel<8, 16>, a);
}

// Enough for X of any type and any groups; none where the products are small.
size_t matvec_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (small_ranks(M, N, K)) return 0;
    size_t most = 0;
    for (int parts = 1; parts <= 2; ++parts) {
        const int nt = parts * M <= 8 ? 1 : parts * M <= 16 ? 2 : 4;
        const int64_t splits = std::max(matvec_splits(M, N, K, nt, matvec_per_sm(nt, 1)),
                                        matvec_splits(M, N, K, nt, matvec_per_sm(nt, 2)));
        most = std::max(most, (size_t)(part_chunks(K) * (kChunk / 16 * nt * 256 + 64) +
                                       (splits > 1 ? splits * M * round_up(N, kCtaCols) * 4 : 0)));
    }
    return (size_t)round_up((int64_t)most, 256);
}

cudaError_t launch_wgroups_matvec(const void *X, int dtype, int64_t ldx, const uint8_t *Q,
                                  int64_t ldq, const float *scale, int64_t lds, int64_t group,
                                  int64_t M, int64_t N, int64_t K, int relu, void *Y, int64_t ldy,
                                  void *ws, int32_t *dstatus, cudaStream_t st) {
    // one group to a column ends wherever it likes
    if (group >= K) group = round_up(K, kUnit);
    if (const int ranks = small_ranks(M, N, K)) {
        const SmallArgs s{X, ldx, Q, ldq, scale, lds, Y, ldy, dstatus, (int)group, (int)M, (int)N, (int)K, relu, ranks,
                          (reinterpret_cast<uintptr_t>(Q) | (uintptr_t)ldq) % 4 == 0};
        return with_dtype(dtype, [&](auto t) {
            using T = decltype(t);
            return M == 1   ? launch_small<T, 1>(s, st)
                   : M == 2 ? launch_small<T, 2>(s, st)
                            : launch_small<T, 4>(s, st);
        });
    }
    const int64_t groups = (K + group - 1) / group;
    MatvecArgs a{{}, {}, nullptr, nullptr, nullptr, 0, 1, Q, ldq, scale, lds, Y, ldy, dstatus, (int)group, (int)M, (int)N, (int)K, relu, 0, 0};
    if (reinterpret_cast<uintptr_t>(Q) % 16 == 0 && ldq % 16 == 0)
        a.tma_q = make_tmap_2d(&a.q_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, Q, (uint64_t)(N + 1) / 2, (uint64_t)K,
                               (uint64_t)ldq, kBoxCols / 2, kUnit, CU_TENSOR_MAP_SWIZZLE_128B);
    if (reinterpret_cast<uintptr_t>(scale) % 16 == 0 && lds % 4 == 0)
        a.tma_s = make_tmap_2d(&a.s_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, scale, (uint64_t)N, (uint64_t)groups,
                               (uint64_t)lds, kBoxCols, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const int slots = (int)M * (sizeof(T) == 4 ? 2 : 1);
        const T *x = static_cast<const T *>(X);
        if (slots <= 8) return launch_matvec<T, 1>(a, x, ldx, ws, st);
        if (slots <= 16) return launch_matvec<T, 2>(a, x, ldx, ws, st);
        if constexpr (sizeof(T) == 4) return launch_matvec<T, 4>(a, x, ldx, ws, st);
        return cudaErrorInvalidValue;
    });
}

}  // namespace bsg

// wcols.cu -- products of any number of tokens with a weight stored as int8 codes and
// one scale per column: each token quantized by itself, exact sums of code products.
//
// "The verified INT8 units", steps 1 to 3, on a weight that keeps its codes: step 1 for
// the tokens alone, into the f16 operand that the tensor-core GEMM reads (every code is
// exact in f16), the weight's codes laid out as the other operand, then the GEMM.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <string.h>

#include "bsg_internal.h"
#include "bsg_ptx.cuh"
#include "serve.cuh"
#include "wcols_runs.h"

namespace bsg {
namespace {

// Step 1 of a token, THREADS each: its values in registers between the maximum and the codes
// (up to 32 a thread; longer rows are read again).  VEC: values of 16 bytes, where every row
// begins on 16; 1 otherwise.
constexpr int kTokenKept = 32;
template <typename T, int VEC, int THREADS>
__global__ void __launch_bounds__(THREADS < 128 ? 128 : THREADS)
    wcols_tokens_kernel(const T *__restrict__ X, int64_t ldx, int64_t M, int K, int ldk, __half *__restrict__ op,
                        float *__restrict__ scale, uint4 *__restrict__ zero, int64_t zeros,
                        int32_t *dstatus) {
    constexpr int kBlock = THREADS < 128 ? 128 : THREADS;
    __shared__ uint32_t red[THREADS / 32];
    const int64_t row = (int64_t)blockIdx.x * (kBlock / THREADS) + threadIdx.x / THREADS;
    const int tid = threadIdx.x % THREADS;
    griddep_launch_dependents();
    // what the next launch adds into
    for (int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x; i < zeros; i += (int64_t)gridDim.x * kBlock)
        zero[i] = make_uint4(0, 0, 0, 0);
    if (row >= M) return;
    const T *x = X + row * ldx;
    constexpr int kPer = kTokenKept / VEC, kStep = THREADS * VEC;
    struct alignas(VEC * sizeof(T)) Piece {
        T v[VEC];
    };
    Piece piece[kPer];
    uint32_t m = 0;  // the largest |x|, as bits: Inf and NaN are the largest of all
    auto read = [&](int k, Piece &p) {
        if (VEC > 1 && k + VEC <= K) {
            p = *reinterpret_cast<const Piece *>(x + k);
        } else {
#pragma unroll
            for (int u = 0; u < VEC; ++u) p.v[u] = k + u < K ? x[k + u] : from_f32<T>(0.0f);
        }
    };
    auto largest = [&](const Piece &p) {
#pragma unroll
        for (int u = 0; u < VEC; ++u) m = max(m, __float_as_uint(to_f32(p.v[u])) & 0x7fffffffu);
    };
    const int k0 = tid * VEC;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (i * kStep < K) read(k0 + i * kStep, piece[i]);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (i * kStep < K) largest(piece[i]);
    for (int k = k0 + kPer * kStep; k < K; k += kStep) {
        Piece p;
        read(k, p);
        largest(p);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (THREADS > 32) {
        if (tid % 32 == 0) red[tid / 32] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) m = max(m, red[i]);
    }
    // the unit's quotients, whose f32 divisions equal the f64 ones rounded
    const float s = fmaxf(__fdiv_rn(__uint_as_float(m), 127.0f), 1e-8f), inv = __fdiv_rn(1.0f, s);
    // A row with Inf or NaN has codes of 0 and no number for its scale: codes that are none (a NaN's
    // scale is the least one) would overflow its sums, which share words with another token's.
    const bool finite = m < 0x7f800000u;
    auto write = [&](int k, const Piece &p) {
        __half h[VEC];
#pragma unroll
        for (int u = 0; u < VEC; ++u) {  // the unit's code: floors below 2^23 are exact in f32
            const float c = finite ? floorf(__fadd_rn(__fmul_rn(to_f32(p.v[u]), inv), 0.5f)) : 0.0f;
            h[u] = __float2half_rn(c);
        }
        if (k < ldk) {  // (a whole number of pieces)
            if constexpr (VEC == 8)
                *reinterpret_cast<uint4 *>(op + row * ldk + k) = *reinterpret_cast<const uint4 *>(h);
            else if constexpr (VEC == 4)
                *reinterpret_cast<uint2 *>(op + row * ldk + k) = *reinterpret_cast<const uint2 *>(h);
            else
                op[row * ldk + k] = h[0];
        }
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (i * kStep < ldk) {
            if (i * kStep >= K) read(K, piece[i]);  // zeros past the end
            write(k0 + i * kStep, piece[i]);
        }
    for (int k = k0 + kPer * kStep; k < ldk; k += kStep) {
        Piece p;
        read(k, p);
        write(k, p);
    }
    if (tid == 0) {
        scale[row] = finite ? s : __uint_as_float(0x7fffffffu);
        if (!finite) set_status(dstatus, BSG_DSTATUS_NONFINITE);
    }
}

template <typename T, int VEC, int THREADS>
cudaError_t launch_tokens_as(const T *X, int64_t ldx, int64_t M, int K, int ldk, __half *op, float *scale, uint4 *zero,
                             int64_t zeros, int32_t *dstatus, cudaStream_t st) {
    // a CTA to a token or four, and some more where there is much to clear
    constexpr int kBlock = THREADS < 128 ? 128 : THREADS, kRowsOf = kBlock / THREADS;
    int64_t clear = zeros / (4 * kBlock), ctas = (M + kRowsOf - 1) / kRowsOf;
    clear = clear < 1024 ? clear : 1024;
    if (ctas < clear) ctas = clear;
    wcols_tokens_kernel<T, VEC, THREADS><<<(unsigned)ctas, kBlock, 0, st>>>(X, ldx, M, K, ldk, op, scale, zero, zeros, dstatus);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_tokens(const T *X, int64_t ldx, int64_t M, int K, int ldk, __half *op, float *scale, uint4 *zero,
                          int64_t zeros, int32_t *dstatus, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    const bool aligned = (reinterpret_cast<uintptr_t>(X) | (uintptr_t)(ldx * (int64_t)sizeof(T))) % 16 == 0;
    // many rows: as few threads as keep one (8192 rows of 768 bf16: 11 us by 128 threads, 8 by 32);
    // few: as many as make it quick
    if (M >= 512 && K <= 32 * kTokenKept)
        return aligned ? launch_tokens_as<T, VEC, 32>(X, ldx, M, K, ldk, op, scale, zero, zeros, dstatus, st)
                       : launch_tokens_as<T, 1, 32>(X, ldx, M, K, ldk, op, scale, zero, zeros, dstatus, st);
    if (K <= (M >= 512 ? 128 * kTokenKept : 1024))
        return aligned ? launch_tokens_as<T, VEC, 128>(X, ldx, M, K, ldk, op, scale, zero, zeros, dstatus, st)
                       : launch_tokens_as<T, 1, 128>(X, ldx, M, K, ldk, op, scale, zero, zeros, dstatus, st);
    if (M >= 512 && K <= 256 * kTokenKept)
        return aligned ? launch_tokens_as<T, VEC, 256>(X, ldx, M, K, ldk, op, scale, zero, zeros, dstatus, st)
                       : launch_tokens_as<T, 1, 256>(X, ldx, M, K, ldk, op, scale, zero, zeros, dstatus, st);
    return aligned ? launch_tokens_as<T, VEC, 512>(X, ldx, M, K, ldk, op, scale, zero, zeros, dstatus, st)
                   : launch_tokens_as<T, 1, 512>(X, ldx, M, K, ldk, op, scale, zero, zeros, dstatus, st);
}

// ---- a few tokens: the weight's codes turned into operands on their way ---------
//
// kFewTokens tokens at a time (more: each block of them on its own, the codes then from L2).
// D[column][token] += W^T X^T with the weight as the A operand, 128 columns as its rows: W lies k
// by k, columns side by side, which is A's "MN-major" form, so codes become f16 where they are,
// without a transposition.  All k-blocks (128 x 128 codes) of
// all column tiles form one list that the CTAs share in equal runs; a run ends a tile's sums
// where it ends, and what is not a whole tile is added up in L2, in integers, so that the order
// does not matter; the last to add writes Y.  Sums are exact: f32 sums of at most 1024
// products, then int32.
//
// Roles: warps 0-7 take sums out of tensor memory, half of the tokens each four; warps 8-23,
// in two teams that take blocks in turn (a block's chain of waits, reads and writes is some
// 1300 clocks, twice what its MMAs take), fetch codes (cp.async into a ring of each warp's own,
// two of its blocks ahead) and turn them into operands; warp 24 issues the MMAs; warp 25
// sends for the tokens (TMA).  Blocks are this deep because every wait of the MMAs' warp costs
// some 100 clocks, its barrier complete or not.
//
// What bounds it: the tokens, which every CTA reads again from L2 for each of its blocks (as many
// bytes as the codes), and the chain of waits of the MMAs' warp; HBM is at 0.35 and the tensor
// cores at 0.13 of their rates.  61 tokens, 8192 x 12288 bf16 38 us (the floor's bytes 15), 8191 x
// 12289 51: rows that begin anywhere take nine pieces of 16 bytes where others take eight, from
// DRAM half as many bytes again (145 MB), and shifts.  (64 tokens' sums spill some 50 bytes a thread:
// 72 registers are what 832 threads leave.)  8192 x 8192 (floor 10): 16 tokens 22, 64
// tokens 29.  Measured and not kept: rings
// of three and four blocks, two stages of operands, four teams of 64-deep blocks.
constexpr int kFewTokens = 64;
constexpr int kSumWarps = 8, kCodeWarps = 16;
constexpr int kFewThreads = (kSumWarps + kCodeWarps + 2) * 32;
constexpr int kDeep = 128;     // k of a block
constexpr int kTeam = 8, kTeams = kCodeWarps / kTeam, kRows = kDeep / kTeam;  // rows of a block, to a warp
constexpr int kAhead = 2;      // blocks of a warp's ring
constexpr int kPitch = 144;    // of a row of codes in the ring: 128 and its overhang
constexpr int kRingBytes = kCodeWarps * kAhead * kRows * kPitch;
template <int kCols>
struct FewCfg {
    static constexpr int kWBytes = 128 * kDeep * 2, kXBytes = kCols * kDeep * 2, kStageBytes = kWBytes + kXBytes;
    static constexpr int kStages = kCols == 16 ? 4 : 3;
    static constexpr int kBytes = kStages * kStageBytes + kRingBytes + 256 + 1024;
    static_assert(kXBytes % 1024 == 0 && kBytes <= 232448, "shared memory");
};

struct FewArgs {
    const int8_t *Q;
    int64_t ldq;
    const float *token_scale, *scale;
    int M, Mp, N, K, blocks;  // Mp: tokens rounded up to 16; blocks of kDeep of K
    int64_t all;              // blocks of all column tiles
    int relu, dtype;
    void *Y;
    int64_t ldy;
    unsigned long long *sums;  // [block of tokens][tile][Mp / 2][128]: two tokens' sums in one word
    unsigned int *counts;      // [block of tokens][tile]: blocks added
    int32_t *dstatus;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void few_store(const FewArgs &a, int m, int n, int32_t s, float sw) {
    float y = __fmul_rn(__fmul_rn(__int2float_rn(s), __ldg(a.token_scale + m)), sw);
    if (a.relu) y = y > 0.0f ? y : 0.0f;
    const int64_t at = (int64_t)m * a.ldy + n;
    if (a.dtype == BSG_F32)
        static_cast<float *>(a.Y)[at] = y;
    else if (a.dtype == BSG_F16)
        static_cast<__half *>(a.Y)[at] = __float2half_rn(y);
    else
        static_cast<__nv_bfloat16 *>(a.Y)[at] = __float2bfloat16_rn(y);
}

// The barrier of the warps that take sums: whether `x` holds for every thread of theirs.
__device__ __forceinline__ bool sums_barrier_all(bool x) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)x), "n"(kSumWarps * 32)
        : "memory");
    return all != 0;
}

// A place in the list of blocks.
struct FewAt {
    int tile, block;
    __device__ __forceinline__ FewAt(const FewArgs &a, int64_t b) : tile((int)(b / a.blocks)), block((int)(b - (int64_t)tile * a.blocks)) {}
    __device__ __forceinline__ void next(const FewArgs &a) {
        if (++block == a.blocks) block = 0, ++tile;
    }
};

// ALIGNED: every row of codes begins on 16 bytes.  kCols: columns of sums in a thread's
// registers (tokens, rounded up).
template <int kCols, bool ALIGNED>
__global__ void __launch_bounds__(kFewThreads, 1)
    wcols_few_kernel(const __grid_constant__ FewArgs a, const __grid_constant__ CUtensorMap tokens) {
    using C = FewCfg<kCols>;
    constexpr int kStages = C::kStages, kWBytes = C::kWBytes, kStageBytes = C::kStageBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    uint8_t *ring_s = smem + kStages * kStageBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring_s + kRingBytes);
    uint64_t *full = bars, *empty = bars + kStages, *sum_full = bars + 2 * kStages, *sum_empty = sum_full + 2;
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(sum_empty + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_ptr + 1);
    volatile int *last_s = reinterpret_cast<volatile int *>(tmem_ptr + 2);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    // this CTA's run of the list
    const int64_t b0 = a.all * blockIdx.x / gridDim.x, b1 = a.all * (blockIdx.x + 1) / gridDim.x;
    const int n_blocks = (int)(b1 - b0);
    const int m0 = blockIdx.y * kFewTokens, rows = min(a.M - m0, kFewTokens);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], kTeam + 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sum_full[s], 1);
            mbar_init(&sum_empty[s], kSumWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
        fence_async_shared();
    }
    constexpr int kMmaWarp = kSumWarps + kCodeWarps;
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_ptr, 2 * kFewTokens);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_ptr;
    auto all_wait = [&](uint64_t *bar, uint32_t parity) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
        if (!ok && lane == 0) {
            *abort_flag = 1;
            set_status(a.dstatus, BSG_DSTATUS_TIMEOUT);
        }
        return ok;
    };
    // Blocks that one accumulator takes from block b on: to the end of the tile, of the run, or
    // of 1024 products.
    auto chunk_of = [&](int block, int left) { return min(min(a.blocks - block, kChunkK / kDeep), left); };

    if (warp > kMmaWarp) {
        // ---- tokens
        if (lane == 0) {
            prefetch_tmap(&tokens);
            griddep_wait();
            FewAt at(a, b0);
            for (int i = 0; i < n_blocks; ++i, at.next(a)) {
                const int stage = i % kStages;
                if (!mbar_wait(&empty[stage], (i / kStages & 1) ^ 1, abort_flag)) {
                    *abort_flag = 1;
                    break;
                }
                mbar_arrive_expect_tx(&full[stage], a.Mp * kDeep * 2);
                uint8_t *x = smem + stage * kStageBytes + kWBytes;
#pragma unroll
                for (int u = 0; u < kDeep / 64; ++u)  // (past the operand's end: zeros)
                    tma_load_2d(&tokens, &full[stage], x + u * (kCols * 128), at.block * kDeep + 64 * u, m0);
            }
            if (*abort_flag) {  // let the copies land
                const long long t0 = clock64();
                while (clock64() - t0 < 2000000) {
                }
            }
        }
    } else if (warp == kMmaWarp) {
        // ---- MMAs
        const uint32_t idesc = idesc_f16_f32(128, a.Mp) | kIdescAMn;
        const uint64_t w_desc = sdesc_mn128(smem_u32(smem), kDeep * 128), x_desc = sdesc_k128(smem_u32(smem) + kWBytes);
        const bool one = elect_one();
        bool ok = true;
        int block = FewAt(a, b0).block, stage = 0;
        uint32_t phase = 0;
#pragma unroll 1
        for (int i = 0, c = 0; i < n_blocks && ok; ++c) {
            const int n = chunk_of(block, n_blocks - i), buffer = c & 1;
            block = block + n == a.blocks ? 0 : block + n;
            if (!(ok = all_wait(&sum_empty[buffer], (c >> 1 & 1) ^ 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < n && ok; ++j, ++i) {
                if (!(ok = all_wait(&full[stage], phase))) break;
                tc_fence_after();
                const uint64_t wd = w_desc + stage * (kStageBytes / 16), xd = x_desc + stage * (kStageBytes / 16);
                if (one) {
#pragma unroll
                    for (int k = 0; k < kDeep / 16; ++k)
                        mma_f16_ss(tmem + buffer * kFewTokens, wd + k * 128, xd + k / 4 * (kCols * 8) + k % 4 * 2, idesc, j + k > 0);
                    mma_commit(&empty[stage]);
                    if (j == n - 1) mma_commit(&sum_full[buffer]);
                }
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
        }
        if (!ok && one) {  // wait until every MMA issued so far has finished
            mma_commit(&sum_full[0]);
            const long long t0 = clock64();
            while (clock64() - t0 < 2000000) {
            }
        }
        __syncwarp();
    } else if (warp >= kSumWarps) {
        // ---- codes: rows kRows w .. of every other block, 8 pieces of 16 columns each, and one
        // more where the row begins inside its first.  Rows kDeep apart begin alike.
        const int w = (warp - kSumWarps) % kTeam, team = (warp - kSumWarps) / kTeam;
        uint8_t *const own = ring_s + (warp - kSumWarps) * kAhead * kRows * kPitch;
        const uint32_t ring = smem_u32(own);
        FewAt ahead(a, b0);
        for (int i = 0; i < team; ++i) ahead.next(a);
        int in_ahead = 0;
        auto fetch = [&](int i) {
            if (i < n_blocks) {
                const int k0 = ahead.block * kDeep + kRows * w;
                const uint32_t dst = ring + in_ahead * (kRows * kPitch);
                const int64_t n0 = (int64_t)ahead.tile * 128;
                const int cols = (int)min((int64_t)128, a.N - n0);
                const int8_t *first = a.Q + n0 + k0 * a.ldq, *last = a.Q + n0 + (int64_t)(a.K - 1) * a.ldq;
                for (int u = 0; u < kTeams; ++u) ahead.next(a);
                auto piece = [&](int row, int c) {
                    // rows past K repeat the last: the tokens are 0 there
                    const int8_t *p = k0 + row < a.K ? first + row * a.ldq : last;
                    const uintptr_t from = (reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15) + 16 * c;
                    // only pieces that hold some of the row's columns
                    if (from < reinterpret_cast<uintptr_t>(p) + cols)
                        copy16(dst + row * kPitch + 16 * c, reinterpret_cast<const void *>(from));
                };
#pragma unroll
                for (int u = 0; u < kRows / 4; ++u) piece(4 * u + lane / 8, lane % 8);
                if (!ALIGNED && lane < kRows) piece(lane, 8);
            }
            in_ahead = in_ahead + 1 == kAhead ? 0 : in_ahead + 1;
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // The lane's pieces: eight lanes store to two rows of either parity, which spreads them
        // over all banks.
        const int row0 = lane / 16 * 2 + lane % 8 / 4, c = lane % 4 + lane / 8 % 2 * 4;
        uint32_t shift[kRows / 4];  // where the row begins in its first 16 bytes
#pragma unroll
        for (int u = 0; u < kRows / 4; ++u)
            shift[u] = ALIGNED ? 0 : (uint32_t)(reinterpret_cast<uintptr_t>(a.Q) + (uint64_t)(kRows * w + row0 + 4 * u) * a.ldq) & 15;
#pragma unroll 1
        for (int i = 0; i < kAhead; ++i) fetch(team + i * kTeams);
        int stage = team % kStages, in_ring = 0;
        uint32_t phase = (team / kStages & 1) ^ 1;
#pragma unroll 1
        for (int i = team; i < n_blocks; i += kTeams) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            __syncwarp();
            const uint8_t *src = own + in_ring * (kRows * kPitch) + row0 * kPitch + 16 * c;
            uint4 x[kRows / 4], y[kRows / 4];
#pragma unroll
            for (int u = 0; u < kRows / 4; ++u) {
                x[u] = *reinterpret_cast<const uint4 *>(src + 4 * u * kPitch);
                if (!ALIGNED) y[u] = *reinterpret_cast<const uint4 *>(src + 4 * u * kPitch + 16);
            }
            __syncwarp();  // every lane has what the next copies replace
            fetch(i + kAhead * kTeams);
            if (!all_wait(&empty[stage], phase)) break;
            uint8_t *line = smem + stage * kStageBytes + c / 4 * (kDeep * 128) + (kRows * w + row0) * 128;
#pragma unroll
            for (int u = 0; u < kRows / 4; ++u) {
                uint32_t v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                if (!ALIGNED) {
                    uint32_t t[8] = {x[u].x, x[u].y, x[u].z, x[u].w, y[u].x, y[u].y, y[u].z, y[u].w};
#pragma unroll
                    for (int q = 0; q < 6; ++q) t[q] = shift[u] & 8 ? t[q + 2] : t[q];
#pragma unroll
                    for (int q = 0; q < 5; ++q) t[q] = shift[u] & 4 ? t[q + 1] : t[q];
                    const uint32_t sel = 0x3210 + (shift[u] & 3) * 0x1111;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = __byte_perm(t[q], t[q + 1], sel);
                }
                uint32_t h[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {  // code + 128, as f16 1024 + that, less 1152
                    const uint32_t z = v[q] ^ 0x80808080u, bias = 0x64806480u;
                    const uint32_t lo = __byte_perm(z, 0x64646464u, 0x4140), hi = __byte_perm(z, 0x64646464u, 0x4342);
                    const __half2 l = __hsub2(*reinterpret_cast<const __half2 *>(&lo), *reinterpret_cast<const __half2 *>(&bias));
                    const __half2 g = __hsub2(*reinterpret_cast<const __half2 *>(&hi), *reinterpret_cast<const __half2 *>(&bias));
                    h[2 * q] = *reinterpret_cast<const uint32_t *>(&l);
                    h[2 * q + 1] = *reinterpret_cast<const uint32_t *>(&g);
                }
                const int at = c % 4 * 2, row = row0 + 4 * u;
                *reinterpret_cast<uint4 *>(line + 4 * u * 128 + ((at ^ row % 8) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(line + 4 * u * 128 + ((at + 1 ^ row % 8) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[stage]);
            stage += kTeams;
            if (stage >= kStages) stage -= kStages, phase ^= 1;
            in_ring = in_ring + 1 == kAhead ? 0 : in_ring + 1;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
        // ---- sums: a column and half of the tokens (from t0 on) to a thread
        constexpr int kMine = kCols / 2;
        const int t0 = warp / 4 * kMine, quad = warp % 4, n_of = quad * 32 + lane;
        const uint32_t sums_at = tmem + ((uint32_t)(quad * 32) << 16) + t0;
        int32_t s[kMine];
        bool ok = true;
        int c = 0;
        FewAt at(a, b0);
        int left = n_blocks;
#pragma unroll 1
        while (left > 0 && ok) {
            // the run's part of a tile
            const int tile = at.tile, part = min(a.blocks - at.block, left);
#pragma unroll
            for (int m = 0; m < kMine; ++m) s[m] = 0;
#pragma unroll 1
            for (int done = 0; done < part; ++c) {
                done += chunk_of(at.block + done, left - done);
                // One warp polls, the others are out of the way of those that work, and its answer is
                // what the barrier gives to all: any other role may give up between two threads' reads
                // of the flag, and those that went on would wait at the next barrier for those that left.
                bool came = true;
                if (warp == 0) came = all_wait(&sum_full[c & 1], c >> 1 & 1);
                if (!(ok = sums_barrier_all(came))) break;
                tc_fence_after();
#pragma unroll
                for (int m = 0; m < kMine; m += 8) {
                    if (t0 + m >= a.Mp) break;
                    uint32_t x[8];
                    tmem_ld8(sums_at + (c & 1) * kFewTokens + m, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int u = 0; u < 8; ++u) s[m + u] += __float2int_rn(__uint_as_float(x[u]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sum_empty[c & 1]);
            }
            at.block = 0, ++at.tile;
            left -= part;
            if (!ok) break;
            const int64_t n = (int64_t)tile * 128 + n_of, tiles = (a.N + 127) / 128, of = blockIdx.y * tiles + tile;
            const float sw = n < a.N ? __ldg(a.scale + n) : 0.0f;
            griddep_wait();  // the tokens' scales, and zeros to add to
            if (part == a.blocks) {
                if (n < a.N)
#pragma unroll
                    for (int m = 0; m < kMine; ++m)
                        if (t0 + m < rows) few_store(a, m0 + t0 + m, (int)n, s[m], sw);
                continue;
            }
            unsigned long long *sums = a.sums + (of * (a.Mp / 2) + t0 / 2) * 128 + n_of;
#pragma unroll
            for (int m = 0; m < kMine; m += 2)
                // the lower sum's borrow comes out of the upper one, and goes back when they are read
                if (t0 + m < rows)
                    atomicAdd(sums + m / 2 * 128, (unsigned long long)((long long)s[m] + ((long long)s[m + 1] << 32)));
            __threadfence();
            asm volatile("bar.sync 1, %0;" ::"n"(kSumWarps * 32) : "memory");
            if (threadIdx.x == 0)
                *last_s = atomicAdd(a.counts + of, (unsigned)part) + (unsigned)part == (unsigned)a.blocks;
            asm volatile("bar.sync 1, %0;" ::"n"(kSumWarps * 32) : "memory");
            if (!*last_s) continue;
            __threadfence();
#pragma unroll
            for (int m = 0; m < kMine; m += 2)
                if (t0 + m < rows) {
                    const long long v = (long long)__ldcg(sums + m / 2 * 128);
                    s[m] = (int32_t)v, s[m + 1] = (int32_t)((v - s[m]) >> 32);
                }
            if (n < a.N)
#pragma unroll
                for (int m = 0; m < kMine; ++m)
                    if (t0 + m < rows) few_store(a, m0 + t0 + m, (int)n, s[m], sw);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * kFewTokens);
    }
}

template <int kCols, bool ALIGNED>
cudaError_t launch_few_as(const FewArgs &a, const CUtensorMap &map, cudaStream_t st) {
    static bool set[64] = {false};  // this kernel's shared memory, on each device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !set[dev]) {
        e = cudaFuncSetAttribute(wcols_few_kernel<kCols, ALIGNED>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewCfg<kCols>::kBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) set[dev] = true;
    }
    const int64_t sms = device_sm_count();
    cudaLaunchConfig_t cfg = {};
    const int64_t blocks = (a.M + kFewTokens - 1) / kFewTokens;
    cfg.gridDim = dim3((unsigned)wcols_runs(a.all, blocks, sms), (unsigned)blocks);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = FewCfg<kCols>::kBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, wcols_few_kernel<kCols, ALIGNED>, a, map);
}

cudaError_t launch_few(const FewArgs &a, const CUtensorMap &map, cudaStream_t st) {
    const bool aligned = (reinterpret_cast<uintptr_t>(a.Q) | (uintptr_t)a.ldq) % 16 == 0;
    if (a.Mp <= 16) return aligned ? launch_few_as<16, true>(a, map, st) : launch_few_as<16, false>(a, map, st);
    return aligned ? launch_few_as<64, true>(a, map, st) : launch_few_as<64, false>(a, map, st);
}

// Where the weight's codes are turned into operands on their way, for each 64 tokens again, rather
// than once into an operand in memory (5 bytes moved for each code) for the unit's GEMM: the
// latter's chain of k-blocks is what short columns have little of.  Both in us, bf16:
//   K x N         tokens: on the way, operand
//   768 x 2304    16: 7.9, 10.2    32: 12.1, 10.2   128: 18.4, 12.6
//   768 x 50304   16: 17, 51       64: 29, 49       256: 78, 52
//   2048 x 8192   16: 14, 27       64: 20, 21       128: 23, 22      256: 32, 24
//   2304 x 2304                    64: 18, 19       128: 19, 19      192: 26, 21
//   2600 x 4096                                     128: 22, 22      160: 24, 23      256: 27, 24
//   3500 x 8192                                                      160: 38, 42      256: 45, 43
//   4096 x 4096                    64: 21, 29       128: 23, 29      192: 32, 31      256: 31, 31
//   4096 x 12288                                                     160: 49, 71      256: 61, 72
//   8192 x 8192                    64: 29, 90       128: 45, 91      192: 60, 94      256: 71, 96     320: 156, 100
//   16384 x 4096                                    128: 43, 117     192: 60, 120     256: 71, 121
bool few_form(int64_t M, int64_t N, int64_t K) {
    return M <= 16 || (M <= 64 && (K > 1024 || N * K > 1 << 23)) || (M <= 128 && K > 2560) || (M <= 256 && K > 3200);
}

// ---- a token or a few and a small weight: one launch ------------------------------
//
// A CTA takes 16 columns and all of K, so that most of the card has a part of a small
// weight: a thread a row of codes in every kSmallThreads (sent for first), times the tokens'
// codes, which every CTA makes for itself; int32 sums over the threads.  What bounds it is a
// launch, one round of loads and a block's few barriers.
constexpr int kSmallThreads = 256, kSmallTokens = 4, kSmallK = 2048;

template <typename T, int kTokens>
__global__ void __launch_bounds__(kSmallThreads)
    wcols_small_kernel(const T *__restrict__ X, int64_t ldx, const int8_t *__restrict__ Q, int64_t ldq,
                       const float *__restrict__ scale, int M, int N, int K, int relu, T *__restrict__ Y,
                       int64_t ldy, int32_t *dstatus) {
    constexpr int kWarps = kSmallThreads / 32, kPer = kSmallK / kSmallThreads;
    __shared__ int32_t sums[kWarps][kTokens][16];
    __shared__ uint32_t red[kTokens][kWarps];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int cols = min(16, N - (int)n0);
    uint32_t w[kPer][4];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int k = tid + i * kSmallThreads;
        if (i * kSmallThreads >= K) break;
        const int8_t *row = Q + (int64_t)min(k, K - 1) * ldq + n0;
        if (reinterpret_cast<uintptr_t>(row) % 16 == 0 && cols == 16) {
            const uint4 v = *reinterpret_cast<const uint4 *>(row);
            w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
        } else {
            // words that hold some of the row's columns, put together
            const uintptr_t p = reinterpret_cast<uintptr_t>(row), end = p + cols;
            const uint32_t *at = reinterpret_cast<const uint32_t *>(p & ~(uintptr_t)3);
            uint32_t x[5];
#pragma unroll
            for (int u = 0; u < 5; ++u) x[u] = reinterpret_cast<uintptr_t>(at + u) < end ? __ldg(at + u) : 0u;
#pragma unroll
            for (int u = 0; u < 4; ++u) w[i][u] = __funnelshift_r(x[u], x[u + 1], 8 * (uint32_t)(p & 3));
        }
    }
    float x[kTokens][kPer];
    uint32_t most[kTokens];  // the largest |x|, as bits
#pragma unroll
    for (int m = 0; m < kTokens; ++m) {
        most[m] = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int k = tid + i * kSmallThreads;
            x[m][i] = k < K && m < M ? to_f32(X[m * ldx + k]) : 0.0f;
            most[m] = max(most[m], __float_as_uint(x[m][i]) & 0x7fffffffu);
        }
        most[m] = __reduce_max_sync(0xffffffffu, most[m]);
        if (lane == 0) red[m][warp] = most[m];
    }
    __syncthreads();
    float token_scale[kTokens];
    int32_t s[kTokens][16];
#pragma unroll
    for (int m = 0; m < kTokens; ++m) {
#pragma unroll
        for (int i = 0; i < kWarps; ++i) most[m] = max(most[m], red[m][i]);
        token_scale[m] = fmaxf(__fdiv_rn(__uint_as_float(most[m]), 127.0f), 1e-8f);
        const float inv = __fdiv_rn(1.0f, token_scale[m]);
        if (blockIdx.x == 0 && tid == 0 && m < M && most[m] >= 0x7f800000u) set_status(dstatus, BSG_DSTATUS_NONFINITE);
#pragma unroll
        for (int c = 0; c < 16; ++c) s[m][c] = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (i * kSmallThreads >= K) break;
            const int q = (int)(int8_t)unit_code(x[m][i], inv);  // 0 past K
#pragma unroll
            for (int c = 0; c < 16; ++c) s[m][c] += q * (int)(int8_t)(w[i][c / 4] >> (8 * (c % 4)));
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            const int32_t all = __reduce_add_sync(0xffffffffu, s[m][c]);
            if (lane == c) sums[warp][m][c] = all;
        }
    }
    __syncthreads();
    if (tid < 16 * kTokens) {
        const int m = tid / 16, c = tid % 16;
        int32_t all = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) all += sums[i][m][c];
        if (m < M && c < cols) {
            float sm = token_scale[0];
#pragma unroll
            for (int u = 1; u < kTokens; ++u) sm = m == u ? token_scale[u] : sm;
            float y = __fmul_rn(__fmul_rn(__int2float_rn(all), sm), __ldg(scale + n0 + c));
            if (relu) y = y > 0.0f ? y : 0.0f;
            Y[m * ldy + n0 + c] = from_f32<T>(y);
        }
    }
}

// Where one launch beats two: few tokens, K in a thread's registers, and no more than 2^23
// products, which the threads make one by one (768 x 2304: 1 token 3.1 us on the device, 4 tokens
// 6.2, against 7.1 and 7.3 by the form above; 2048 x 2048: 1 token 4.0, 4 tokens 10.0 against 9.0).
bool small_form(int64_t M, int64_t N, int64_t K) {
    return M <= kSmallTokens && K <= kSmallK && N <= (8 << 20) / (K * M) && N <= (4 << 20) / K;
}

template <typename T>
cudaError_t launch_small(const T *X, int64_t ldx, const int8_t *Q, int64_t ldq, const float *scale, int M, int N, int K,
                         int relu, T *Y, int64_t ldy, int32_t *dstatus, cudaStream_t st) {
    const unsigned grid = (unsigned)((N + 15) / 16);
    if (M == 1)
        wcols_small_kernel<T, 1><<<grid, kSmallThreads, 0, st>>>(X, ldx, Q, ldq, scale, M, N, K, relu, Y, ldy, dstatus);
    else if (M == 2)
        wcols_small_kernel<T, 2><<<grid, kSmallThreads, 0, st>>>(X, ldx, Q, ldq, scale, M, N, K, relu, Y, ldy, dstatus);
    else
        wcols_small_kernel<T, 4><<<grid, kSmallThreads, 0, st>>>(X, ldx, Q, ldq, scale, M, N, K, relu, Y, ldy, dstatus);
    count_launches(1);
    return cudaGetLastError();
}

int few_rows(int64_t M) { return M > kFewTokens ? kFewTokens : (int)round_up(M, 16); }

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// The workspace: the tokens' operand and scales; then sums and counts, or the weight's operand,
// its scales and the GEMM's tile counter.
struct Layout {
    int64_t ldk, zeros;  // zeros: 16-byte pieces from `zero` on that the tokens' launch clears
    size_t token_scale, zero, counts, weights, col_scale, bytes;
};
Layout layout(int64_t M, int64_t N, int64_t K) {
    Layout l = {};
    l.ldk = operand_ld(K);
    l.token_scale = up256((size_t)M * l.ldk * 2);
    l.zero = l.token_scale + up256((size_t)round_up(M, kBM) * 4);
    if (few_form(M, N, K)) {
        const size_t tiles = (size_t)(N + 127) / 128, blocks = (size_t)(M + kFewTokens - 1) / kFewTokens;
        l.counts = l.zero + blocks * tiles * few_rows(M) * 128 * 4;
        l.bytes = l.counts + up256(blocks * tiles * 4);
        l.zeros = (int64_t)(l.bytes - l.zero) / 16;
    } else {
        l.zeros = 1;  // the tile counter
        l.weights = l.zero + 256;
        l.col_scale = l.weights + up256((size_t)N * l.ldk * 2);
        l.bytes = l.col_scale + up256((size_t)(round_up(N, kBN) + kBN) * 4);
    }
    return l;
}

}  // namespace

size_t wcols_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    return small_form(M, N, K) ? 0 : layout(M, N, K).bytes;
}

cudaError_t launch_wcols_matmul(const void *X, int dtype, int64_t ldx, const int8_t *Q, int64_t ldq,
                                const float *scale, int64_t M, int64_t N, int64_t K, int relu,
                                void *Y, int64_t ldy, void *ws, int32_t *dstatus, cudaStream_t st) {
    if (small_form(M, N, K))
        return with_dtype(dtype, [&](auto t) {
            using T = decltype(t);
            return launch_small(static_cast<const T *>(X), ldx, Q, ldq, scale, (int)M, (int)N, (int)K, relu,
                                static_cast<T *>(Y), ldy, dstatus, st);
        });
    const Layout l = layout(M, N, K);
    uint8_t *w = static_cast<uint8_t *>(ws);
    __half *aop = reinterpret_cast<__half *>(w);
    float *sa = reinterpret_cast<float *>(w + l.token_scale);
    cudaError_t e = with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return launch_tokens(static_cast<const T *>(X), ldx, M, (int)K, (int)l.ldk, aop, sa,
                             reinterpret_cast<uint4 *>(w + l.zero), l.zeros, dstatus, st);
    });
    if (e != cudaSuccess) return e;
    if (few_form(M, N, K)) {
        FewArgs a{Q, ldq, sa, scale, (int)M, few_rows(M), (int)N, (int)K, (int)((K + kDeep - 1) / kDeep), 0, relu, dtype,
                  Y, ldy, reinterpret_cast<unsigned long long *>(w + l.zero), reinterpret_cast<unsigned int *>(w + l.counts), dstatus};
        a.all = (N + 127) / 128 * a.blocks;
        CUtensorMap map;
        memset(&map, 0, sizeof(map));
        if (!make_tmap_2d(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, aop, (uint64_t)l.ldk, (uint64_t)M, (uint64_t)l.ldk,
                          64, (uint32_t)a.Mp))
            return cudaErrorInvalidValue;
        return launch_few(a, map, st);
    }
    __half *bop = reinterpret_cast<__half *>(w + l.weights);
    float *sb = reinterpret_cast<float *>(w + l.col_scale);
    // (the GEMM reads whole tiles of scales)
    e = launch_i8_cols_to_half(Q, K, N, ldq, bop, l.ldk, st, scale, sb, true);
    if (e != cudaSuccess) return e;
    return launch_gemm_tc(aop, bop, M, N, K, sa, sb, relu, dtype == BSG_F32 ? 0 : dtype == BSG_F16 ? 2 : 3, Y,
                          ldy, dstatus, reinterpret_cast<unsigned int *>(w + l.zero), st);
}

}  // namespace bsg

// kv8_tiles.cuh -- attention of many query rows over the int8 cache on the tcgen05 tensor
// cores: prompts through a window with sinks, and the prefix that a batch shares.
//
// A CTA takes up to kM x 128 rows (queries of one key/value head: the heads of its group
// times tokens) and walks the tiles of kN positions that some of them see:
//   S = Q K^T          128 x kN, in tensor memory, one place that the groups of 128 rows use in turn
//   p' = 2^(S ks mul + log2 vs - ref)   a thread to a row, in f16, half a tile at a time
//   O += P V           P (f32, f16: two f16 parts, 22 bits; bf16: one, 11) read from tensor memory, O stays there
// with ks, vs the page's scales (one for each 16 positions of a tile), mul the row's
// multiplier, ref the row's running reference, which follows the maximum only when that is
// above 2^15 (what f16 holds) and makes it 2^9 then: O is rescaled where it lies, a few times
// in a row's life.  Sums of p = p' / vs in f32.
// bf16's one part: each p is off by 2^-11 of itself at most, an output by 2^-11 of sum p |v|, where its own
// rounding is 2^-8 of itself; two prompts of 16384 through a window of 4096 and 64 sequences
// behind 32768 shared tokens are 1.669e-3 off 64 bits (norms), 1.659e-3 with two parts (and with f32
// throughout), which take 2.19 ms in place of 1.54 and 72 us in place of 60.  Where values cancel, an output smaller than sum p |v| / 8 shows it: such sums want f16 or f32.
// Codes are exact in f16, so K and V are too; queries are relative to a power of two near
// their row's largest, f32's as two f16 parts (22 bits).
//
// Roles, four warps each, the registers split among them (setmaxnreg):
//   0-3, 4-7   softmax, a row to a thread (4-7: the second 128 rows), the row's scores of a
//              tile in registers;
//   8-11       codes into f16 operands, in a ring of shared memory that K and V tiles take
//              in turn; each tile's loads are sent two fills ahead;
//   12, 14     issue the MMAs of a group of rows each: S of a tile as soon as the one before
//              it has been read into registers, P V of each half tile as it comes;
//   13         finds where the tiles' pages lie, and their scales, some tiles at a time.
//
// What bounds it: the chain of a tile (S, its way into registers, maximum, exponentials, P, O) that
// the two groups of rows take in turn; no one pipe (a prompt of 4096 through a window of 2048:
// tensor 0.39 of the active cycles, ALU 0.40, XU 0.20).  Two prompts of up to 16384, window 4096,
// 32/8 heads of 128, bf16: 1.54 ms, 0.56 of the products' floor; 64 rows behind 131071 shared
// positions, 8 heads of 128, f16 (two parts of P): 167 us of the call's 185, tensor 0.55; ragged
// prompts of up to 1021, 5 heads of 64, f32: 46 us, three rounds of CTAs of five tiles, whose start
// and end take some 10 of each 16 us.  Prompts of 16384 without a window: bf16 3.4 ms, f16 4.9, f32 7.9;
// f16's and f32's softmax threads spill 40 to 200 bytes each (-Xptxas -v), bf16's 20 to 40.
// Why so: S in registers and a split of these by role 3.6 -> 2.06 ms (S read from tensor memory
// in pieces spilled or came twice); MMAs issued by a converged warp, descriptors in uniform
// registers 1.91; P apart from S, so that the next S does not wait for P V, by halves, so that P V
// begins early, 1.76; a warp to issue for each group of rows, barriers and maxima side by side
// 1.54.  P in S's place without a pass for the maximum (sums above 2^15 tell) took 1.87, P by
// quarters 188 us where halves take 175 (f16).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bsg_internal.h"
#include "bsg_ptx.cuh"
#include "kv8_more.h"
#include "kv8_seen.cuh"
#include "serve.cuh"

namespace bsg {
namespace {

struct TileArgs {
    bsg_kv8_cache c;
    const int32_t *table;      // of the sequences, or the prefix's pages
    int64_t table_ld;
    const int32_t *lens, *counts;  // prefix: lens is the prefix's length
    bsg_tokens q, out;
    int tokens, heads, window, sinks;
    int rows, row_blocks;      // of a key/value head (and sequence); CTAs that they take
    int64_t groups;            // key/value heads (of all sequences)
    int splits, later;         // chunks of a CTA's tiles; 1: what is found is joined later
    float scale;
    float *lse;
    float *part_o;             // [sequence][head][row][split][D]: outputs before the division by the sum,
    float2 *part_ml;           // and the reference and sum (0: nothing seen); where splits > 1 or later
    int32_t *dstatus;
};

constexpr float kTileTop = 9.0f, kTileMost = 15.0f;  // exponents of a new reference's largest p', and of any
constexpr int kAtSlots = 4;
constexpr int kWaitTries = 1 << 23;  // of some tens of clocks at least: far above any wait here

__device__ __forceinline__ float tile_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x f + off for two values; f and off twice in a pair each.
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t f, uint64_t off) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(f), "l"(off));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[32]) { tmem_st32(at, r); }
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[16]) { tmem_st16(at, r); }

// The lowest n bits.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

template <int D, int kQParts, int kPParts, bool kLong>
struct TileCfg {
    static constexpr int kM = D == 256 ? 1 : 2;
    static constexpr int kN = D == 256 ? 64 : 128;
    static constexpr int kBlocks = (D + 63) / 64;             // of 64 dims (128 bytes of f16)
    static constexpr int kQBytes = kBlocks * 128 * 128;       // one part of 128 rows
    static constexpr int kStageBytes = kBlocks * kN * 128;    // a K or V tile
    static constexpr int kRoom = 229376 - kM * kQParts * kQBytes;
    static constexpr int kStages = kRoom / kStageBytes >= 6 ? 6 : kRoom / kStageBytes == 5 ? 4 : kRoom / kStageBytes;
    static constexpr int kGroups = kN / 16;
    static constexpr int kOffStage = kM * kQParts * kQBytes;
    static constexpr int kOffAt = kOffStage + kStages * kStageBytes;
    static constexpr int kOffBar = kOffAt + kAtSlots * kGroups * 16;
    static constexpr int kBars = 2 * kStages + 2 * kAtSlots + 8 * kM;
    static constexpr int kUsed = kOffBar + kBars * 8 + 16;
    static constexpr int kBytes = (kUsed > 118000 ? kUsed : 118000) + 1024;  // one CTA on an SM (all its tensor memory)
    static_assert(kStages >= 2 && kBytes <= 232448, "shared memory");
    // Columns of tensor memory.  S in one place that the groups of rows use in turn, P's two
    // halves and O of each group; where that is more than there is (two parts of P, 96 or 128
    // dims), each group has a place for S, which its P takes afterwards.
    static constexpr int kPCols = kPParts * kN / 2;
    static constexpr bool kInPlace = kN + kM * (kPCols + D) > 512;
    static constexpr int kSStep = kInPlace ? kN : 0;                     // from one group's S to the next's
    static constexpr int kP0 = kInPlace ? 0 : kN, kPStep = kInPlace ? kN : kPCols;
    static constexpr int kO0 = kInPlace ? kM * kN : kN + kM * kPCols;
    static_assert(kO0 + kM * D <= 512 && kPCols <= kN, "tensor memory");
    // What the tensor cores add to an f32 sum is cut off below its last bit, not rounded: some 2^-24
    // of O is lost with each product of 16 positions, always towards 0; and the sum of p, of as many
    // terms, rounds the same way each time where they are alike.  Both are therefore added (rounded)
    // to a second set, which lies in local memory, every kFlush tiles and begun anew, but for the last
    // quarter as many more.  Off 64 bits on the mean, with equal scores and values of one sign: f32, 65536
    // positions, 1.2e-6 (the sum of p in one piece 1.7e-5); f16, 131072, 5e-5 (in one piece of 65536
    // 4.2e-4; its rounding 4.9e-4 at most); bf16, 524288, 2.5e-4 (3.7e-3; 3.9e-3).  Between runs of
    // tiles and not within the loop over them: prompts of 16384 without a window, f16 5.5 -> 4.9 ms, f32
    // 8.0 -> 7.9 (16 sequences of 16384 by 48 rows 421 -> 445 us).  In local memory a warp's second set
    // lies side by side; f32's in the outputs' rows took 11.2 ms there.
    static constexpr int kFlush = (kQParts == 2 ? 512 : kPParts == 2 ? 8192 : 32768) / kN;  // tiles
    static constexpr int kFlushMost = kFlush + kFlush / 4;
    static __device__ bool flush_at(int i, int tiles) {
        return kLong && i > 0 && i % kFlush == 0 && tiles - i > kFlush / 4;
    }
};

constexpr int kTileThreads = 512;
// Registers of a softmax, a converting and another thread; together no more than four
// times the 128 that the block is launched with.
constexpr int kSoftRegs = 176, kConvRegs = 112, kOtherRegs = 48;
static_assert(2 * kSoftRegs + kConvRegs + kOtherRegs <= 4 * 128, "register split");
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 16 bytes of codes, in the order of the program.
__device__ __forceinline__ uint4 load_codes(const int8_t *p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// PREFIX: rows are those of all sequences (rows = B x tokens x heads of a group), every one
// sees the positions below *lens; what a CTA finds is joined later.  The report of bad lengths
// is the first CTA's.
template <int D, int kQParts, int kPParts, bool PREFIX, bool kLong>
__global__ void __launch_bounds__(kTileThreads, 1)
    kv8_tiles_kernel(const __grid_constant__ TileArgs a) {
    using C = TileCfg<D, kQParts, kPParts, kLong>;
    constexpr int kM = C::kM, kN = C::kN, kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    // of a tile's groups of 16 positions: key scale, log2 of the value scale, its reciprocal,
    // and the place in the pool (in groups; unseen: exponents of -inf, any place)
    float4 *at_s = reinterpret_cast<float4 *>(smem + C::kOffAt);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *kv_full = bars, *kv_empty = bars + kStages, *at_full = bars + 2 * kStages;
    uint64_t *at_empty = at_full + kAtSlots, *s_empty = at_empty + kAtSlots, *s_full = s_empty + kM;
    uint64_t *o_full = s_full + kM, *p_full = o_full + kM, *p_empty = p_full + 2 * kM;  // [m][slot]
    uint64_t *q_full = p_empty + 2 * kM;
    constexpr int kHalf = kN / 2;  // P goes to the tensor cores by halves of a tile
    constexpr bool kInPlace = C::kInPlace;
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(bars + C::kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_ptr + 1);

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
    const unsigned block = blockIdx.x / (unsigned)a.groups, group = blockIdx.x - block * (unsigned)a.groups;
    const int b = (int)(group / (unsigned)a.c.heads), hk = (int)(group - (unsigned)b * a.c.heads), split = blockIdx.y;
    const int share = a.heads / a.c.heads, P = a.c.page_tokens;
    // later rows see more: they go first
    const int r0 = (a.row_blocks - 1 - (int)block) * (kM * 128);
    const int64_t most = a.table_ld * P;

    // The rows that are there, and what they see.
    int count = a.tokens, len;
    if (PREFIX) {
        len = __ldg(a.lens);
    } else {
        len = __ldg(a.lens + b);
        if (a.counts) count = __ldg(a.counts + b);
    }
    const bool report = tid == 0 && split == 0 && r0 == 0;
    if (len < 0 || len > most) {
        if (report) set_status(a.dstatus, BSG_DSTATUS_RANGE);
        len = len < 0 ? 0 : (int)most;
    }
    int rows = a.rows;  // of all CTAs
    if (!PREFIX && a.counts) {
        if (count < 0 || count > a.tokens) {
            if (report) set_status(a.dstatus, BSG_DSTATUS_RANGE);
            count = 0;
        }
        rows = count * share;
    }
    rows = min(rows - r0, kM * 128);
    if (rows <= 0) return;
    const int pos0 = PREFIX ? 0 : len - count;  // token 0's position
    const Seen seen = PREFIX ? seen_by<kN>(0, len - 1, 0, 0)
                             : seen_by<kN>(pos0 + r0 / share, pos0 + (r0 + rows - 1) / share, a.window, a.sinks);
    const int begin = (int)((int64_t)seen.tiles * split / a.splits);
    const int tiles = (int)((int64_t)seen.tiles * (split + 1) / a.splits) - begin;
    if (tiles == 0 && split > 0) {  // the join reads no output of such a chunk
        if (tid < rows)
            a.part_ml[(((int64_t)b * a.c.heads + hk) * a.rows + r0 + tid) * a.splits + split] = make_float2(0.0f, 0.0f);
        if (PREFIX) griddep_wait();
        return;
    }
    const int groups = rows > 128 ? kM : 1;  // of 128 rows
    auto position = [&](int i) { return seen.tile(begin + i) * kN; };  // of the CTA's tile i

    if (tid < C::kBars) {
        int count = 4;                                             // kv_full, s_empty, p_full, q_full: the warps of a role
        if (bars + tid >= kv_empty) count = groups;                // the MMAs' warps
        if (bars + tid >= at_full) count = 1;
        if (bars + tid >= at_empty) count = 4 + 4 * groups;        // the warps that read a slot
        if (bars + tid >= s_empty) count = 4;
        if (bars + tid >= s_full) count = 1;                       // and o_full: commits
        if (bars + tid >= p_full) count = 4;
        if (bars + tid >= p_empty) count = 1;
        if (bars + tid >= q_full) count = 4;
        mbar_init(bars + tid, count);
        fence_mbar_init();
    }
    if (tid == 0) *abort_flag = 0;
    constexpr int kMmaWarp = 12;
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_ptr, 512);
        tmem_relinquish();
    }
    griddep_launch_dependents();

    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // all 512 columns are this CTA's: they begin at column 0
    auto give_up = [&]() {
        *abort_flag = 1;
        set_status(a.dstatus, BSG_DSTATUS_TIMEOUT);
    };
    // a whole warp's wait
    auto all_wait = [&](uint64_t *bar, uint32_t parity) {
        bool ok = mbar_try_wait(bar, parity);
        // (some twenty copies of this: as little code as may be, for the instruction caches)
#pragma unroll 1
        for (int n = 0; !ok && n < kWaitTries && !*abort_flag; ++n) ok = mbar_try_wait(bar, parity);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) give_up();
        return ok;
    };

    if (warp >= 12) {
        fewer_registers<kOtherRegs>();
        const int m = (warp - kMmaWarp) / 2;  // of the MMAs' warps
        if (warp % 2 == 0 && m < groups && tiles > 0) {
            // ------------------------------------------------ MMA issuers
            // The whole warp goes along, so that descriptors stay in uniform registers (one
            // lane alone took 90 clocks to issue an MMA of 64); one lane issues.  A warp to
            // each group of rows: every wait costs some 100 clocks, its barrier complete or
            // not, and one warp's for both took longer than the MMAs.
            constexpr uint32_t kIdescS = idesc_f16_f32(128, kN), kIdescO = idesc_f16_f32(128, D) | kIdescBMn;
            const uint32_t stage0 = smem_u32(smem + C::kOffStage);
            const uint64_t q_desc = sdesc_k128(smem_u32(smem) + m * (kQParts * C::kQBytes)), k_desc = sdesc_k128(stage0);
            const uint64_t v_desc = sdesc_mn128(stage0, kN * 128);
            const int n = __reduce_max_sync(0xffffffffu, tiles);
            const bool two = __reduce_max_sync(0xffffffffu, groups) > 1;
            const bool one = elect_one();
            const uint32_t s_at = m * C::kSStep, o_at = C::kO0 + m * D;
            bool ok = true;
            // S of tiles and rows in turn take one place, each when the one before it has been
            // read, and P V of a tile follows the S of the next; in place S follows the P V.
            int k_stage = 0, v_stage = 1;  // fills K 0, V 0, K 1, V 1, ...
            uint32_t k_phase = 0, v_phase = 0;
            auto step = [&](int &stage, uint32_t &phase) {
                stage += 2;
                if (stage >= kStages) stage -= kStages, phase ^= 1;
            };
            ok = all_wait(&q_full[m], 0);
            int s_next = 0;
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
#pragma unroll 1
                while (s_next < n && s_next <= i + (kInPlace ? 0 : 1)) {
                    if (!(ok = all_wait(&kv_full[k_stage], k_phase))) break;
                    if (kInPlace) {
                    } else if (two && m == 1) {  // after the first rows' S of this tile
                        ok = all_wait(&s_empty[0], s_next & 1);
                    } else if (s_next > 0) {  // after the S before: the other rows', or this group's own
                        ok = all_wait(&s_empty[two ? kM - 1 : 0], (s_next - 1) & 1);
                    }
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t kd = k_desc + k_stage * (C::kStageBytes / 16);
                    if (one) {
#pragma unroll
                        for (int part = kQParts - 1; part >= 0; --part)  // the small part first: sums are cut to 24 bits
#pragma unroll
                            for (int j = 0; j < D / 16; ++j)
                                mma_f16_ss(s_at, q_desc + part * (C::kQBytes / 16) + j / 4 * 1024 + 2 * (j % 4),
                                           kd + j / 4 * (kN * 8) + 2 * (j % 4), kIdescS, part < kQParts - 1 || j > 0);
                        mma_commit(&s_full[m]);
                        mma_commit(&kv_empty[k_stage]);
                    }
                    step(k_stage, k_phase);
                    ++s_next;
                }
                if (!ok || !(ok = all_wait(&kv_full[v_stage], v_phase))) break;
                const uint64_t v = v_desc + v_stage * (C::kStageBytes / 16);
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {  // P V of tile i
                    if (!(ok = all_wait(&p_full[2 * m + half], i & 1))) break;
                    tc_fence_after();
                    const uint32_t p_at = C::kP0 + m * C::kPStep + half * (C::kPCols / 2);
                    const uint64_t vd = v + half * (kHalf / 16 * 128);
                    if (one) {
#pragma unroll
                        for (int j = 0; j < kHalf / 16; ++j)
#pragma unroll
                            for (int part = 0; part < kPParts; ++part)
                                mma_f16_ts(o_at, p_at + part * (kHalf / 2) + 8 * j, vd + j * 128, kIdescO,
                                           j + part > 0 ? 1 : half > 0 || (i > 0 && !C::flush_at(i, n)));
                        if (!kInPlace) mma_commit(&p_empty[2 * m + half]);
                    }
                }
                if (one) {
                    mma_commit(&kv_empty[v_stage]);
                    if (i + 1 == n) mma_commit(&o_full[m]);
                }
                step(v_stage, v_phase);
            }
            if (!ok && one) {  // wait until every MMA issued so far has finished
                mma_commit(&o_full[m]);
                const long long t0 = clock64();
                while (!mbar_try_wait(&o_full[m], 0) && clock64() - t0 < kWaitLimitCycles) {
                }
            }
        } else if (warp == 13) {
            // ------------------------------------------------ pages and scales
            constexpr int kBatch = 32 / C::kGroups;  // tiles at a time, a lane to each group of 16 positions
            const int32_t *table = a.table + b * a.table_ld;
            bool ok = true;
#pragma unroll 1
            for (int i0 = 0; i0 < tiles && ok; i0 += kBatch) {
                const int i = i0 + lane / C::kGroups;
                float4 at = make_float4(0.0f, -INFINITY, 0.0f, __int_as_float(0));
                if (i < tiles) {
                    const int pos = position(i) + lane % C::kGroups * 16;
                    // a page that no row sees is not looked up
                    if (pos < seen.see && (pos + 16 > seen.low || pos < a.sinks)) {
                        const int page = __ldg(table + pos / P);
                        if (page < 0 || page >= a.c.pages) {
                            set_status(a.dstatus, BSG_DSTATUS_RANGE);
                        } else {
                            const int64_t ph = (int64_t)page * a.c.heads + hk;
                            // finite: a masked score of -inf and the logarithm of Inf would be no number
                            // for rows that do not see the page (NaN: the least scale)
                            const float v = fminf(fmaxf(__ldg(a.c.v_scale + ph), 1e-30f), 3e38f);
                            at = make_float4(__ldg(a.c.k_scale + ph), log2f(v), __frcp_rn(v),
                                             __int_as_float((int)(ph * (P / 16) + pos % P / 16)));
                        }
                    }
                }
#pragma unroll 1
                for (int u = 0; u < kBatch && i0 + u < tiles; ++u) {
                    const int slot = (i0 + u) % kAtSlots;
                    if (!(ok = all_wait(&at_empty[slot], ((i0 + u) / kAtSlots & 1) ^ 1))) break;
                    if (lane / C::kGroups == u) at_s[slot * C::kGroups + lane % C::kGroups] = at;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&at_full[slot]);
                }
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ---------------------------------------------------- codes to f16 operands
        fewer_registers<kConvRegs>();
        constexpr int kChunks = D / 16;           // 16-byte pieces of a row
        constexpr int kPer = kN * kChunks / 128;  // of a thread and tile
        const uint32_t ctid = tid - 256;
        // Piece j of a thread: which 16 bytes of which row.  Eight lanes store to two rows, of
        // either parity, so that the swizzle spreads them over all banks; a thread's pieces
        // are whole groups of 16 rows apart, or even parts of one (but for 96 dims).
        constexpr uint32_t kStep = D == 96 ? 0 : 2048 / D;  // rows
        const uint32_t row0 = kChunks % 4 ? ctid / kChunks : ctid / (2 * kChunks) * 2 + ctid % 8 / 4;
        const uint32_t chunk0 = kChunks % 4 ? ctid % kChunks : ctid % 4 + ctid / 8 % (kChunks / 4 ? kChunks / 4 : 1) * 4;
        auto group_of = [&](uint32_t j) {
            return D == 96 ? (ctid + j * 128) / kChunks / 16 : kStep >= 16 ? row0 / 16 + j * (kStep / 16) : j / (16 / (kStep ? kStep : 1));
        };
        auto row_of = [&](uint32_t j) {  // of the group
            return D == 96 ? (ctid + j * 128) / kChunks % 16 : kStep >= 16 ? row0 % 16 : row0 + j % (16 / (kStep ? kStep : 1)) * kStep;
        };
        auto chunk_of = [&](uint32_t j) { return D == 96 ? (ctid + j * 128) % kChunks : chunk0; };
        uint4 buf[2][kPer];  // of K and V tiles
        auto load = [&](uint4 (&x)[kPer], const int8_t *codes, int i) {
            const float4 *at = at_s + i % kAtSlots * C::kGroups;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int place = __float_as_int(at[group_of(j)].w);
                x[j] = load_codes(codes + (row_of(j) * D + chunk_of(j) * 16) + (int64_t)place * (16 * D));
            }
        };
        bool ok = true;
        if (tiles > 0 && (ok = all_wait(&at_full[0], 0))) {
            load(buf[0], a.c.k, 0);
            load(buf[1], a.c.v, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&at_empty[0]);
        }
        int stage = 0;
        uint32_t phase = 0;
#pragma unroll 1
        for (int i = 0; i < tiles && ok; ++i) {
            const bool more = i + 1 < tiles;
            const int slot = (i + 1) % kAtSlots;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                if (!ok || !(ok = all_wait(&kv_empty[stage], phase ^ 1))) break;
                uint8_t *tile = smem + C::kOffStage + stage * C::kStageBytes;
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const uint32_t row = row_of(j), chunk = chunk_of(j);
                    uint32_t h[8];
                    const uint32_t w[4] = {buf[side][j].x, buf[side][j].y, buf[side][j].z, buf[side][j].w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {  // code + 128, as f16 1024 + that, less 1152
                        const uint32_t x = w[u] ^ 0x80808080u, bias = 0x64806480u;
                        const uint32_t lo = __byte_perm(x, 0x64646464u, 0x4140), hi = __byte_perm(x, 0x64646464u, 0x4342);
                        const __half2 l = __hsub2(*reinterpret_cast<const __half2 *>(&lo), *reinterpret_cast<const __half2 *>(&bias));
                        const __half2 g = __hsub2(*reinterpret_cast<const __half2 *>(&hi), *reinterpret_cast<const __half2 *>(&bias));
                        h[2 * u] = *reinterpret_cast<const uint32_t *>(&l);
                        h[2 * u + 1] = *reinterpret_cast<const uint32_t *>(&g);
                    }
                    uint8_t *line = tile + group_of(j) * 2048 + (chunk / 4 * (kN * 128) + row * 128);
                    const uint32_t c = chunk % 4 * 2;
                    *reinterpret_cast<uint4 *>(line + ((c ^ row % 8) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4 *>(line + ((c + 1 ^ row % 8) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&kv_full[stage]);
                if (++stage == kStages) stage = 0, phase ^= 1;
                if (more) {  // the next tile's, into the registers that are free
                    if (side == 0 && !(ok = all_wait(&at_full[slot], (i + 1) / kAtSlots & 1))) break;
                    load(buf[side], side ? a.c.v : a.c.k, i + 1);
                    __syncwarp();
                    if (side == 1 && lane == 0) mbar_arrive(&at_empty[slot]);
                }
            }
        }
    } else {
        // ---------------------------------------------------- softmax, a row a thread
        more_registers<kSoftRegs>();
        const int m = warp / 4, r = tid;
        if (m < groups) {
        const uint32_t quad = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t s_at = m * C::kSStep + quad, p_at = C::kP0 + m * C::kPStep + quad, o_at = C::kO0 + m * D + quad;
        const int pos = PREFIX ? len - 1 : pos0 + (r0 + r) / share;
        const int see = r < rows ? pos + 1 : 0;
        const int low = !PREFIX && a.window && pos >= a.window ? pos - a.window + 1 : 0;
        // rows m: tiles from `all_low` to `all_see` are seen by every one
        const int last = min(rows, m * 128 + 128) - 1;
        const int all_see = PREFIX ? len : pos0 + (r0 + m * 128) / share + 1;
        const int last_pos = PREFIX ? 0 : pos0 + (r0 + last) / share;
        const int all_low = !PREFIX && a.window && last_pos >= a.window ? last_pos - a.window + 1 : 0;
        // Queries, the warp's own rows: each relative to a power of two near its largest |q| (with
        // the sign of the scale), in f16 parts, rows of 64 dims in the 128-byte swizzle.
        float mul = 0.0f;
        auto load_queries = [&](auto type) {
            using T = decltype(type);
            constexpr int kAhead = D == 256 ? 8 : 16;
            const int n = (r0 + r) / share, h = (r0 + r) % share;  // where row `lane` is
            const int64_t where = (PREFIX ? n / a.tokens * a.q.stride_batch + n % a.tokens * a.q.stride_token
                                          : b * a.q.stride_batch + n * a.q.stride_token) + (hk * share + h) * a.q.stride_head;
            uint8_t *const tile = smem + m * kQParts * C::kQBytes;
#pragma unroll 1
            for (int r1 = 0; r1 < 32; r1 += kAhead) {
                float q[kAhead][D / 32];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const T *row = static_cast<const T *>(a.q.data) + __shfl_sync(0xffffffffu, where, r1 + i) + lane;
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) q[i][j] = warp * 32 + r1 + i < rows ? to_f32(row[32 * j]) : 0.0f;
                }
                bool bad = false;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    float x = 0.0f;
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        bad |= !isfinite(q[i][j]);
                        x = fmaxf(x, fabsf(q[i][j]));
                    }
                    x = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
                    // 2^e with x 2^e in [2^13, 2^14); e <= 126 leaves subnormal rows their small error
                    const int e = max(-126, min(126, 13 + 127 - (int)(__float_as_uint(x) >> 23)));
                    const float up = copysignf(__uint_as_float((uint32_t)(e + 127) << 23), a.scale);
                    const int at_r = warp % 4 * 32 + r1 + i;
                    if (lane == r1 + i)
                        mul = fabsf(a.scale) * 1.4426950408889634f * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        const int d = lane + 32 * j;
                        const int at = d / 64 * 16384 + at_r * 128 + ((d % 64 / 8 ^ at_r % 8) << 4) + d % 8 * 2;
                        const float y = q[i][j] * up;
                        const __half hi = __float2half_rn(y);
                        *reinterpret_cast<__half *>(tile + at) = hi;
                        if (kQParts == 2)
                            *reinterpret_cast<__half *>(tile + C::kQBytes + at) = __float2half_rn(y - __half2float(hi));
                    }
                }
                if (bad) set_status(a.dstatus, BSG_DSTATUS_NONFINITE);
            }
        };
        // The same by 16 bytes, where rows begin on them and a row's pieces are 1 to 32 lanes, a power
        // of two.
        auto load_pieces = [&](auto type) {
            using T = decltype(type);
            constexpr int kE = 16 / sizeof(T), kL = D / kE, kR = 32 / kL, kAhead = kQParts == 2 ? 8 : 32 / kR < 8 ? 32 / kR : 8;
            const int n = (r0 + r) / share, h = (r0 + r) % share;
            const int64_t where = (PREFIX ? n / a.tokens * a.q.stride_batch + n % a.tokens * a.q.stride_token
                                          : b * a.q.stride_batch + n * a.q.stride_token) + (hk * share + h) * a.q.stride_head;
            uint8_t *const tile = smem + m * kQParts * C::kQBytes;
            struct alignas(16) Piece {
                T v[kE];
            };
#pragma unroll 1
            for (int r1 = 0; r1 < 32; r1 += kR * kAhead) {
                Piece q[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int row = r1 + i * kR + lane / kL;
                    const int64_t at = __shfl_sync(0xffffffffu, where, row);
                    if (warp * 32 + row < rows) {
                        q[i] = *reinterpret_cast<const Piece *>(static_cast<const T *>(a.q.data) + at + lane % kL * kE);
                    } else {
#pragma unroll
                        for (int j = 0; j < kE; ++j) q[i].v[j] = from_f32<T>(0.0f);
                    }
                }
                bool bad = false;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    // the row's largest |q|: bits order as magnitudes do, Inf and NaN above all
                    float x, y[kE];
                    const uint32_t *bits = reinterpret_cast<const uint32_t *>(&q[i]);
                    if constexpr (sizeof(T) == 2) {
                        uint32_t most = __vmaxu2(__vmaxu2(bits[0] & 0x7fff7fffu, bits[1] & 0x7fff7fffu),
                                                 __vmaxu2(bits[2] & 0x7fff7fffu, bits[3] & 0x7fff7fffu));
                        most = max(most >> 16, most & 0xffffu);
#pragma unroll
                        for (int o = kL / 2; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
                        const uint16_t h = (uint16_t)most;
                        x = to_f32(*reinterpret_cast<const T *>(&h));
                    } else {
                        uint32_t most = max(max(bits[0] & 0x7fffffffu, bits[1] & 0x7fffffffu),
                                            max(bits[2] & 0x7fffffffu, bits[3] & 0x7fffffffu));
#pragma unroll
                        for (int o = kL / 2; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
                        x = __uint_as_float(most);
                    }
                    bad |= !isfinite(x);
#pragma unroll
                    for (int j = 0; j < kE; ++j) y[j] = to_f32(q[i].v[j]);
                    const int e = max(-126, min(126, 13 + 127 - (int)(__float_as_uint(x) >> 23)));
                    const float up = copysignf(__uint_as_float((uint32_t)(e + 127) << 23), a.scale);
                    const float its = fabsf(a.scale) * 1.4426950408889634f * __uint_as_float((uint32_t)(127 - e) << 23);
                    const float from = __shfl_sync(0xffffffffu, its, (lane - r1 - i * kR) * kL & 31);
                    if (lane >= r1 + i * kR && lane < r1 + (i + 1) * kR) mul = from;
                    const int at_r = warp % 4 * 32 + r1 + i * kR + lane / kL, d = lane % kL * kE;
                    uint8_t *const to = tile + d / 64 * 16384 + at_r * 128 + ((d % 64 / 8 ^ at_r % 8) << 4) + d % 8 * 2;
                    __half2 hi[kE / 2], lo[kE / 2];
#pragma unroll
                    for (int j = 0; j < kE / 2; ++j) {
                        const float y0 = y[2 * j] * up, y1 = y[2 * j + 1] * up;
                        hi[j] = __floats2half2_rn(y0, y1);
                        const float2 back = __half22float2(hi[j]);
                        lo[j] = __floats2half2_rn(y0 - back.x, y1 - back.y);
                    }
                    if constexpr (kQParts == 2) {
                        *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<const uint2 *>(hi);
                        *reinterpret_cast<uint2 *>(to + C::kQBytes) = *reinterpret_cast<const uint2 *>(lo);
                    } else {
                        *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(hi);
                    }
                }
                if (bad) set_status(a.dstatus, BSG_DSTATUS_NONFINITE);
            }
        };
        auto load_any = [&](auto type) {
            using T = decltype(type);
            constexpr bool kPieces = D != 96 && (D * (int)sizeof(T)) / 16 <= 32;
            const uintptr_t all = reinterpret_cast<uintptr_t>(a.q.data) | (uintptr_t)(a.q.stride_batch * (int64_t)sizeof(T)) |
                                  (uintptr_t)(a.q.stride_token * (int64_t)sizeof(T)) | (uintptr_t)(a.q.stride_head * (int64_t)sizeof(T));
            if constexpr (kPieces) {
                if (all % 16 == 0) {
                    load_pieces(type);
                    return;
                }
            }
            load_queries(type);
        };
        if constexpr (kQParts == 2) {
            load_any(float{});
        } else if constexpr (kPParts == 2) {
            load_any(__half{});
        } else {
            load_any(__nv_bfloat16{});
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[m]);
        float ref = 0.0f, sum = 0.0f;
        bool none = true, ok = true;
        // What O was before it was begun anew, the sum, and the reference then (a row that had seen
        // nothing: -inf, no part of it): in local memory, and in no register from one time to the next.
        volatile float kept[D + 2];
        // runs of tiles between which the sums are begun anew
#pragma unroll 1
        for (int i = 0; i < tiles;) {
            if (C::flush_at(i, tiles)) {
                // O is at rest once the last P of the tile before is used up (in place: as the next S is there)
                if (kInPlace) ok = all_wait(&s_full[m], i & 1);
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (!kInPlace && ok) ok = all_wait(&p_empty[2 * m + u], (i - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const bool some_kept = i > C::kFlush;
                const float f = some_kept ? tile_exp2(kept[D + 1] - ref) : 0.0f;
                kept[D] = some_kept ? fmaf(kept[D], f, sum) : sum;
                kept[D + 1] = none ? -INFINITY : ref;
                sum = 0.0f;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    float before[32];
                    __syncwarp();
                    tmem_ld32(o_at + 32 * c, o);
#pragma unroll
                    for (int u = 0; u < 32; ++u) before[u] = some_kept ? kept[32 * c + u] : 0.0f;
                    tmem_ld_wait32(o);
#pragma unroll
                    for (int u = 0; u < 32; ++u) kept[32 * c + u] = fmaf(before[u], f, __uint_as_float(o[u]));
                }
            }
            const int stop = C::flush_at(i + C::kFlush, tiles) ? i + C::kFlush : tiles;
#pragma unroll 1
            for (; i < stop; ++i) {
                const int tile = position(i), slot = i % kAtSlots;
                const float4 *of_s = at_s + slot * C::kGroups;
                if (!(ok = all_wait(&at_full[slot], i / kAtSlots & 1) && all_wait(&s_full[m], i & 1))) break;
                tc_fence_after();
                const bool edge = tile + kN > all_see || (tile < all_low && tile + kN > a.sinks);
                if (edge) {  // what the row does not see, where S lies (seldom; rolled up)
#pragma unroll 1
                    for (int c = 0; c < kN / 16; ++c) {
                        const int j = tile + 16 * c;
                        const uint32_t mask = below(see - j) & (~below(low - j) | below(a.sinks - j));
                        uint32_t x[16];
                        tmem_ld16(s_at + 16 * c, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int u = 0; u < 16; ++u)
                            if (!(mask & 1u << u)) x[u] = 0xff800000u;
                        tmem_st16(s_at + 16 * c, x);
                    }
                    tmem_st_wait();
                }
                uint32_t v[kN / 32][32];  // the row's scores
#pragma unroll
                for (int c = 0; c < kN / 32; ++c) tmem_ld32(s_at + 32 * c, v[c]);
#pragma unroll
                for (int c = 0; c < kN / 32; ++c) tmem_ld_wait32(v[c]);
                tc_fence_before();
                __syncwarp();
                if (!kInPlace && lane == 0) mbar_arrive(&s_empty[m]);
                // the largest exponent, relative to the reference
                float y[C::kGroups], top = -INFINITY;
#pragma unroll
                for (int g = 0; g < C::kGroups; ++g) y[g] = __uint_as_float(v[g / 2][g % 2 * 16]);
#pragma unroll
                for (int u = 1; u < 16; ++u)  // the groups side by side, not one after another
#pragma unroll
                    for (int g = 0; g < C::kGroups; ++g) y[g] = fmaxf(y[g], __uint_as_float(v[g / 2][g % 2 * 16 + u]));
                // (a score of -inf times 0 would be no number)
#pragma unroll
                for (int g = 0; g < C::kGroups; ++g) {
                    const float2 of = *reinterpret_cast<const float2 *>(of_s + g);
                    top = fmaxf(top, fmaf(y[g], fmaxf(of.x * mul, 1e-37f), of.y - ref));
                }
                const bool move = none ? top > -INFINITY : top > kTileMost;
                if (__any_sync(0xffffffffu, move)) {
                    float keep = 1.0f;
                    if (move) {  // each row by itself: no other row's values move its reference
                        if (!none) keep = tile_exp2(kTileTop - top);
                        ref += top - kTileTop;
                        sum *= keep;
                        none = false;
                    }
                    if (i > 0) {
                        // O is at rest once the last P of the tile before is used up (in place: as S is there)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            if (!kInPlace && ok) ok = all_wait(&p_empty[2 * m + u], (i - 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(o_at + 16 * c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * keep);
                            tmem_st16(o_at + 16 * c, o);
                        }
                    }
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t hi[kHalf / 2], lo[kHalf / 2];
#pragma unroll
                    for (int g = 0; g < kHalf / 16; ++g) {
                        const float4 of = of_s[half * (kHalf / 16) + g];
                        const float f = fmaxf(of.x * mul, 1e-37f), off = of.y - ref;
                        const uint64_t ff = pair_of(f, f), oo = pair_of(off, off);
                        const uint32_t *x = v[(half * kHalf + 16 * g) / 32] + (half * kHalf + 16 * g) % 32;
                        float p[16];
#pragma unroll
                        for (int u = 0; u < 16; u += 2) {
                            unpair(fma2(pair_of(__uint_as_float(x[u]), __uint_as_float(x[u + 1])), ff, oo), p[u], p[u + 1]);
                            p[u] = tile_exp2(p[u]), p[u + 1] = tile_exp2(p[u + 1]);
                        }
                        uint64_t part[2] = {pair_of(p[0], p[1]), pair_of(p[2], p[3])};
#pragma unroll
                        for (int u = 4; u < 16; u += 2) part[u / 2 % 2] = add2(part[u / 2 % 2], pair_of(p[u], p[u + 1]));
                        float even, odd;
                        unpair(add2(part[0], part[1]), even, odd);
                        sum = fmaf(even + odd, of.z, sum);
#pragma unroll
                        for (int u = 0; u < 16; u += 2) {
                            const __half2 h = __floats2half2_rn(p[u], p[u + 1]);
                            hi[8 * g + u / 2] = *reinterpret_cast<const uint32_t *>(&h);
                            if (kPParts == 2) {
                                const float2 back = __half22float2(h);
                                const __half2 rest = __floats2half2_rn(p[u] - back.x, p[u + 1] - back.y);
                                lo[8 * g + u / 2] = *reinterpret_cast<const uint32_t *>(&rest);
                            }
                        }
                    }
                    // its place is free when what was there has been multiplied
                    if (!kInPlace && i > 0 && !(ok = all_wait(&p_empty[2 * m + half], (i - 1) & 1))) break;
                    tc_fence_after();
                    tmem_store(p_at + half * (C::kPCols / 2), hi);
                    if (kPParts == 2) tmem_store(p_at + half * (C::kPCols / 2) + kHalf / 2, lo);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * m + half]);
                }
                if (!ok) break;
                if (lane == 0) mbar_arrive(&at_empty[slot]);
            }
            if (!ok) break;
        }
        if (ok && tiles > 0) {
            ok = all_wait(&o_full[m], 0);
            tc_fence_after();
        }
        // ---- the row's outputs
        const int64_t n = (r0 + r) / share;
        const int head = hk * share + (r0 + r) % share;
        const bool direct = !PREFIX && a.splits == 1 && !a.later;
        const int64_t part = (((int64_t)b * a.c.heads + hk) * a.rows + r0 + r) * a.splits + split;
        const bool there = r < rows && ok;
        const bool some_kept = C::flush_at(C::kFlush, tiles);
        const float of_kept = some_kept ? tile_exp2(kept[D + 1] - ref) : 0.0f;
        if (some_kept) sum = fmaf(kept[D], of_kept, sum);
        const bool some = sum > 0.0f || sum != sum;
        const float inv = some ? __frcp_rn(sum) : 0.0f;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            __syncwarp();
            if (tiles > 0) {
                tmem_ld32(o_at + 32 * c, v);
                tmem_ld_wait32(v);
            }
            if (!there) continue;
            float o[32];
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = tiles == 0 || (!some && direct) ? 0.0f : __uint_as_float(v[u]);
            if (some_kept)
#pragma unroll
                for (int u = 0; u < 32; ++u) o[u] = fmaf(kept[32 * c + u], of_kept, o[u]);
            if (direct) {
                auto store = [&](auto type) {
                    using T = decltype(type);
                    T *dst = static_cast<T *>(a.out.data) + b * a.out.stride_batch + n * a.out.stride_token +
                             head * a.out.stride_head + 32 * c;
                    T y[32];
#pragma unroll
                    for (int u = 0; u < 32; ++u) y[u] = from_f32<T>(o[u] * inv);
                    if (reinterpret_cast<uintptr_t>(dst) % 16 == 0) {
#pragma unroll
                        for (int u = 0; u < 32 * (int)sizeof(T) / 16; ++u)
                            reinterpret_cast<uint4 *>(dst)[u] = reinterpret_cast<const uint4 *>(y)[u];
                    } else {
#pragma unroll
                        for (int u = 0; u < 32; ++u) dst[u] = y[u];
                    }
                };
                if constexpr (kQParts == 2) {
                    store(float{});
                } else if constexpr (kPParts == 2) {
                    store(__half{});
                } else {
                    store(__nv_bfloat16{});
                }
            } else {
                float4 *dst = reinterpret_cast<float4 *>(a.part_o + part * D + 32 * c);
#pragma unroll
                for (int u = 0; u < 8; ++u) dst[u] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
            }
        }
        if (there && !direct) a.part_ml[part] = make_float2(ref, sum);
        if (there && direct && a.lse)
            a.lse[((int64_t)b * a.tokens + n) * a.heads + head] =
                some ? (ref + log2f(sum)) * 0.69314718055994531f : -INFINITY;
        tc_fence_before();
        }
    }
    __syncthreads();
    if (PREFIX) griddep_wait();  // this grid never ends before the one that it was launched beside
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(0, 512);
    }
}

template <int D, int kQ, int kP, bool PREFIX, bool kLong>
cudaError_t launch_tiles_as(const TileArgs &a, cudaStream_t st) {
    using C = TileCfg<D, kQ, kP, kLong>;
    static bool set[64] = {false};  // this kernel's shared memory, on each device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !set[dev]) {
        e = cudaFuncSetAttribute(kv8_tiles_kernel<D, kQ, kP, PREFIX, kLong>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) set[dev] = true;
    }
    const int64_t blocks = a.row_blocks * a.groups;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)a.splits);
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = C::kBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PREFIX ? 1 : 0;  // beside the sequences' own positions' launch
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kv8_tiles_kernel<D, kQ, kP, PREFIX, kLong>, a);
}

// most: tiles of a chunk.  Chunks that one sum takes need none of the code that begins it anew, which
// 16-bit types' registers have little room for (f16, prompts of 16384 through a window of 4096: 2541
// us without, 2727 with).
template <int D, int kQ, int kP, bool PREFIX>
cudaError_t launch_tiles_long(const TileArgs &a, int most, cudaStream_t st) {
    if constexpr (kQ == 1)
        if (most <= TileCfg<D, kQ, kP, true>::kFlushMost) return launch_tiles_as<D, kQ, kP, PREFIX, false>(a, st);
    return launch_tiles_as<D, kQ, kP, PREFIX, true>(a, st);
}

template <int D, bool PREFIX>
cudaError_t launch_tiles_dim(const TileArgs &a, int dtype, int most, cudaStream_t st) {
    if (dtype == BSG_F32) return launch_tiles_long<D, 2, 2, PREFIX>(a, most, st);
    if (dtype == BSG_F16) return launch_tiles_long<D, 1, 2, PREFIX>(a, most, st);
    return launch_tiles_long<D, 1, 1, PREFIX>(a, most, st);
}

template <bool PREFIX>
cudaError_t launch_tiles(const KvCall &k, const KvPlan &p, cudaStream_t st) {
    const TileArgs a{k.c, k.table, k.table_ld, k.lens, k.counts, k.q, k.out, k.tokens, k.heads, k.window, k.sinks,
                     (int)k.rows, p.row_blocks, k.B * k.c.heads, p.splits, k.later, k.scale, k.lse, k.part_o, k.part_ml, k.dstatus};
    switch (k.c.dim) {
        case 32: return launch_tiles_dim<32, PREFIX>(a, k.dtype, p.tiles, st);
        case 64: return launch_tiles_dim<64, PREFIX>(a, k.dtype, p.tiles, st);
        case 96: return launch_tiles_dim<96, PREFIX>(a, k.dtype, p.tiles, st);
        case 128: return launch_tiles_dim<128, PREFIX>(a, k.dtype, p.tiles, st);
        default: return launch_tiles_dim<256, PREFIX>(a, k.dtype, p.tiles, st);
    }
}

}  // namespace
}  // namespace bsg

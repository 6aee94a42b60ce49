// kv8_tiles.cuh -- attention of many query rows over the int8 cache on the tcgen05 tensor
// cores: prompts through a window with sinks, and the prefix that a batch shares.
//
// A CTA takes up to kM x 128 rows (queries of one key/value head: the heads of its group
// times tokens) and walks the tiles of kN positions that some of them see:
//   S = Q K^T          one accumulator of 128 x kN per 128 rows, in tensor memory
//   p' = 2^(S ks mul + log2 vs - ref)   a thread to a row, in f16, in S's place
//   O += P V           P read from tensor memory, O stays there
// with ks, vs the page's scales (one for each 16 positions of a tile), mul the row's
// multiplier, ref the row's running reference, which follows the maximum only when that is
// more than 2^4 above it (O is then rescaled where it lies); sums of p = p' / vs in f32.
// Codes are exact in f16, so K and V are too; queries are relative to a power of two near
// their row's largest, f32's as two f16 parts (22 bits).
//
// Roles: warps 0-3 (and 4-7 for the second 128 rows) softmax, one row a thread; 4 warps
// turn codes into f16 operands in a ring of shared memory, their loads a tile ahead in
// registers; one thread issues the MMAs.  The two groups of rows alternate: while one's
// softmax runs, the tensor cores work for the other.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bsg_internal.h"
#include "bsg_ptx.cuh"
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

constexpr float kTileTop = 11.0f, kTileMost = 15.0f;
constexpr int kScaleSlots = 6;

__device__ __forceinline__ float tile_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a CTA of some rows sees: `sink_tiles` tiles from the first, then those from `first`.
struct Seen {
    int tiles, sink_tiles, first;
    int low, see;  // the lowest position of the window part, and the end
};
template <int kN>
__device__ __forceinline__ Seen seen_by(int first_pos, int last_pos, int window, int sinks) {
    Seen s;
    s.see = last_pos + 1;
    s.low = window && first_pos >= window ? first_pos - window + 1 : 0;
    if (s.see <= 0) {
        s.tiles = s.sink_tiles = s.first = 0;
        return s;
    }
    const int k = min(sinks, s.low);
    s.sink_tiles = (k + kN - 1) / kN;
    s.first = max(s.sink_tiles, s.low / kN);
    s.tiles = s.sink_tiles + max(0, (s.see + kN - 1) / kN - s.first);
    return s;
}

template <int D, int kQParts>
struct TileCfg {
    static constexpr int kM = D == 256 ? 1 : 2;
    static constexpr int kN = D == 256 ? 64 : 128;
    static constexpr int kBlocks = (D + 63) / 64;             // of 64 dims (128 bytes of f16)
    static constexpr int kQBytes = kBlocks * 128 * 128;       // one part of 128 rows
    static constexpr int kStageBytes = kBlocks * kN * 128;    // a K or V tile
    static constexpr int kRoom = 229376 - kM * kQParts * kQBytes;
    static constexpr int kStages = kRoom / kStageBytes < 6 ? kRoom / kStageBytes : 6;
    static constexpr int kGroups = kN / 16;
    static constexpr int kSoftWarps = 4 * kM, kConvWarps = 4;
    static constexpr int kThreads = (kSoftWarps + kConvWarps + 1) * 32;
    static constexpr int kOffStage = kM * kQParts * kQBytes;
    static constexpr int kOffScale = kOffStage + kStages * kStageBytes;
    static constexpr int kOffMul = kOffScale + kScaleSlots * kGroups * 16;
    static constexpr int kOffBar = kOffMul + kM * 128 * 4;
    static constexpr int kBars = 2 * kStages + kScaleSlots + 3 * kM;
    static constexpr int kUsed = kOffBar + kBars * 8 + 16;
    static constexpr int kBytes = (kUsed > 118000 ? kUsed : 118000) + 1024;  // one CTA on an SM (all its tensor memory)
    static_assert(kStages >= 2 && kBytes <= 232448, "shared memory");
    static_assert(kScaleSlots >= kStages / 2 + 3, "a slot is free before it is written again");
    static __device__ constexpr int kS(int m) { return m * kN; }               // columns of tensor memory
    static __device__ constexpr int kO(int m) { return kM * kN + m * D; }
};

// PREFIX: rows are those of all sequences (rows = B x tokens x heads of a group), every one
// sees the positions below *lens; what a CTA finds is joined later.  The report of bad lengths
// is the first CTA's.
template <int D, int kQParts, int kPParts, bool PREFIX>
__global__ void __launch_bounds__(TileCfg<D, kQParts>::kThreads, 1)
    kv8_tiles_kernel(const __grid_constant__ TileArgs a) {
    using C = TileCfg<D, kQParts>;
    constexpr int kM = C::kM, kN = C::kN, kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    float4 *scale_s = reinterpret_cast<float4 *>(smem + C::kOffScale);
    float *mul_s = reinterpret_cast<float *>(smem + C::kOffMul);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *kv_full = bars, *kv_empty = bars + kStages, *sc_full = bars + 2 * kStages;
    uint64_t *s_full = sc_full + kScaleSlots, *p_full = s_full + kM, *o_full = p_full + kM;
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(bars + C::kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_ptr + 1);

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t group = blockIdx.x % a.groups;
    const int hk = (int)(group % a.c.heads), b = (int)(group / a.c.heads), split = blockIdx.y;
    const int share = a.heads / a.c.heads, P = a.c.page_tokens;
    // later rows see more: they go first
    const int r0 = (a.row_blocks - 1 - (int)(blockIdx.x / a.groups)) * (kM * 128);
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
    const int groups = rows > 128 ? kM : 1;  // of 128 rows
    auto position = [&](int i) {  // of the CTA's tile i
        const int v = begin + i;
        return (v < seen.sink_tiles ? v : v - seen.sink_tiles + seen.first) * kN;
    };

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&kv_full[s], C::kConvWarps);
            mbar_init(&kv_empty[s], 1);
        }
        for (int s = 0; s < kScaleSlots; ++s) mbar_init(&sc_full[s], 1);
        for (int m = 0; m < kM; ++m) {
            mbar_init(&s_full[m], 1);
            mbar_init(&p_full[m], 4);
            mbar_init(&o_full[m], 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    constexpr int kMmaWarp = C::kSoftWarps + C::kConvWarps;
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_ptr, 512);
        tmem_relinquish();
    }
    griddep_launch_dependents();

    // Queries: each row relative to a power of two near its largest |q| (with the sign of
    // the scale), in f16 parts, rows of 64 dims in the 128-byte swizzle.
    auto load_queries = [&](auto type) {
        using T = decltype(type);
        constexpr int kAhead = 4;
        for (int rr = warp * kAhead; rr < groups * 128; rr += C::kThreads / 32 * kAhead) {
            float q[kAhead][D / 32];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int r = r0 + rr + i;
                const int64_t n = r / share;
                const int64_t at = PREFIX ? n / a.tokens * a.q.stride_batch + n % a.tokens * a.q.stride_token
                                          : b * a.q.stride_batch + n * a.q.stride_token;
                const T *row = static_cast<const T *>(a.q.data) + at + (hk * share + r % share) * a.q.stride_head + lane;
#pragma unroll
                for (int j = 0; j < D / 32; ++j) q[i][j] = rr + i < rows ? to_f32(row[32 * j]) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
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
                const int e = max(-126, min(126, 13 + 127 - (int)(__float_as_uint(m) >> 23)));
                const float up = copysignf(__uint_as_float((uint32_t)(e + 127) << 23), a.scale);
                const int r = rr + i;
                if (lane == 0) mul_s[r] = fabsf(a.scale) * 1.4426950408889634f * __uint_as_float((uint32_t)(127 - e) << 23);
                uint8_t *tile = smem + r / 128 * kQParts * C::kQBytes;
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const int d = lane + 32 * j;
                    const int at = d / 64 * 16384 + r % 128 * 128 + ((d % 64 / 8 ^ r % 8) << 4) + d % 8 * 2;
                    const float y = q[i][j] * up;
                    const __half hi = __float2half_rn(y);
                    *reinterpret_cast<__half *>(tile + at) = hi;
                    if (kQParts == 2)
                        *reinterpret_cast<__half *>(tile + C::kQBytes + at) = __float2half_rn(y - __half2float(hi));
                }
            }
        }
    };
    if constexpr (kQParts == 2) {
        load_queries(float{});
    } else if constexpr (kPParts == 2) {
        load_queries(__half{});
    } else {
        load_queries(__nv_bfloat16{});
    }
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_ptr;
    auto give_up = [&]() {
        *abort_flag = 1;
        set_status(a.dstatus, BSG_DSTATUS_TIMEOUT);
    };

    if (warp == kMmaWarp) {
        // ---------------------------------------------------- MMA issuer
        if (lane == 0 && tiles > 0) {
            constexpr uint32_t kIdescS = idesc_f16_f32(128, kN), kIdescO = idesc_f16_f32(128, D) | kIdescBMn;
            const uint32_t stage0 = smem_u32(smem + C::kOffStage);
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (ok && !mbar_wait(bar, parity, abort_flag)) {
                    give_up();
                    ok = false;
                }
                tc_fence_after();
            };
            auto products = [&](int m, int i) {  // S of rows m and tile i
                const uint32_t k = stage0 + 2 * i % kStages * C::kStageBytes;
#pragma unroll
                for (int part = 0; part < kQParts; ++part)
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
                        mma_f16_ss(tmem + C::kS(m),
                                   sdesc_k128(smem_u32(smem) + (m * kQParts + part) * C::kQBytes + j / 4 * 16384) + 2 * (j % 4),
                                   sdesc_k128(k + j / 4 * (kN * 128)) + 2 * (j % 4), kIdescS, part + j > 0);
                mma_commit(&s_full[m]);
            };
            wait(&kv_full[0], 0);
            if (ok) {
                products(0, 0);
                if (groups > 1) products(kM - 1, 0);
                mma_commit(&kv_empty[0]);
            }
            for (int i = 0; i < tiles && ok; ++i) {
                const int vs = (2 * i + 1) % kStages, ks = (2 * i + 2) % kStages;
                const uint32_t vphase = (2 * i + 1) / kStages & 1, kphase = (2 * i + 2) / kStages & 1;
                for (int m = 0; m < groups; ++m) {
                    wait(&p_full[m], i & 1);
                    if (m == 0) wait(&kv_full[vs], vphase);
                    if (!ok) break;
                    const uint32_t v = stage0 + vs * C::kStageBytes;
#pragma unroll
                    for (int j = 0; j < kN / 16; ++j)
#pragma unroll
                        for (int part = 0; part < kPParts; ++part)
                            mma_f16_ts(tmem + C::kO(m), tmem + C::kS(m) + j / 2 * 32 + j % 2 * 8 + part * 16,
                                       sdesc_mn128(v + j * 2048, kN * 128), kIdescO, i + j + part > 0);
                    if (m == groups - 1) mma_commit(&kv_empty[vs]);
                    if (i + 1 == tiles) {
                        mma_commit(&o_full[m]);
                        continue;
                    }
                    if (m == 0) wait(&kv_full[ks], kphase);
                    if (!ok) break;
                    products(m, i + 1);
                    if (m == groups - 1) mma_commit(&kv_empty[ks]);
                }
            }
            if (!ok) {  // wait until every MMA issued so far has finished
                mma_commit(&o_full[0]);
                const long long t0 = clock64();
                while (!mbar_try_wait(&o_full[0], 0) && clock64() - t0 < kWaitLimitCycles) {
                }
            }
        }
        __syncwarp();
    } else if (warp >= C::kSoftWarps) {
        // ---------------------------------------------------- codes to f16 operands
        constexpr int kChunks = D / 16;                             // 16-byte pieces of a row
        constexpr int kPer = kN * kChunks / (C::kConvWarps * 32);   // of a thread and tile
        const int ctid = tid - C::kSoftWarps * 32;
        const int32_t *table = a.table + b * a.table_ld;
        uint4 kbuf[kPer], vbuf[kPer];
        int64_t at = -1, at_next = -1;  // of group `lane` of a tile, in bytes of the pool; -1: nowhere
        float4 sc, sc_next;
        // Where the groups of tile i lie, a lane each.  A page that no row sees is not looked up.
        auto look_up = [&](int i) {
            at_next = -1;
            sc_next = make_float4(0.0f, -INFINITY, 0.0f, 1.0f);
            if (i >= tiles || lane >= C::kGroups) return;
            const int pos = position(i) + lane * 16;
            if (pos >= seen.see || (pos + 16 <= seen.low && pos >= a.sinks)) return;
            const int page = __ldg(table + pos / P);
            if (page < 0 || page >= a.c.pages) {
                set_status(a.dstatus, BSG_DSTATUS_RANGE);
                return;
            }
            const int64_t ph = (int64_t)page * a.c.heads + hk;
            at_next = (ph * P + pos % P) * D;
            const float ks = __ldg(a.c.k_scale + ph), vs = __ldg(a.c.v_scale + ph), v = fmaxf(fabsf(vs), 1e-30f);
            // w: the signs, which go to the codes
            sc_next = make_float4(fabsf(ks), log2f(v), __frcp_rn(v),
                                  __uint_as_float((ks < 0.0f ? 1u : 0u) | (vs < 0.0f ? 2u : 0u)));
        };
        auto load = [&](uint4 (&buf)[kPer], const int8_t *codes, int64_t where) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int e = ctid + j * (C::kConvWarps * 32), row = e / kChunks;
                const int64_t base = __shfl_sync(0xffffffffu, where, row / 16);
                buf[j] = make_uint4(0x0u, 0x0u, 0x0u, 0x0u);
                if (base >= 0)
                    buf[j] = __ldg(reinterpret_cast<const uint4 *>(codes + base + row % 16 * D) + e % kChunks);
            }
        };
        auto convert = [&](const uint4 (&buf)[kPer], int fill, uint32_t bit, float4 of) {
            const int stage = fill % kStages;
            const bool ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[stage], (fill / kStages & 1) ^ 1, abort_flag));
            if (!ok) {
                if (lane == 0) give_up();
                return false;
            }
            uint8_t *tile = smem + C::kOffStage + stage * C::kStageBytes;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int e = ctid + j * (C::kConvWarps * 32), row = e / kChunks, chunk = e % kChunks;
                const uint32_t signs = __float_as_uint(__shfl_sync(0xffffffffu, of.w, row / 16));
                const __half2 sign = __float2half2_rn(signs & bit ? -1.0f : 1.0f);
                const __half2 bias = __float2half2_rn(signs & bit ? 1152.0f : -1152.0f);
                uint32_t h[8];
                const uint32_t w[4] = {buf[j].x, buf[j].y, buf[j].z, buf[j].w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t x = w[u] ^ 0x80808080u;
                    const uint32_t lo = __byte_perm(x, 0x64646464u, 0x4140), hi = __byte_perm(x, 0x64646464u, 0x4342);
                    const __half2 l = __hfma2(*reinterpret_cast<const __half2 *>(&lo), sign, bias);
                    const __half2 g = __hfma2(*reinterpret_cast<const __half2 *>(&hi), sign, bias);
                    h[2 * u] = *reinterpret_cast<const uint32_t *>(&l);
                    h[2 * u + 1] = *reinterpret_cast<const uint32_t *>(&g);
                }
                uint8_t *line = tile + chunk / 4 * (kN * 128) + row * 128;
                const int c = chunk % 4 * 2;
                *reinterpret_cast<uint4 *>(line + ((c ^ row % 8) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(line + ((c + 1 ^ row % 8) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&kv_full[stage]);
            return true;
        };
        look_up(0);
        at = at_next, sc = sc_next;
        load(kbuf, a.c.k, at);
        for (int i = 0; i < tiles; ++i) {
            load(vbuf, a.c.v, at);
            look_up(i + 1);
            // the scales' slot was read by the softmax of tile i - kScaleSlots, whose P V a
            // value tile filled earlier has waited for
            if (warp == C::kSoftWarps) {
                if (lane < C::kGroups) scale_s[i % kScaleSlots * C::kGroups + lane] = sc;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_full[i % kScaleSlots]);
            }
            if (!convert(kbuf, 2 * i, 1u, sc)) break;
            load(kbuf, a.c.k, at_next);
            if (!convert(vbuf, 2 * i + 1, 2u, sc)) break;
            at = at_next, sc = sc_next;
        }
    } else if (warp / 4 < groups) {
        // ---------------------------------------------------- softmax, a row a thread
        const int m = warp / 4, r = tid;
        const uint32_t quad = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t s_at = tmem + C::kS(m) + quad, o_at = tmem + C::kO(m) + quad;
        const int pos = PREFIX ? len - 1 : pos0 + (r0 + r) / share;
        const int see = r < rows ? pos + 1 : 0;
        const int low = !PREFIX && a.window && pos >= a.window ? pos - a.window + 1 : 0;
        // rows m: tiles from `all_low` to `all_see` are seen by every one
        const int last = min(rows, m * 128 + 128) - 1;
        const int all_see = PREFIX ? len : pos0 + (r0 + m * 128) / share + 1;
        const int last_pos = PREFIX ? 0 : pos0 + (r0 + last) / share;
        const int all_low = !PREFIX && a.window && last_pos >= a.window ? last_pos - a.window + 1 : 0;
        const float mul = mul_s[r];
        float ref = 0.0f, sum = 0.0f;
        bool none = true, ok = true;
        uint32_t v[2][32];
        for (int i = 0; i < tiles; ++i) {
            const int tile = position(i);
            const float4 *sc = scale_s + i % kScaleSlots * C::kGroups;
            ok = __all_sync(0xffffffffu, mbar_wait(&sc_full[i % kScaleSlots], i / kScaleSlots & 1, abort_flag) &&
                                             mbar_wait(&s_full[m], i & 1, abort_flag));
            if (!ok) {
                if (lane == 0) give_up();
                break;
            }
            tc_fence_after();
            const bool edge = tile + kN > all_see || (tile < all_low && tile + kN > a.sinks);
            auto hidden = [&](int j) { return j >= see || (j < low && j >= a.sinks); };
            // the largest exponent, relative to the reference
            float top = -INFINITY;
            tmem_ld32(s_at, v[0]);
#pragma unroll
            for (int c = 0; c < kN / 32; ++c) {
                tmem_ld_wait32(v[c % 2]);
                if (c + 1 < kN / 32) tmem_ld32(s_at + 32 * (c + 1), v[(c + 1) % 2]);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float4 of = sc[2 * c + g];
                    const float f = of.x * mul, off = of.y - ref;
                    float x = -INFINITY;
                    if (edge) {
#pragma unroll
                        for (int u = 0; u < 16; ++u)
                            if (!hidden(tile + 32 * c + 16 * g + u)) x = fmaxf(x, __uint_as_float(v[c % 2][16 * g + u]));
                    } else {
#pragma unroll
                        for (int u = 0; u < 16; ++u) x = fmaxf(x, __uint_as_float(v[c % 2][16 * g + u]));
                    }
                    if (x > -INFINITY) top = fmaxf(top, fmaf(x, f, off));
                }
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
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        tmem_ld32(o_at + 32 * c, v[0]);
                        tmem_ld_wait32(v[0]);
#pragma unroll
                        for (int u = 0; u < 32; ++u) v[0][u] = __float_as_uint(__uint_as_float(v[0][u]) * keep);
                        tmem_st32(o_at + 32 * c, v[0]);
                    }
                }
            }
            tmem_ld32(s_at, v[0]);
#pragma unroll
            for (int c = 0; c < kN / 32; ++c) {
                tmem_ld_wait32(v[c % 2]);
                if (c + 1 < kN / 32) tmem_ld32(s_at + 32 * (c + 1), v[(c + 1) % 2]);
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float4 of = sc[2 * c + g];
                    const float f = of.x * mul, off = of.y - ref;
                    float part = 0.0f;
#pragma unroll
                    for (int u = 0; u < 16; u += 2) {
                        float x[2], p[2];
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            x[w] = fmaf(__uint_as_float(v[c % 2][16 * g + u + w]), f, off);
                            if (edge && hidden(tile + 32 * c + 16 * g + u + w)) x[w] = -INFINITY;
                            p[w] = tile_exp2(x[w]);
                        }
                        part += p[0] + p[1];
                        const __half2 h = __floats2half2_rn(p[0], p[1]);
                        hi[8 * g + u / 2] = *reinterpret_cast<const uint32_t *>(&h);
                        if (kPParts == 2) {
                            const float2 back = __half22float2(h);
                            const __half2 rest = __floats2half2_rn(p[0] - back.x, p[1] - back.y);
                            lo[8 * g + u / 2] = *reinterpret_cast<const uint32_t *>(&rest);
                        }
                    }
                    sum = fmaf(part, of.z, sum);
                }
                // in the place of the 32 columns of S that were read
                tmem_st16(s_at + 32 * c, hi);
                if (kPParts == 2) tmem_st16(s_at + 32 * c + 16, lo);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[m]);
        }
        if (ok && tiles > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&o_full[m], 0, abort_flag));
            if (!ok && lane == 0) give_up();
            tc_fence_after();
        }
        // ---- the row's outputs
        const int64_t n = (r0 + r) / share;
        const int head = hk * share + (r0 + r) % share;
        const bool there = r < rows && ok;
        const bool direct = !PREFIX && a.splits == 1 && !a.later;
        const int64_t part = (((int64_t)b * a.c.heads + hk) * a.rows + r0 + r) * a.splits + split;
        const bool some = sum > 0.0f || sum != sum;
        const float inv = some ? __frcp_rn(sum) : 0.0f;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            __syncwarp();
            if (tiles > 0) {
                tmem_ld32(o_at + 32 * c, v[0]);
                tmem_ld_wait32(v[0]);
            }
            if (!there) continue;
            float *o = reinterpret_cast<float *>(v[0]);
            if (tiles == 0 || (!some && direct)) {
#pragma unroll
                for (int u = 0; u < 32; ++u) o[u] = 0.0f;
            }
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
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace
}  // namespace bsg

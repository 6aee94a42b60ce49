// kv8.cu -- the int8 key/value cache: appending tokens, and attention over it.
//
// A page holds page_tokens tokens of every head; each page and head has one
// f32 scale for its keys and one for its values.  The codes follow the unit's
// ("Verification", section "The verified INT8 units", step 1: scale =
// max / 127 floored at 1e-8, floor(x inv + 0.5)) over a block of tokens in
// place of a row; the scale is one f32 product with f32(1/127).
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsg_internal.h"
#include "bsg_ptx.cuh"
#include "serve.cuh"

namespace bsg {
namespace {

template <int N>
__device__ __forceinline__ float block_max(float x, float *red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int i = 1; i < N / 32; ++i) x = fmaxf(x, red[i]);
    __syncthreads();
    return x;
}

template <int N>
__device__ __forceinline__ float block_sum(float x, float *red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int i = 1; i < N / 32; ++i) x += red[i];
    __syncthreads();
    return x;
}

// One CTA per touched page of a sequence, head, and side (keys or values).
template <typename T>
__global__ void __launch_bounds__(128)
    kv8_append_kernel(bsg_kv8_cache c, const int32_t *__restrict__ table, int64_t table_ld,
                      const int32_t *__restrict__ starts, const int32_t *__restrict__ counts,
                      bsg_tokens tk, bsg_tokens tv, int blocks, int tokens,
                      int32_t *__restrict__ dstatus) {
    __shared__ float red[4];
    const int b = blockIdx.x / blocks, h = blockIdx.y, t = threadIdx.x;
    const int start = starts[b], count = counts ? counts[b] : tokens;
    if (start < 0 || count < 0 || count > tokens) {
        if (t == 0) set_status(dstatus, BSG_DSTATUS_RANGE);
        return;
    }
    const int P = c.page_tokens, D = c.dim;
    const int64_t end = (int64_t)start + count;
    const int64_t j = start / P + blockIdx.x % blocks;  // the sequence's page
    if (j * P >= end) return;
    int page = -1;
    if (j < table_ld) page = table[b * table_ld + j];
    if (page < 0 || page >= c.pages) {
        if (t == 0) set_status(dstatus, BSG_DSTATUS_RANGE);
        return;
    }
    const bsg_tokens &tok = blockIdx.z ? tv : tk;
    const int64_t ph = (int64_t)page * c.heads + h;
    int8_t *codes = (blockIdx.z ? c.v : c.k) + ph * P * D;
    float *scale = (blockIdx.z ? c.v_scale : c.k_scale) + ph;
    const int lo = (int)(start > j * P ? start - j * P : 0);              // new tokens: [lo, hi)
    const int hi = (int)(end < (j + 1) * P ? end - j * P : P);
    const T *x = (const T *)tok.data + b * tok.stride_batch + h * tok.stride_head +
                 (j * P - start) * tok.stride_token;
    float m = 0.0f;
    bool bad = false;
    for (int i = lo * D + t; i < hi * D; i += 128) {
        const float v = to_f32(x[(i / D) * tok.stride_token + i % D]);
        bad |= !isfinite(v);
        m = fmaxf(m, fabsf(v));
    }
    if (bad) set_status(dstatus, BSG_DSTATUS_NONFINITE);
    m = block_max<128>(m, red);
    float s = kv8_scale(m);
    if (lo > 0) {
        const float old = *scale;
        if (old < s) {
            const float r = __fdiv_rn(old, s);
            for (int i = t; i < lo * D; i += 128) codes[i] = (int8_t)unit_code(codes[i], r);
        } else {
            s = old;
        }
    }
    const float inv = __fdiv_rn(1.0f, s);
    for (int i = lo * D + t; i < hi * D; i += 128)
        codes[i] = (int8_t)unit_code(to_f32(x[(i / D) * tok.stride_token + i % D]), inv);
    __syncthreads();  // every thread has read the old scale
    if (t == 0) *scale = s;
}

// ---- attention ----------------------------------------------------------------
//
// out = sum_j p_j v_j over one sequence and key/value head, for the rows (query
// tokens x query heads) that share it.  The work is reading 2 len dim bytes of
// codes once; a CTA takes a chunk of the positions, its warps every kWarps-th
// tile of 16 positions each, and all is joined at the end.  Per tile and warp:
//
//   S^T (16 positions x 8 slots) = K (16 x dim) . Q^T      mma m16n8k16, f32 sums
//   p = 2^(S' - ref),  S' = S * page scale * softmax scale * log2 e
//   O^T (dim x 8 slots) += page scale * (V^T (dim x 16) . P^T (16 x 8 slots))
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
// (a power of two), so two parts keep 2^-22 of it; probabilities keep 2^-22 of
// themselves.  16-bit types have one part: their queries are exact in it, and
// their probabilities keep 11 bits, as many as the output can show.
//
// The running reference `ref` follows a row's maximum only when that is more
// than 2^8 above it: probabilities stay below 2^8 (f16 holds 2^15) and the
// outputs are rescaled a few times per row instead of at every tile.

constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr float kRefNone = -3.0e38f;  // the reference of a row that has seen nothing
constexpr float kSlack = 8.0f;

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

// D = A B + C, A 16 x 16 f16 (row), B 16 x 8 f16 (column), C and D f32.
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

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Two codes, already + 128 (unsigned bytes `sel` picks of x), as f16.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_half2(uint32_t x) {
    const uint32_t m = __byte_perm(x, 0x64646464u, SEL);
    const uint32_t bias = 0x64806480u;  // 1152, 1152
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&m),
                              *reinterpret_cast<const __half2 *>(&bias));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Which dim the lane's word `w` of a key row starts at (t = lane % 4), and of a
// value row (g = lane / 4): 16-byte pieces of 64 (128) bytes, then smaller ones.
template <int D>
__host__ __device__ constexpr int key_dim(int w, int t) {
    return w < D / 64 * 4 ? w / 4 * 64 + 16 * t + w % 4 * 4 : D / 64 * 64 + 8 * t + (w - D / 64 * 4) * 4;
}
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
    int dtype, tokens, heads, rows, row_tiles, chunk, splits;
    float scale;
    float *lse, *part_o, *part_ml;
    int32_t *dstatus;
};

__device__ __forceinline__ float load_any(const void *p, int64_t i, int dtype) {
    return dtype == BSG_F32   ? static_cast<const float *>(p)[i]
           : dtype == BSG_F16 ? __half2float(static_cast<const __half *>(p)[i])
                              : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
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
    const int len = a.lens[b];
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
              a.dtype, l > 0.0f || l != l ? __fdividef(o, l) : 0.0f);
    if (d == 0 && a.lse)
        a.lse[((int64_t)b * a.tokens + at.token) * a.heads + at.head] =
            l > 0.0f || l != l ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// Shared memory: the queries, then the warps' rings, whose place the partial
// outputs take at the end.
template <int D, int NT, int kParts>
constexpr int attend_smem() {
    constexpr int rings = kWarps * kStages * 32 * D;
    constexpr int join = kWarps * (8 * NT / kParts) * (D + 2) * 4;
    return NT * (D / 16) * 32 * 8 + (rings > join ? rings : join);
}

// grid (splits, heads x row tiles, B)
template <int D, int NT, int kParts>
__global__ void __launch_bounds__(kWarps * 32) kv8_attend_kernel(const AttendArgs a) {
    constexpr int kRows = 8 * NT / kParts;  // rows of a CTA
    constexpr int kStep = D / 16;           // k16 steps of q.k, m16 tiles of the output
    extern __shared__ __align__(16) uint8_t smem[];
    uint2 *q_s = reinterpret_cast<uint2 *>(smem);                   // [NT][kStep][32 lanes]
    uint8_t *ring_s = smem + NT * kStep * 32 * 8;                   // [warp][stage][K, V tile]
    float *o_s = reinterpret_cast<float *>(ring_s);                 // [warp][row][D + 2]: l last
    __shared__ float4 scales_s[kWarps][kStages];                    // of a stage's tile; z: 1 if there
    __shared__ float mul_s[kRows];                                  // score multiplier of each row
    __shared__ float max_s[kRows][kWarps];
    const int b = blockIdx.z, hk = blockIdx.y / a.row_tiles;
    const int r0 = blockIdx.y % a.row_tiles * kRows;
    const int rows = min(kRows, a.rows - r0);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
    const int len = length_of(a, b, blockIdx.x == 0 && tid == 0);
    const int j0 = blockIdx.x * a.chunk;
    if (j0 >= len && (blockIdx.x > 0 || a.splits > 1)) return;  // the join knows that it has no part
    const int j1 = min(len, j0 + a.chunk);

    // The pages and scales of the warp's next 32 tiles, one to a lane.
    const int P = a.c.page_tokens;
    const int32_t *table = a.table + b * a.table_ld;
    const int tiles = (j1 + 15) / 16;
    int first = j0 / 16 + warp;             // the tile of lane 0
    int my_page = -1;
    float my_ks = 0.0f, my_vs = 0.0f;
    auto look_up = [&]() {
        const int tile = first + lane * kWarps;
        my_page = -1;
        if (tile < tiles) {
            const int p = table[tile * 16 / P];
            if (p >= 0 && p < a.c.pages) {
                my_page = p;
                my_ks = a.c.k_scale[(int64_t)p * a.c.heads + hk];
                my_vs = a.c.v_scale[(int64_t)p * a.c.heads + hk];
            } else {
                set_status(a.dstatus, BSG_DSTATUS_RANGE);
            }
        }
    };
    look_up();
    // Copy the warp's next tile into a stage (nothing past the last, or where
    // the page is none); a group of copies each time, so that they count.
    uint8_t *ring = ring_s + warp * kStages * 32 * D;
    int next = first, in_batch = 0;
    auto fetch = [&](int stage) {
        if (in_batch == 32) {
            in_batch = 0;
            first = next;
            look_up();
        }
        const int page = __shfl_sync(0xffffffffu, my_page, in_batch);
        if (lane == in_batch) scales_s[warp][stage] = make_float4(my_ks, my_vs, page < 0 ? 0.0f : 1.0f, 0.0f);
        if (page >= 0) {
            const int64_t at = (((int64_t)page * a.c.heads + hk) * P + next * 16 % P) * D;
            const uint32_t dst = smem_u32(ring + stage * 32 * D);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int e = (i * 32 + lane) * 16, r = e / D, col = e % D;
                copy16(dst + tile_at<D>(r, col), a.c.k + at + e);
                copy16(dst + 16 * D + tile_at<D>(r, col), a.c.v + at + e);
            }
        }
        copies_commit();
        ++in_batch;
        next += kWarps;
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(i);

    // Queries: each row relative to a power of two near its largest |q|, in
    // f16 parts, laid out as the B operand.
    for (int r = warp; r < kRows; r += kWarps) {
        float m = 0.0f, x[(D + 31) / 32];
        bool bad = false;
        const RowAt ra = row_at(a, hk, min(r0 + r, a.rows - 1));
        const int64_t base = b * a.q.stride_batch + ra.token * a.q.stride_token +
                             ra.head * a.q.stride_head;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            x[i] = r < rows ? load_any(a.q.data, base + lane + 32 * i, a.dtype) : 0.0f;
            bad |= !isfinite(x[i]);
            m = fmaxf(m, fabsf(x[i]));
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
        for (int i = 0; i < D / 32; ++i) {
            const int d = lane + 32 * i;
            // the step and lane whose word covers dim d
            int w, tt;
            if (d < D / 64 * 64)
                w = d / 64 * 4 + d % 16 / 4, tt = d % 64 / 16;
            else
                w = D / 64 * 4 + d % 8 / 4, tt = d % 32 / 8;
            const float y = x[i] * up;
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
    int see[NT][2];
    float acc[NT][kStep][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = (8 * n + 2 * t + u) / kParts;
            mul[n][u] = mul_s[r];
            ref[n][u] = kRefNone;
            sum[n][u] = 0.0f;
            see[n][u] = r < rows ? len - a.tokens + row_at(a, hk, r0 + r).token + 1 : 0;
        }
#pragma unroll
        for (int i = 0; i < kStep; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[n][i][u] = 0.0f;
    }

    int stage = 0;
    for (int tile = j0 / 16 + warp; tile < tiles; tile += kWarps) {
        copies_wait<kStages - 1>();
        __syncwarp();
        const uint8_t *kt = ring + stage * 32 * D, *vt = kt + 16 * D;
        const float4 of_tile = scales_s[warp][stage];
        const float ks = of_tile.x, vs = of_tile.y;
        if (of_tile.z == 0.0f) {
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

        // Scores in powers of two; kParts = 2: one row's in s[n][0] and s[n][2].
        bool above = false;
        const bool edge = tile * 16 + 16 > len - a.tokens;  // some row may not see all of it
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (kParts == 2) {
                s[n][0] = fmaf(s[n][1], 0x1p-11f, s[n][0]) * (ks * mul[n][0]);
                s[n][2] = fmaf(s[n][3], 0x1p-11f, s[n][2]) * (ks * mul[n][0]);
            } else {
                s[n][0] *= ks * mul[n][0], s[n][1] *= ks * mul[n][1];
                s[n][2] *= ks * mul[n][0], s[n][3] *= ks * mul[n][1];
            }
            if (edge) {
                const int p0 = tile * 16 + g;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (p0 + u / 2 * 8 >= see[n][u % 2]) s[n][u] = -INFINITY;
            }
#pragma unroll
            for (int u = 0; u < 4; u += kParts) above |= s[n][u] > ref[n][u % 2] + kSlack;
        }
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float keep[2];
#pragma unroll
                for (int u = 0; u < 2; u += kParts) {
                    float m = fmaxf(s[n][u], s[n][u + 2]);
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    keep[u] = 1.0f;
                    if (m > ref[n][u] + kSlack) {  // of this row alone
                        keep[u] = exp2_fast(ref[n][u] - m);
                        ref[n][u] = m;
                        sum[n][u] *= keep[u];
                    }
                }
                if (kParts == 2) keep[1] = keep[0];
#pragma unroll
                for (int i = 0; i < kStep; ++i)
#pragma unroll
                    for (int u = 0; u < 4; ++u) acc[n][i][u] *= keep[u % 2];
            }
        }
        // Probabilities, as the B operand of the second product.
        uint32_t p01[NT], p89[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (kParts == 2) {
                const float pa = exp2_fast(s[n][0] - ref[n][0]);
                const float pb = exp2_fast(s[n][2] - ref[n][0]);
                sum[n][0] += pa + pb;
                const float ha = __half2float(__float2half_rn(pa));
                const float hb = __half2float(__float2half_rn(pb));
                p01[n] = transpose8(pack_half2(ha, (pa - ha) * 2048.0f));
                p89[n] = transpose8(pack_half2(hb, (pb - hb) * 2048.0f));
            } else {
                float p[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) p[u] = exp2_fast(s[n][u] - ref[n][u % 2]);
                sum[n][0] += p[0] + p[2];
                sum[n][1] += p[1] + p[3];
                p01[n] = transpose8(pack_half2(p[0], p[1]));
                p89[n] = transpose8(pack_half2(p[2], p[3]));
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
                for (int n = 0; n < NT; ++n) {
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma_16816(d, a0, a1, a2, a3, p01[n], p89[n]);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        acc[n][2 * w + h][u] = fmaf(d[u], vs, acc[n][2 * w + h][u]);
                }
            }
        }
        __syncwarp();  // every lane has read the stage
        fetch(stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    copies_wait<0>();
    __syncthreads();  // the rings are free

    // Join the warps: sums over the lanes of a column, then over the warps,
    // each relative to the largest reference.
    float *mine = o_s + warp * kRows * (D + 2);
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
                mine[r * (D + 2) + D] = l;
                max_s[r][warp] = ref[n][u];
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
                *reinterpret_cast<float2 *>(mine + r * (D + 2) + d) = o;
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < rows * D; e += kWarps * 32) {
        const int r = e / D, d = e % D;
        float m = max_s[r][0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = fmaxf(m, max_s[r][w]);
        float o = 0.0f, l = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2_fast(max_s[r][w] - m);
            o = fmaf(o_s[(w * kRows + r) * (D + 2) + d], f, o);
            l = fmaf(o_s[(w * kRows + r) * (D + 2) + D], f, l);
        }
        if (a.splits == 1) {
            store_row(a, b, hk, r0 + r, d, o, m, l);
        } else {
            const int64_t part =
                (((int64_t)b * a.c.heads + hk) * a.rows + r0 + r) * a.splits + blockIdx.x;
            a.part_o[part * D + d] = o;
            if (d == 0) a.part_ml[2 * part] = m, a.part_ml[2 * part + 1] = l;
        }
    }
}

// Joins the splits of one row: grid (rows, heads, B), dim threads.
__global__ void kv8_join_kernel(const AttendArgs a) {
    const int r = blockIdx.x, hk = blockIdx.y, b = blockIdx.z, d = threadIdx.x, D = blockDim.x;
    const int len = length_of(a, b, false);
    const int n = (len + a.chunk - 1) / a.chunk;
    const int64_t part = (((int64_t)b * a.c.heads + hk) * a.rows + r) * a.splits;
    const float *ml = a.part_ml + 2 * part, *po = a.part_o + part * D + d;
    float m = kRefNone;
    for (int i = 0; i < n; ++i) m = fmaxf(m, ml[2 * i]);
    float o = 0.0f, l = 0.0f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float f = exp2_fast(ml[2 * i] - m);
        o = fmaf(po[(int64_t)i * D], f, o);
        l = fmaf(ml[2 * i + 1], f, l);
    }
    store_row(a, b, hk, r, d, o, m, l);
}

}  // namespace

cudaError_t launch_kv8_append(const bsg_kv8_cache &c, const int32_t *table, int64_t table_ld,
                              const int32_t *starts, const int32_t *counts, const bsg_tokens &k,
                              const bsg_tokens &v, int dtype, int64_t B, int64_t T,
                              int32_t *dstatus, cudaStream_t st) {
    // T tokens from any position touch at most this many pages
    const int64_t blocks = (T - 2 + c.page_tokens) / c.page_tokens + 1;
    if (B * blocks > INT32_MAX) return cudaErrorInvalidValue;
    return with_dtype(dtype, [&](auto t) {
        using E = decltype(t);
        const dim3 grid((unsigned)(B * blocks), (unsigned)c.heads, 2);
        kv8_append_kernel<E><<<grid, 128, 0, st>>>(c, table, table_ld, starts, counts, k, v,
                                                   (int)blocks, (int)T, dstatus);
        count_launches(1);
        return cudaGetLastError();
    });
}

// How a call is laid out: slots of 8 that a CTA holds, and how the positions
// are split.  Splits follow the table's width alone (lengths are in device
// memory).
struct AttendPlan {
    int parts, nt, rows, row_tiles, chunk, splits;
};
static AttendPlan attend_plan(const bsg_kv8_cache &c, int64_t table_ld, int64_t B, int64_t T,
                              int heads, int parts) {
    AttendPlan p;
    p.parts = parts;
    p.rows = (int)T * (heads / c.heads);
    const int slots = p.rows * parts;
    p.nt = slots <= 8 ? 1 : slots <= 16 || c.dim == 256 ? 2 : 4;
    p.row_tiles = (slots + 8 * p.nt - 1) / (8 * p.nt);
    const int64_t groups = B * c.heads * p.row_tiles, most = table_ld * c.page_tokens;
    const int64_t ctas = (int64_t)device_sm_count() * 16;
    int64_t splits = (ctas + groups - 1) / groups;
    const int64_t least = 64;  // positions of a split: one tile for each warp
    if (splits > (most + least - 1) / least) splits = (most + least - 1) / least;
    if (splits > 1024) splits = 1024;
    const int64_t chunk = ((most + splits - 1) / splits + least - 1) / least * least;
    p.chunk = (int)chunk;
    p.splits = (int)((most + chunk - 1) / chunk);
    return p;
}

size_t kv8_attend_workspace_bytes(const bsg_kv8_cache &c, int64_t table_ld, int64_t B, int64_t T,
                                  int heads) {
    size_t most = 256;
    for (int parts = 1; parts <= 2; ++parts) {
        const AttendPlan p = attend_plan(c, table_ld, B, T, heads, parts);
        const size_t n = (size_t)B * c.heads * p.rows * p.splits * (c.dim + 2) * 4;
        if (p.splits > 1 && n > most) most = n;
    }
    return (most + 255) / 256 * 256;
}

template <int D, int NT, int kParts>
static cudaError_t launch_attend(const AttendArgs &a, const dim3 &grid, cudaStream_t st) {
    constexpr int smem = attend_smem<D, NT, kParts>();
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kv8_attend_kernel<D, NT, kParts>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kv8_attend_kernel<D, NT, kParts><<<grid, kWarps * 32, smem, st>>>(a);
    return cudaGetLastError();
}

template <int D>
static cudaError_t launch_attend_dim(const AttendArgs &a, const AttendPlan &p, const dim3 &grid,
                                     cudaStream_t st) {
    if (p.parts == 1) {
        if (p.nt == 1) return launch_attend<D, 1, 1>(a, grid, st);
        if (p.nt == 2) return launch_attend<D, 2, 1>(a, grid, st);
        if constexpr (D < 256) return launch_attend<D, 4, 1>(a, grid, st);
    } else {
        if (p.nt == 1) return launch_attend<D, 1, 2>(a, grid, st);
        if (p.nt == 2) return launch_attend<D, 2, 2>(a, grid, st);
        if constexpr (D < 256) return launch_attend<D, 4, 2>(a, grid, st);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv8_attend(const bsg_kv8_cache &c, const int32_t *table, int64_t table_ld,
                              const int32_t *lens, const bsg_tokens &q, const bsg_tokens &out,
                              int dtype, int64_t B, int64_t T, int heads, float scale, float *lse,
                              void *ws, int32_t *dstatus, cudaStream_t st) {
    const AttendPlan p = attend_plan(c, table_ld, B, T, heads, dtype == BSG_F32 ? 2 : 1);
    AttendArgs a{c, table, table_ld, lens, q, out, dtype, (int)T, heads, p.rows, p.row_tiles,
                 p.chunk, p.splits, scale, lse, nullptr, nullptr, dstatus};
    a.part_o = static_cast<float *>(ws);
    a.part_ml = a.part_o + (size_t)B * c.heads * p.rows * p.splits * c.dim;
    if ((int64_t)c.heads * p.row_tiles > 65535) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)p.splits, (unsigned)(c.heads * p.row_tiles), (unsigned)B);
    cudaError_t e;
    switch (c.dim) {
        case 32: e = launch_attend_dim<32>(a, p, grid, st); break;
        case 64: e = launch_attend_dim<64>(a, p, grid, st); break;
        case 96: e = launch_attend_dim<96>(a, p, grid, st); break;
        case 128: e = launch_attend_dim<128>(a, p, grid, st); break;
        default: e = launch_attend_dim<256>(a, p, grid, st); break;
    }
    if (e != cudaSuccess) return e;
    count_launches(1);
    if (p.splits > 1) {
        kv8_join_kernel<<<dim3((unsigned)p.rows, (unsigned)c.heads, (unsigned)B), c.dim, 0, st>>>(a);
        count_launches(1);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace bsg

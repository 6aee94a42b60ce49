// serving_api.cu -- the C ABI of the serving calls: argument checks, then the
// launchers of wgroups.cu, kv8.cu and logprobs.cu.
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsg_internal.h"
#include "bsgemm.h"

namespace bsg {
namespace {

bsg_status done(cudaError_t e) { return e == cudaSuccess ? BSG_OK : BSG_ERR_CUDA; }

cudaStream_t stream_of(void *s) { return static_cast<cudaStream_t>(s); }

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool ws_ok(const void *ws, size_t have, size_t need) {
    return need == 0 || (ws != nullptr && aligned(ws, 256) && have >= need);
}

// A known type, and a pointer on one of its elements.
bool typed(const void *p, bsg_dtype t) {
    return p != nullptr && (t == BSG_F32 || t == BSG_F16 || t == BSG_BF16) &&
           aligned(p, t == BSG_F32 ? 4 : 2);
}

// Element counts and offsets stay inside the kernels' 64-bit arithmetic:
// rows and columns below 2^31.
bool size_ok(int64_t n) { return n >= 1 && n <= INT32_MAX; }

bool group_ok(int group) { return group >= 0 && group % 32 == 0; }

bool cache_ok(const bsg_kv8_cache *c) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return false;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) ||
        !aligned(c->v_scale, 4))
        return false;
    if (c->pages < 1 || c->pages > INT32_MAX || c->heads < 1 || c->heads > 65535) return false;
    if (c->page_tokens < 16 || c->page_tokens > 1024 || c->page_tokens % 16) return false;
    return c->dim == 32 || c->dim == 64 || c->dim == 96 || c->dim == 128 || c->dim == 256;
}

// Batches fill a grid's y or z; a sequence's positions stay in int32.
bool table_ok(const bsg_kv8_cache *c, const int32_t *table, int64_t table_ld, int64_t B) {
    return table && aligned(table, 4) && B >= 1 && B <= 65535 && table_ld >= 1 &&
           table_ld <= (INT32_MAX / 2) / c->page_tokens;
}

}  // namespace
}  // namespace bsg

using namespace bsg;

extern "C" {

bsg_status bsg_wquant_groups(const float *W, int64_t K, int64_t N, int64_t ldw, int group,
                             uint8_t *Q, int64_t ldq, float *scale, int64_t lds,
                             int32_t *dstatus, void *stream) {
    if (!typed(W, BSG_F32) || !Q || !typed(scale, BSG_F32) || !size_ok(K) || !size_ok(N) ||
        ldw < N || ldq < (N + 1) / 2 || lds < N || !group_ok(group))
        return BSG_ERR_ARG;
    const bsg_status s = check_device();
    if (s != BSG_OK) return s;
    return done(launch_wquant_groups(W, K, N, ldw, group ? group : K, Q, ldq, scale, lds, dstatus,
                                     stream_of(stream)));
}

size_t bsg_wgroups_matvec_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M < 1 || M > BSG_MATVEC_MAX_M || N < 1 || N > (1 << 25) || K < 1 || K > (1 << 30)) return 0;
    return matvec_workspace_bytes(M, N, K);
}

bsg_status bsg_wgroups_matvec(const void *X, bsg_dtype dtype, int64_t ldx, const uint8_t *Q,
                              int64_t ldq, const float *scale, int64_t lds, int group, int64_t M,
                              int64_t N, int64_t K, int relu, void *Y, int64_t ldy,
                              void *workspace, size_t ws_bytes, int32_t *dstatus, void *stream) {
    if (!typed(X, dtype) || !typed(Y, dtype) || !Q || !typed(scale, BSG_F32) || M < 1 ||
        M > BSG_MATVEC_MAX_M || N < 1 || N > (1 << 25) || K < 1 || K > (1 << 30) || ldx < K || ldy < N ||
        ldq < (N + 1) / 2 || lds < N || !group_ok(group) || (relu != 0 && relu != 1))
        return BSG_ERR_ARG;
    if (!ws_ok(workspace, ws_bytes, matvec_workspace_bytes(M, N, K))) return BSG_ERR_WORKSPACE;
    const bsg_status s = check_device();
    if (s != BSG_OK) return s;
    return done(launch_wgroups_matvec(X, dtype, ldx, Q, ldq, scale, lds, group ? group : K, M, N,
                                      K, relu, Y, ldy, workspace, dstatus, stream_of(stream)));
}

bsg_status bsg_kv8_append(const bsg_kv8_cache *cache, const int32_t *table, int64_t table_ld,
                          const int32_t *starts, const int32_t *counts, const bsg_tokens *k,
                          const bsg_tokens *v, bsg_dtype dtype, int64_t B, int64_t T,
                          int32_t *dstatus, void *stream) {
    if (!cache_ok(cache) || !table_ok(cache, table, table_ld, B) || !starts || !k || !v ||
        !typed(k->data, dtype) || !typed(v->data, dtype) || T < 1 || T > INT32_MAX / 2)
        return BSG_ERR_ARG;
    const bsg_status s = check_device();
    if (s != BSG_OK) return s;
    return done(launch_kv8_append(*cache, table, table_ld, starts, counts, *k, *v, dtype, B, T,
                                  dstatus, stream_of(stream)));
}

size_t bsg_kv8_attend_workspace_size(const bsg_kv8_cache *cache, int64_t table_ld, int64_t B,
                                     int64_t T, int heads) {
    static const int32_t any = 0;
    if (!cache_ok(cache) || !table_ok(cache, &any, table_ld, B) || T < 1 || T > BSG_KV8_MAX_T ||
        heads < 1 || heads % cache->heads)
        return 0;
    return kv8_attend_workspace_bytes(*cache, table_ld, B, T, heads);
}

bsg_status bsg_kv8_attend(const bsg_kv8_cache *cache, const int32_t *table, int64_t table_ld,
                          const int32_t *lens, const bsg_tokens *q, const bsg_tokens *out,
                          bsg_dtype dtype, int64_t B, int64_t T, int heads, float scale,
                          float *lse, void *workspace, size_t ws_bytes, int32_t *dstatus,
                          void *stream) {
    if (!cache_ok(cache) || !table_ok(cache, table, table_ld, B) || !lens || !q || !out ||
        !typed(q->data, dtype) || !typed(out->data, dtype) || T < 1 || T > BSG_KV8_MAX_T ||
        heads < 1 || heads > 65535 || heads % cache->heads || !(scale - scale == 0.0f))
        return BSG_ERR_ARG;
    if (!ws_ok(workspace, ws_bytes, kv8_attend_workspace_bytes(*cache, table_ld, B, T, heads)))
        return BSG_ERR_WORKSPACE;
    const bsg_status s = check_device();
    if (s != BSG_OK) return s;
    return done(launch_kv8_attend(*cache, table, table_ld, lens, *q, *out, dtype, B, T, heads,
                                  scale, lse, workspace, dstatus, stream_of(stream)));
}

bsg_status bsg_logprobs(const void *logits, bsg_dtype dtype, int64_t M, int64_t V, int64_t ldl,
                        const int64_t *target, int top, float *logprob, float *entropy,
                        float *lse, float *top_logprob, int32_t *top_id, int32_t *dstatus,
                        void *stream) {
    if (!typed(logits, dtype) || !size_ok(M) || !size_ok(V) || ldl < V || top < 0 ||
        top > BSG_MAX_TOP || top > V || (top > 0 && (!top_logprob || !top_id)))
        return BSG_ERR_ARG;
    const bsg_status s = check_device();
    if (s != BSG_OK) return s;
    return done(launch_logprobs(logits, dtype, M, V, ldl, target, top, logprob, entropy, lse,
                                top_logprob, top_id, dstatus, stream_of(stream)));
}

bsg_status bsg_logprobs_backward(const void *logits, bsg_dtype dtype, int64_t M, int64_t V,
                                 int64_t ldl, const int64_t *target, const float *lse,
                                 const float *entropy, const float *g_logprob,
                                 const float *g_entropy, void *dlogits, int64_t ldd,
                                 int32_t *dstatus, void *stream) {
    if (!typed(logits, dtype) || !typed(dlogits, dtype) || !size_ok(M) || !size_ok(V) ||
        ldl < V || ldd < V || !lse || (g_entropy && !entropy))
        return BSG_ERR_ARG;
    if (dlogits == logits && ldd != ldl) return BSG_ERR_ARG;
    const bsg_status s = check_device();
    if (s != BSG_OK) return s;
    return done(launch_logprobs_backward(logits, dtype, M, V, ldl, target, lse, entropy, g_logprob,
                                         g_entropy, dlogits, ldd, dstatus, stream_of(stream)));
}

}  // extern "C"

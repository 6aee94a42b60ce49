"""Plain definitions of the calls for prompts, windows and shared prefixes, in numpy
(64 bits), for the tests.  Each follows include/bsgemm.h and shares no code with the
library."""
import numpy as np
import torch


def codes_of(x):
    """(codes, scale) of float32 rows by the unit's step 1, every rounding to float32
    written out."""
    f = np.float32
    m = np.abs(x).max(1).astype(np.float64)
    s = np.maximum(m / 127.0, 1e-8).astype(f)
    inv = (1.0 / s.astype(np.float64)).astype(f)
    q = np.floor((x.astype(f) * inv[:, None]).astype(f) + f(0.5))
    return q.astype(np.int64), s


def matmul(x, codes, scale, relu, dtype):
    """The product's bits: x float32 (M, K), codes int8 (K, N), scale float32 (N,)."""
    q, s = codes_of(x)
    S = q.astype(np.float64) @ codes.astype(np.float64)        # whole numbers below 2^31: exact
    y = (S.astype(np.float32) * s[:, None]).astype(np.float32) * scale[None].astype(np.float32)
    if relu:
        y = np.where(y > 0, y, np.float32(0))
    return torch.from_numpy(np.ascontiguousarray(y, np.float32)).to(dtype)


def cached(cache, pages, n, head):
    """(k, v) of the first n tokens in these pages, 64 bits."""
    D = cache[0].shape[3]
    return [(cache[i][pages, head].astype(np.float64)
             * cache[i + 2][pages, head].astype(np.float64)[:, None, None]).reshape(-1, D)[:n] for i in (0, 1)]


def softmax_attend(q, k, v, see, scale, parts):
    """(out, lse, tol, lse_tol) of rows q (R, D) over k, v (n, D) where see (R, n).

    tol, what float32 scores and sums may be off: scores by 2^-20 of sum |q k| for the
    products and their float32 sums and 2^-21 of max|q| sum |k| for q's parts, exp's
    argument by 2^-21 |s - max|, sums by 2^-20; and, where probabilities are one f16
    part (parts = 1), each by 2^-11 of itself.  f16 ends in steps of 2^-24, and a row's
    largest probability is kept as 2^9 or more: half a step, 2^-25, is 2^-34 of it.  lse_tol: the mean of the
    scores' errors, 2^-20 of the sum and of lse itself."""
    R, D = q.shape
    out, tol, lse, lse_tol = np.zeros((R, D)), np.zeros((R, D)), np.full(R, -np.inf), np.zeros(R)
    some = see.any(1)
    if not some.any():
        return out, lse, tol, lse_tol
    q, see = q[some], see[some]
    s = scale * (q @ k.T)
    s = np.where(see, s, -np.inf)
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    l = e.sum(1, keepdims=True)
    p = e / l
    ds = abs(scale) * (2.0 ** -20 * (np.abs(q) @ np.abs(k).T)
                       + 2.0 ** -21 * np.abs(q).max(1, keepdims=True) * np.abs(k).sum(1)[None])
    ds = np.where(see, ds + 2.0 ** -21 * np.minimum(np.abs(np.where(see, s, 0) - m), 100), 0)
    w = p * (ds + (p * ds).sum(1, keepdims=True) + 2.0 ** -20 + (2.0 ** -11 if parts == 1 else 0)) + np.where(see, 2.0 ** -34, 0) / l
    out[some], lse[some] = p @ v, (m + np.log(l))[:, 0]
    tol[some] = w @ np.abs(v)
    lse_tol[some] = (p * ds).sum(1) + 2.0 ** -20 * (2 + np.abs(lse[some]))
    return out, lse, tol, lse_tol


def window(q, cache, table, lens, counts, window, sinks, scale, parts=2):
    """(out, lse, tol, lse_tol), zeros where a token is not there."""
    B, T, H, D = q.shape
    Hk, P = cache[0].shape[1], cache[0].shape[2]
    out, tol, lse, lt = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, T, H)), np.zeros((B, T, H))
    for b in range(B):
        n, c = int(lens[b]), int(counts[b])
        i = np.arange(n - c, n)[:, None]
        j = np.arange(n)[None]
        see = (j <= i) & ((j > i - (window or 1 << 40)) | (j < sinks))
        pages = table[b, : -(-n // P)]
        for h in range(H if c else 0):
            g = h // (H // Hk)
            k, v = cached(cache, np.clip(pages, 0, cache[0].shape[0] - 1), n, g)
            out[b, :c, h], lse[b, :c, h], tol[b, :c, h], lt[b, :c, h] = softmax_attend(q[b, :c, h], k, v, see, scale, parts)
    return out, lse, tol, lt


def shared(q, cache, prefix, prefix_len, table, lens, scale, parts=2):
    B, T, H, D = q.shape
    Hk, P = cache[0].shape[1], cache[0].shape[2]
    out, tol, lse, lt = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, T, H)), np.zeros((B, T, H))
    for h in range(H):
        g = h // (H // Hk)
        k0, v0 = cached(cache, prefix, prefix_len, g)
        for b in range(B):
            n = int(lens[b])
            k1, v1 = cached(cache, table[b, : -(-n // P)], n, g)
            i, j = np.arange(n - T, n)[:, None], np.arange(n)[None]
            see = np.concatenate([np.broadcast_to(i >= 0, (T, prefix_len)), j <= i], 1)
            out[b, :, h], lse[b, :, h], tol[b, :, h], lt[b, :, h] = softmax_attend(
                q[b, :, h], np.concatenate([k0, k1]), np.concatenate([v0, v1]), see, scale, parts)
    return out, lse, tol, lt

"""Plain definitions of the serving calls, in numpy (64 bits), for the tests.

Each follows include/bsgemm.h and shares no code with the library."""
import numpy as np
import torch

UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
IDS = ["f32", "f16", "bf16"]


def f64(t):
    return t.detach().double().cpu().numpy()


def rounding(y, dtype):
    """Half a unit in the last place of results y in dtype."""
    tiny = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
    return np.abs(y) * UNIT[dtype] + tiny[dtype]


def within(got, want, tol, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = ~(np.abs(got - want) <= tol)
    if off.any():
        i = tuple(int(v) for v in np.argwhere(off)[0])
        t = np.broadcast_to(tol, got.shape)[i]
        raise AssertionError(f"{what}: {int(off.sum())} of {off.size} outside; first {i}: "
                             f"{got[i]!r}, want {want[i]!r} +- {t!r}")


# ---- int4 weights with group scales
def unpack4(Q, N):
    Q = np.asarray(Q).astype(np.int64)
    q = np.stack([Q & 15, Q >> 4], 2).reshape(Q.shape[0], -1)[:, :N]
    return q - 16 * (q >= 8)


def stored(Q, scale, N, group):
    """The stored weight, 64 bits."""
    K = Q.shape[0]
    return unpack4(Q, N) * np.asarray(scale, np.float64)[np.arange(K) // (group or K)]


# ---- int8 cache
def append(k, v, cache, table, starts, counts):
    """The cache (k, v int8; k_scale, v_scale f32 arrays, changed in place)
    after the append, with every rounding to float32 written out.  k, v:
    float32 arrays (B, T, H, D)."""
    f = np.float32
    P = cache[0].shape[2]
    for x, codes, scales in ((k, cache[0], cache[2]), (v, cache[1], cache[3])):
        for b in range(x.shape[0]):
            p, end = int(starts[b]), int(starts[b]) + int(counts[b])
            while p < end:
                to = min(end, (p // P + 1) * P)
                page = int(table[b, p // P])
                lo, hi = p % P, p % P + to - p
                new = x[b, p - starts[b]: to - starts[b]].astype(f)      # tokens, heads, dim
                for h in range(x.shape[2]):
                    m = np.abs(new[:, h]).max().astype(f)
                    s = max(f(m * f(1 / 127)), f(1e-8))
                    if lo > 0:
                        s0 = scales[page, h]
                        if s0 < s:
                            r = f(s0 / s)
                            old = codes[page, h, :lo].astype(f)
                            codes[page, h, :lo] = np.floor((old * r).astype(f) + f(0.5))
                        else:
                            s = s0
                    inv = f(1.0 / np.float64(s))
                    codes[page, h, lo:hi] = np.floor((new[:, h] * inv).astype(f) + f(0.5))
                    scales[page, h] = s
                p = to
    return cache


def attend(q, cache, table, lens, scale):
    """(out, lse, tol): 64-bit attention, and the error that f32 scores and
    sums may have (see the tests)."""
    B, T, H, D = q.shape
    Hk, P = cache[0].shape[1], cache[0].shape[2]
    out, tol = np.zeros((B, T, H, D)), np.zeros((B, T, H, D))
    lse = np.full((B, T, H), -np.inf)
    for b in range(B):
        for i in range(T):
            see = int(lens[b]) - T + i + 1
            if see <= 0:
                continue
            pages = table[b, : (see + P - 1) // P]
            for h in range(H):
                g = h // (H // Hk)
                k = (cache[0][pages, g].astype(np.float64)
                     * cache[2][pages, g].astype(np.float64)[:, None, None]).reshape(-1, D)[:see]
                v = (cache[1][pages, g].astype(np.float64)
                     * cache[3][pages, g].astype(np.float64)[:, None, None]).reshape(-1, D)[:see]
                s = scale * (k @ q[b, i, h])
                m = s.max()
                e = np.exp(s - m)
                out[b, i, h] = (e / e.sum()) @ v
                lse[b, i, h] = m + np.log(e.sum())
                # scores: 2^-20 of sum |q k| for the products and their f32 sums,
                # 2^-21 of max|q| sum |k| for q's parts; 2^-21 |s - m| for exp's argument
                ds = abs(scale) * (2.0 ** -20 * (np.abs(k) @ np.abs(q[b, i, h]))
                                   + 2.0 ** -21 * np.abs(q[b, i, h]).max() * np.abs(k).sum(1))
                ds = ds + 2.0 ** -21 * np.minimum(np.abs(s - m), 100)
                p = e / e.sum()
                tol[b, i, h] = (p * (ds + (p * ds).sum() + 2.0 ** -20)) @ np.abs(v)
    return out, lse, tol


# ---- log probabilities
def logprobs(x, target, top):
    """(logprob, entropy, lse, top_logprob, top_id) of float64 logits."""
    M, V = x.shape
    lse, H, lp = np.zeros(M), np.zeros(M), np.zeros(M)
    ids = np.zeros((M, top), np.int64)
    tl = np.zeros((M, top))
    for r in range(M):
        m = x[r].max()
        none = m == -np.inf
        d = np.where(x[r] == -np.inf, -np.inf, x[r] - (0 if none else m))
        e = np.exp(d)
        lse[r] = -np.inf if none else m + np.log(e.sum())
        with np.errstate(invalid="ignore"):
            y = np.where(d == -np.inf, -np.inf, d - np.log(e.sum()))   # not x - lse: all may be near -1e38
        p = np.exp(y)
        H[r] = 0.0 if none else -(p[p > 0] * y[p > 0]).sum()
        if target is not None and target[r] >= 0:
            lp[r] = y[target[r]]
        ids[r] = np.lexsort((np.arange(V), -x[r]))[:top]
        tl[r] = y[ids[r]]
    return lp, H, lse, tl, ids


def logprobs_grad(x, target, lse, H, gl, gh):
    """The gradient formula at the given lse and entropy (64 bits), and the
    size that its rounding errors are relative to."""
    with np.errstate(invalid="ignore"):
        y = np.where(x == -np.inf, -np.inf, x - lse[:, None])
    p = np.exp(y)
    yf = np.where(p > 0, y, 0.0)
    has = target >= 0
    g = np.where(has, gl, 0.0)[:, None]
    dx = -p * (g + gh[:, None] * (yf + H[:, None]))
    size = p * (np.abs(g) + np.abs(gh[:, None]) * (np.abs(yf) + np.abs(H[:, None]))) * (1 + np.abs(yf) + np.abs(lse[:, None]))
    rows = np.arange(x.shape[0])[has]
    dx[rows, target[has]] += gl[has]
    size[rows, target[has]] += np.abs(gl[has])
    dx[np.isneginf(lse)] = size[np.isneginf(lse)] = 0.0
    return dx, size

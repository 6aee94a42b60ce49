"""Products of few rows whose activations differ in size along K: zeros, tiny and huge
stretches in every order, in one split of K and in many.

Tolerance: 2^-20 of sum |x w| for the f32 sums and for the parts' 22 bits, and 2^-38 of each
256 k's largest |x| times their sum |w|, the least step of the first f16 part relative to that
largest; then one rounding to the output's type."""
import numpy as np
import pytest
import torch

import verifiable_quantize_rows_gb300 as bsg
from gpu_util import dev, host
from serving_ref import DTYPES, IDS, f64, rounding, stored, within

pytestmark = pytest.mark.gpu
CHUNK = 256

# What each 256 k of a row is multiplied by (the last one for all that follow).
ORDERS = {
    "large then zeros": [2000, 2000, 0],
    "zeros then large": [0, 0, 0, 2000],
    "huge then zeros": [1e30, 0],
    "huge then ordinary": [1e30, 1, 1, 1e-3],
    "ordinary then huge": [1, 1e-3, 1, 1, 1e30],
    "tiny then ordinary": [1e-30, 1e-30, 1],
    "ordinary then tiny": [1, 1e-30, 0, 1e-30],
    "down": [2.0 ** (30 - 15 * i) for i in range(9)],
    "up": [2.0 ** (-70 + 15 * i) for i in range(9)],
    "in turn": [1e8, 0, 1, 0, 1e-8, 0, 0, 1e8],
    "one place": [0, 0, 3e4, 0],
}


def activations(M, K, dtype, first):
    """M rows, each of an order of its own, from the `first` order on."""
    rng = np.random.default_rng(M + K)
    x = rng.standard_normal((M, K))
    names = list(ORDERS)
    for m in range(M):
        by = ORDERS[names[(first + m) % len(names)]]
        for c in range(0, K, CHUNK):
            x[m, c:c + CHUNK] *= by[min(c // CHUNK, len(by) - 1)]
    if dtype == torch.float16:
        x = np.clip(x, -6e4, 6e4)
    return dev(x.astype(np.float32)).to(dtype)


def check(X, W, group, columns):
    Q, sc = bsg.wquant_groups(W, group)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    Y = bsg.wgroups_matvec(X, Q, sc, group=group, dstatus=st)
    assert int(st.item()) == 0
    x, N = f64(X), sc.shape[1]
    for c0 in columns:  # a stretch of columns is enough
        c1 = min(N, c0 + 200)
        w = stored(host(Q[:, c0 // 2:(c1 + 1) // 2].contiguous()), host(sc[:, c0:c1].contiguous()), c1 - c0, group)
        want = x @ w
        tol = 2.0 ** -20 * (np.abs(x) @ np.abs(w))
        for k in range(0, x.shape[1], CHUNK):
            tol += 2.0 ** -38 * np.abs(x[:, k:k + CHUNK]).max(1)[:, None] * np.abs(w[k:k + CHUNK]).sum(0)[None, :]
        got, most = f64(Y[:, c0:c1]), torch.finfo(X.dtype).max
        beyond = np.abs(want) + tol > most  # of f16: its largest, or Inf, is what the type has there
        assert (np.abs(got[beyond]) >= most * (1 - 2.0 ** -8)).all() and (got[beyond] * want[beyond] > 0).all()
        within(np.where(beyond, 0, got), np.where(beyond, 0, want), tol + rounding(want, X.dtype))


def weight(K, N, size):
    return torch.randn((K, N), generator=torch.Generator("cuda").manual_seed(K + N), device="cuda") * size


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("M,first", [(5, 0), (5, 6), (8, 3), (16, 0)])
@pytest.mark.parametrize("K,N", [(2048, 233472), (2100, 240000), (4096, 50304), (9000, 300), (1500, 9001)])
@pytest.mark.parametrize("size,group", [(0.02, 64), (1.0, 32), (0.02, 0)])
def test_sizes_that_change_along_k(dtype, M, first, K, N, size, group):
    check(activations(M, K, dtype, first), weight(K, N, size), group, [0, N // 2 // 2 * 2, (N - 200) // 2 * 2])


def test_a_large_sum_before_zeros_is_kept():
    """Sums made by the first rows of K alone, of 2^12 and far more, and nothing after them."""
    K, N = 2048, 233472
    X = torch.zeros((5, K), device="cuda")
    X[0, :256], X[1, :256], X[2, 0], X[3, 255], X[4, 256:300] = 1e5, 2000.0, 1e30, 3e38, -5e33
    W = torch.full((K, N), 0.02, device="cuda")
    Q, sc = bsg.wquant_groups(W, 64)
    Y = bsg.wgroups_matvec(X, Q, sc)
    want = X.double().sum(1, keepdim=True) * float(sc[0, 0]) * 7
    assert torch.isfinite(Y).all()
    assert ((Y.double() - want).abs() <= 2.0 ** -20 * want.abs()).all()


@pytest.mark.parametrize("M,K,N", [(1, 768, 2304), (2, 768, 768), (4, 300, 1000), (3, 300, 1001)])
def test_values_near_the_largest_in_the_small_form(M, K, N):
    """X times a code is beyond f32 here; X times the weight is not."""
    X = torch.zeros((M, K), device="cuda")
    X[:, 5], X[:, K - 1] = 3e38, -1e38
    Q, sc = bsg.wquant_groups(torch.full((K, N), 0.02, device="cuda"), 64)
    Y = bsg.wgroups_matvec(X, Q, sc)
    want = X.double().sum(1, keepdim=True) * float(sc[0, 0]) * 7
    assert ((Y.double() - want).abs() <= 2.0 ** -20 * 4e38 * float(sc[0, 0]) * 7).all()

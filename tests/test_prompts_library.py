"""The calls for prompts, windows and shared prefixes without a GPU: exported, and every bad
argument refused before anything touches CUDA; the definitions they are tested against."""
import numpy as np
import pytest
import torch

import prompts_ref
import verifiable_quantize_rows_gb300 as bsg
from test_serving_library import ARG, BAD_CACHES, D, WORKSPACE, cache, lib, refused, tokens  # noqa: F401


def test_declared():
    names = bsg.exported_symbols()
    for n in ("bsg_wcols_matmul", "bsg_wcols_matmul_workspace_size", "bsg_kv8_attend_window", "bsg_kv8_attend_window_workspace_size",
              "bsg_kv8_attend_shared", "bsg_kv8_attend_shared_workspace_size"):
        assert n in names


def test_wcols_matmul(lib):  # noqa: F811
    size = lib.bsg_wcols_matmul_workspace_size(300, 7, 100)
    good = dict(X=D, dtype=1, ldx=100, Q=D, ldq=7, scale=D, M=300, N=7, K=100, relu=0, Y=2 * D, ldy=7, ws=D, n=size, st=None, stream=None)
    refused(lib.bsg_wcols_matmul, good,
            [("X", None), ("X", D + 1), ("dtype", 3), ("ldx", 99), ("Q", None), ("ldq", 6), ("scale", None), ("scale", D + 2), ("M", 0), ("N", 0),
             ("M", 1 << 31), ("N", 1 << 31), ("K", 0), ("relu", 2), ("relu", -1), ("Y", None), ("Y", D), ("Y", D + 1), ("ldy", 6)])
    refused(lib.bsg_wcols_matmul, good, [("ws", None), ("ws", D + 16), ("n", size - 1)], WORKSPACE)
    assert lib.bsg_wcols_matmul(*dict(good, K=bsg.MAX_K + 1, ldx=1 << 20).values()) == 2
    for bad in ((0, 5, 5), (5, 0, 5), (5, 5, 0), (5, 5, bsg.MAX_K + 1), (1 << 31, 5, 5), (1 << 30, 1 << 30, 5)):
        assert lib.bsg_wcols_matmul_workspace_size(*bad) == 0


def test_kv8_attend_window(lib):  # noqa: F811
    for T in (3, 300):
        size = lib.bsg_kv8_attend_window_workspace_size(cache(), 4, 2, T, 4, 100, 3)
        assert size > 0
        for bad in BAD_CACHES:
            assert lib.bsg_kv8_attend_window_workspace_size(cache(**bad), 4, 2, T, 4, 100, 3) == 0
        for bad in ((0, 2, T, 4, 1, 1), (4, 0, T, 4, 1, 1), (4, 2, 0, 4, 1, 1), (4, 2, T, 3, 1, 1), (4, 2, T, 0, 1, 1), (4, 2, T, 4, -1, 1),
                    (4, 2, T, 4, 1, -1), (4, 2, 1 << 30, 4, 1, 1)):
            assert lib.bsg_kv8_attend_window_workspace_size(cache(), *bad) == 0
        good = dict(cache=cache(), table=D, ld=4, lens=D, counts=None, q=tokens(), out=tokens(2 * D), dtype=0, B=2, T=T, heads=4, window=100,
                    sinks=3, scale=0.1, lse=None, ws=D, n=size, st=None, stream=None)
        refused(lib.bsg_kv8_attend_window, good,
                [("cache", None), *[("cache", cache(**c)) for c in BAD_CACHES], ("table", None), ("ld", 0), ("lens", None), ("lens", D + 2),
                 ("counts", D + 1), ("q", None), ("out", None), ("q", tokens(D + 2)), ("out", tokens(None)), ("out", tokens(D)), ("dtype", 3),
                 ("B", 0), ("B", 65536), ("T", 0), ("T", 1 << 31), ("heads", 3), ("heads", 0), ("heads", 1 << 17), ("window", -1), ("sinks", -1),
                 ("scale", float("inf")), ("scale", float("nan")), ("lse", D + 2)])
        refused(lib.bsg_kv8_attend_window, good, [("ws", None), ("ws", D + 128), ("n", size - 1), ("n", 0)], WORKSPACE)


def test_kv8_attend_shared(lib):  # noqa: F811
    for B in (2, 200):
        size = lib.bsg_kv8_attend_shared_workspace_size(cache(), 9, 4, B, 3, 4)
        assert size > 0
        for bad in BAD_CACHES:
            assert lib.bsg_kv8_attend_shared_workspace_size(cache(**bad), 9, 4, B, 3, 4) == 0
        for bad in ((0, 4, B, 3, 4), (9, 0, B, 3, 4), (9, 4, 0, 3, 4), (9, 4, B, 17, 4), (9, 4, B, 0, 4), (9, 4, B, 3, 3), (1 << 30, 4, B, 3, 4)):
            assert lib.bsg_kv8_attend_shared_workspace_size(cache(), *bad) == 0
        good = dict(cache=cache(), prefix=D, pages=9, prefix_len=D, table=D, ld=4, lens=D, q=tokens(), out=tokens(2 * D), dtype=0, B=B, T=3,
                    heads=4, scale=0.1, lse=None, ws=D, n=size, st=None, stream=None)
        refused(lib.bsg_kv8_attend_shared, good,
                [("cache", None), *[("cache", cache(**c)) for c in BAD_CACHES], ("prefix", None), ("prefix", D + 2), ("pages", 0), ("pages", 1 << 30),
                 ("prefix_len", None), ("prefix_len", D + 1), ("table", None), ("ld", 0), ("lens", None), ("q", None), ("out", None),
                 ("q", tokens(D + 2)), ("out", tokens(None)), ("out", tokens(D)), ("dtype", 3), ("B", 0), ("T", 0), ("T", 17), ("heads", 3),
                 ("scale", float("inf")), ("lse", D + 2)])
        refused(lib.bsg_kv8_attend_shared, good, [("ws", None), ("ws", D + 128), ("n", size - 1)], WORKSPACE)


def test_the_binding_refuses_host_tensors():
    x = torch.ones(2, 64)
    for call in (lambda: bsg.wcols_matmul(x, x, x), lambda: bsg.kv8_attend_window(x[None, None], (x, x, x, x), x, x),
                 lambda: bsg.kv8_attend_shared(x[None, None], (x, x, x, x), x, x, x, x)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()


def test_the_definition_of_codes_is_the_oracles(orc):
    """prompts_ref's step 1, beside the oracle's."""
    x = np.random.default_rng(1).standard_normal((20, 300)).astype(np.float32) * np.exp2(np.arange(20) - 10)[:, None].astype(np.float32)
    x[3] = 0
    q, s = prompts_ref.codes_of(x)
    want = orc.quantize_rows(x)
    assert np.array_equal(q, np.asarray(want[0], np.int64)) and np.array_equal(s, np.asarray(want[1]))


def test_the_definition_masks_windows():
    """A plain loop beside the definition's masks."""
    rng = np.random.default_rng(2)
    cache = [rng.integers(-127, 128, (4, 1, 16, 32)).astype(np.int8) for _ in range(2)] + [np.full((4, 1), 0.01, np.float32)] * 2
    table, q, W, S, n, T = np.array([[2, 0, 3]]), rng.standard_normal((1, 9, 1, 32)), 7, 3, 40, 9
    out, lse, _, _ = prompts_ref.window(q, cache, table, [n], [T], W, S, 0.2)
    for t in range(T):
        i, e, o = n - T + t, 0.0, 0.0
        for j in range(n):
            if j <= i and (j > i - W or j < S):
                page = table[0, j // 16]
                w = np.exp(0.2 * q[0, t, 0] @ (cache[0][page, 0, j % 16] * np.float64(cache[2][page, 0])))
                e, o = e + w, o + w * cache[1][page, 0, j % 16] * np.float64(cache[3][page, 0])
        assert np.allclose(out[0, t, 0], o / e) and np.isclose(lse[0, t, 0], np.log(e))

"""Log probabilities, entropy and top alternatives against 64 bits, and their
gradient against the formula and against differences.

Tolerances: x - m carries 2^-24 of its size, exp and the f32 sums 2^-21 of
theirs, log 2^-22; so 2^-20 (1 + |x - lse|) for a log probability and
2^-20 (1 + log V) for lse (relative to it where it is large) and the entropy.
Of the gradient, 2^-19 of |its terms| (1 + |x - lse| + |lse|), then one
rounding to the type."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import verifiable_quantize_rows_gb300 as bsg
from gpu_util import dev, host
from serving_ref import DTYPES, IDS, f64, rounding, within

pytestmark = pytest.mark.gpu


def rows(M, V, dtype, seed, spread=2.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, V)) * spread * np.exp(rng.random((M, 1)))
    return dev(x.astype(np.float32)).to(dtype)


def check(x, target=None, top=0, want_status=0):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = bsg.logprobs(x, None if target is None else dev(np.int64(target)), top=top, dstatus=st)
    torch.cuda.synchronize()
    assert int(st.item()) == want_status
    lp, H, lse, tl, ti = ref.logprobs(f64(x), target, top)
    V = x.shape[1]
    assert (host(r.top_id) == ti).all(), "top ids"
    with np.errstate(invalid="ignore"):
        for name, got, want, tol in (
                ("logprob", r.logprob, lp, 2.0 ** -20 * (1 + np.abs(lp))),
                ("entropy", r.entropy, H, 2.0 ** -20 * (1 + np.log(V))),
                ("lse", r.lse, lse, 2.0 ** -20 * (1 + np.log(V)) + 2.0 ** -23 * np.abs(lse)),
                ("top", r.top_logprob, tl, 2.0 ** -20 * (1 + np.abs(tl)))):
            g = f64(got)
            inf = np.isinf(want)
            assert (g[inf] == want[inf]).all(), name
            within(np.where(inf, 0, g), np.where(inf, 0, want), np.where(inf, 0, tol), name)
    return r


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("M,V", [(1, 1), (1, 2), (2, 31), (3, 32), (1, 33), (5, 255), (4, 1000),
                                 (7, 1025), (1, 4099), (2, 50304), (200, 777), (400, 130), (160, 9000)],
                         ids=lambda v: str(v))
def test_against_64_bits(dtype, M, V):
    rng = np.random.default_rng(M + V)
    target = rng.integers(0, V, M)
    target[M // 2] = -1 if M > 1 else V - 1
    check(rows(M, V, dtype, V), target, min(V, 20))


@pytest.mark.parametrize("top", [0, 1, 2, 5, 31, 32])
@pytest.mark.parametrize("M", [1, 3, 300])
def test_top_counts(top, M):
    check(rows(M, 3001, torch.float32, top), None, top)


@pytest.mark.parametrize("M", [1, 200])
@pytest.mark.parametrize("kind", ["equal", "zeros", "rising", "falling", "few", "one"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_ties_and_orders(dtype, kind, M):
    """All equal, +0 and -0, sorted either way (each value a new maximum),
    a handful of levels, one far above the rest."""
    V = 5000
    i = np.arange(V)
    x = {"equal": np.full(V, -3.5), "zeros": np.where(i % 3 == 1, 0.0, -0.0),
         "rising": i / 64.0, "falling": -i / 64.0, "few": (i * 7919 % 5).astype(float),
         "one": np.where(i == 4097, 60.0, 0.0)}[kind]
    x = dev(np.tile(x.astype(np.float32), (M, 1))).to(dtype)
    check(x, np.full(M, 4097), 32)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("M", [1, 200])
def test_masked_logits(dtype, M):
    """-inf here and there, in whole stretches, in all but one or three
    places, and everywhere; the type's lowest value as a mask."""
    V = 6000
    x = rows(M + 6, V, dtype, 3)
    low = torch.finfo(dtype).min
    x[0, ::2] = -float("inf")
    x[1, :5000] = -float("inf")
    x[2, :] = -float("inf")
    x[2, 5999] = 1.5
    x[3, :] = -float("inf")
    x[3, [5, 4000, 4001]] = torch.tensor([1.0, 1.0, -2.0], dtype=dtype, device="cuda")
    x[4, :] = -float("inf")
    x[5, 100:] = low
    x[6, :] = low
    target = np.random.default_rng(1).integers(0, V, M + 6)
    target[0], target[2], target[4] = 2, 5999, 17
    for sel in ([0], [1], [2], [3], [4], [5], [6], list(range(M + 6))):
        check(x[sel], target[sel], 20)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("M", [2, 180])
def test_strided_and_unaligned_rows(dtype, M):
    V = 1500
    wide = rows(M, V + 37, dtype, 9)
    for off in (0, 1, 3, 8):
        check(wide[:, off: off + V], np.full(M, V - 1), 7)


@pytest.mark.parametrize("M", [1, 170])
def test_large_and_tiny_values(M):
    x = rows(M, 2000, torch.float32, 2)
    check(x * 1e4, np.zeros(M, np.int64), 5)
    check(x + 1e6, np.zeros(M, np.int64), 5)
    check(x * 1e-30, np.zeros(M, np.int64), 5)


@pytest.mark.parametrize("M", [3, 200])
def test_status_bits(M):
    x = rows(M, 300, torch.float32, 2)
    good = bsg.logprobs(x, dev(np.full(M, 5)), top=3)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[1, 299] = bad
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        r = bsg.logprobs(y, dev(np.full(M, 5)), top=3, dstatus=st)
        assert int(st.item()) == bsg.DSTATUS_NONFINITE
        keep = [i for i in range(M) if i != 1]
        for a, b in zip(r, good):
            assert torch.equal(a[keep], b[keep])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    target = np.full(M, 5)
    target[1] = 300
    r = bsg.logprobs(x, dev(target), top=3, dstatus=st)
    assert int(st.item()) == bsg.DSTATUS_RANGE
    assert torch.isnan(r.logprob[1]) and torch.equal(r.lse, good.lse)


@pytest.mark.parametrize("M", [1, 40])
def test_the_same_bits_every_time(M):
    x = rows(M, 50304, torch.bfloat16, 2)
    a = bsg.logprobs(x, top=32)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(10):
        b = bsg.logprobs(x, top=32, stream=s if i % 2 else None)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_a_row_is_the_same_alone_and_in_a_batch():
    """Within the tolerance of both, and with the same tokens on top."""
    x = rows(500, 5000, torch.float32, 12)
    a = bsg.logprobs(x, top=8)
    for i in (0, 250, 499):
        b = bsg.logprobs(x[i: i + 1], top=8)
        assert torch.equal(a.top_id[i: i + 1], b.top_id)
        assert torch.allclose(a.lse[i: i + 1], b.lse, rtol=0, atol=2.0 ** -18)


def test_offsets_past_32_bits():
    M, V = 3, 1000
    wide = torch.empty((M, (1 << 30) + 64), device="cuda")      # rows 4 GB apart
    x = rows(M, V, torch.float32, 1)
    wide[:, :V] = x
    r = check(wide[:, :V], np.full(M, 999), 5)
    g = torch.ones(M, device="cuda")
    dx = bsg.logprobs_backward(wide[:, :V], dev(np.full(M, 999)), r.lse, r.entropy, g, g)
    assert torch.equal(dx, bsg.logprobs_backward(x, dev(np.full(M, 999)), r.lse, r.entropy, g, g))


# ---------------------------------------------------------------------------
def grad_check(x, target, gl, gh, **kw):
    r = bsg.logprobs(x, dev(np.int64(target)))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx = bsg.logprobs_backward(x, dev(np.int64(target)), r.lse, r.entropy, dev(gl), dev(gh),
                               dstatus=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and dx.dtype == x.dtype
    xs = f64(x) if "out" not in kw or kw["out"] is not x else None
    if xs is not None:
        want, size = ref.logprobs_grad(xs, target, f64(r.lse), f64(r.entropy),
                                       gl.astype(np.float64), gh.astype(np.float64))
        within(f64(dx), want, 2.0 ** -19 * size + rounding(want, x.dtype), "dx")
    return dx


def cotangents(M, seed):
    rng = np.random.default_rng(seed)
    return rng.standard_normal(M).astype(np.float32), rng.standard_normal(M).astype(np.float32)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("M,V", [(1, 1), (1, 2), (3, 33), (5, 1000), (97, 1289), (2, 50304), (300, 257)],
                         ids=lambda v: str(v))
def test_gradient_against_the_formula(dtype, M, V):
    target = np.random.default_rng(V).integers(0, V, M)
    if M > 1:
        target[M - 1] = -1
    grad_check(rows(M, V, dtype, M), target, *cotangents(M, 1))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gradient_of_masked_rows(dtype):
    """-inf takes no gradient; a row of nothing else none at all; the lowest
    value as a mask."""
    x = rows(4, 700, dtype, 5)
    x[0, ::3] = -float("inf")
    x[1, :] = -float("inf")
    x[2, 5:] = torch.finfo(dtype).min
    x[3, :] = -float("inf")
    x[3, 9] = 2.0
    dx = grad_check(x, np.array([1, 3, 2, 9]), *cotangents(4, 2))
    assert (dx[0, ::3] == 0).all() and (dx[1] == 0).all()


def test_gradient_strided_in_place_and_without_parts():
    M, V = 9, 801
    target = np.arange(M) * 5
    gl, gh = cotangents(M, 3)
    wide = rows(M, V + 6, torch.float32, 4)
    x = wide[:, 3: 3 + V]
    out = torch.full((M, V + 5), 7.0, device="cuda")
    dx = grad_check(x, target, gl, gh, out=out[:, 2: 2 + V])
    assert (out[:, :2] == 7).all() and (out[:, 2 + V:] == 7).all()
    r = bsg.logprobs(x, dev(target))
    lp = bsg.logprobs_backward(x, dev(target), r.lse, g_logprob=dev(gl))
    en = bsg.logprobs_backward(x, None, r.lse, r.entropy, g_entropy=dev(gh))
    zero = np.zeros(M, np.float32)
    assert torch.equal(lp, bsg.logprobs_backward(x, dev(target), r.lse, r.entropy, dev(gl), dev(zero)))
    assert torch.equal(en, bsg.logprobs_backward(x, dev(target), r.lse, r.entropy, dev(zero), dev(gh)))
    none = bsg.logprobs_backward(x, dev(target), r.lse)
    assert (none == 0).all()
    y = x.clone()
    assert bsg.logprobs_backward(y, dev(target), r.lse, r.entropy, dev(gl), dev(gh), out=y) is y
    assert torch.equal(y, dx)


def test_gradient_against_differences():
    """(f(x + h u) - f(x - h u)) / 2h in 64 bits along random directions, with
    f = sum g_lp logprob + g_H entropy: off by O(h^2) = 1e-8 and the f32
    gradient's 2^-19 of the terms."""
    M, V, h = 3, 50, 1e-4
    x = rows(M, V, torch.float32, 6, 1.0)
    target = np.array([4, -1, 49])
    gl, gh = cotangents(M, 5)
    dx = f64(grad_check(x, target, gl, gh))
    rng = np.random.default_rng(8)

    def f(z):
        lp, H, *_ = ref.logprobs(z, target, 0)
        return (gl * lp).sum() + (gh * H).sum()

    for _ in range(20):
        u = rng.standard_normal((M, V))
        want = (f(f64(x) + h * u) - f(f64(x) - h * u)) / (2 * h)
        assert abs((dx * u).sum() - want) < 1e-5 * (1 + np.abs(dx * u).sum())


@pytest.mark.parametrize("M", [2, 200])
def test_gradient_status_bits(M):
    x = rows(M, 500, torch.float32, 2)
    target = np.full(M, 7)
    gl, gh = cotangents(M, 1)
    good = grad_check(x, target, gl, gh)
    r = bsg.logprobs(x, dev(target))
    target[1] = 500
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx = bsg.logprobs_backward(x, dev(target), r.lse, r.entropy, dev(gl), dev(gh), dstatus=st)
    assert int(st.item()) == bsg.DSTATUS_RANGE
    assert torch.isnan(dx[1]).all() and torch.equal(dx[0], good[0]) and torch.equal(dx[2:], good[2:])
    target[1] = 7
    x[1, 3] = float("nan")
    st.zero_()
    dx = bsg.logprobs_backward(x, dev(target), r.lse, r.entropy, dev(gl), dev(gh), dstatus=st)
    assert int(st.item()) == bsg.DSTATUS_NONFINITE
    assert torch.equal(dx[0], good[0]) and torch.equal(dx[2:], good[2:])

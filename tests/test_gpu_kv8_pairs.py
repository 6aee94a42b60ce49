"""How many bits a probability keeps on its way to the values, seen through sums that cancel.

Positions stand in pairs: keys that differ by one code of one dim, values that are each other's
negatives.  An output is then the sum of what little the pairs' probabilities differ by, and the
rounding of 16-bit outputs hides nothing of them.  With 22 bits a call is within the tolerance that
prompts_ref derives for two parts; probabilities of 11 bits are far outside it, which the test
without a GPU shows on the definition."""
import numpy as np
import pytest
import torch

import prompts_ref as ref
import verifiable_quantize_rows_gb300 as bsg
from gpu_util import dev
from serving_ref import DTYPES, IDS, f64, rounding, within

PAGE = 16
gpu = pytest.mark.gpu
# Calls whose probabilities have two parts: up to 16 query rows of a key/value head whatever the
# type, and f16 and f32 with any number of rows.
CALLS = [(T, dt) for T in (1, 3, 8, 40, 150) for dt in DTYPES if T <= 8 or dt != torch.bfloat16]


def pairs(B, T, H, Hk, D, n, seed):
    rng = np.random.default_rng(seed)
    per = -(-n // PAGE)
    codes = [rng.integers(-100, 101, (B * per, Hk, PAGE, D)).astype(np.int8) for _ in range(2)]
    codes[0][:, :, 1::2] = codes[0][:, :, ::2]
    codes[0][:, :, 1::2, 0] += 1
    codes[1][:, :, 1::2] = -codes[1][:, :, ::2]
    scales = [(0.005 + 0.01 * rng.random((B * per, Hk))).astype(np.float32) for _ in range(2)]
    table = rng.permutation(B * per).reshape(B, per).astype(np.int32)
    return rng.standard_normal((B, T, H, D)).astype(np.float32), codes + scales, table


def test_eleven_bits_would_be_seen():
    """Probabilities rounded to 11 bits, in the definition's place: most outputs leave the tolerance."""
    D, n = 64, 96
    q, cache, table = pairs(1, 4, 1, 1, D, n, 1)
    q = q[0, :, 0].astype(np.float64)
    k, v = ref.cached(cache, table[0], n, 0)
    see = np.ones((4, n), bool)
    out, _, tol, _ = ref.softmax_attend(q, k, v, see, D ** -0.5, 2)
    s = D ** -0.5 * (q @ k.T)
    p = np.exp(s - s.max(1, keepdims=True)).astype(np.float64)
    coarse = (p * 512).astype(np.float16).astype(np.float64) / 512
    got = torch.from_numpy(coarse @ v / p.sum(1, keepdims=True)).to(torch.bfloat16).double().numpy()
    fine = torch.from_numpy(out).to(torch.bfloat16).double().numpy()
    limit = tol * 1.001 + rounding(out, torch.bfloat16)
    assert (np.abs(fine - out) <= limit).all()
    assert (np.abs(got - out) > limit).mean() > 0.5


@gpu
@pytest.mark.parametrize("D", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("T,dtype", CALLS, ids=lambda x: IDS[DTYPES.index(x)] if x in DTYPES else str(x))
def test_windows(T, dtype, D):
    for share, n, window, sinks in ((1, 300, 0, 0), (2, 300, 96, 4), (2, 900, 0, 0), (1, 48, 0, 0)):
        if T > n:
            continue
        q, cache, table = pairs(3, T, 2 * share, 2, D, n, T + D + n)
        qd = dev(q).to(dtype)
        lens = [n, n - 2 if n - 2 >= T else n, max(T, n // 2)]
        y = bsg.kv8_attend_window(qd, bsg.Kv8Cache(*map(dev, cache)), dev(table), dev(np.int32(lens)), window=window, sinks=sinks)
        want, _, tol, _ = ref.window(f64(qd), cache, table, lens, [T] * 3, window, sinks, D ** -0.5, 2)
        within(f64(y), want, tol * 1.001 + rounding(want, dtype), (share, n, window))


@gpu
@pytest.mark.parametrize("D", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("B,T,dtype", [(B, T, dt) for B, T in ((1, 1), (5, 1), (2, 8), (3, 5), (20, 2), (40, 4)) for dt in DTYPES
                                       if B * T <= 16 or dt != torch.bfloat16], ids=lambda x: IDS[DTYPES.index(x)] if x in DTYPES else str(x))
def test_shared_beginnings(B, T, dtype, D):
    n0, own = 240, 64
    q, cache, table = pairs(B + 1, T, 2, 2, D, n0, B + T + D)
    prefix, table = table[0].copy(), table[1:, : own // PAGE].copy()
    qd = dev(q[:B]).to(dtype)
    lens = [own - 2 * (b % 20) for b in range(B)]
    y = bsg.kv8_attend_shared(qd, bsg.Kv8Cache(*map(dev, cache)), dev(prefix), dev(np.int32([n0])), dev(table), dev(np.int32(lens)))
    want, _, tol, _ = ref.shared(f64(qd), cache, prefix, n0, table, lens, D ** -0.5, 2)
    within(f64(y), want, tol * 1.001 + rounding(want, dtype))

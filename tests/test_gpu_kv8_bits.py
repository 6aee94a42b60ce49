"""Attention of 16-bit types: what their probabilities lose on the way to the values.

A probability goes to the second product as two f16 parts of p' = 2^(S - ref), whose
largest is at least 2^11 in every warp: what the parts leave out of p' is at most
2^-24 p' (the second part's rounding) or 2^-25 (half of the least f16 step), whichever is
larger.  So beside the scores' errors (serving_ref.attend) an output may be off by 2^-23 of
sum p |v|, and by 2^-36 of the largest p times its value scale for each position's
largest code (128), and is rounded once to its type."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import verifiable_quantize_rows_gb300 as bsg
from gpu_util import dev, host
from serving_ref import f64, rounding, within

pytestmark = pytest.mark.gpu
HALVES = pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])


def pool(pages, heads, page, dim, seed, value=0.02):
    rng = np.random.default_rng(seed)
    codes = [rng.integers(-127, 128, (pages, heads, page, dim)).astype(np.int8) for _ in range(2)]
    scales = [(rng.random((pages, heads)) * s + s / 20).astype(np.float32) for s in (0.02, value)]
    return codes + scales


def parts_error(q, cache, table, lens, scale):
    """The bound above, of every output element."""
    B, T, H, D = q.shape
    Hk, P = cache[0].shape[1], cache[0].shape[2]
    tol = np.zeros((B, T, H, D))
    for b in range(B):
        for i in range(T):
            see = int(lens[b]) - T + i + 1
            if see <= 0:
                continue
            pages = table[b, : (see + P - 1) // P]
            for h in range(H):
                g = h // (H // Hk)
                ks, vs = (np.repeat(cache[n][pages, g].astype(np.float64), P)[:see] for n in (2, 3))
                k, v = (cache[n][pages, g].reshape(-1, D)[:see].astype(np.float64) for n in (0, 1))
                s = scale * ks * (k @ q[b, i, h])
                p = np.exp(s - s.max())
                p /= p.sum()
                tol[b, i, h] = 2.0 ** -23 * ((p * vs) @ np.abs(v)) + see * 2.0 ** -36 * (p * vs).max() * 128
    return tol


def check(q, cache, table, lens, scale=None):
    s = q.shape[3] ** -0.5 if scale is None else scale
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = bsg.kv8_attend(q, bsg.Kv8Cache(*[dev(x) for x in cache]), dev(table), dev(np.int32(lens)), scale=scale, dstatus=st)
    assert int(st.item()) == 0
    want, _, tol = ref.attend(f64(q), cache, table, lens, s)
    within(f64(o), want, tol + parts_error(f64(q), cache, table, lens, s) + rounding(want, q.dtype))


def queries(shape, dtype, seed, scale=1.0):
    x = np.random.default_rng(seed).standard_normal(shape) * scale
    return dev(x.astype(np.float32)).to(dtype)


def table_for(batch, per, pages, seed):
    return np.random.default_rng(seed).permutation(pages)[: batch * per].reshape(batch, per).astype(np.int32)


@HALVES
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("share,T", [(1, 1), (4, 1), (4, 4), (8, 4)])
def test_heads_and_tokens(dtype, dim, share, T):
    lens = [0, 3, 47, 130, 700]
    cache = pool(5 * 44, 2, 16, dim, dim + share)
    check(queries((5, T, 2 * share, dim), dtype, T + dim), cache, table_for(5, 44, 220, T), lens)


@HALVES
@pytest.mark.parametrize("B,length", [(1, 5001), (2, 9000), (1, 40000), (60, 900)])
def test_lengths_in_many_and_in_few_chunks(dtype, B, length):
    per = length // 64 + 1
    cache = pool(B * per, 2, 64, 64, length)
    check(queries((B, 1, 4, 64), dtype, length), cache, table_for(B, per, B * per, 2), [length] * B)


@HALVES
@pytest.mark.parametrize("qscale", [0.0, 1e-3, 30.0])
def test_flat_and_peaked(dtype, qscale):
    cache = pool(40, 2, 32, 64, 8)
    cache[3][::3] *= 50            # pages of very different value scales
    cache[2][1::3] *= 0.01
    check(queries((4, 2, 4, 64), dtype, 8, qscale), cache, table_for(4, 10, 40, 8), [320, 319, 33, 2])


@HALVES
@pytest.mark.parametrize("above", [8, 16])
def test_one_position_far_above_the_rest_with_nothing_to_say(dtype, above):
    """A position that takes nearly all of the probability and whose value is 0: the
    output is what the others leave, some e^-above of the values' size."""
    B, D, page = 400, 64, 16
    rng = np.random.default_rng(above)
    lens = [int(n) for n in rng.integers(40, 400, B)]
    per = 25
    cache = pool(B * per, 1, page, D, above, 1.0)
    cache[2][:] = 0.01
    table = table_for(B, per, B * per, 1)
    u = np.where(rng.random(D) < 0.5, 1.0, -1.0)
    cache[0][table[:, 0], 0, 0] = (127 * u).astype(np.int8)
    cache[1][table[:, 0], 0, 0] = 0
    # score of the first: scale 0.01 127 D c; of the others: about 1 / 14 of it either way
    c = above / (D ** -0.5 * 0.01 * 127 * D)
    q = dev(np.float32(np.broadcast_to(c * u, (B, 1, 2, D)))).to(dtype)
    check(q, cache, table, lens)

"""Sums of attention over many positions, where what each addition loses adds up.

Equal scores and values of one sign, each page with a value scale of its own, none a power of
two (with powers of two and whole codes every partial sum is exact and nothing can be lost).
The output is then sum(vs c) / n, off by, relative to it:

- 2^-19 for the probabilities: the value scale's logarithm, in (-8, -4), by half a step of 2^-21
  and its difference to the reference by as much, in units of log 2; exp2 by 2^-22, their two f16
  parts by 2^-22, 1 / vs by 2^-24: 2^-20.2 of each, of which what is common to all cancels and the
  rest is at most twice that;
- 2^-22 with each product of 16 positions that one sum of the tensor cores takes (cut off below
  the last of 24 bits where it is added, and as much where its terms are aligned): RUN of them;
- 2^-24 with each f32 addition, of outputs and of the probabilities' sum: RUN in a run at most,
  one for each run, and 16 for the joins of warps, lanes and chunks.

Each output is rounded once to its type."""
import numpy as np
import pytest
import torch

import prompts_ref
import verifiable_quantize_rows_gb300 as bsg
from gpu_util import dev
from serving_ref import DTYPES, IDS, f64, rounding, within

pytestmark = pytest.mark.gpu
F32, F16, BF16 = DTYPES
PAGE = 64


def cache_of(pages, heads, dim, seed):
    rng = np.random.default_rng(seed)
    codes = [np.ones((pages, heads, PAGE, dim), np.int8), rng.integers(90, 128, (pages, heads, PAGE, dim)).astype(np.int8)]
    return codes + [np.full((pages, heads), 0.01, np.float32), ((0.6 + rng.random((pages, heads))) / 128).astype(np.float32)]


def means(cache, order, n):
    """sum(vs c) / n over the first n positions of the pages in `order`: (heads, dim)."""
    v = cache[1].astype(np.float64) * cache[3].astype(np.float64)[:, :, None, None]
    full = np.bincount(order[: n // PAGE], minlength=len(v))
    total = np.einsum("p,phtd->hd", full, v)
    if n % PAGE:
        total += v[order[n // PAGE], :, : n % PAGE].sum(1)
    return total / n


def equal_scores(call, dtype, B, T, Hk, D, n, run, runs, pool=256):
    rng = np.random.default_rng(n + D)
    cache = cache_of(pool, Hk, D, D)
    order = rng.integers(0, pool, -(-n // PAGE)).astype(np.int32)      # a page may stand in a table often
    table = dev(np.broadcast_to(order, (B, len(order))).copy())
    q = torch.zeros(B, T, Hk, D, dtype=dtype, device="cuda")
    lse = torch.empty(B, T, Hk, device="cuda")
    out = call(q, bsg.Kv8Cache(*map(dev, cache)), table, torch.full((B,), n, dtype=torch.int32, device="cuda"), lse=lse)
    off = 2.0 ** -19 + run * 2.0 ** -22 + 2 * (run + runs + 16) * 2.0 ** -24
    for t in {0, T - 1}:
        want = np.broadcast_to(means(cache, order, n - T + 1 + t), (B, Hk, D))
        within(f64(out[:, t]), want, np.abs(want) * off * 1.01 + rounding(want, dtype), f"token {t}")
        # log n; the sum's error, and f32's in the reference and the logarithm (prompts_ref's 2^-20)
        want = np.full((B, Hk), np.log(n - T + 1 + t))
        within(f64(lse[:, t]), want, off + 2.0 ** -20 * (2 + want), f"lse of token {t}")


# Sequences enough that a chunk is a whole sequence or a good part of one; a warp takes every
# fourth of its tiles of 16 positions, 32 of them to a sum (16-bit types: 128, with two products each).
@pytest.mark.parametrize("call", [bsg.kv8_attend, bsg.kv8_attend_window], ids=["attend", "window"])
@pytest.mark.parametrize("dtype,B,T,D,n", [(F32, 512, 1, 128, 16384), (F32, 512, 1, 128, 131072), (F32, 400, 8, 64, 40000), (F32, 64, 1, 128, 131072),
                                           (F32, 300, 4, 256, 30000), (F16, 512, 1, 64, 1 << 20), (F16, 512, 4, 32, 1 << 20)])
def test_few_rows(call, dtype, B, T, D, n):
    run = 32 if dtype == F32 else 256
    equal_scores(call, dtype, B, T, 8, D, n, run, -(-n // (64 * (32 if dtype == F32 else 128))))


# A sum of the tensor cores' takes 640 positions at most (f16: 10240, bf16: 40960), two products to each 16 (bf16: one).
@pytest.mark.parametrize("dtype,B,T,D,n", [(F32, 40, 64, 64, 1 << 18), (F32, 40, 64, 256, 1 << 17), (F32, 40, 33, 32, 40000), (F16, 40, 64, 64, 1 << 16),
                                           (F16, 40, 17, 96, 1 << 18), (F16, 40, 200, 256, 1 << 17), (BF16, 40, 64, 64, 1 << 19)])
def test_many_rows(dtype, B, T, D, n):
    run, positions = {F32: (80, 512), F16: (1280, 8192), BF16: (2560, 32768)}[dtype]
    equal_scores(bsg.kv8_attend_window, dtype, B, T, 4, D, n, run, -(-n // positions))


@pytest.mark.parametrize("dtype,n", [(F32, 1 << 17), (F16, 1 << 18), (BF16, 1 << 19)])
def test_a_long_prefix(dtype, n):
    """The prefix's positions in one chunk, by equal scores; the own token is one position more."""
    B, Hk, D, pool = 1024, 8, 64, 256
    cache = cache_of(pool, Hk, D, 9)
    order = np.random.default_rng(1).integers(0, pool, n // PAGE).astype(np.int32)
    q = torch.zeros(B, 4, Hk, D, dtype=dtype, device="cuda")
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    y = bsg.kv8_attend_shared(q, bsg.Kv8Cache(*map(dev, cache)), dev(order), dev(np.int32([n])), table, torch.full((B,), 4, dtype=torch.int32, device="cuda"))
    own = cache[1][0, :, 0].astype(np.float64) * cache[3][0].astype(np.float64)[:, None]       # the first own position
    want = np.broadcast_to((means(cache, order, n) * n + own) / (n + 1), (B, Hk, D))
    run, positions = {F32: (80, 512), F16: (1280, 8192), BF16: (2560, 32768)}[dtype]
    off = 2.0 ** -19 + run * 2.0 ** -22 + 2 * (run + n // positions + 16) * 2.0 ** -24
    within(f64(y[:, 0]), want, want * off * 1.01 + rounding(want, dtype))


def test_own_tokens_behind_a_prefix():
    prefix, n0 = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    equal_scores(lambda q, c, table, lens, lse: bsg.kv8_attend_shared(q, c, prefix, n0, table, lens, lse=lse), F32, 400, 1, 8, 128, 65536, 32, 32)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T", [1, 3, 40])
@pytest.mark.parametrize("scores", ["rise", "fall", "any"])
def test_references_that_move_between_sums(scores, T, dtype):
    """Long chunks whose scores rise all along, fall, or do neither, against the definition."""
    B, Hk, D, n = 304, 8, 128, 18000
    rng = np.random.default_rng(7)
    pages = -(-n // PAGE)
    cache = cache_of(pages, Hk, D, 3)
    cache[1] = rng.integers(-127, 128, cache[1].shape).astype(np.int8)
    if scores == "any":
        cache[0] = rng.integers(-127, 128, cache[0].shape).astype(np.int8)
    else:
        at = np.arange(pages) if scores == "rise" else pages - 1 - np.arange(pages)
        cache[0][:] = np.minimum(127, at * 120 // pages + 1)[:, None, None, None]
    q3 = rng.standard_normal((3, T, Hk, D)).astype(np.float32) if scores == "any" else np.full((3, T, Hk, D), 0.1, np.float32) * np.float32([1, 2, 5])[:, None, None, None]
    q = dev(np.tile(q3, (-(-B // 3), 1, 1, 1))[:B]).to(dtype)
    order = np.arange(pages, dtype=np.int32)
    table = np.broadcast_to(order, (B, pages)).copy()
    lens = [n] * B
    y = bsg.kv8_attend_window(q, bsg.Kv8Cache(*map(dev, cache)), dev(table), dev(np.int32(lens)), scale=1.0)
    want, _, tol, _ = prompts_ref.window(f64(q[:3]), cache, table[:3], lens[:3], [T] * 3, 0, 0, 1.0)
    within(f64(y[:3]), want, tol * 1.001 + rounding(want, dtype))
    for b in range(3, B):
        assert torch.equal(y[b], y[b % 3])


@pytest.mark.parametrize("gone", [[32], [127, 128], [128], [32, 33, 64, 128, 256], list(range(30, 200))], ids=str)
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_pages_that_are_skipped_where_sums_begin_anew(dtype, gone):
    """Page i of 64 positions holds turn i of each of the four warps, which begin anew at turns 32 and
    128 and as many on; a page out of range is skipped, as if its positions were not there."""
    B, Hk, D, n = 304, 8, 128, 18500
    cache = cache_of(300, Hk, D, 5)
    order = np.random.default_rng(5).permutation(300).astype(np.int32)[: -(-n // PAGE)]
    table = np.broadcast_to(order, (B, len(order))).copy()
    table[:, gone] = -1
    kept = np.delete(order, gone)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(B, 1, Hk, D, dtype=dtype, device="cuda")
    given = bsg.Kv8Cache(*map(dev, cache))
    for y in (bsg.kv8_attend_window(q, given, dev(table), torch.full((B,), n, dtype=torch.int32, device="cuda"), dstatus=st),
              bsg.kv8_attend(q, given, dev(table), torch.full((B,), n, dtype=torch.int32, device="cuda"), dstatus=st)):
        assert int(st) == bsg.DSTATUS_RANGE
        want = np.broadcast_to(means(cache, kept, n - PAGE * len(gone)), (B, 1, Hk, D))
        run, runs = (32, 10) if dtype == F32 else (256, 3)
        within(f64(y), want, want * (2.0 ** -19 + run * 2.0 ** -22 + 2 * (run + runs + 16) * 2.0 ** -24) * 1.01 + rounding(want, dtype))

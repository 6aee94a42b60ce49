"""Attention through a window with sinks, for any number of tokens, against 64 bits.

Tolerances: prompts_ref.softmax_attend derives them; every output is rounded once to
its type."""
import numpy as np
import pytest
import torch

import prompts_ref as ref
import verifiable_quantize_rows_gb300 as bsg
from gpu_util import dev, host
from serving_ref import DTYPES, IDS, f64, rounding, within

pytestmark = pytest.mark.gpu
KEPT = -77.0        # what out holds before


def pool(pages, heads, page, dim, seed):
    rng = np.random.default_rng(seed)
    codes = [rng.integers(-127, 128, (pages, heads, page, dim)).astype(np.int8) for _ in range(2)]
    scales = [(rng.random((pages, heads)) * 0.02 + 0.001).astype(np.float32) for _ in range(2)]
    return codes + scales


def case(B, T, H, Hk, D, page, lens, dtype, seed=0, q_scale=1.0):
    rng = np.random.default_rng(seed)
    per = max(1, -(-max(lens) // page))
    pages = B * per + 3
    cache = pool(pages, Hk, page, D, seed)
    table = rng.permutation(pages)[: B * per].reshape(B, per).astype(np.int32)
    q = dev((rng.standard_normal((B, T, H, D)) * q_scale).astype(np.float32)).to(dtype)
    return q, cache, table


def check(q, cache, table, lens, counts=None, window=0, sinks=0, scale=None, status=0, given=None, **kw):
    """One call against the definition; returns (out, lse)."""
    B, T, H, D = q.shape
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, KEPT) if kw.get("out") is None else kw.pop("out")
    lse = torch.full((B, T, H), KEPT, device="cuda")
    y = bsg.kv8_attend_window(q, given or bsg.Kv8Cache(*map(dev, cache)), dev(table), dev(np.int32(lens)), window=window, sinks=sinks,
                              counts=None if counts is None else dev(np.int32(counts)), scale=scale, out=out, lse=lse, dstatus=st, **kw)
    torch.cuda.synchronize()
    assert y is out and int(st) == status
    c = [T] * B if counts is None else [n if 0 <= n <= T else 0 for n in counts]
    lens = np.clip(lens, 0, table.shape[1] * cache[0].shape[2])
    parts = 1 if q.dtype == torch.bfloat16 else 2
    want, wlse, tol, lt = ref.window(f64(q), cache, table, lens, c, window, sinks, D ** -0.5 if scale is None else scale, parts)
    there = (np.arange(T)[None] < np.array(c)[:, None])
    want[~there], wlse[~there] = KEPT, KEPT
    within(f64(y), want, np.where(there[:, :, None, None], tol * 1.001 + rounding(want, q.dtype), 0), "out")
    g = f64(lse)
    none = np.isneginf(wlse)
    assert (np.isneginf(g) == none).all()
    within(np.where(none, 0, g), np.where(none, 0, wlse), np.where(there[:, :, None], 1.001 * lt, 0), "lse")
    return y, lse


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("D", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("T,window,sinks", [(1, 50, 4), (1, 0, 0), (5, 33, 1), (16, 100, 20), (17, 0, 0), (40, 64, 130), (150, 7, 4), (300, 129, 0)])
def test_ragged(T, window, sinks, D, dtype):
    B, H, Hk, page = 4, 4, 2, 16
    counts = [T, T // 2, 1, 0]
    lens = [T, T // 2 + 211, 400, 30]
    q, cache, table = case(B, T, H, Hk, D, page, lens, dtype, T + D)
    check(q, cache, table, lens, counts, window, sinks)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (8, 1), (14, 2), (40, 5)])
@pytest.mark.parametrize("T", [1, 3, 70, 129])
def test_heads(T, H, Hk, dtype):
    lens = [T, 313, 1000]
    q, cache, table = case(3, T, H, Hk, 64, 48, lens, dtype, H)
    check(q, cache, table, lens, None, 200, 3)
    check(q, cache, table, lens, None, 0, 0)


@pytest.mark.parametrize("page", [16, 32, 48, 128, 1024])
@pytest.mark.parametrize("T", [1, 257])
def test_pages(page, T):
    lens = [1500, T]
    q, cache, table = case(2, T, 4, 2, 128, page, lens, torch.float16, page)
    for window, sinks in ((0, 0), (1, 0), (16, 16), (333, 1), (1 << 30, 1 << 30), (5, 10_000), (1499, 0)):
        check(q, cache, table, lens, None, window, sinks)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T", [2, 16, 60, 200])
def test_rows_that_see_nothing(T, dtype):
    """More new tokens than are cached: those at negative positions give zeros; a length of 0."""
    lens = [0, 1, T - 1, T]
    q, cache, table = case(4, T, 4, 2, 64, 16, [300] * 4, dtype, T)
    y, lse = check(q, cache, table, lens, None, 9, 2)
    assert bool((y[0] == 0).all()) and bool(torch.isneginf(lse[0]).all())
    check(q, cache, table, lens, None, 0, 0)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,B", [(2, 1), (3, 70), (8, 40), (16, 150), (150, 3)])
def test_windows_that_begin_behind_a_tile_another_row_sees(T, B, dtype):
    """The rows of a CTA begin to see at different tiles, in whatever order they come: few chunks
    and many (by the batch's size), windows that begin at the ends of tiles, sinks and none."""
    for window, sinks in ((150, 0), (145, 3), (209, 17), (16 * T // 2 + 1, 0)):
        lens = [T + 16 * i % 256 + 160 for i in range(B)]
        q, cache, table = case(B, T, 2, 1, 32, 16, lens, dtype, window)
        check(q, cache, table, lens, None, window, sinks)


@pytest.mark.parametrize("T", [1, 5, 64, 300])
def test_a_window_of_one_gives_the_newest_value(T):
    """Exactly: code x scale, rounded; whatever the scores are."""
    for dtype in DTYPES:
        q, cache, table = case(2, T, 2, 2, 64, 16, [T, 301], dtype, 1, q_scale=30.0)
        y, _ = check(q, cache, table, [T, 301], None, 1, 0)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T", [1, 33, 180])
def test_sizes_of_scores(T, dtype):
    """Peaked rows, nearly flat ones, rows of zeros, of subnormal and of large values; scales 0 and below."""
    lens = [500, T]
    q, cache, table = case(2, T, 4, 2, 64, 32, lens, dtype, 3)
    for f in (50.0, 1e-3):
        check((q.float() * f).to(dtype), cache, table, lens, None, 150, 4)
    z = q.clone()
    z[0, 0] = 0
    z[1, -1] = torch.finfo(dtype).tiny
    check(z, cache, table, lens, None, 0, 0)
    check(q, cache, table, lens, None, 90, 0, scale=0.0)
    check(q, cache, table, lens, None, 90, 1, scale=-0.3)
    if dtype != torch.float16:
        z[0, 0] = 1e30
        check(z, cache, table, lens, None, 90, 0, scale=1e-30)


@pytest.mark.parametrize("T", [1, 20, 140])
def test_a_maximum_that_grows_all_along(T):
    """Later keys score far above earlier ones, so that the running maximum moves at every tile."""
    lens, D = [900], 64
    q, cache, table = case(1, T, 2, 1, D, 16, lens, torch.float32, 9)
    q = dev(np.ones((1, T, 2, D), np.float32))
    for i, page in enumerate(table[0]):
        cache[0][page] = np.minimum(127, 2 * i + np.arange(16) // 8)[None, :, None]
        cache[2][page] = 0.02
    check(q, cache, table, lens, None, 0, 0, scale=1.0)
    for i, page in enumerate(table[0]):
        cache[0][page] *= -1
    check(q, cache, table, lens, None, 0, 0, scale=1.0)
    check(q, cache, table, lens, None, 500, 5, scale=1.0)


@pytest.mark.parametrize("T", [1, 24, 150])
def test_strides(T):
    """q a slice of a fused projection, one element off; out with strides of its own."""
    B, H, D = 2, 4, 64
    for dtype in DTYPES:
        lens = [T + 100, T]
        q, cache, table = case(B, T, H, 2, D, 16, lens, dtype, 2)
        for shift in (0, 1):
            fused = torch.zeros((B, T, 3 * H * D + 8), dtype=dtype, device="cuda")
            view = fused[:, :, shift:shift + H * D].unflatten(2, (H, D))
            view.copy_(q)
            store = torch.full((T, B, H + 1, D + 2), KEPT, dtype=dtype, device="cuda")
            out = store[:, :, :H, shift:shift + D].permute(1, 0, 2, 3)
            check(view, cache, table, lens, None, 40, 2, out=out)
            left = store.clone()
            left[:, :, :H, shift:shift + D] = KEPT
            assert bool((left == KEPT).all())


@pytest.mark.parametrize("T", [1, 5, 50, 200])
def test_pages_out_of_the_window_may_be_gone(T):
    """Table entries that no query sees may be anything, and so may their pages' scales; those
    that one sees are reported and skipped."""
    lens, window, sinks, page = [1000, 700], 100, 5, 16
    q, cache, table = case(2, T, 4, 2, 64, page, lens, torch.float32, T)
    gone = table.copy()
    for b, n in enumerate(lens):
        first = max(1, (n - T - window + 1) // page)
        gone[b, 1:first] = np.resize([-1, 1 << 30, -5], first - 1)
        gone[b, -(-n // page):] = 1 << 29
    # the definition reads clipped entries at positions that it masks
    check(q, cache, gone, lens, None, window, sinks)
    for b, n in enumerate(lens):
        for i in range(1, max(1, (n - T - window + 1) // page)):
            cache[2][table[b, i]] = cache[3][table[b, i]] = np.nan
    clean = [np.nan_to_num(x, nan=1.0) if x.dtype == np.float32 else x for x in cache]
    check(q, clean, table, lens, None, window, sinks, given=bsg.Kv8Cache(*map(dev, cache)))
    bad = table.copy()
    bad[0, (lens[0] - 1) // page] = -1          # the newest page
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = bsg.kv8_attend_window(q, bsg.Kv8Cache(*map(dev, clean)), dev(bad), dev(np.int32(lens)), window=window, sinks=sinks, dstatus=st)
    assert int(st) == bsg.DSTATUS_RANGE and bool(torch.isfinite(y).all())
    want, _, tol, _ = ref.window(f64(q[1:]), clean, table[1:], lens[1:], [T], window, sinks, 64 ** -0.5)
    within(f64(y[1:]), want, tol * 1.001 + rounding(want, q.dtype))


@pytest.mark.parametrize("T", [1, 8, 100])
def test_lengths_and_counts_out_of_range(T):
    page = 16
    q, cache, table = case(5, T, 2, 1, 64, page, [20 * page] * 5, torch.float16, T)
    lens, counts = [-3, 20 * page + 1, 100, 100, 100], [T, T, -1, T + 1, T]
    check(q, cache, table, lens, counts, 50, 3, status=bsg.DSTATUS_RANGE)
    check(q, cache, table, [0, 100, 1 << 30, 5, 100], None, 0, 0, status=bsg.DSTATUS_RANGE)


@pytest.mark.parametrize("T", [1, 30, 140])
def test_reports_nonfinite_and_keeps_the_other_rows(T):
    for dtype in DTYPES:
        lens = [300, T]
        q, cache, table = case(2, T, 4, 2, 64, 16, lens, dtype, T)
        args = bsg.Kv8Cache(*map(dev, cache)), dev(table), dev(np.int32(lens))
        want = bsg.kv8_attend_window(q, *args, window=90, sinks=2)
        for bad in (float("inf"), float("nan")):
            z = q.clone()
            z[0, T // 2, 1, 7] = bad
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            y = bsg.kv8_attend_window(z, *args, window=90, sinks=2, dstatus=st)
            assert int(st) == bsg.DSTATUS_NONFINITE
            keep = torch.ones(q.shape[:3], dtype=torch.bool, device="cuda")
            keep[0, T // 2, 1] = False
            assert torch.equal(y[keep], want[keep])


def test_tokens_that_are_not_there_are_not_read():
    for T in (8, 200):
        q, cache, table = case(2, T, 4, 2, 64, 16, [200, T], torch.float32, 4)
        q[0, 3:] = float("nan")
        check(q, cache, table, [200, T], [3, T], 50, 1)


def test_no_window_is_kv8_attend():
    for dtype in DTYPES:
        for T in (1, 16):
            lens = [1, 17, 900]
            q, cache, table = case(3, T, 8, 2, 128, 32, lens, dtype, T)
            c = bsg.Kv8Cache(*map(dev, cache))
            y, _ = check(q, cache, table, lens, None, 0, 0)
            z = bsg.kv8_attend(q, c, dev(table), dev(np.int32(lens)))
            # each is within the derived tolerance of the definition, so they are within two of one another
            want, _, tol, _ = ref.window(f64(q), cache, table, lens, [T] * 3, 0, 0, 128 ** -0.5, 1 if dtype == torch.bfloat16 else 2)
            within(f64(y), f64(z), 2 * (tol * 1.001 + rounding(want, dtype)) * 1.01)


def test_long_lengths():
    """Positions and offsets past 2^31 bytes of a cache; many chunks."""
    B, Hk, D, page, n = 2, 2, 256, 1024, 1 << 20
    pages = n // page + 2
    k = torch.zeros((2 * pages, Hk, page, D), dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    assert v.numel() > 1 << 30
    v[:, :, :, :] = torch.arange(2 * pages, device="cuda").remainder(100).to(torch.int8)[:, None, None, None]
    s = torch.full((2 * pages, Hk), 0.5, device="cuda")
    table = torch.arange(2 * pages - 1, -1, -1, dtype=torch.int32, device="cuda").view(2, pages)
    lens = torch.tensor([n, n - 77], dtype=torch.int32, device="cuda")
    for T in (1, 70):
        q = torch.randn((B, T, 4, D), device="cuda")
        y = bsg.kv8_attend_window(q, (k, v, s, s), table, lens, window=3000, sinks=6)
        for b in range(B):
            for t in (0, T - 1):
                i = int(lens[b]) - T + t
                j = torch.cat((torch.arange(6), torch.arange(i - 2999, i + 1)))
                want = float((table[b].cpu().long()[j // page] % 100).double().mean()) * 0.5
                assert float((y[b, t].double() - want).abs().max()) < 1e-4 * want
    y = bsg.kv8_attend_window(torch.randn((B, 1, 4, D), device="cuda"), (k, v, s, s), table, lens)
    want = float((table[0].cpu().long()[torch.arange(n) // page] % 100).double().mean()) * 0.5
    assert float((y[0].double() - want).abs().max()) < 1e-4 * want


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("gap", [0, 1])
def test_f32_sums_do_not_drift(D, gap):
    """Equal scores and values of one sign, where what a sum of f32 loses adds up.  Tensor cores
    lose less than 2^-23 of a sum with each product of 16 positions, two products to each (the
    probability's parts), and a sum of theirs takes 640 positions at most: 80 times 2^-23.  The
    rest: 16384 / 512 sums of those by 2^-24 each, and 2^-20 for what a score and a probability of
    22 bits are off.  (The scales are powers of two: the sum of the probabilities is exact.)"""
    B, T, Hk, n, page = 40, 64, 4, 16384, 64
    rng = np.random.default_rng(D)
    codes = [np.ones((n // page, Hk, page, D), np.int8), rng.integers(90, 128, (n // page, Hk, page, D)).astype(np.int8)]
    cache = codes + [np.full((n // page, Hk), 2.0 ** -7, np.float32)] * 2
    given = bsg.Kv8Cache(*map(dev, cache))
    table = dev(np.tile(np.arange(n // page, dtype=np.int32), (B, 1)))   # all sequences' positions are the same ones
    q = torch.zeros(B, T, Hk, D, device="cuda")
    out = torch.full((B, T, Hk, D + gap), KEPT, device="cuda")[..., :D]
    bsg.kv8_attend_window(q, given, table, dev(np.full(B, n, np.int32)), out=out)
    v = codes[1].astype(np.float64).transpose(1, 0, 2, 3).reshape(Hk, n, D) * 2.0 ** -7
    sums = np.cumsum(v, 1)[:, n - T:] / np.arange(n - T + 1, n + 1)[:, None]
    want = np.broadcast_to(sums.transpose(1, 0, 2)[None], q.shape)
    within(f64(out), want, np.abs(want) * (80 * 2.0 ** -23 + 32 * 2.0 ** -24 + 2.0 ** -20), "out")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_tables_far_wider_than_what_they_hold(dtype):
    """Room for 8 chunks of 65536 positions (bf16: one of 524288) in each of 80 sequences: some hold two of
    them, most less than a tile, one nothing."""
    B, T, page, width = 80, 17, 1024, 512
    lens = [0, 17, 70000, 65536, 131073] + [100 + 3 * b for b in range(B - 5)]
    rng = np.random.default_rng(5)
    cache = pool(160, 1, page, 32, 5)
    table = np.full((B, width), -1, np.int32)
    for b, n in enumerate(lens):
        table[b, : -(-n // page)] = rng.permutation(160)[: -(-n // page)]
    q = dev(rng.standard_normal((B, T, 1, 32)).astype(np.float32)).to(dtype)
    check(q, cache, table, lens)
    check(q, cache, table, lens, counts=[T if b % 3 else b % T for b in range(B)])


def test_graph_and_streams():
    """Captured, replayed at other lengths; calls on several streams at once."""
    for T in (1, 6, 130):
        lens = [T + 5, 777]
        q, cache, table = case(2, T, 4, 2, 64, 16, [1000, 1000], torch.float16, 6)
        c, tb = bsg.Kv8Cache(*map(dev, cache)), dev(table)
        ln = dev(np.int32(lens))
        ws = bsg.Workspace(q.device)
        out = bsg.kv8_attend_window(q, c, tb, ln, window=300, sinks=4, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            bsg.kv8_attend_window(q, c, tb, ln, window=300, sinks=4, out=out, workspace=ws)
        for lens in ([1000, 0], [T, 400]):
            ln.copy_(dev(np.int32(lens)))
            out.zero_()
            g.replay()
            first = out.clone()
            assert torch.equal(first, bsg.kv8_attend_window(q, c, tb, ln, window=300, sinks=4))
            want, _, tol, _ = ref.window(f64(q), cache, table, lens, [T, T], 300, 4, 64 ** -0.5)
            within(f64(first), want, tol * 1.001 + rounding(want, q.dtype))
        want = out.clone()
        torch.cuda.synchronize()
        got = []
        for st in [torch.cuda.Stream() for _ in range(3)]:
            with torch.cuda.stream(st):
                got.append(bsg.kv8_attend_window(q, c, tb, ln, window=300, sinks=4))
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) for x in got)


def test_refusals():
    q, cache, table = case(2, 3, 4, 2, 64, 16, [50, 60], torch.float32)
    c, tb, ln = bsg.Kv8Cache(*map(dev, cache)), dev(table), dev(np.int32([50, 60]))
    for call, error in ((lambda: bsg.kv8_attend_window(q, c, tb, ln, window=-1), ValueError),
                        (lambda: bsg.kv8_attend_window(q, c, tb, ln, sinks=-1), ValueError),
                        (lambda: bsg.kv8_attend_window(q, c, tb, ln, window=1 << 31), ValueError),
                        (lambda: bsg.kv8_attend_window(q, c, tb, ln.long()), TypeError),
                        (lambda: bsg.kv8_attend_window(q, c, tb, ln, counts=ln[:1]), ValueError),
                        (lambda: bsg.kv8_attend_window(q, c, tb[:1], ln), ValueError),
                        (lambda: bsg.kv8_attend_window(q[:, :, :3], c, tb, ln), ValueError),
                        (lambda: bsg.kv8_attend_window(q, c, tb, ln, out=q), ValueError),
                        (lambda: bsg.kv8_attend_window(q, c, tb, ln, scale=float("inf")), bsg.BsgError),
                        (lambda: bsg.kv8_attend_window(q.double(), c, tb, ln), TypeError)):
        with pytest.raises(error):
            call()

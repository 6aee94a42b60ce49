"""Attention behind a prefix that all sequences share, against 64 bits; tolerances as in
test_gpu_kv8_window."""
import numpy as np
import pytest
import torch

import prompts_ref as ref
import verifiable_quantize_rows_gb300 as bsg
from gpu_util import dev
from serving_ref import DTYPES, IDS, f64, rounding, within
from test_gpu_kv8_window import pool

pytestmark = pytest.mark.gpu


def case(B, T, H, Hk, D, page, n, lens, dtype, seed=0):
    rng = np.random.default_rng(seed)
    per, pre = max(1, -(-max(lens) // page)), max(1, -(-n // page))
    pages = B * per + pre + 2
    order = rng.permutation(pages).astype(np.int32)
    cache = pool(pages, Hk, page, D, seed)
    q = dev(rng.standard_normal((B, T, H, D)).astype(np.float32)).to(dtype)
    return q, cache, order[:pre].copy(), order[pre:pre + B * per].reshape(B, per).copy()


def check(q, cache, prefix, n, table, lens, scale=None, status=0, given=None, out=None, **kw):
    B, T, H, D = q.shape
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.empty((B, T, H), device="cuda")
    y = bsg.kv8_attend_shared(q, given or bsg.Kv8Cache(*map(dev, cache)), dev(prefix), dev(np.int32([n])), dev(table), dev(np.int32(lens)),
                              scale=scale, out=out, lse=lse, dstatus=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == status
    page = cache[0].shape[2]
    n, lens = min(max(n, 0), len(prefix) * page), np.clip(lens, 0, table.shape[1] * page)
    parts = 1 if q.dtype == torch.bfloat16 else 2
    want, wlse, tol, lt = ref.shared(f64(q), cache, prefix, n, table, lens, D ** -0.5 if scale is None else scale, parts)
    within(f64(y), want, tol * 1.001 + rounding(want, q.dtype), "out")
    g, none = f64(lse), np.isneginf(wlse)
    assert (np.isneginf(g) == none).all()
    within(np.where(none, 0, g), np.where(none, 0, wlse), 1.001 * lt, "lse")
    return y


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("D", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("B,T,n", [(1, 1, 100), (3, 5, 33), (5, 1, 1000), (9, 16, 300), (40, 2, 700), (70, 1, 513)])
def test_batches(B, T, n, D, dtype):
    lens = [T + 7 * i for i in range(B)]
    lens[0] = 0 if B > 1 else T             # an idle slot
    check(*case(B, T, 4, 2, D, 16, n, lens, dtype, B + D)[:3], n, *case(B, T, 4, 2, D, 16, n, lens, dtype, B + D)[3:], lens)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (8, 1), (14, 2), (40, 5)])
@pytest.mark.parametrize("B", [2, 17])
def test_heads(B, H, Hk, dtype):
    lens = [1 + 13 * i for i in range(B)]
    q, cache, prefix, table = case(B, 1, H, Hk, 64, 48, 400, lens, dtype, H)
    check(q, cache, prefix, 400, table, lens)


@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 127, 128, 129, 2000])
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_prefix_lengths(n, page):
    for B, T in ((2, 3), (40, 4)):
        lens = [T + i for i in range(B)]
        q, cache, prefix, table = case(B, T, 4, 2, 128, page, max(n, 1), lens, torch.float16, n)
        check(q, cache, prefix, n, table, lens)


@pytest.mark.parametrize("B", [3, 50])
def test_queries_before_the_first_own_token_see_nothing(B):
    T = 5
    lens = [i % 7 for i in range(B)]
    q, cache, prefix, table = case(B, T, 4, 2, 64, 16, 100, [7] * B, torch.float32, 1)
    y = check(q, cache, prefix, 100, table, lens)
    assert bool((y[0] == 0).all()) and bool((y[1, :4] == 0).all())


@pytest.mark.parametrize("B", [3, 60])
def test_values(B):
    """Garbage behind the prefix's end in its last page; NaN in scales of pages that nothing reads;
    scales 0 and below; scores that differ much between prefix and own tokens."""
    lens = [1 + 5 * i for i in range(B)]
    q, cache, prefix, table = case(B, 1, 8, 2, 64, 32, 300, lens, torch.float32, 2)
    for b in range(B):
        for i in range(-(-lens[b] // 32), table.shape[1]):
            cache[2][table[b, i]] = cache[3][table[b, i]] = np.nan
    clean = [np.nan_to_num(x, nan=1.0) if x.dtype == np.float32 else x for x in cache]
    given = bsg.Kv8Cache(*map(dev, cache))
    check(q, clean, prefix, 300, table, lens, given=given)
    check(q, clean, prefix, 300, table, lens, scale=0.0)
    check(q, clean, prefix, 300, table, lens, scale=-0.2)
    check(q * 40, clean, prefix, 300, table, lens)
    clean[2][prefix] *= 1e-6
    check(q, clean, prefix, 300, table, lens, scale=1.0)
    clean[2][prefix] *= 1e8
    check(q, clean, prefix, 300, table, lens, scale=0.05)


def test_out_of_range():
    for B in (3, 60):
        lens = [20 + i for i in range(B)]
        q, cache, prefix, table = case(B, 1, 4, 2, 64, 16, 100, lens, torch.float32, 5)
        check(q, cache, prefix, 16 * len(prefix) + 1, table, lens, status=bsg.DSTATUS_RANGE)
        check(q, cache, prefix, -1, table, lens, status=bsg.DSTATUS_RANGE)
        check(q, cache, prefix, 50, table, [-1, 1 << 30] + lens[2:], status=bsg.DSTATUS_RANGE)
        bad = prefix.copy()
        bad[1] = -1                         # skipped: as if its positions were not there
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = bsg.kv8_attend_shared(q, bsg.Kv8Cache(*map(dev, cache)), dev(bad), dev(np.int32([48])), dev(table), dev(np.int32(lens)), dstatus=st)
        assert int(st) == bsg.DSTATUS_RANGE
        want, _, tol, _ = ref.shared(f64(q), cache, prefix[[0, 2]], 32, table, lens, 64 ** -0.5)
        within(f64(y), want, tol * 1.001 + rounding(want, q.dtype))
        st.zero_()
        bsg.kv8_attend_shared(q, bsg.Kv8Cache(*map(dev, cache)), dev(bad), dev(np.int32([16])), dev(table), dev(np.int32(lens)), dstatus=st)
        assert int(st) == 0                 # the bad page is not read


@pytest.mark.parametrize("B", [2, 70])
def test_reports_nonfinite_and_keeps_the_other_rows(B):
    for dtype in DTYPES:
        lens = [30 + i for i in range(B)]
        q, cache, prefix, table = case(B, 2, 4, 2, 64, 16, 200, lens, dtype, 8)
        args = bsg.Kv8Cache(*map(dev, cache)), dev(prefix), dev(np.int32([200])), dev(table), dev(np.int32(lens))
        want = bsg.kv8_attend_shared(q, *args)
        z = q.clone()
        z[1, 0, 2, 5] = float("nan")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = bsg.kv8_attend_shared(z, *args, dstatus=st)
        assert int(st) == bsg.DSTATUS_NONFINITE
        keep = torch.ones(q.shape[:3], dtype=torch.bool, device="cuda")
        keep[1, 0, 2] = False
        assert torch.equal(y[keep], want[keep])


@pytest.mark.parametrize("B,T", [(3, 1), (40, 3)])
def test_strides_graph_and_streams(B, T):
    H, D = 4, 64
    for dtype in DTYPES:
        lens = [T + 3 * i for i in range(B)]
        q, cache, prefix, table = case(B, T, H, 2, D, 16, 333, lens, dtype, 3)
        fused = torch.zeros((B, T, 3 * H * D + 8), dtype=dtype, device="cuda")
        view = fused[:, :, 1:1 + H * D].unflatten(2, (H, D))
        view.copy_(q)
        store = torch.full((T, B, H + 1, D + 2), 5.0, dtype=dtype, device="cuda")
        out = store[:, :, :H, 1:1 + D].permute(1, 0, 2, 3)
        y = check(view, cache, prefix, 333, table, lens, out=out)
        left = store.clone()
        left[:, :, :H, 1:1 + D] = 5
        assert bool((left == 5).all())
        c, pf, n, tb, ln = bsg.Kv8Cache(*map(dev, cache)), dev(prefix), dev(np.int32([333])), dev(table), dev(np.int32(lens))
        ws = bsg.Workspace(q.device)
        out = bsg.kv8_attend_shared(q, c, pf, n, tb, ln, workspace=ws)
        assert torch.equal(out, y)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            bsg.kv8_attend_shared(q, c, pf, n, tb, ln, out=out, workspace=ws)
        n.fill_(77)
        ln.sub_(1)
        out.zero_()
        g.replay()
        want = bsg.kv8_attend_shared(q, c, pf, n, tb, ln)
        assert torch.equal(out, want)
        torch.cuda.synchronize()
        got = []
        for st in [torch.cuda.Stream() for _ in range(3)]:
            with torch.cuda.stream(st):
                got.append(bsg.kv8_attend_shared(q, c, pf, n, tb, ln))
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) for x in got)


def test_equals_the_whole_sequence_in_one_table():
    """A prefix of whole pages and the same pages at the head of each table: the same attention."""
    B, T, page, n = 20, 2, 16, 320
    lens = [T + 11 * i for i in range(B)]
    q, cache, prefix, table = case(B, T, 8, 2, 128, page, n, lens, torch.float32, 4)
    y = check(q, cache, prefix, n, table, lens)
    whole = np.concatenate([np.broadcast_to(prefix, (B, len(prefix))), table], 1).copy()
    z = bsg.kv8_attend(q, bsg.Kv8Cache(*map(dev, cache)), dev(whole), dev(np.int32(lens) + n))
    # each is within the derived tolerance of the definition, so they are within two of one another
    want, _, tol, _ = ref.shared(f64(q), cache, prefix, n, table, lens, 128 ** -0.5)
    within(f64(y), f64(z), 2 * (tol * 1.001 + rounding(want, q.dtype)))


def test_refusals():
    q, cache, prefix, table = case(2, 3, 4, 2, 64, 16, 50, [5, 6], torch.float32)
    c, pf, n, tb, ln = bsg.Kv8Cache(*map(dev, cache)), dev(prefix), dev(np.int32([50])), dev(table), dev(np.int32([5, 6]))
    for call, error in ((lambda: bsg.kv8_attend_shared(q, c, pf[:0], n, tb, ln), ValueError),
                        (lambda: bsg.kv8_attend_shared(q, c, pf, 50, tb, ln), TypeError),
                        (lambda: bsg.kv8_attend_shared(q, c, pf.long(), n, tb, ln), TypeError),
                        (lambda: bsg.kv8_attend_shared(q, c, pf[None], n, tb, ln), ValueError),
                        (lambda: bsg.kv8_attend_shared(q, c, pf, n, tb, ln, out=q), ValueError),
                        (lambda: bsg.kv8_attend_shared(q.expand(2, 3, 4, 64).repeat(1, 6, 1, 1), c, pf, n, tb, ln), ValueError),
                        (lambda: bsg.kv8_attend_shared(q, c, pf, n, tb, ln, scale=float("nan")), bsg.BsgError)):
        with pytest.raises(error):
            call()

"""The int8 key/value cache: append against the stated roundings (bitwise),
attention against 64 bits.

Tolerance of attention: serving_ref.attend derives it per element from the
scores' errors; outputs of 16-bit types may also have probabilities rounded to
11 bits (2^-11 of sum p |v|), and every output is rounded once to its type."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import verifiable_quantize_rows_gb300 as bsg
from gpu_util import dev, host
from serving_ref import DTYPES, IDS, f64, rounding, within

pytestmark = pytest.mark.gpu


def pool(pages, heads, page, dim, seed):
    rng = np.random.default_rng(seed)
    codes = [rng.integers(-127, 128, (pages, heads, page, dim)).astype(np.int8) for _ in range(2)]
    scales = [(rng.random((pages, heads)) * 0.02 + 0.001).astype(np.float32) for _ in range(2)]
    return codes + scales


def table_for(batch, per, pages, seed):
    return np.random.default_rng(seed).permutation(pages)[: batch * per].reshape(batch, per).astype(np.int32)


def on_gpu(cache):
    return bsg.Kv8Cache(*[dev(x) for x in cache])


def run_append(k, v, cache, table, starts, counts, want_status=0, **kw):
    """The library's append on a copy of `cache`; returns host arrays."""
    c = on_gpu(cache)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsg.kv8_append(k, v, c, dev(table), dev(np.int32(starts)),
                   None if counts is None else dev(np.int32(counts)), dstatus=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == want_status
    return [host(x) for x in c]


def same_cache(got, want):
    for name, g, w in zip(("k", "v", "k_scale", "v_scale"), got, want):
        bad = np.argwhere(g.view(np.uint8 if g.itemsize == 1 else np.uint32)
                          != w.view(np.uint8 if w.itemsize == 1 else np.uint32))
        assert not len(bad), (name, len(bad), bad[0], g[tuple(bad[0])], w[tuple(bad[0])])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("page,T", [(16, 1), (16, 37), (32, 5), (48, 100), (64, 64), (128, 300)])
def test_append(dtype, dim, page, T):
    B, H = 5, 3
    starts = [0, 1, page - 1, page, 2 * page + 7]
    counts = [T, T, max(T - 1, 0), 0, T]
    per = (max(starts) + T) // page + 1
    pages = B * per + 2
    cache = pool(pages, H, page, dim, dim + T)
    # new values smaller and larger than the old blocks', so that some scales grow
    rng = np.random.default_rng(T)
    k, v = (dev((rng.standard_normal((B, T, H, dim)) * s).astype(np.float32)).to(dtype)
            for s in (0.4, 2.0))
    table = table_for(B, per, pages, 3)
    got = run_append(k, v, cache, table, starts, counts)
    want = ref.append(k.float().cpu().numpy(), v.float().cpu().numpy(),
                      [x.copy() for x in cache], table, starts, counts)
    same_cache(got, want)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_append_reads_slices_of_a_fused_projection(dtype):
    """k and v as strided views of one (batch, tokens, 3 heads dim) tensor,
    aligned and one element off."""
    B, T, H, D, page = 2, 19, 4, 64, 16
    for shift in (0, 1):
        fused = dev(np.random.default_rng(1).standard_normal((B, T, 3 * H * D + 8)).astype(np.float32)).to(dtype)
        k = fused[:, :, shift + H * D: shift + 2 * H * D].unflatten(2, (H, D))
        v = fused[:, :, shift + 2 * H * D: shift + 3 * H * D].unflatten(2, (H, D))
        cache = pool(9, H, page, D, 2)
        table = table_for(B, 3, 9, 1)
        got = run_append(k, v, cache, table, [3, 16], None)
        want = ref.append(k.float().cpu().numpy(), v.float().cpu().numpy(),
                          [x.copy() for x in cache], table, [3, 16], [T, T])
        same_cache(got, want)


def test_append_token_by_token_and_ties():
    """One token at a time into the same pages, with zeros, the floor, exact
    ties (x inv = n + 1/2), and a growing scale on most steps."""
    H, D, page, n = 2, 32, 16, 40
    cache = pool(4, H, page, D, 5)
    table = table_for(1, 3, 4, 0)
    rng = np.random.default_rng(7)
    x = rng.standard_normal((n, H, D)).astype(np.float32) * np.linspace(0.1, 3, n).astype(np.float32)[:, None, None]
    x[0] = 0.0
    x[16] = 1e-9
    x[17] = np.resize(np.float32([0.5, 1.5, -0.5, -2.5, 127.0]), D)     # scale 1: ties
    x[18] = -0.0
    c = on_gpu(cache)
    want = [a.copy() for a in cache]
    for i in range(n):
        k = dev(x[None, i: i + 1])
        bsg.kv8_append(k, -k, c, dev(table), dev(np.int32([i])))
        ref.append(x[None, i: i + 1], -x[None, i: i + 1], want, table, [i], [1])
    same_cache([host(a) for a in c], want)


def test_append_out_of_range_writes_nothing():
    """Negative starts, counts above T, positions past the table and pages
    outside the pool: reported, and everything else is as without them."""
    B, T, H, D, page = 7, 3, 2, 64, 16
    cache = pool(8, H, page, D, 1)
    table = np.array([[0], [1], [2], [3], [8], [-1], [4]], np.int32)
    starts, counts = [-1, 2, 14, 16, 0, 0, 5], [3, 4, 3, 1, 3, 3, 3]
    k = dev(np.random.default_rng(2).standard_normal((B, T, H, D)).astype(np.float32))
    got = run_append(k, k, cache, table, starts, counts, want_status=bsg.DSTATUS_RANGE)
    kh = host(k)
    want = [x.copy() for x in cache]
    ref.append(kh[2:3], kh[2:3], want, table[2:3], [14], [2])      # the tokens inside the table
    ref.append(kh[6:], kh[6:], want, table[6:], [5], [3])
    same_cache(got, want)
    got = run_append(k[2:3], k[2:3], cache, table[2:3], [2 ** 31 - 1], [3], want_status=bsg.DSTATUS_RANGE)
    same_cache(got, cache)


def test_append_reports_nonfinite():
    H, D, page = 2, 64, 16
    cache = pool(3, H, page, D, 1)
    table = np.array([[0], [2]], np.int32)
    x = np.ones((2, 4, H, D), np.float32)
    x[1, 2, 0, 5] = np.inf
    got = run_append(dev(x), dev(np.ones_like(x)), cache, table, [0, 0], None,
                     want_status=bsg.DSTATUS_NONFINITE)
    want = ref.append(np.ones_like(x), np.ones_like(x), [a.copy() for a in cache], table, [0, 0], [4, 4])
    got[0][2, 0], got[2][2, 0] = want[0][2, 0], want[2][2, 0]          # the page and head with the Inf
    same_cache(got, want)


# ---------------------------------------------------------------------------
def check(q, cache, table, lens, scale=None, heads_out=None, what="", want_status=0, **kw):
    B, T, H, D = q.shape
    c = cache if isinstance(cache, bsg.Kv8Cache) else on_gpu(cache)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.full((B, T, H), 3.0, device="cuda")
    s = D ** -0.5 if scale is None else scale
    o = bsg.kv8_attend(q, c, dev(table), dev(np.int32(lens)), scale=scale, lse=lse, dstatus=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == want_status
    want, wl, tol = ref.attend(f64(q), [host(x) for x in c], table, lens, s)
    if q.dtype != torch.float32:
        # probabilities in 11 bits: 2^-11 of sum p|v|, at most max |v| of the cache's codes
        vmax = float((c.v.float().abs().amax((0, 2, 3)) * c.v_scale.amax(0)).max())
        tol = tol + 2.0 ** -11 * np.minimum(vmax, vmax * (wl[..., None] > -np.inf))
    within(f64(o), want, tol + rounding(want, q.dtype), what)
    seen = wl > -np.inf
    got = host(lse)
    assert (got[~seen] == -np.inf).all()
    # lse: the scores' errors (bounded with |q| and |k| at their largest) and the sum's
    kmax = 127 * float(c.k_scale.max())
    qa = np.abs(f64(q))
    dl = abs(s) * kmax * (2.0 ** -20 * qa.sum(3) + 2.0 ** -21 * D * qa.max(3)) + 2.0 ** -19
    within(got[seen], wl[seen], (dl + 2.0 ** -22 * np.abs(wl))[seen], what + " lse")
    assert (f64(o)[~seen] == 0).all()
    return o


def queries(shape, dtype, seed, scale=1.0):
    x = np.random.default_rng(seed).standard_normal(shape) * scale
    return dev(x.astype(np.float32)).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("share,T", [(1, 1), (1, 3), (2, 1), (4, 1), (4, 4), (5, 3), (8, 1), (8, 16), (3, 16)])
def test_attend_heads_and_tokens(dtype, dim, share, T):
    """Shared heads, several queries, and a dim of every kind, at ragged
    lengths: empty, shorter than T, one page, several."""
    B, Hk, page = 6, 2, 16
    lens = [0, 1, 2, 16, 47, 130]
    pages = B * 9 + 1
    cache = pool(pages, Hk, page, dim, dim + share)
    table = table_for(B, 9, pages, T)
    check(queries((B, T, Hk * share, dim), dtype, T + dim), cache, table, lens)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 128, 1024])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_attend_every_tail(page, dtype):
    """Lengths around every boundary of tiles and pages."""
    lens = [1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 500, 511, 513, 1000, 1024]
    per = 1024 // page + (1024 % page > 0)
    pages = len(lens) * per
    cache = pool(pages, 1, page, 64, page)
    table = table_for(len(lens), per, pages, 1)
    check(queries((len(lens), 2, 2, 64), dtype, 4), cache, table, lens)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16], ids=["f32", "f16"])
@pytest.mark.parametrize("B,length", [(1, 1), (1, 300), (1, 5001), (3, 9000), (1, 40000)])
def test_attend_long(dtype, B, length):
    per = length // 64 + 2
    cache = pool(B * per, 2, 64, 64, length)
    table = table_for(B, per, B * per, 2)
    check(queries((B, 1, 8, 64), dtype, length), cache, table, [length] * B)


def test_attend_many_sequences_one_long():
    """150 sequences of which one is much longer than the rest."""
    B, per = 150, 64
    lens = [(7 * i) % 40 for i in range(B)]
    lens[77] = 1000
    cache = pool(400, 2, 16, 32, 3)
    table = np.random.default_rng(1).integers(0, 400, (B, per)).astype(np.int32)
    check(queries((B, 1, 4, 32), torch.float32, 1), cache, table, lens)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("qscale,scale", [(1e-3, None), (30.0, None), (1.0, -0.3), (1.0, 0.0), (100.0, 1.0)])
def test_attend_flat_and_peaked(dtype, qscale, scale):
    """Softmaxes from flat to one-hot, and a negative or zero scale."""
    cache = pool(40, 2, 32, 64, 8)
    cache[3][::3] *= 50            # pages of very different value scales
    cache[2][1::3] *= 0.01
    table = table_for(4, 10, 40, 8)
    check(queries((4, 2, 4, 64), dtype, 8, qscale), cache, table, [320, 319, 33, 2], scale)


def test_attend_rising_scores():
    """Every position's score above all before it: the running maximum moves
    in every tile, up to hundreds."""
    H, D, page, n = 1, 32, 16, 512
    cache = pool(n // page, H, page, D, 4)
    cache[0][:] = 1
    cache[2][:, 0] = np.linspace(0.01, 4, n // page)
    q = queries((1, 1, 2, D), torch.float32, 0)
    q[:] = torch.tensor([[[[2.0] * D, [8.0] * D]]], device="cuda")
    table = np.arange(n // page, dtype=np.int32)[None]
    check(q, cache, table, [n], 1.0)
    check(q, cache, table[:, ::-1].copy(), [n - 5], 1.0)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_attend_strided_queries_and_outputs(dtype):
    """q inside a fused projection (one element off alignment), out inside a
    wider tensor whose other elements stay."""
    B, T, H, D = 3, 2, 4, 64
    cache = pool(30, 2, 16, D, 6)
    table = table_for(B, 10, 30, 6)
    fused = queries((B, T, 3 * H * D + 1), dtype, 5)
    q = fused[:, :, 1: 1 + H * D].unflatten(2, (H, D))
    wide = torch.full((B, T, H, D + 8), 7.0, dtype=dtype, device="cuda")
    check(q, cache, table, [100, 160, 3], out=wide[..., :D])
    assert (wide[..., D:] == 7).all()


def test_attend_what_a_page_holds_beyond_the_length_does_not_matter():
    cache = pool(6, 2, 32, 64, 6)
    table = np.array([[0, 1, 2], [3, 4, 5]], np.int32)
    q = queries((2, 1, 4, 64), torch.float32, 1)
    a = check(q, cache, table, [33, 5])
    cache[0][1, :, 1:], cache[1][1, :, 1:] = -128, -128
    cache[0][3, :, 5:], cache[1][3, :, 5:] = 127, -128
    for s in (cache[2], cache[3]):
        s[2] = s[4] = s[5] = np.nan                              # pages that nothing has been written to
    table[0, 2], table[1, 1:] = 10 ** 6, -5                      # and table entries not filled in
    b = bsg.kv8_attend(q, on_gpu(cache), dev(table), dev(np.int32([33, 5])))
    assert torch.equal(a, b)


def test_attend_out_of_range_is_reported():
    """Lengths beyond the table count as the table's, negative ones as empty;
    pages outside the pool are left out."""
    cache = pool(6, 2, 16, 64, 6)
    q = queries((3, 1, 4, 64), torch.float32, 1)
    table = np.array([[0, 1], [2, 3], [4, 5]], np.int32)
    c = on_gpu(cache)
    want = bsg.kv8_attend(q, c, dev(table), dev(np.int32([32, 0, 7])))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bsg.kv8_attend(q, c, dev(table), dev(np.int32([33, -4, 7])), dstatus=st)
    assert int(st.item()) == bsg.DSTATUS_RANGE and torch.equal(got, want)
    st.zero_()
    bad = np.array([[0, 6], [2, 3], [-1, 5]], np.int32)
    got = bsg.kv8_attend(q, c, dev(bad), dev(np.int32([32, 0, 7])), dstatus=st)
    assert int(st.item()) == bsg.DSTATUS_RANGE
    ok = bsg.kv8_attend(q, c, dev(table), dev(np.int32([16, 0, 0])))
    assert torch.allclose(got[0], ok[0], rtol=1e-5, atol=1e-6) and (got[1:] == 0).all()


def test_attend_rows_do_not_affect_each_other_and_nonfinite_is_reported():
    cache = pool(30, 2, 16, 64, 6)
    table = table_for(3, 10, 30, 6)
    q = queries((3, 2, 8, 64), torch.float32, 1)
    a = check(q, cache, table, [100, 160, 3])
    q2 = q.clone()
    q2[1, 0, 3, 9] = float("nan")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    b = bsg.kv8_attend(q2, on_gpu(cache), dev(table), dev(np.int32([100, 160, 3])), dstatus=st)
    assert int(st.item()) == bsg.DSTATUS_NONFINITE
    b[1, 0, 3] = a[1, 0, 3]
    assert torch.equal(a, b)


def test_attend_offsets_past_32_bits():
    """Pages beyond 2^32 bytes into the pool."""
    pages, H, page, D = 36000, 8, 64, 256                       # 4.7 GB of keys
    c = bsg.Kv8Cache.empty(pages, H, page, D)
    far = [pages - 1, pages - 3, 3]
    rng = np.random.default_rng(3)
    small = pool(3, H, page, D, 3)
    for dst, src in zip(c, small):
        dst[torch.tensor(far, device="cuda")] = dev(src)
    q = queries((1, 1, 8, D), torch.float32, 3)
    got = bsg.kv8_attend(q, c, dev(np.int32([far])), dev(np.int32([150])))
    want = check(q, small, np.array([[0, 1, 2]], np.int32), [150])
    assert torch.equal(got, want)
    k = queries((1, 70, H, D), torch.float32, 4)
    bsg.kv8_append(k, k, c, dev(np.int32([far])), dev(np.int32([10])))
    wantc = ref.append(host(k), host(k), [x.copy() for x in small], np.array([[0, 1, 2]]), [10], [70])
    same_cache([host(x[torch.tensor(far, device="cuda")]) for x in c], wantc)


def test_attend_the_same_bits_every_time_and_on_another_stream():
    cache = on_gpu(pool(400, 2, 64, 64, 6))
    table = dev(table_for(2, 200, 400, 6))
    lens = dev(np.int32([12000, 700]))
    q = queries((2, 1, 8, 64), torch.float16, 2)
    a = bsg.kv8_attend(q, cache, table, lens)
    torch.cuda.synchronize()
    s, ws = torch.cuda.Stream(), bsg.Workspace()
    for i in range(20):
        b = bsg.kv8_attend(q, cache, table, lens, stream=s if i % 2 else None, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(a, b)


def test_attend_in_a_graph_with_new_lengths():
    """A captured step replays with the lengths and tables of its buffers."""
    cache = on_gpu(pool(60, 2, 16, 64, 6))
    tb = table_for(2, 30, 60, 6)
    table, lens = dev(tb), dev(np.int32([480, 100]))
    q = queries((2, 1, 4, 64), torch.float32, 2)
    ws = bsg.Workspace()
    out = bsg.kv8_attend(q, cache, table, lens, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsg.kv8_attend(q, cache, table, lens, out=out, workspace=ws)
    for n in ([480, 100], [3, 0], [77, 480]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, bsg.kv8_attend(q, cache, table, lens))

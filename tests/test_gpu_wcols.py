"""Products of tokens with int8 weights, bit for bit against the definition."""
import numpy as np
import pytest
import torch

import prompts_ref as ref
import verifiable_quantize_rows_gb300 as bsg
from gpu_util import dev
from serving_ref import DTYPES, IDS

pytestmark = pytest.mark.gpu


def inputs(M, K, N, dtype, seed=0, spread=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)).astype(np.float32)
    if spread:      # rows of very different sizes, outliers in them
        x *= np.exp2(rng.integers(-8, 6, (M, 1))).astype(np.float32)
        x[rng.random((M, K)) < 0.01] *= 20
    w = rng.integers(-127, 128, (K, N)).astype(np.int8)
    return dev(x).to(dtype), dev(w), dev((rng.random(N) * 0.01 + 1e-4).astype(np.float32))


def same(x, w, s, relu=False, status=0, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = bsg.wcols_matmul(x, w, s, relu=relu, dstatus=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == status
    assert y.dtype == x.dtype and y.shape == (x.shape[0], w.shape[1])
    want = ref.matmul(x.float().cpu().numpy(), w.cpu().numpy(), s.cpu().numpy(), relu, x.dtype)
    got = y.cpu()
    bad = (got != want).nonzero()
    assert not len(bad), (len(bad), bad[0].tolist(), got[tuple(bad[0])], want[tuple(bad[0])])
    return y


SIZES = [(1, 1, 1), (1, 768, 2304), (2, 17, 5), (3, 64, 128), (5, 1023, 255), (8, 1024, 256), (9, 1025, 257), (16, 130, 1),
         (17, 2048, 384), (31, 333, 1000), (33, 4097, 129), (61, 777, 1229), (64, 64, 64), (65, 1100, 512), (100, 2049, 131),
         (127, 300, 700), (128, 512, 640), (129, 640, 512), (200, 300, 1100), (256, 1536, 272), (257, 1024, 128), (300, 96, 2000),
         (513, 770, 515), (1000, 1000, 1000)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("M,K,N", SIZES)
def test_sizes(M, K, N, dtype):
    same(*inputs(M, K, N, dtype, M + K + N), relu=bool(N % 2))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("M", [1, 7, 40, 150, 400])
def test_strides(M, dtype):
    """Slices of wider rows, aligned and one element off; the weight's rows too."""
    K, N = 320, 336
    x, w, s = inputs(M, K, N, dtype)
    for shift in (0, 1, 8):
        wide = torch.zeros((M, K + 16), dtype=dtype, device="cuda")
        wide[:, shift:shift + K] = x
        rows = torch.full((K, N + 32), -128, dtype=torch.int8, device="cuda")
        rows[:, shift:shift + N] = w
        out = torch.full((M, N + 16), 7.0, dtype=dtype, device="cuda")
        y = same(wide[:, shift:shift + K], rows[:, shift:shift + N], s, out=out[:, shift:shift + N])
        assert y.data_ptr() == out[:, shift:].data_ptr()
        rest = torch.cat((out[:, :shift], out[:, shift + N:]), 1)
        assert bool((rest == 7).all())


LONG = [(17, 1030, 300), (40, 700, 12289), (64, 769, 11000), (64, 1025, 129), (65, 2049, 129), (100, 2300, 1000), (128, 2304, 384),
        (129, 4097, 200), (193, 2050, 1), (200, 2100, 700), (256, 8191, 272), (256, 2304, 768)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("M,K,N", LONG)
def test_sizes_of_long_columns_and_wide_weights(M, K, N, dtype):
    same(*inputs(M, K, N, dtype, M + K + N), relu=bool(N % 2))


@pytest.mark.parametrize("M", [40, 150])
def test_strides_of_long_columns(M):
    K, N = 2100, 336
    x, w, s = inputs(M, K, N, torch.bfloat16)
    for shift in (0, 1, 8):
        wide = torch.zeros((M, K + 16), dtype=torch.bfloat16, device="cuda")
        wide[:, shift:shift + K] = x
        rows = torch.full((K, N + 32), -128, dtype=torch.int8, device="cuda")
        rows[:, shift:shift + N] = w
        out = torch.full((M, N + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        same(wide[:, shift:shift + K], rows[:, shift:shift + N], s, out=out[:, shift:shift + N])
        assert bool((torch.cat((out[:, :shift], out[:, shift + N:]), 1) == 7).all())


@pytest.mark.parametrize("M", [1, 30, 200, 300])
def test_long_sums_and_largest_codes(M):
    """The largest K, every product 127 x 127: the sums fill 31 bits."""
    K, N = bsg.MAX_K, 40
    x = torch.full((M, K), 3.0, device="cuda")
    x[:, 1::2] = -3.0
    w = torch.full((K, N), 127, dtype=torch.int8, device="cuda")
    w[1::2, 1:] = -127
    same(x, w, torch.ones(N, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("M", [1, 20, 260])
def test_values(M, dtype):
    """Zero rows (the scale's floor), subnormal rows, ties, the largest finite ones, negative zeros."""
    K, N = 256, 128
    x, w, s = inputs(M, K, N, dtype, 5)
    x[0] = 0
    if M > 5:
        x[1] = -0.0
        x[2] = torch.finfo(dtype).tiny / 2
        x[3] = 0.5
        x[3, ::2] = 1.5
        x[3, 0] = 127.0
        x[4, 0] = torch.finfo(dtype).max
    same(x, w, s, relu=True)
    same(x, w, s)


def test_reports_nonfinite_and_keeps_the_other_rows():
    for M in (4, 40, 300):
        for bad in (float("inf"), float("-inf"), float("nan")):
            x, w, s = inputs(M, 200, 96, torch.float32)
            want = bsg.wcols_matmul(x, w, s).clone()
            x[2, 77] = bad
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            y = bsg.wcols_matmul(x, w, s, dstatus=st)
            assert int(st) == bsg.DSTATUS_NONFINITE
            keep = torch.arange(M, device="cuda") != 2
            assert torch.equal(y[keep], want[keep])


def test_a_row_does_not_depend_on_the_others():
    x, w, s = inputs(700, 1500, 300, torch.bfloat16)
    y = bsg.wcols_matmul(x, w, s)
    for n in (1, 8, 16, 17, 64, 128, 129, 256, 257):
        assert torch.equal(bsg.wcols_matmul(x[:n], w, s), y[:n])


def test_takes_what_wquant_cols_stores():
    W = torch.randn(500, 260, generator=torch.Generator("cuda").manual_seed(3), device="cuda") * 0.02
    x = torch.randn(50, 500, generator=torch.Generator("cuda").manual_seed(4), device="cuda")
    Q, s = bsg.wquant_cols(W, bits=8)
    y = same(x, Q, s)
    assert float((y - x @ W).abs().max()) < 0.05    # two roundings to 8 bits of 500 products of size 0.02


def test_graph_and_streams():
    """Captured, replayed with new inputs; calls on two streams at once; two graphs with a workspace each."""
    sets = [inputs(M, 900, 400, torch.float16, M) for M in (3, 90, 300)]
    want = [bsg.wcols_matmul(*i).clone() for i in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for st, i in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(bsg.wcols_matmul(*i))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for x, w, s in sets:
        x2 = torch.flip(x, (0,))
        buf = x.clone()
        ws = bsg.Workspace(x.device)
        out = bsg.wcols_matmul(buf, w, s, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            bsg.wcols_matmul(buf, w, s, out=out, workspace=ws)
        buf.copy_(x2)
        for _ in range(3):
            out.zero_()
            g.replay()
            assert torch.equal(out, torch.flip(bsg.wcols_matmul(x, w, s), (0,)))


def test_refusals():
    x, w, s = inputs(4, 64, 48, torch.float32)
    for call, error in ((lambda: bsg.wcols_matmul(x.double(), w, s), TypeError), (lambda: bsg.wcols_matmul(x, w.float(), s), TypeError),
                        (lambda: bsg.wcols_matmul(x, w, s.double()), TypeError), (lambda: bsg.wcols_matmul(x[:, 1:], w, s), ValueError),
                        (lambda: bsg.wcols_matmul(x, w.t(), s), ValueError), (lambda: bsg.wcols_matmul(x, w, s[1:]), ValueError),
                        (lambda: bsg.wcols_matmul(x, w, s, out=torch.empty(4, 47, device="cuda")), ValueError),
                        (lambda: bsg.wcols_matmul(x, w.cpu(), s), TypeError), (lambda: bsg.wcols_matmul(x[0].expand(4, 64), w, s), ValueError),
                        (lambda: bsg.wcols_matmul(x[0], w, s), ValueError), (lambda: bsg.wcols_matmul(x, w[:, :0], s[:0]), ValueError)):
        with pytest.raises(error):
            call()
    sq = torch.zeros(4, 4, device="cuda")
    with pytest.raises(ValueError, match="share"):
        bsg.wcols_matmul(sq, torch.zeros(4, 4, dtype=torch.int8, device="cuda"), s[:4].contiguous(), out=sq)

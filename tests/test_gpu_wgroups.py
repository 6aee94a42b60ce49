"""int4 weights with group scales: the storage against exact rationals' oracle
(bitwise), and products of a few rows with it against 64 bits.

Tolerance of a product (f32 sums of exact products): 2^-20 of sum |x w| for
the sums' roundings, and 2^-21 of a group's largest |x| times its sum |w| for
activations taken to the tensor cores in parts relative to that largest; then
one rounding to the output's type."""
import numpy as np
import pytest
import torch

import verifiable_quantize_rows_gb300 as bsg
from gpu_util import assert_bits_equal, dev, host
from serving_ref import DTYPES, IDS, f64, rounding, stored, unpack4, within

pytestmark = pytest.mark.gpu


def weight(K, N, seed):
    W = (np.random.default_rng(seed).standard_normal((K, N)) * 0.02).astype(np.float32)
    if N > 3:
        W[:, 0] = 0.0                                    # every group all zero
        W[K // 2:, 1] = 0.0
        W[:, 2] = np.float32(2.0 ** -149)                # the scale rounds to zero
    return W


@pytest.mark.parametrize("shape", [(1, 1), (32, 2), (33, 7), (200, 66), (1000, 129), (768, 300)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("group", [0, 32, 64, 96, 128, 4096])
def test_storage_is_the_column_storage_of_each_block(orc, shape, group):
    K, N = shape
    W = weight(K, N, K + N)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    Q, sc = bsg.wquant_groups(dev(W), group, dstatus=st)
    assert Q.shape == (K, (N + 1) // 2) and Q.stride(0) % 16 == 0
    G = group or K
    assert sc.shape == ((K + G - 1) // G, N)
    for g in range(sc.shape[0]):
        Qo, so, rc = orc.wquant_cols(np.ascontiguousarray(W[g * G:(g + 1) * G]), 4, False)
        assert rc == 0
        assert_bits_equal(host(sc[g]), so, "scales")
        assert (host(Q[g * G:(g + 1) * G].contiguous()) == orc.pack_int4(Qo)).all()
    assert int(st.item()) == 0


@pytest.mark.parametrize("K,N", [(5000, 130), (2049, 131), (129, 517)])
@pytest.mark.parametrize("group", [0, 64, 128, 160, 1056, 2048])
def test_storage_of_halves_and_tiny_scales(orc, K, N, group):
    """Quotients on and next to half-integers, and columns whose scale is near
    or below the least normal number (there the oracle says that it had to clamp)."""
    rng = np.random.default_rng(K + group)
    s = np.float32(rng.random((1, N)) + 0.5)
    n = rng.integers(-7, 7, (K, N))
    W = np.float32(s * (n + 0.5))
    W = np.nextafter(W, np.float32(W * rng.integers(0, 3, W.shape)), dtype=np.float32)
    W[0::32] = 7 * s
    W[:, 3::7] *= np.float32(2.0 ** -125)
    W[:, 4::7] *= np.float32(2.0 ** -147)
    Q, sc = bsg.wquant_groups(dev(W), group)
    G = group or K
    for g in range(sc.shape[0]):
        Qo, so, _ = orc.wquant_cols(np.ascontiguousarray(W[g * G:(g + 1) * G]), 4, False)
        assert_bits_equal(host(sc[g]), so, "scales")
        assert (host(Q[g * G:(g + 1) * G].contiguous()) == orc.pack_int4(Qo)).all()


def test_storage_reads_strided_weights_and_reports_nonfinite(orc):
    W = weight(100, 50, 1)
    wide = dev(np.concatenate([W, W], 1))
    Q, sc = bsg.wquant_groups(wide[:, 50:], 32)
    Q2, sc2 = bsg.wquant_groups(dev(W), 32)
    assert torch.equal(Q, Q2) and torch.equal(sc, sc2)
    W[40, 3] = np.nan
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    Q3, sc3 = bsg.wquant_groups(dev(W), 32, dstatus=st)
    assert int(st.item()) == bsg.DSTATUS_NONFINITE
    assert torch.equal(Q3[:32], Q2[:32]) and torch.equal(sc3[0], sc2[0])


def check(X, Q, sc, group, relu=False, what="", **kw):
    N = sc.shape[1]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    Y = bsg.wgroups_matvec(X, Q, sc, group=group, relu=relu, dstatus=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert Y.dtype == X.dtype and Y.shape == (X.shape[0], N)
    x, w = f64(X), stored(host(Q.contiguous()), host(sc.contiguous()), N, group)
    want = x @ w
    tol = 2.0 ** -20 * (np.abs(x) @ np.abs(w))
    G = group or x.shape[1]
    for k in range(0, x.shape[1], G):
        tol += (2.0 ** -21 * np.abs(x[:, k:k + G]).max(1)[:, None]
                * np.abs(w[k:k + G]).sum(0)[None, :])
    if relu:
        want = np.maximum(want, 0)
    within(f64(Y), want, tol + rounding(want, X.dtype), what)
    return Y


def activations(M, K, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.where(rng.random((M, K)) < 0.01, 20, 1)
    return dev(x.astype(np.float32)).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9, 13, 16])
@pytest.mark.parametrize("K,N,group", [(768, 2304, 64), (100, 70, 32), (1, 1, 0), (65, 130, 64),
                                       (511, 257, 128), (2050, 1000, 0)],
                         ids=lambda v: str(v))
def test_products(dtype, M, K, N, group):
    Q, sc = bsg.wquant_groups(dev(weight(K, N, K * 3 + N)), group)
    check(activations(M, K, dtype, M + K), Q, sc, group, relu=(M % 3 == 0))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("K", [1, 15, 16, 17, 31, 32, 33, 63, 64, 127, 500, 1023, 4097, 9000])
@pytest.mark.parametrize("group", [0, 32, 96])
def test_every_tail_of_k(dtype, K, group):
    Q, sc = bsg.wquant_groups(dev(weight(K, 200, K)), group)
    check(activations(3, K, dtype, K), Q, sc, group)


@pytest.mark.parametrize("N", [1, 2, 3, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 1001])
@pytest.mark.parametrize("tight", [False, True])
def test_every_tail_of_n(N, tight):
    K = 300
    Q, sc = bsg.wquant_groups(dev(weight(K, N, N)), 64)
    if tight:
        Q = Q.contiguous()
    check(activations(2, K, torch.float32, N), Q, sc, 64)


@pytest.mark.parametrize("offset", [1, 2, 4, 8])
def test_unaligned_and_strided_operands(offset):
    """Q at any byte, rows of every operand inside wider ones, and Y's
    neighbours untouched."""
    K, N, M, group = 200, 333, 4, 32
    Q, sc = bsg.wquant_groups(dev(weight(K, N, 5)), group)
    half = (N + 1) // 2
    wide = torch.full((K, half + 2 * offset + 3), 0x5A, dtype=torch.uint8, device="cuda")
    wide[:, offset:offset + half] = Q
    scw = torch.full((sc.shape[0], N + 5), float("nan"), device="cuda")
    scw[:, offset:offset + N] = sc[:, :N] if offset <= 5 else 0
    if offset > 5:
        scw[:, :N] = sc
    scv = scw[:, offset:offset + N] if offset <= 5 else scw[:, :N]
    X = torch.full((M, K + 9), float("nan"), device="cuda")
    X[:, offset:offset + K] = activations(M, K, torch.float32, 2)
    out = torch.full((M, N + 9), 7.0, device="cuda")
    Y = check(X[:, offset:offset + K], wide[:, offset:offset + half], scv, group,
              out=out[:, offset:offset + N])
    assert Y.data_ptr() == out.data_ptr() + 4 * offset
    assert (out[:, :offset] == 7).all() and (out[:, offset + N:] == 7).all()


@pytest.mark.parametrize("K", [1, 15, 16, 17, 31, 33, 64, 127, 255, 256, 257, 1023])
@pytest.mark.parametrize("N", [1, 63, 130, 513])
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_five_rows(K, N, offset):
    """The tails again with more rows than the small form takes, whose products
    run on the tensor cores at any size."""
    Q, sc = bsg.wquant_groups(dev(weight(K, N, K + N)), 32)
    half = (N + 1) // 2
    wide = torch.full((K, half + offset + 3), 0x5A, dtype=torch.uint8, device="cuda")
    wide[:, offset:offset + half] = Q
    X = torch.full((5, K + 9), float("nan"), device="cuda")
    X[:, offset:offset + K] = activations(5, K, torch.float32, K)
    check(X[:, offset:offset + K], wide[:, offset:offset + half], sc, 32)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("M,K,N", [(1, 4096, 2048), (1, 4096, 2049), (1, 4097, 2048), (2, 2048, 2048),
                                   (2, 2047, 2051), (3, 1031, 2035), (4, 1031, 2033), (4, 9001, 233),
                                   (2, 4096, 2048), (2, 2049, 4096), (4, 2048, 2048), (3, 2048, 2049),
                                   (1, 2048, 2048), (1, 2049, 2048), (2, 1024, 2048), (2, 1024, 2049),
                                   (4, 1024, 1024), (3, 1024, 1025),
                                   (1, 65537, 128), (1, 65537, 127), (1, 1, 70001), (1, 7, 1198372)])
def test_either_side_of_small(dtype, M, K, N):
    Q, sc = bsg.wquant_groups(dev(weight(K, N, K + N)), 96)
    check(activations(M, K, dtype, M), Q, sc, 96)


def test_column_storage_is_group_zero():
    """A weight that wquant_cols stored in 4 bits goes in as it is."""
    W = dev(weight(700, 131, 8))
    Q, sc = bsg.wquant_cols(W, bits=4)
    check(activations(2, 700, torch.float16, 1), Q, sc.view(1, -1), 0)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_scales_and_activations_of_any_size(dtype):
    """Groups of very different sizes in one row, zeros, and values near the
    type's ends."""
    K, N, group = 256, 96, 32
    big, small = (1e30, 1e-30) if dtype != torch.float16 else (3e4, 1e-6)
    x = np.random.default_rng(3).standard_normal((3, K))
    x[0, :32] *= big / 4
    x[0, 32:64] *= small
    x[1, :] = 0.0
    x[2, ::2] *= small
    W = weight(K, N, 9)
    W[:32] *= 1e-20
    Q, sc = bsg.wquant_groups(dev(W), group)
    check(dev(x.astype(np.float32)).to(dtype), Q, sc, group)


def test_codes_reach_minus_eight():
    """Codes that the storage never writes, -8, are still two's complement."""
    Q = torch.full((64, 8), 0x88, dtype=torch.uint8, device="cuda")
    sc = torch.ones((2, 16), device="cuda")
    Y = bsg.wgroups_matvec(torch.ones((1, 64), device="cuda"), Q, sc, group=32)
    assert (Y == -512).all()


def test_rows_do_not_affect_each_other_and_nonfinite_is_reported():
    K, N = 500, 300
    Q, sc = bsg.wquant_groups(dev(weight(K, N, 4)), 64)
    X = activations(5, K, torch.float32, 4)
    Y = bsg.wgroups_matvec(X, Q, sc)
    for bad in (float("inf"), float("nan")):
        X2 = X.clone()
        X2[3, 499] = bad
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        Y2 = bsg.wgroups_matvec(X2, Q, sc, dstatus=st)
        assert int(st.item()) == bsg.DSTATUS_NONFINITE
        keep = [0, 1, 2, 4]
        assert torch.equal(Y2[keep], Y[keep])


def test_the_same_bits_every_time_and_on_another_stream():
    K, N = 4096, 640
    Q, sc = bsg.wquant_groups(dev(weight(K, N, 6)), 64)
    X = activations(6, K, torch.bfloat16, 6)
    Y = bsg.wgroups_matvec(X, Q, sc)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for i in range(20):
        Z = bsg.wgroups_matvec(X, Q, sc, stream=s if i % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(Y, Z)


def test_offsets_past_32_bits():
    """A weight whose codes and rows lie beyond 2^32 bytes from its start."""
    K, N, group = 1100, 8, 0
    rows = torch.empty((K, 4 << 20), dtype=torch.uint8, device="cuda")
    small, sc = bsg.wquant_groups(dev(weight(K, N, 2)), group)
    rows[:, :4] = small
    check(activations(2, K, torch.float32, 2), rows[:, :4], sc, group)


@pytest.mark.parametrize("given", [False, True], ids=["current", "given"])
def test_calls_on_two_streams(given):
    """Calls that overlap on two streams, each with its stream's own workspace."""
    K, N = 2048, 5000
    sides = []
    for i in range(2):
        Q, sc = bsg.wquant_groups(dev(weight(K, N, i)), 64)
        X = activations(8, K, torch.float32, i)
        sides.append((X, Q, sc, check(X, Q, sc, 64), torch.cuda.Stream()))
    torch.cuda.synchronize()
    out = []
    for _ in range(50):
        for X, Q, sc, want, stream in sides:
            if given:
                out.append((bsg.wgroups_matvec(X, Q, sc, stream=stream), want))
            else:
                with torch.cuda.stream(stream):
                    out.append((bsg.wgroups_matvec(X, Q, sc), want))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y, want in out)

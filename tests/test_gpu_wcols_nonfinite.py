"""A token with Inf or NaN leaves every other token's bits as they were, however many parts its
sums come in."""
import pytest
import torch

import verifiable_quantize_rows_gb300 as bsg
from serving_ref import DTYPES, IDS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")], ids=str)
@pytest.mark.parametrize("M,K,N", [(3, 1500, 128), (16, 8192, 128), (17, 8192, 200), (64, 8192, 128), (200, 8192, 128), (300, 8192, 128)])
def test_sums_of_one_sign_beside_a_row_that_is_not_finite(M, K, N, bad, dtype):
    """All products have one sign, so a row whose codes are no codes sums to more than 31 bits; two
    tokens' sums travel in one word, the even one's below, and each of some 64 runs adds its part."""
    x = torch.ones(M, K, device="cuda").mul_(torch.arange(1, M + 1, device="cuda")[:, None]).to(dtype)
    w = torch.ones(K, N, dtype=torch.int8, device="cuda")
    s = torch.full((N,), 2.0 ** -9, device="cuda")
    want = bsg.wcols_matmul(x, w, s).clone()
    for sign in (1, -1):
        for row in {0, 1, M - 1 - M % 2, M - 1}:
            y = x.clone() * sign
            y[row, K // 3] = bad
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            got = bsg.wcols_matmul(y, w, s, dstatus=st)
            assert int(st) == bsg.DSTATUS_NONFINITE
            keep = torch.arange(M, device="cuda") != row
            assert torch.equal(got[keep], sign * want[keep]), row

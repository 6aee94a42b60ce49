"""Scales that are no numbers, on pages that some tokens of a call see and others do not.

A token with Inf or NaN leaves its page and head unspecified for those that see it; a query before
it, or one whose window has passed it, keeps its bits."""
import numpy as np
import pytest
import torch

import verifiable_quantize_rows_gb300 as bsg
from gpu_util import dev
from serving_ref import DTYPES, IDS
from test_gpu_kv8_window import case

pytestmark = pytest.mark.gpu
BAD = [float("inf"), float("-inf"), float("nan")]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("D", [32, 96, 128, 256])
@pytest.mark.parametrize("T,window,sinks", [(8, 0, 0), (8, 5, 0), (100, 0, 0), (300, 0, 0), (300, 70, 3), (300, 33, 0)])
def test_rows_that_do_not_see_a_page_keep_their_bits(T, window, sinks, D, dtype):
    page, lens = 16, [T + 20, T]
    q, cache, table = case(2, T, 4, 2, D, page, lens, dtype, T + D)
    given = bsg.Kv8Cache(*map(dev, cache))
    args = dict(window=window, sinks=sinks)
    want = bsg.kv8_attend_window(q, given, dev(table), dev(np.int32(lens)), **args)
    for at in {1, (T // 2) // page, (lens[0] - 1) // page}:      # pages of either sequence, the last one among them
        for which, bad in [(i, b) for i in (2, 3) for b in BAD]:
            spoilt = bsg.Kv8Cache(*[x.clone() for x in given])
            for b in range(2):
                if at < table.shape[1]:
                    spoilt[which][table[b, at]] = bad
            got = bsg.kv8_attend_window(q, spoilt, dev(table), dev(np.int32(lens)), **args)
            for b, n in enumerate(lens):
                i = np.arange(n - T, n)
                last = np.minimum(i, at * page + page - 1)       # the newest position of the page that row i could see
                sees = (at * page <= i) & ((last > i - window if window else True) | (at * page < sinks))
                keep = torch.from_numpy(~sees).cuda()
                assert torch.equal(got[b][keep], want[b][keep]), (at, which, bad, b)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("B", [3, 60])
def test_of_other_sequences_behind_a_shared_beginning(B, dtype):
    """A token that is no number in one sequence's own pages: the others keep their bits, and so do
    that sequence's tokens before it."""
    T, page, lens = 4, 16, [20 + b % 7 for b in range(B)]
    q, cache, table = case(B + 1, T, 4, 2, 64, page, [32] * (B + 1), dtype, B)
    prefix, table, q = table[B], table[:B], q[:B]
    lens[1] = 18                                                  # positions 14 to 17: two of its tokens on its second page
    given = bsg.Kv8Cache(*map(dev, cache))
    rest = dev(prefix), dev(np.int32([32])), dev(table.copy()), dev(np.int32(lens))
    want = bsg.kv8_attend_shared(q, given, *rest)
    for which, bad in [(i, b) for i in (2, 3) for b in BAD]:
        spoilt = bsg.Kv8Cache(*[x.clone() for x in given])
        spoilt[which][table[1, 1]] = bad
        got = bsg.kv8_attend_shared(q, spoilt, *rest)
        keep = torch.ones(B, T, dtype=torch.bool, device="cuda")
        keep[1, 2:] = False
        assert torch.equal(got[keep], want[keep]), (which, bad)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_a_prompt_whose_values_overflow(dtype):
    """Appended as it comes: a value of Inf from token 50 on leaves the 48 tokens of the pages before
    as they are."""
    T, H, D, page = 120, 2, 64, 16
    gen = torch.Generator(device="cuda").manual_seed(4)
    q, k, v = (torch.randn(1, T, H, D, generator=gen, device="cuda").to(dtype) for _ in range(3))
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    out = []
    for bad in (None, *BAD):
        w = v.clone()
        if bad is not None:
            w[0, 50, 1, 3] = bad
        cache = bsg.Kv8Cache.empty(8, H, page, D)
        bsg.kv8_append(k, w, cache, table, torch.zeros_like(lens))
        out.append(bsg.kv8_attend_window(q, cache, table, lens))
    for y in out[1:]:
        assert torch.equal(y[:, :48], out[0][:, :48]) and torch.equal(y[:, :, 0], out[0][:, :, 0])

"""The small decoder against 64 bits: the calls together.

The reference takes the decoder's stored weights and, of each block, the cache
as the step left it, and computes the newest token's logits.  Each product's
error is at most about 2^-20 of the sum of its terms' magnitudes (some 2^5 of
the result's), and a step of two blocks is nine products, so 2^-10 of the
largest logit holds them with room; a wrong position, page, scale or head is
of the logits' own size."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import verifiable_quantize_rows_gb300 as bsg
from gpu_util import host
from serving_ref import f64
from verifiable_quantize_rows_gb300.decode import Decoder, Shape

pytestmark = pytest.mark.gpu

SHAPES = [Shape(layers=2, heads=4, kv_heads=4, dim=32, hidden=200, vocab=1000, positions=200),
          Shape(layers=2, heads=6, kv_heads=2, dim=64, hidden=333, vocab=1003, positions=150, group=32)]


def norm(x):
    x = x - x.mean(-1, keepdims=True)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)


def newest(model, b, token):
    """The logits of the newest token of sequence b, 64 bits; each block's new
    key and value in the cache are checked to be the token's."""
    s, n = model.shape, int(model.lens[b])
    pages = host(model.table)[b]
    x = f64(model.embed[token]) + f64(model.place[n - 1])
    for cache, weights in zip(model.caches, model.blocks):
        P = cache[0].shape[2]
        W = [ref.stored(host(q.contiguous()), host(sc.contiguous()), sc.shape[1], s.group) for q, sc in weights]
        y = (norm(x) @ W[0]).reshape(-1, s.dim)
        q, new = y[:s.heads], (y[s.heads:s.heads + s.kv_heads], y[s.heads + s.kv_heads:])
        kv = []
        for codes, scales, mine in zip(cache[:2], cache[2:], new):
            c, sc = f64(codes[pages.tolist()]), f64(scales[pages.tolist()])
            all_ = (c * sc[:, :, None, None]).transpose(0, 2, 1, 3).reshape(-1, s.kv_heads, s.dim)[:n]
            half = 0.51 * sc[(n - 1) // P][:, None] + 1e-3 * np.abs(mine).max()
            assert (np.abs(all_[-1] - mine) <= half).all()
            kv.append(np.repeat(all_, s.heads // s.kv_heads, 1))
        z = np.einsum("hd,nhd->hn", q, kv[0]) * s.dim ** -0.5
        p = np.exp(z - z.max(1, keepdims=True))
        a = np.einsum("hn,nhd->hd", p / p.sum(1, keepdims=True), kv[1]).reshape(-1)
        x = x + a @ W[1]
        x = x + np.maximum(norm(x) @ W[2], 0) @ W[3]
    q, sc = model.head
    logits = norm(x) @ ref.stored(host(q.contiguous()), host(sc.contiguous()), s.vocab, s.group)
    return logits + f64(model.bias)


def log_softmax(z):
    return z - z.max() - np.log(np.exp(z - z.max()).sum())


@pytest.mark.parametrize("shape", SHAPES, ids=["heads", "shared"])
@pytest.mark.parametrize("lengths", [(1, 37, 64), (100,), (17, 5, 2, 33, 1)], ids=str)
def test_decoder(shape, lengths):
    model = Decoder(shape, len(lengths), page_tokens=32)
    rng = torch.Generator().manual_seed(len(lengths))
    last = []
    for b, n in enumerate(lengths):
        ids = torch.randint(shape.vocab, (n,), generator=rng).cuda()
        logits = model.prompt(ids, b)
        want = newest(model, b, int(ids[-1]))
        assert logits.shape == (n, shape.vocab)
        assert np.abs(f64(logits[-1]) - want).max() <= 2.0 ** -10 * np.abs(want).max()
        last.append(logits[-1].argmax())
    steps = 40
    answer = model.generate(torch.stack(last), steps, top=3)
    assert answer.tokens.shape == (len(lengths), steps)
    assert host(model.lens).tolist() == [n + steps for n in lengths]
    for b in range(len(lengths)):
        want = newest(model, b, int(answer.tokens[b, -2]))
        tol = 2.0 ** -9 * np.abs(want).max()
        lp = log_softmax(want)
        tokens = answer.top_token[b, -1].tolist()
        assert np.abs(f64(answer.top_logprob[b, -1]) - lp[tokens]).max() <= tol
        assert np.abs(lp[tokens] - np.sort(lp)[::-1][:3]).max() <= tol
        assert int(answer.tokens[b, -1]) == tokens[0]


def test_score_and_bias():
    model = Decoder(SHAPES[0])
    ids = torch.randint(1000, (50,), generator=torch.Generator().manual_seed(2)).cuda()
    logits = model.prompt(ids)
    z = f64(logits[:-1])
    lse = np.log(np.exp(z).sum(1))
    lp, entropy = model.score(logits, ids)
    at = (np.arange(49), host(ids)[1:])
    assert np.abs(f64(lp) - (z[at] - lse)).max() <= 1e-5
    p = np.exp(z - lse[:, None])
    assert np.abs(f64(entropy) - (p * (lse[:, None] - z)).sum(1)).max() <= 1e-5
    means = model.fit_bias(logits, ids, rate=2.0, steps=1)
    g = -p / 49
    np.add.at(g, at, 1 / 49)
    assert np.abs(f64(model.bias) - 2 * g.sum(0)).max() <= 1e-6
    assert abs(means[0] - (z[at] - lse).mean()) <= 1e-5
    now = z + f64(model.bias)
    assert abs(means[1] - (now[at] - np.log(np.exp(now).sum(1))).mean()) <= 1e-5
    assert model.fit_bias(logits, ids, steps=5)[-1] > means[1] > means[0]


def test_refusals():
    with pytest.raises(ValueError, match="sequences"):
        Decoder(SHAPES[0], 17)
    with pytest.raises(ValueError, match="multiple"):
        Decoder(SHAPES[0]._replace(kv_heads=3))
    model = Decoder(SHAPES[0], 2)
    with pytest.raises(ValueError, match="at most 200"):
        model.prompt(torch.zeros(201, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="at most 200"):
        model.generate(torch.zeros(2, dtype=torch.int64, device="cuda"), 201)

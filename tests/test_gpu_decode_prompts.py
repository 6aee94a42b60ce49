"""The small decoder with int8 weights, windows and shared beginnings, against 64 bits.

The reference takes the decoder's stored weights and, of each block, the cache as the step
left it, quantizes each product's input by the definition and computes the newest token's
logits.  Where an input lies within float32's error of a rounding border, the decoder's code may
be the neighbour: one of K inputs moves by 1/127 of the row's largest, some 3 / 127, and an output
by that times a weight of at most some 0.08: 2e-3, where the largest logit is about 1.  2^-8 of it
holds two such moves (they are rare: a border within 2^-18 of a value); a wrong mask moves logits by
2^-7 of the largest and more (tested below), a wrong position, page, scale or head by their own size."""
import numpy as np
import pytest
import torch

import prompts_ref
from gpu_util import host
from serving_ref import f64
from test_gpu_decode import log_softmax, norm
from verifiable_quantize_rows_gb300.decode import Decoder, Shape

pytestmark = pytest.mark.gpu

SHAPES = [Shape(layers=2, heads=4, kv_heads=4, dim=32, hidden=200, vocab=1000, positions=400),
          Shape(layers=2, heads=6, kv_heads=2, dim=64, hidden=333, vocab=1003, positions=350)]


def linear(x, weight):
    q, s = prompts_ref.codes_of(np.float32(x)[None])
    return ((q.astype(np.float64) @ f64(weight[0])) * np.float64(s)[:, None] * f64(weight[1]))[0]


def newest(model, b, token):
    """The logits of the newest token of sequence b, 64 bits; the cache holds its key and value."""
    s, own, pre = model.shape, int(model.lens[b]), model.shared
    n = own + pre
    seen = np.arange(n) >= (n - model.window if model.window else 0)
    seen[: model.sinks] = True
    x = f64(model.embed[token]) + f64(model.place[n - 1])
    for cache, weights in zip(model.caches, model.blocks):
        page = cache[0].shape[2]
        y = linear(norm(x), weights[0]).reshape(-1, s.dim)
        q, new = y[:s.heads], (y[s.heads:s.heads + s.kv_heads], y[s.heads + s.kv_heads:])
        kv = []
        for side in (0, 1):
            parts = []
            for pages, count in ((host(model.beginning), pre), (host(model.table)[b], own)):
                c, sc = f64(cache[side][pages.tolist()]), f64(cache[2 + side][pages.tolist()])
                parts.append((c * sc[:, :, None, None]).transpose(0, 2, 1, 3).reshape(-1, s.kv_heads, s.dim)[:count])
            all_ = np.concatenate(parts)
            step = f64(cache[2 + side][int(host(model.table)[b, (own - 1) // page])])[:, None]
            # half a step, and what the product's own codes may be off by
            assert (np.abs(all_[-1] - new[side]) <= 0.51 * step + 2.0 ** -5 * np.abs(new[side]).max()).all()
            kv.append(np.repeat(all_, s.heads // s.kv_heads, 1))
        z = np.where(seen, np.einsum("hd,nhd->hn", q, kv[0]) * s.dim ** -0.5, -np.inf)
        p = np.exp(z - z.max(1, keepdims=True))
        a = np.einsum("hn,nhd->hd", p / p.sum(1, keepdims=True), kv[1]).reshape(-1)
        x = x + linear(a, weights[1])
        x = x + linear(np.maximum(linear(norm(x), weights[2]), 0), weights[3])
    return linear(norm(x), model.head) + f64(model.bias)


def close(logits, want):
    assert np.abs(f64(logits) - want).max() <= 2.0 ** -8 * np.abs(want).max()


def run(model, lengths, steps, seed):
    """Prompts, then tokens in a graph; the newest logits of both against the reference."""
    rng = torch.Generator().manual_seed(seed)
    last = []
    for b, n in enumerate(lengths):
        ids = torch.randint(model.shape.vocab, (n,), generator=rng).cuda()
        logits = model.prompt(ids, b)
        assert logits.shape == (n, model.shape.vocab)
        close(logits[-1], newest(model, b, int(ids[-1])))
        last.append(logits[-1].argmax())
    answer = model.generate(torch.stack(last), steps, top=3)
    assert host(model.lens).tolist() == [n + steps for n in lengths]
    for b in range(len(lengths)):
        want = newest(model, b, int(answer.tokens[b, -2]))
        lp = log_softmax(want)
        tokens = answer.top_token[b, -1].tolist()
        assert np.abs(f64(answer.top_logprob[b, -1]) - lp[tokens]).max() <= 2.0 ** -7 * np.abs(want).max()
    model.check()


@pytest.mark.parametrize("shape", SHAPES, ids=["heads", "shared heads"])
@pytest.mark.parametrize("lengths", [(1, 37, 270), (100,), (17, 5, 2, 33, 1)], ids=str)
def test_whole_prompts(shape, lengths):
    run(Decoder(shape, len(lengths), page_tokens=32, codes=8), lengths, 30, len(lengths))


@pytest.mark.parametrize("shape", SHAPES, ids=["heads", "shared heads"])
@pytest.mark.parametrize("window,sinks", [(40, 4), (16, 0), (1, 1)])
def test_windows(shape, window, sinks):
    run(Decoder(shape, 3, page_tokens=16, codes=8, window=window, sinks=sinks), (3, 200, 61), 30, window)


@pytest.mark.parametrize("shape", SHAPES, ids=["heads", "shared heads"])
@pytest.mark.parametrize("n", [1, 33, 150])
def test_a_shared_beginning(shape, n):
    model = Decoder(shape, 3, page_tokens=16, codes=8, prefix=150)
    logits = model.share(torch.randint(shape.vocab, (n,), generator=torch.Generator().manual_seed(n)).cuda())
    assert logits.shape == (n, shape.vocab)
    run(model, (1, 40, 7), 30, n)


def test_many_sequences_and_half_precision():
    """More sequences than int4 products take; 16-bit activations for running, with every step a graph's."""
    for dtype in (torch.float16, torch.bfloat16):
        model = Decoder(SHAPES[1], 40, page_tokens=16, codes=8, dtype=dtype, prefix=64)
        model.share(torch.arange(64, device="cuda"))
        ids = torch.arange(40, device="cuda")
        first = model.step(ids[:, None])
        assert first.dtype == dtype and bool(torch.isfinite(first).all())
        answer = model.generate(first.argmax(1), 10)
        assert answer.tokens.shape == (40, 10)
        model.check()


def test_int4_weights_take_windows_and_shared_beginnings():
    """The same calls with the other weights: 16 tokens at a time."""
    model = Decoder(SHAPES[0], 2, page_tokens=16, window=30, sinks=2)
    ids = torch.arange(100, device="cuda")
    a = model.prompt(ids)
    whole = Decoder(SHAPES[0], 2, page_tokens=16).prompt(ids)
    # within the window nothing is different but for the kernels' sums
    assert float((a[:30] - whole[:30]).abs().max()) <= 2.0 ** -10 * float(whole.abs().max())
    assert float((a[60:] - whole[60:]).abs().max()) > 2.0 ** -7 * float(whole.abs().max())
    model = Decoder(SHAPES[0], 2, page_tokens=16, prefix=48)
    model.share(ids[:48])
    b = model.prompt(ids[48:], 1)
    # the same tokens in the same blocks of 16, so the same codes; the sums in another order
    assert float((b - whole[48:]).abs().max()) <= 2.0 ** -10 * float(whole.abs().max())


def test_refusals():
    s = SHAPES[0]
    for kw, what in ((dict(codes=2), "codes"), (dict(sequences=17), "sequences"), (dict(window=5, prefix=5), "window")):
        with pytest.raises(ValueError, match=what):
            Decoder(s, **kw)
    model = Decoder(s, 2, codes=8, prefix=20)
    for n in (21,):
        with pytest.raises(ValueError, match="at most 20"):
            model.share(torch.zeros(n, dtype=torch.int64, device="cuda"))
    model.share(torch.zeros(20, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="once"):
        model.share(torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="at most 400"):
        model.prompt(torch.zeros(381, dtype=torch.int64, device="cuda"))

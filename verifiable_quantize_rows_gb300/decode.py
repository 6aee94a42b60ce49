"""A small decoder served from codes: the serving calls together, as a program uses them.

GPT-2-shaped (pre-norm blocks, learned positions, a ReLU between the two
linears of the MLP; optionally fewer key/value heads than query heads) with
random weights.  Every weight is stored in int4 codes by wquant_groups or in int8
codes by wquant_cols, the keys and values in a Kv8Cache, and a step is

    products (QKV) -> kv8_append -> attention -> products (output)
    -> products (fc, ReLU) -> products (proj)                  in each block,
    products (head) -> logprobs                                at the end.

Embeddings, norms and residuals are plain PyTorch.  With int4 weights
(wgroups_matvec) prompts go in by up to 16 tokens at a time; with int8 weights
(wcols_matmul) a prompt goes in whole, its attention by kv8_attend_window.  Tokens are
then made for all sequences at once, the step in a CUDA graph.  A window with
sinks bounds what a long stream reads, and share() lets all sequences begin with
one prompt whose keys and values are kept and read once (kv8_attend_shared).
score() gives the log probabilities of given tokens and fit_bias() uses
logprobs_backward to fit a bias on the logits to them.

    python -m verifiable_quantize_rows_gb300.decode [--sequences 4] [--tokens 64] [--codes 8]
"""
from __future__ import annotations

import argparse
import time
from typing import NamedTuple

import torch

import verifiable_quantize_rows_gb300 as bsg
from verifiable_quantize_rows_gb300 import inputs

__all__ = ["Shape", "GPT2_SMALL", "Decoder"]


class Shape(NamedTuple):
    layers: int
    heads: int
    kv_heads: int
    dim: int        # of a head
    hidden: int
    vocab: int
    positions: int
    group: int = 64

    @property
    def width(self) -> int:
        return self.heads * self.dim


GPT2_SMALL = Shape(layers=12, heads=12, kv_heads=12, dim=64, hidden=3072, vocab=50304, positions=1024)


class Answer(NamedTuple):
    tokens: torch.Tensor        # (sequences, n): the likeliest at each place
    top_logprob: torch.Tensor   # (sequences, n, top)
    top_token: torch.Tensor


class Decoder:
    """`sequences` sequences of up to `positions` tokens; at most MATVEC_MAX_M with int4
    weights (codes=4).  window, sinks: kv8_attend_window's (0: every position).  prefix:
    tokens that a beginning shared by all sequences may have."""

    def __init__(self, shape: Shape, sequences: int = 1, page_tokens: int = 64, dtype=torch.float32,
                 seed: int = 0, device="cuda", codes: int = 4, window: int = 0, sinks: int = 0, prefix: int = 0):
        if codes not in (4, 8):
            raise ValueError("codes must be 4 or 8")
        if sequences < 1 or codes == 4 and sequences > bsg.MATVEC_MAX_M:
            raise ValueError(f"sequences must be 1 to {bsg.MATVEC_MAX_M}")
        if window and prefix:
            raise ValueError("a shared beginning is seen by every token: there is no window with it")
        if shape.heads % shape.kv_heads:
            raise ValueError("heads must be a multiple of kv_heads")
        self.shape, self.dtype, self.device = shape, dtype, torch.device(device)
        self.dstatus = torch.zeros(1, dtype=torch.int32, device=device)
        self.workspace = bsg.Workspace(self.device)
        s, E = shape, shape.width
        count = iter(range(seed, 1 << 31))

        self.codes, self.window, self.sinks = codes, window, sinks

        def store(K, N):
            W = inputs.gpt2_weights(K, N, next(count)).to(device)
            if codes == 8:
                return bsg.wquant_cols(W, bits=8, dstatus=self.dstatus)
            return bsg.wquant_groups(W, s.group, dstatus=self.dstatus)

        qkv = (s.heads + 2 * s.kv_heads) * s.dim
        self.blocks = [(store(E, qkv), store(E, E), store(E, s.hidden), store(s.hidden, E)) for _ in range(s.layers)]
        self.head = store(E, s.vocab)
        self.embed = inputs.normal((s.vocab, E), 1.0, next(count)).to(device, dtype)
        self.place = inputs.normal((s.positions, E), 0.1, next(count)).to(device, dtype)
        self.bias = torch.zeros(s.vocab, dtype=dtype, device=device)
        # each sequence's pages; a server would hand them out as sequences grow
        pages = -(-s.positions // page_tokens)
        self.table = torch.randperm(sequences * pages, generator=torch.Generator().manual_seed(seed)) \
            .to(torch.int32).view(sequences, pages).to(device)
        shared = -(-prefix // page_tokens)
        self.beginning = torch.arange(sequences * pages, sequences * pages + shared, dtype=torch.int32, device=device)
        self.begun = torch.zeros(1, dtype=torch.int32, device=device)  # tokens of the shared beginning
        self.shared, self.prefix = 0, prefix
        self.caches = [bsg.Kv8Cache.empty(sequences * pages + shared, s.kv_heads, page_tokens, s.dim, device)
                       for _ in range(s.layers)]
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=device)

    def _linear(self, x, weight, relu=False):
        if self.codes == 8:
            return bsg.wcols_matmul(x, *weight, relu=relu, dstatus=self.dstatus, workspace=self.workspace)
        return bsg.wgroups_matvec(x, *weight, group=self.shape.group, relu=relu, dstatus=self.dstatus,
                                  workspace=self.workspace)

    def _norm(self, x):
        return torch.nn.functional.layer_norm(x, (self.shape.width,))

    def _attend(self, q, cache, table, lens):
        kw = dict(dstatus=self.dstatus, workspace=self.workspace)
        if self.shared and table is not self.beginning:
            return bsg.kv8_attend_shared(q, cache, self.beginning, self.begun, table, lens, **kw)
        table = table.view(-1, table.shape[-1])
        if self.window or q.shape[1] > bsg.KV8_MAX_T:
            return bsg.kv8_attend_window(q, cache, table, lens, self.window, self.sinks, **kw)
        return bsg.kv8_attend(q, cache, table, lens, **kw)

    def _feed(self, ids, table, lens, at):
        """The tokens' logits, their keys and values appended; lens counts them already."""
        s, (B, T) = self.shape, ids.shape
        starts = lens - T
        x = (self.embed[ids] + self.place[at]).view(B * T, s.width)
        for cache, (qkv, out, fc, proj) in zip(self.caches, self.blocks):
            y = self._linear(self._norm(x), qkv).view(B, T, -1, s.dim)
            q, k, v = y.split((s.heads, s.kv_heads, s.kv_heads), 2)
            bsg.kv8_append(k, v, cache, table.view(B, -1), starts, dstatus=self.dstatus)
            a = self._attend(q, cache, table, lens)
            x = x + self._linear(a.view(B * T, s.width), out)
            x = x + self._linear(self._linear(self._norm(x), fc, relu=True), proj)
        return self._linear(self._norm(x), self.head) + self.bias

    def step(self, ids, first: int = 0):
        """Feed ids (sequences, tokens), the next tokens of sequences first,
        first + 1 and so on; returns logits (sequences * tokens, vocab)."""
        s, (B, T) = self.shape, ids.shape
        table, lens = self.table[first:first + B], self.lens[first:first + B]
        at = (self.shared + lens[:, None] + torch.arange(T, device=self.device)).clamp_(max=s.positions - 1)
        lens += T
        return self._feed(ids, table, lens, at)

    def _rows(self, behind: bool) -> int:
        """Tokens of one sequence that a step takes."""
        if self.codes == 4:
            return min(bsg.MATVEC_MAX_M, bsg.KV8_MAX_T)
        return bsg.KV8_MAX_T if behind else self.shape.positions

    def prompt(self, ids, sequence: int = 0):
        """Feed a prompt (tokens,) to one sequence, as many tokens at a time as a step
        takes; returns the logits of each of its tokens (tokens, vocab)."""
        if self.shared + int(self.lens[sequence]) + len(ids) > self.shape.positions:
            raise ValueError(f"at most {self.shape.positions} tokens a sequence")
        return torch.cat([self.step(part.view(1, -1), sequence) for part in ids.split(self._rows(self.shared > 0))])

    def share(self, ids):
        """Begin every sequence with these tokens (tokens,), before anything else is fed;
        returns their logits (tokens, vocab)."""
        if self.shared or int(self.lens.max()):
            raise ValueError("a shared beginning comes once, before anything else")
        if len(ids) > self.prefix or len(ids) >= self.shape.positions:
            raise ValueError(f"at most {min(self.prefix, self.shape.positions - 1)} tokens of a shared beginning")
        logits = []
        for part in ids.split(self._rows(False)):
            at = self.begun[:, None] + torch.arange(len(part), device=self.device)
            self.begun += len(part)
            logits.append(self._feed(part.view(1, -1), self.beginning, self.begun, at))
        self.shared = len(ids)
        return torch.cat(logits)

    def generate(self, last, n: int, top: int = 5) -> Answer:
        """n >= 2 more tokens for every sequence, whose newest tokens (not fed
        yet) are `last` (sequences,): the likeliest each time."""
        if self.shared + int(self.lens.max()) + n > self.shape.positions:
            raise ValueError(f"at most {self.shape.positions} tokens a sequence")
        ids = last.view(-1, 1).clone()
        made = []

        def one():
            r = bsg.logprobs(self.step(ids), top=top, dstatus=self.dstatus)
            ids.copy_(r.top_id[:, :1].clamp(0, self.shape.vocab - 1))  # (a row without numbers names any)
            return r.top_logprob, r.top_id

        made.append([t.clone() for t in one()])  # sizes the workspace, too
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            result = one()
        for _ in range(n - 1):
            graph.replay()
            made.append([t.clone() for t in result])
        self.check()
        lp, tok = (torch.stack(part, 1) for part in zip(*made))
        return Answer(tok[:, :, 0], lp, tok)

    def score(self, logits, ids):
        """The log probabilities of ids[1:], given the logits that prompt(ids)
        returned, and their entropies."""
        r = bsg.logprobs(logits[:-1], ids[1:], dstatus=self.dstatus)
        return r.logprob, r.entropy

    def fit_bias(self, logits, ids, rate: float = 10.0, steps: int = 10):
        """Fit the logits' bias to ids by gradient ascent on their mean log
        probability, the model itself left alone; returns that mean, before each
        step and at the end."""
        plain, target = logits[:-1] - self.bias, ids[1:].contiguous()
        g = torch.full((len(target),), 1.0 / len(target), device=self.device)
        means = []
        for _ in range(steps):
            now = plain + self.bias
            r = bsg.logprobs(now, target, dstatus=self.dstatus)
            means.append(r.logprob.mean())
            d = bsg.logprobs_backward(now, target, r.lse, g_logprob=g, out=now, dstatus=self.dstatus)
            self.bias += rate * d.sum(0)
        means.append(bsg.logprobs(plain + self.bias, target, dstatus=self.dstatus).logprob.mean())
        self.check()
        return torch.stack(means).tolist()

    def check(self):
        """Raise if a kernel met a value or an index that it refuses."""
        if int(self.dstatus):
            raise RuntimeError(f"device status {int(self.dstatus):#x}")


def main(argv=None):
    p = argparse.ArgumentParser(description="A GPT-2-small-shaped decoder with random weights, served from codes.")
    p.add_argument("--sequences", type=int, default=4)
    p.add_argument("--prompt", type=int, default=100, help="tokens of each prompt")
    p.add_argument("--tokens", type=int, default=64, help="tokens to make for each sequence")
    p.add_argument("--codes", type=int, default=4, choices=(4, 8), help="bits of the weights' codes")
    p.add_argument("--window", type=int, default=0, help="positions that a token sees, and four first ones (0: all)")
    p.add_argument("--share", type=int, default=0, help="tokens of a beginning that the sequences share")
    a = p.parse_args(argv)
    s = GPT2_SMALL
    model = Decoder(s, a.sequences, codes=a.codes, window=a.window, sinks=4 if a.window else 0, prefix=a.share)
    if a.share:
        model.share(torch.randint(s.vocab, (a.share,), generator=torch.Generator().manual_seed(2)).cuda())
    prompts = torch.randint(s.vocab, (a.sequences, a.prompt), generator=torch.Generator().manual_seed(1)).cuda()
    for b in range(a.sequences):
        logits = model.prompt(prompts[b], b)
    lp, entropy = model.score(logits, prompts[-1])
    print(f"prompt of {a.prompt} tokens: mean log probability {lp.mean():.3f}, entropy {entropy.mean():.3f}")
    last = logits[-1:].argmax(1).expand(a.sequences)
    model.generate(last, 2)
    torch.cuda.synchronize()
    t = time.perf_counter()
    answer = model.generate(last, a.tokens)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t) * 1e3
    print(f"{a.sequences} x {a.tokens} tokens in {ms:.1f} ms, the graph's capture among them; "
          f"the likeliest had a mean log probability of {answer.top_logprob[:, :, 0].mean():.3f}")
    means = model.fit_bias(logits, prompts[-1])
    print(f"bias fitted to the prompt: mean log probability {means[0]:.3f} -> {means[-1]:.3f}")


if __name__ == "__main__":
    main()

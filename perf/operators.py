"""The serving operators' cases: what is timed, on which inputs, and what the answers are.

A decode step of a model that is stored in codes: products of a few rows with
4-bit weights that carry group scales ("matvec"), new keys and values into an
8-bit cache ("append"), attention over that cache ("attend"), and what is
reported of the logits, log probabilities of given tokens with entropy and the
top alternatives ("logprobs"), with its gradient for training on them
("logprobs_backward").

`run` computes each in its plain form, elementary torch operations in 32 bits;
with `own` set it makes the calls a user makes of verifiable_quantize_rows_gb300.
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# --------------------------------------------------------------------------
# cases
def listed():
    return [
        # One token through GPT-2 small's QKV projection: the smallest call, latency counts.
        dict(name="matvec qkv 1 row", op="matvec", m=1, k=768, n=2304, group=64, dtype="f32", relu=False, tight=False),
        # A verification step of five tokens through an odd-sized layer; nothing divides anything.
        dict(name="matvec ragged 5 rows", op="matvec", m=5, k=8191, n=12289, group=128, dtype="bf16", relu=True, tight=False),
        # A large layer for a batch of eight f32 rows, small groups of weights.
        dict(name="matvec 16384 8 rows", op="matvec", m=8, k=16384, n=16384, group=64, dtype="f32", relu=False, tight=False),
        # One new token for each of 64 sequences, GPT-2 small's heads, f32.
        dict(name="append 64 tokens", op="append", batch=64, tokens=1, kv_heads=12, dim=64, page=16, start_min=1, start_max=1023, dtype="f32"),
        # Prompts of up to 4096 tokens of different lengths into empty pages, bf16.
        dict(name="append prompts", op="append", batch=16, tokens=4096, kv_heads=8, dim=128, page=64, start_min=0, start_max=0, dtype="bf16"),
        # One sequence of GPT-2 small near its full context: one new token, latency counts.
        dict(name="attend gpt2 1 sequence", op="attend", batch=1, tokens=1, heads=12, kv_heads=12, dim=64, page=16, len_min=1001, len_max=1001, dtype="f32"),
        # A serving batch of ragged lengths, an idle slot (length 0) in it, four query heads to a key head.
        dict(name="attend batch ragged", op="attend", batch=64, tokens=1, heads=32, kv_heads=8, dim=128, page=32, len_min=0, len_max=8190, dtype="bf16"),
        # Long contexts with four draft tokens to verify: the longest axis, split over the whole card.
        dict(name="attend long 4 tokens", op="attend", batch=2, tokens=4, heads=32, kv_heads=8, dim=128, page=64, len_min=131071, len_max=262143, dtype="f16"),
        # The LM head's logits of one sampled token, the vocabulary padded to 50304 with -inf.
        dict(name="logprobs 1 row", op="logprobs", rows=1, vocab=50304, pad=47, top=5, dtype="f32"),
        # Scoring 8192 tokens with the twenty best alternatives each.
        dict(name="logprobs 8192 rows", op="logprobs", rows=8192, vocab=50304, pad=47, top=20, dtype="f32"),
        # The gradient of a few rows over an odd vocabulary, bf16.
        dict(name="logprobs backward ragged", op="logprobs_backward", rows=97, vocab=12289, pad=0, dtype="bf16"),
        # The gradient of 8192 scored tokens.
        dict(name="logprobs backward 8192", op="logprobs_backward", rows=8192, vocab=50304, pad=47, dtype="f32"),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    dtype = rng.choice(["f32", "f16", "bf16"])
    op = rng.choice(["matvec", "matvec", "append", "attend", "attend", "logprobs", "logprobs_backward"])
    if op == "matvec":
        k, n = log_int(300, 16384), log_int(300, 16384)
        return dict(op=op, m=rng.randint(1, min(16, 8 * 16384**2 // (k * n))), k=k, n=n, group=rng.choice([32, 64, 128, 0]), dtype=dtype,
                    relu=rng.random() < 0.3, tight=rng.random() < 0.25)
    if op == "append":
        batch, tokens = log_int(1, 128), rng.choice([1, 1, rng.randint(2, 8), log_int(16, 256)])
        return dict(op=op, batch=batch, tokens=tokens, kv_heads=rng.choice([1, 2, 8, 12]), dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                    start_min=rng.randint(0, 40), start_max=rng.randint(41, 700), dtype=dtype)
    if op == "attend":
        kv = rng.choice([1, 2, 5, 8, 12])
        batch, tokens, heads, dim = log_int(1, 128), rng.choice([1, 1, 1, 2, 5, 16]), kv * rng.choice([1, 1, 4, 7, 8]), rng.choice([32, 64, 96, 128, 256])
        # no more to read or to compute than the longest listed case has
        most = log_int(16, max(17, min(65536, 393_000 * min(8 * 128 / (kv * dim), 4 * 32 * 128 / (tokens * heads * dim)) // batch)))
        return dict(op=op, batch=batch, tokens=tokens, heads=heads, kv_heads=kv, dim=dim,
                    page=rng.choice([16, 32, 64, 128]), len_min=rng.randint(0, most), len_max=most, dtype=dtype)
    vocab = log_int(2000, 60000)
    case = dict(op=op, rows=log_int(1, min(6000, 200_000_000 // vocab)), vocab=vocab, pad=rng.choice([0, 0, 47, 200]), dtype=dtype)
    return dict(case, top=rng.choice([0, 1, 5, 20, 32])) if op == "logprobs" else case


def lengths(lo, hi, n):
    """n whole numbers spread evenly over lo..hi (hi alone where n is 1)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "matvec":
        m, k, n = case["m"], case["k"], case["n"]
        groups = -(-k // case["group"]) if case["group"] else 1
        return {"bytes": k * ((n + 1) // 2) + 4 * groups * n + e * m * (k + n), "flops": 2 * m * k * n}
    if case["op"] == "append":
        new = sum(append_counts(case))
        return {"bytes": 2 * new * case["kv_heads"] * case["dim"] * (e + 1) + 8 * case["kv_heads"] * -(-new // case["page"]), "flops": 4 * new * case["kv_heads"] * case["dim"]}
    if case["op"] == "attend":
        lens = lengths(case["len_min"], case["len_max"], case["batch"])
        blocks = sum(-(-x // case["page"]) for x in lens)
        rows = case["batch"] * case["tokens"] * case["heads"]
        return {"bytes": 2 * sum(lens) * case["kv_heads"] * case["dim"] + 8 * blocks * case["kv_heads"] + 2 * e * rows * case["dim"],
                "flops": 4 * sum(lens) * case["tokens"] * case["heads"] * case["dim"]}
    size = case["rows"] * case["vocab"]
    if case["op"] == "logprobs":
        return {"bytes": e * size + case["rows"] * (20 + 8 * case["top"]), "flops": 6 * size}
    return {"bytes": 2 * e * size + case["rows"] * 24, "flops": 6 * size}


def append_counts(case):
    """New tokens of each sequence: `tokens` for all where there are few, ragged prompts from a quarter up to `tokens` otherwise."""
    t = case["tokens"]
    return [t] * case["batch"] if t < 16 else lengths(t // 4, t, case["batch"])


# --------------------------------------------------------------------------
# inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return dict(case=case, **{"matvec": matvec_inputs, "append": append_inputs, "attend": attend_inputs, "logprobs": logit_inputs,
                              "logprobs_backward": logit_inputs}[case["op"]](case, gen))


def normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def matvec_inputs(case, gen):
    m, k, n, group = case["m"], case["k"], case["n"], case["group"] or case["k"]
    # activations with 0.1 % outliers, weights N(0, 0.02): the linears' inputs
    x = normal(gen, m, k)
    x = torch.where(torch.rand((m, k), generator=gen, device="cuda") < 1e-3, 20 * x, x)
    # the stored weight: codes -7..7 with one scale for each group and column, two columns to a byte
    groups = -(-k // group)
    w = normal(gen, k, n).mul_(0.02)
    padded = torch.zeros((groups * group, n), device="cuda")
    padded[:k] = w
    scale = padded.view(groups, group, n).abs().amax(1) / 7
    q = torch.round(padded.view(groups, group, n) / scale[:, None].clamp_min(1e-30)).view(-1, n)[:k].to(torch.int16)
    half = (n + 1) // 2
    low, high = q[:, 0::2] & 15, torch.zeros((k, half), dtype=torch.int16, device="cuda")
    high[:, : n // 2] = q[:, 1::2] & 15
    stride = half if case["tight"] else -(-half // 16) * 16  # rows as bsg.wquant_cols has them, or as bsg.wquant_groups has them
    codes = torch.zeros((k, stride), dtype=torch.uint8, device="cuda")
    codes[:, :half] = (low | high << 4).to(torch.uint8)
    return dict(x=x.to(DTYPE[case["dtype"]]), codes=codes[:, :half], scale=scale.contiguous())


def page_table(case, gen, most):
    """(table, pages): the sequences' pages in an order of their own; a few spare pages in the pool."""
    per = max(1, -(-most // case["page"]))
    pages = case["batch"] * per + 3
    order = torch.randperm(pages, generator=gen, device="cuda")[: case["batch"] * per]
    return order.view(case["batch"], per).to(torch.int32), pages


def cache_inputs(case, gen, pages):
    """A pool whose pages hold N(0, 1) values in codes, each block with a scale of its own."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])

    def codes():
        c = torch.empty(shape, dtype=torch.int8, device="cuda")
        for i in range(0, pages, 4096):
            c[i : i + 4096] = normal(gen, *c[i : i + 4096].shape).mul_(35).round_().clamp_(-127, 127).to(torch.int8)
        return c

    def scales():
        return (0.6 + torch.rand(shape[:2], generator=gen, device="cuda")) / 35

    return codes(), codes(), scales(), scales()


def append_inputs(case, gen):
    starts = lengths(case["start_min"], case["start_max"], case["batch"])
    counts = append_counts(case)
    table, pages = page_table(case, gen, max(s + c for s, c in zip(starts, counts)))
    shape = (case["batch"], case["tokens"], case["kv_heads"], case["dim"])
    return dict(k=normal(gen, *shape).to(DTYPE[case["dtype"]]), v=normal(gen, *shape).to(DTYPE[case["dtype"]]), cache=cache_inputs(case, gen, pages), table=table,
                starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), counts=torch.tensor(counts, dtype=torch.int32, device="cuda"))


def attend_inputs(case, gen):
    lens = torch.tensor(lengths(case["len_min"], case["len_max"], case["batch"]), dtype=torch.int32, device="cuda")
    lens = lens[torch.randperm(case["batch"], generator=gen, device="cuda")]
    table, pages = page_table(case, gen, case["len_max"])
    q = normal(gen, case["batch"], case["tokens"], case["heads"], case["dim"]).to(DTYPE[case["dtype"]])
    return dict(q=q, cache=cache_inputs(case, gen, pages), table=table, lens=lens, scale=case["dim"] ** -0.5)


def logit_inputs(case, gen):
    m, v = case["rows"], case["vocab"]
    logits = normal(gen, m, v)
    # rows from nearly flat to sharply peaked
    logits *= torch.exp(1.5 * torch.rand((m, 1), generator=gen, device="cuda"))
    if case["pad"]:
        logits[:, v - case["pad"] :] = -math.inf  # the vocabulary's padding
    target = torch.randint(0, v - case["pad"], (m,), generator=gen, device="cuda")
    # one row in sixteen is padding of its sequence: no token is given
    target[torch.rand((m,), generator=gen, device="cuda") < 1 / 16] = -1
    state = dict(logits=logits.to(DTYPE[case["dtype"]]), target=target)
    if case["op"] == "logprobs_backward":
        x = state["logits"].double()
        lp = torch.log_softmax(x, 1)
        state["lse"] = torch.logsumexp(x, 1).float()
        state["entropy"] = -(lp.exp() * lp.clamp_min(-1e30)).sum(1).float()
        state["g_logprob"], state["g_entropy"] = normal(gen, m) / m, normal(gen, m) * (0.01 / m)
    return state


# --------------------------------------------------------------------------
# one pass
def run(s):
    return (run_own if own else run_plain)(s)


def run_own(s):
    import verifiable_quantize_rows_gb300 as bsg

    case = s["case"]
    if case["op"] == "matvec":
        return bsg.wgroups_matvec(s["x"], s["codes"], s["scale"], group=case["group"], relu=case["relu"])
    if case["op"] == "append":
        bsg.kv8_append(s["k"], s["v"], s["cache"], s["table"], s["starts"], s["counts"])
        return s["cache"]
    if case["op"] == "attend":
        return bsg.kv8_attend(s["q"], s["cache"], s["table"], s["lens"], scale=s["scale"])
    if case["op"] == "logprobs":
        return bsg.logprobs(s["logits"], s["target"], top=case["top"])
    return bsg.logprobs_backward(s["logits"], s["target"], s["lse"], s["entropy"], s["g_logprob"], s["g_entropy"])


def run_plain(s):
    return {"matvec": plain_matvec, "append": plain_append, "attend": plain_attend, "logprobs": plain_logprobs, "logprobs_backward": plain_backward}[s["case"]["op"]](s)


def unpack(codes, n):
    """4-bit two's complement codes, two columns to a byte, as float32 (K, n)."""
    both = torch.stack((codes & 15, codes >> 4), 2).reshape(codes.shape[0], -1)[:, :n]
    return both.float() - 16 * (both >= 8)


def plain_matvec(s):
    case, scale = s["case"], s["scale"]
    group = case["group"] or case["k"]
    w = unpack(s["codes"], case["n"]) * scale.repeat_interleave(group, 0)[: case["k"]]
    y = s["x"].float() @ w
    if case["relu"]:
        y = y.clamp_min(0)
    return y.to(s["x"].dtype)


def quantize(x, scale):
    """The unit's rounding: floor(x / scale + 1/2) with the reciprocal and each step rounded to float32."""
    return torch.floor(x * (1 / scale) + 0.5)


def plain_append(s):
    """Every block of every sequence as one tensor: old codes rescaled where its scale grows, new tokens in their places, and back."""
    case, table = s["case"], s["table"].long()
    p, (b, blocks) = case["page"], table.shape
    start, count = s["starts"].long()[:, None, None], s["counts"].long()[:, None, None]
    at = torch.arange(blocks * p, device="cuda").view(1, blocks, p)  # positions of each block
    new = (at >= start) & (at < start + count)  # b, blocks, p
    touched = new.any(2)
    source = (at - start).clamp(0, case["tokens"] - 1).expand(b, -1, -1)
    every = torch.arange(b, device="cuda")[:, None, None]
    for x, codes, scales in ((s["k"], s["cache"][0], s["cache"][2]), (s["v"], s["cache"][1], s["cache"][3])):
        fresh = x[every, source].float().transpose(2, 3)  # b, blocks, heads, p, dim
        mine = new[:, :, None, :, None]
        most = torch.where(mine, fresh.abs(), torch.zeros_like(fresh)).amax((3, 4))
        begun = (at[:, :, 0] < start[:, :, 0])[:, :, None]  # the block holds older tokens
        old = scales[table]
        scale = torch.maximum(torch.where(begun, old, torch.zeros_like(old)), (most / 127).clamp_min(1e-8))
        kept = codes[table]
        ratio = torch.where(begun, old / scale, torch.ones_like(scale))
        moved = torch.where((ratio < 1)[..., None, None] & (at < start)[:, :, None, :, None], torch.floor(kept.float() * ratio[..., None, None] + 0.5), kept.float())
        value = torch.where(mine, quantize(fresh, scale[..., None, None]), moved).to(torch.int8)
        codes[table[touched]] = value[touched]
        scales[table[touched]] = scale[touched]
    return s["cache"]


def plain_attend(s):
    case, table, lens = s["case"], s["table"].long(), s["lens"].long()
    b, t, h, d = s["q"].shape
    hk, p = case["kv_heads"], case["page"]

    def cached(codes, scales):  # b, kv heads, length, dim
        x = codes[table].float() * scales[table][..., None, None]
        return x.transpose(1, 2).reshape(b, hk, -1, d)

    q = s["q"].float().view(b, t, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    scores = q @ cached(s["cache"][0], s["cache"][2]).transpose(2, 3) * s["scale"]
    last = lens[:, None] - t + torch.arange(t, device="cuda")  # the last position that each query sees
    seen = torch.arange(scores.shape[3], device="cuda") <= last[:, :, None]  # b, t, length
    seen = seen[:, None, None].expand(b, 1, h // hk, t, -1).reshape(b, 1, -1, scores.shape[3])
    scores = scores.masked_fill(~seen, -math.inf)
    e = torch.exp(scores - scores.amax(3, keepdim=True).clamp_min(-1e30))
    o = e @ cached(s["cache"][1], s["cache"][3]) / e.sum(3, keepdim=True).clamp_min(1e-30)
    return o.view(b, hk, h // hk, t, d).permute(0, 3, 1, 2, 4).reshape(b, t, h, d).to(s["q"].dtype)


def given(target, vocab):
    return target.clamp(0, vocab - 1)[:, None], target >= 0


def plain_logprobs(s):
    case, x = s["case"], s["logits"].float()
    index, has = given(s["target"], case["vocab"])
    top = x.amax(1, keepdim=True)
    d = x - top
    e = torch.exp(d)
    total = e.sum(1)
    log_total = total.log()
    lse = top[:, 0] + log_total
    entropy = log_total - (e * d.clamp_min(-1e30)).sum(1) / total
    logprob = torch.where(has, d.gather(1, index)[:, 0] - log_total, torch.zeros_like(lse))
    # by value, the lowest index first among equals: both in one whole number
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -2147483648 - bits, bits) * 65536 + (65535 - torch.arange(case["vocab"], device="cuda"))
    at = 65535 - key.topk(case["top"], 1).values % 65536
    return logprob, entropy, lse, d.gather(1, at) - log_total[:, None], at.to(torch.int32)


def plain_backward(s):
    case, x = s["case"], s["logits"].float()
    index, has = given(s["target"], case["vocab"])
    lp = x - s["lse"][:, None]
    p = torch.exp(lp)
    g = torch.where(has, s["g_logprob"], torch.zeros_like(s["lse"]))
    dx = -p * (g[:, None] + s["g_entropy"][:, None] * (lp.clamp_min(-1e30) + s["entropy"][:, None]))
    return dx.scatter_add_(1, index, g[:, None]).to(s["logits"].dtype)


# --------------------------------------------------------------------------
# the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matvec":
        x, k, n = s["x"].double(), case["k"], case["n"]
        group = case["group"] or k
        y = torch.zeros((case["m"], n), dtype=torch.float64, device="cuda")
        for g in range(0, k, group):
            byte = s["codes"][g : g + group].long()
            nibble = torch.empty((byte.shape[0], 2 * byte.shape[1]), dtype=torch.long, device="cuda")
            nibble[:, 0::2], nibble[:, 1::2] = byte % 16, byte // 16
            code = ((nibble + 8) % 16 - 8)[:, :n].double()
            y += (x[:, g : g + group] @ code) * s["scale"][g // group].double()
        return torch.relu(y) if case["relu"] else y
    if case["op"] == "append":
        new = [None, None]
        for x, scales in ((s["k"], s["cache"][2]), (s["v"], s["cache"][3])):
            scales = scales.double().cpu()
            table, starts, counts = s["table"].tolist(), s["starts"].tolist(), s["counts"].tolist()
            most = x.double().abs().amax(3).cpu()  # batch, tokens, heads
            for b in range(case["batch"]):
                at, end = starts[b], starts[b] + counts[b]
                while at < end:
                    to = min(end, (at // case["page"] + 1) * case["page"])
                    page = table[b][at // case["page"]]
                    m = (most[b, at - starts[b] : to - starts[b]].amax(0) / 127).clamp_min(1e-8)
                    scales[page] = m if at % case["page"] == 0 else torch.maximum(scales[page], m)
                    at = to
            new.append(scales)
        return new
    if case["op"] == "attend":
        b, t, h, d = s["q"].shape
        out = torch.zeros((b, t, h, d), dtype=torch.float64, device="cuda")
        share = h // case["kv_heads"]
        for i, n in enumerate(s["lens"].tolist()):
            pages = s["table"][i, : -(-n // case["page"])].long()
            for j in range(case["kv_heads"]):
                k = (s["cache"][0][pages, j].double() * s["cache"][2][pages, j].double()[:, None, None]).reshape(-1, d)[:n]
                v = (s["cache"][1][pages, j].double() * s["cache"][3][pages, j].double()[:, None, None]).reshape(-1, d)[:n]
                for u in range(max(0, t - n), t):
                    see = n - t + u + 1
                    w = torch.softmax(s["scale"] * (s["q"][i, u, j * share : (j + 1) * share].double() @ k[:see].T), 1)
                    out[i, u, j * share : (j + 1) * share] = w @ v[:see]
        return out
    x = s["logits"].double()
    lp = torch.log_softmax(x, 1)
    p = lp.exp()
    has = s["target"] >= 0
    index = s["target"].clamp_min(0)[:, None]
    if case["op"] == "logprobs":
        entropy = torch.special.entr(p).sum(1)
        best = lp.topk(case["top"], 1).values
        return torch.where(has, lp.gather(1, index)[:, 0], 0.0), entropy, torch.logsumexp(x, 1), best, None
    g, h = torch.where(has, s["g_logprob"].double(), 0.0), torch.special.entr(p).sum(1)
    dx = -g[:, None] * p + s["g_entropy"].double()[:, None] * (torch.special.entr(p) - p * h[:, None])
    return dx.scatter_add_(1, index, g[:, None])

"""More serving operators: their cases, inputs, plain forms and answers.

What a model stored in codes needs for prompts, for long streams and for
batches that begin alike: products of any number of rows with 8-bit weights,
each token quantised by itself ("matmul"), attention over the 8-bit cache
through a sliding window with a few first tokens that stay visible, for whole
prompts and for single tokens ("window"), and attention of a batch whose
sequences share a prefix ("shared").

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
        dict(name="matmul qkv 1 token", op="matmul", m=1, k=768, n=2304, dtype="f32", relu=False),
        # The tokens of a serving batch through an odd-sized layer; nothing divides anything.
        dict(name="matmul ragged 61 tokens", op="matmul", m=61, k=8191, n=12289, dtype="bf16", relu=True),
        # A batch of 8192 tokens through GPT-2 small's QKV projection.
        dict(name="matmul qkv 8192 tokens", op="matmul", m=8192, k=768, n=2304, dtype="bf16", relu=False),
        # Prompts through a large layer.
        dict(name="matmul 4096 tokens 8192x8192", op="matmul", m=4096, k=8192, n=8192, dtype="f16", relu=False),
        # One stream of GPT-2 small's heads: one new token, latency counts.
        dict(name="window gpt2 1 token", op="window", batch=1, tokens=1, least=1, past_min=1000, past_max=1000, window=256, sinks=4, heads=12, kv_heads=12,
             dim=64, page=16, dtype="f32"),
        # One new token for each of 64 long streams, an idle slot among them.
        dict(name="window 64 streams", op="window", batch=64, tokens=1, least=1, past_min=-1, past_max=65535, window=4096, sinks=4, heads=32, kv_heads=8,
             dim=128, page=32, dtype="bf16"),
        # Short prompts of different lengths behind what is cached, odd sizes, f32.
        dict(name="window ragged prompts", op="window", batch=7, tokens=1021, least=1, past_min=0, past_max=777, window=301, sinks=5, heads=15, kv_heads=5,
             dim=64, page=16, dtype="f32"),
        # Two long prompts into empty caches: the most to compute.
        dict(name="window prompts of 16384", op="window", batch=2, tokens=16384, least=12001, past_min=0, past_max=0, window=4096, sinks=4, heads=32, kv_heads=8,
             dim=128, page=64, dtype="bf16"),
        # Four sequences behind a common prompt of GPT-2 small's size: latency counts.
        dict(name="shared gpt2 4 sequences", op="shared", batch=4, tokens=1, prefix=700, len_min=1, len_max=99, heads=12, kv_heads=12, dim=64, page=16, dtype="f32"),
        # A serving batch behind a long document, an idle slot among its sequences.
        dict(name="shared 64 sequences", op="shared", batch=64, tokens=1, prefix=32768, len_min=0, len_max=511, heads=32, kv_heads=8, dim=128, page=32, dtype="bf16"),
        # Draft tokens of 16 sequences behind a prefix that ends inside a page: the longest axis.
        dict(name="shared long 4 tokens", op="shared", batch=16, tokens=4, prefix=131071, len_min=4, len_max=2047, heads=32, kv_heads=8, dim=128, page=64, dtype="f16"),
    ]


def draw(rng):
    """Sizes over the whole range, drawn again where a case would read, compute or hold more than the largest listed ones."""
    while True:
        case = draw_any(rng)
        most, full = (250_000_000, 550e9) if case["op"] == "matmul" else (520_000_000, 1630e9 if case["op"] == "window" else 138e9), dict(case)
        if case["op"] == "window":
            full.update(least=case["tokens"], past_min=case["past_max"])
        w = work(full)
        if w["bytes"] <= most[0] and w["flops"] <= most[1] and held(case) <= 5_000_000_000:
            return case


def draw_any(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    dtype = rng.choice(["f32", "f16", "bf16"])
    op = rng.choice(["matmul", "window", "window", "shared"])
    if op == "matmul":
        return dict(op=op, m=log_int(1, 16384), k=log_int(300, 16384), n=log_int(300, 16384), dtype=dtype, relu=rng.random() < 0.3)
    kv = rng.choice([1, 2, 5, 8, 12])
    case = dict(op=op, heads=kv * rng.choice([1, 1, 4, 7, 8]), kv_heads=kv, dim=rng.choice([32, 64, 96, 128, 256]), page=rng.choice([16, 32, 64, 128]), dtype=dtype)
    if op == "shared":
        tokens = rng.choice([1, 1, 1, 2, 5, 16])
        return dict(case, batch=log_int(1, 128), tokens=tokens, prefix=log_int(1, 131072), len_min=rng.randint(0, tokens), len_max=tokens + log_int(1, 1000))
    tokens, past = rng.choice([1, 1, 5, 16, log_int(17, 8192), log_int(17, 8192)]), rng.choice([0, log_int(1, 65536), log_int(1, 65536)])
    return dict(case, batch=log_int(1, 64), tokens=tokens, least=rng.choice([tokens, rng.randint(0, tokens)]), past_min=rng.choice([-1, 0, past]), past_max=past,
                window=rng.choice([0, log_int(1, 8192), log_int(16, 8192)]), sinks=rng.choice([0, 1, 4, 4, 130]))


def held(case):
    """Bytes of the cache and of the queries that a case has in hand."""
    if case["op"] == "matmul":
        return 0
    a_sequence = max(streams(case)[1]) if case["op"] == "window" else case["len_max"]
    return 2 * case["batch"] * a_sequence * case["kv_heads"] * case["dim"] + 4 * case["batch"] * case["tokens"] * case["heads"] * case["dim"]


def lengths(lo, hi, n):
    """n whole numbers spread evenly over lo..hi (hi alone where n is 1)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def streams(case):
    """(new tokens, cached tokens with them) of each sequence. One whose past is -1 is an idle slot: nothing is cached."""
    counts = lengths(case["least"], case["tokens"], case["batch"])
    past = lengths(case["past_min"], case["past_max"], case["batch"])[::-1]
    return counts, [0 if p < 0 else p + c for p, c in zip(past, counts)]


def seen(case, count, length):
    """(positions of a sequence that some query sees, pairs of a query and a position that it sees)."""
    window, sinks = case["window"] or length, case["sinks"]
    first = max(0, length - count)
    low = max(0, first - window + 1)
    some = length - low + min(sinks, low)

    def up_to(n):  # the sum of min(i + 1, window) over the positions i below n
        return n * (n + 1) // 2 - max(0, n - window) * (max(0, n - window) + 1) // 2

    pairs = up_to(length) - up_to(first)
    outside = [max(0, min(sinks, i - window + 1)) for i in range(first, length)] if sinks else []
    return (some, pairs + sum(outside)) if length > first else (0, 0)


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "matmul":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": k * n + 4 * n + e * m * (k + n), "flops": 2 * m * k * n}
    width, share = case["kv_heads"] * case["dim"], case["heads"] // case["kv_heads"]
    if case["op"] == "window":
        counts, lens = streams(case)
        each = [seen(case, c, n) for c, n in zip(counts, lens)]
        return {"bytes": sum(2 * s * width + 8 * -(-s // case["page"]) * case["kv_heads"] for s, _ in each) + 2 * e * sum(counts) * width * share,
                "flops": 4 * sum(p for _, p in each) * width * share}
    lens = lengths(case["len_min"], case["len_max"], case["batch"])
    rows = case["batch"] * case["tokens"]
    blocks = sum(-(-n // case["page"]) for n in [case["prefix"], *lens])
    return {"bytes": 2 * (case["prefix"] + sum(lens)) * width + 8 * blocks * case["kv_heads"] + 2 * e * rows * width * share,
            "flops": 4 * (rows * case["prefix"] + case["tokens"] * sum(lens)) * width * share}


# --------------------------------------------------------------------------
# inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return dict(case=case, **{"matmul": matmul_inputs, "window": window_inputs, "shared": shared_inputs}[case["op"]](case, gen))


def normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def matmul_inputs(case, gen):
    m, k, n = case["m"], case["k"], case["n"]
    # activations with 0.1 % outliers, weights N(0, 0.02): the linears' inputs
    x = normal(gen, m, k)
    x = torch.where(torch.rand((m, k), generator=gen, device="cuda") < 1e-3, 20 * x, x)
    # the stored weight, as bsg.wquant_cols has it: codes -127..127, one scale for each column
    w = normal(gen, k, n).mul_(0.02)
    scale = w.abs().amax(0) / 127
    return dict(x=x.to(DTYPE[case["dtype"]]), codes=torch.round(w / scale).to(torch.int8), scale=scale)


def pool(case, gen, pages):
    """A cache whose pages hold N(0, 1) values in codes, each block with a scale of its own."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])

    def codes():
        c = torch.empty(shape, dtype=torch.int8, device="cuda")
        for i in range(0, pages, 4096):
            c[i : i + 4096] = normal(gen, *c[i : i + 4096].shape).mul_(35).round_().clamp_(-127, 127).to(torch.int8)
        return c

    def scales():
        return (0.6 + torch.rand(shape[:2], generator=gen, device="cuda")) / 35

    return codes(), codes(), scales(), scales()


def deal(case, gen, lens, more=0):
    """(the sequences' tables, `more` pages besides, pages of the pool): in an order of their own, a few spare."""
    per = max(1, -(-max(lens) // case["page"]))
    pages = case["batch"] * per + more + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    return order[: case["batch"] * per].view(case["batch"], per), order[pages - more :], pages


def window_inputs(case, gen):
    counts, lens = streams(case)
    table, _, pages = deal(case, gen, lens)
    q = normal(gen, case["batch"], case["tokens"], case["heads"], case["dim"]).to(DTYPE[case["dtype"]])
    ragged = None if case["least"] == case["tokens"] else torch.tensor(counts, dtype=torch.int32, device="cuda")
    # the step's output buffer: what lies behind a sequence's new tokens stays as it is
    return dict(q=q, cache=pool(case, gen, pages), table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), counts=ragged,
                scale=case["dim"] ** -0.5, out=torch.zeros_like(q))


def shared_inputs(case, gen):
    lens = lengths(case["len_min"], case["len_max"], case["batch"])
    table, prefix, pages = deal(case, gen, lens, -(-case["prefix"] // case["page"]))
    q = normal(gen, case["batch"], case["tokens"], case["heads"], case["dim"]).to(DTYPE[case["dtype"]])
    return dict(q=q, cache=pool(case, gen, pages), prefix=prefix, prefix_len=torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda"), table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=case["dim"] ** -0.5)


# --------------------------------------------------------------------------
# one pass
def run(s):
    return (run_own if own else run_plain)(s)


def run_own(s):
    import verifiable_quantize_rows_gb300 as bsg

    case = s["case"]
    if case["op"] == "matmul":
        return bsg.wcols_matmul(s["x"], s["codes"], s["scale"], relu=case["relu"])
    if case["op"] == "window":
        return bsg.kv8_attend_window(s["q"], s["cache"], s["table"], s["lens"], window=case["window"], sinks=case["sinks"], counts=s["counts"],
                                     scale=s["scale"], out=s["out"])
    return bsg.kv8_attend_shared(s["q"], s["cache"], s["prefix"], s["prefix_len"], s["table"], s["lens"], scale=s["scale"])


def run_plain(s):
    return {"matmul": plain_matmul, "window": plain_window, "shared": plain_shared}[s["case"]["op"]](s)


def plain_matmul(s):
    x = s["x"].float()
    # the unit's step 1, each step rounded to float32 but for the two quotients
    scale = (x.abs().amax(1).double() / 127).clamp_min(1e-8).float()
    inverse = (1 / scale.double()).float()
    q = torch.floor(x * inverse[:, None] + 0.5)
    total = torch.zeros((x.shape[0], s["codes"].shape[1]), dtype=torch.float64, device="cuda")
    for k in range(0, x.shape[1], 1024):  # sums of 1024 products of codes are exact in float32
        total += q[:, k : k + 1024] @ s["codes"][k : k + 1024].float()
    y = total.float() * scale[:, None] * s["scale"]
    if s["case"]["relu"]:
        y = y.clamp_min(0)
    return y.to(s["x"].dtype)


def values(codes, scales, table):
    """The cached tokens of each row of pages: (rows, kv heads, tokens, dim) in float32."""
    x = codes[table].float() * scales[table][..., None, None]
    return x.transpose(1, 2).reshape(table.shape[0], codes.shape[1], -1, codes.shape[3])


def by_group(q, kv_heads):
    """(batch, tokens, heads, dim) as (batch, kv heads, heads of the group x tokens, dim) in float32."""
    b, t, h, d = q.shape
    return q.float().view(b, t, kv_heads, h // kv_heads, d).permute(0, 2, 3, 1, 4).reshape(b, kv_heads, -1, d)


def by_head(o, t):
    b, hk, rows, d = o.shape
    return o.view(b, hk, rows // t, t, d).permute(0, 3, 1, 2, 4).reshape(b, t, -1, d)


def softmax_sum(scores, v):
    """softmax(scores) @ v, and zeros for rows of nothing but -inf."""
    e = torch.exp(scores - scores.amax(-1, keepdim=True).clamp_min(-1e30))
    return e @ v / e.sum(-1, keepdim=True).clamp_min(1e-30)


def plain_window(s):
    """Some query tokens of all sequences at a time, over the positions that one of them may see."""
    case, q, out = s["case"], s["q"], s["out"]
    b, t, h, d = q.shape
    k_codes, v_codes, k_scale, v_scale = s["cache"]
    hk, page, sinks, most = case["kv_heads"], case["page"], case["sinks"], s["table"].shape[1] * case["page"]
    window, lens = case["window"] or most, s["lens"].long()
    counts = torch.full_like(lens, t) if s["counts"] is None else s["counts"].long()
    table = s["table"].long()
    head = torch.arange(hk, device="cuda")[None, :, None]
    step = max(1, min(t, 1024, 400_000_000 // (b * h * most)))
    for t0 in range(0, t, step):
        n = min(step, t - t0)
        at = (lens - counts)[:, None] + torch.arange(t0, t0 + n, device="cuda")  # the queries' positions
        low = (at[:, 0] - window + 1).clamp_min(0)
        near = low[:, None] + torch.arange(min(most, window + n - 1), device="cuda")
        first = torch.arange(min(sinks, most), device="cuda").expand(b, -1)
        j = torch.cat((first.where(first < low[:, None], most), near), 1)  # positions; `most` and beyond: none
        place = j.clamp_max(most - 1)
        pages, within = table.gather(1, place // page)[:, None], (place % page)[:, None]
        k = k_codes[pages, head, within].float() * k_scale[pages, head][..., None]  # b, kv heads, positions, dim
        v = v_codes[pages, head, within].float() * v_scale[pages, head][..., None]
        scores = by_group(q[:, t0 : t0 + n], hk) @ k.transpose(2, 3) * s["scale"]
        i, j = at[:, :, None], j[:, None]
        see = (j <= i) & ((j > i - window) | (j < sinks)) & (j < most)  # b, tokens, positions
        scores = scores.view(b, hk, h // hk, n, -1).masked_fill_(~see[:, None, None], -math.inf).view(b, hk, h // hk * n, -1)
        o = by_head(softmax_sum(scores, v), n).to(q.dtype)
        new = torch.arange(t0, t0 + n, device="cuda") < counts[:, None]
        out[:, t0 : t0 + n] = torch.where(new[:, :, None, None], o, out[:, t0 : t0 + n])
    return out


def plain_shared(s):
    """The prefix's scores beside each sequence's own, one softmax over both."""
    case, lens = s["case"], s["lens"].long()
    k_codes, v_codes, k_scale, v_scale = s["cache"]
    b, t, h, d = s["q"].shape
    hk, n = case["kv_heads"], case["prefix"]
    table, prefix = s["table"].long(), s["prefix"].long()[None]
    k0, v0 = values(k_codes, k_scale, prefix)[0, :, :n], values(v_codes, v_scale, prefix)[0, :, :n]
    q = by_group(s["q"], hk)
    rows = q.transpose(0, 1).reshape(hk, -1, d)  # all sequences' queries
    before = (rows @ k0.transpose(1, 2) * s["scale"]).view(hk, b, -1, n).transpose(0, 1)
    after = q @ values(k_codes, k_scale, table).transpose(2, 3) * s["scale"]
    at = lens[:, None] - t + torch.arange(t, device="cuda")  # the queries' own positions; below 0: padding, which sees nothing
    see = (torch.arange(after.shape[3], device="cuda") <= at[:, :, None])[:, None, None].expand(b, 1, h // hk, t, -1).reshape(b, 1, -1, after.shape[3])
    after = after.masked_fill(~see, -math.inf)
    there = (at >= 0)[:, None].expand(b, h // hk, t).reshape(b, 1, -1, 1)
    top = torch.maximum(before.amax(3), after.amax(3))[..., None]
    e0, e1 = torch.exp(before - top), torch.exp(after - top)
    total = e0.sum(3, keepdim=True) + e1.sum(3, keepdim=True)
    o = (e0.transpose(0, 1).reshape(hk, -1, n) @ v0).view(hk, b, -1, d).transpose(0, 1) + e1 @ values(v_codes, v_scale, table)
    return by_head(torch.where(there, o / total, torch.zeros_like(o)), t).to(s["q"].dtype)


# --------------------------------------------------------------------------
# the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matmul":
        x = s["x"].double()
        a = torch.clamp(x.abs().max(1).values / 127, min=1e-8).float()
        r = a.double().reciprocal().float()
        q = ((s["x"].float() * r.unsqueeze(1)) + 0.5).floor().double()  # codes, by their definition in float32 steps
        y = (q @ s["codes"].double()) * a.double().unsqueeze(1) * s["scale"].double()
        return torch.relu(y) if case["relu"] else y
    b, t, h, d = s["q"].shape
    share = h // case["kv_heads"]
    out = torch.zeros((b, t, h, d), dtype=torch.float64, device="cuda")

    def cached(pages, n, j):
        k = (s["cache"][0][pages, j].double() * s["cache"][2][pages, j].double()[:, None, None]).reshape(-1, d)[:n]
        v = (s["cache"][1][pages, j].double() * s["cache"][3][pages, j].double()[:, None, None]).reshape(-1, d)[:n]
        return k, v

    if case["op"] == "window":
        for i, (count, n) in enumerate(zip(*streams(case))):
            pages = s["table"][i, : -(-n // case["page"])].long()
            for j in range(case["kv_heads"] if n else 0):
                k, v = cached(pages, n, j)
                for u in range(0, count, 256):
                    to = min(count, u + 256)
                    at = torch.arange(n - count + u, n - count + to, device="cuda")
                    if n - count + to <= 0:
                        continue
                    low = max(0, n - count + u + 1 - case["window"]) if case["window"] else 0
                    pick = torch.cat((torch.arange(min(case["sinks"], low), device="cuda"), torch.arange(low, n - count + to, device="cuda")))
                    hidden = pick > at[:, None]
                    if case["window"]:
                        hidden |= (pick <= at[:, None] - case["window"]) & (pick >= case["sinks"])
                    z = torch.einsum("tgd,nd->gtn", s["q"][i, u:to, j * share : (j + 1) * share].double(), k[pick]) * s["scale"]
                    w = torch.nan_to_num(torch.softmax(z.masked_fill(hidden, -math.inf), 2))
                    out[i, u:to, j * share : (j + 1) * share] = torch.einsum("gtn,nd->tgd", w, v[pick])
        return out
    lens = lengths(case["len_min"], case["len_max"], case["batch"])
    for j in range(case["kv_heads"]):
        k0, v0 = cached(s["prefix"].long(), case["prefix"], j)
        for i, n in enumerate(lens):
            k1, v1 = cached(s["table"][i, : -(-n // case["page"])].long(), n, j)
            for u in range(max(0, t - n), t):
                see = n - t + u + 1
                k, v = torch.cat((k0, k1[:see])), torch.cat((v0, v1[:see]))
                w = torch.softmax(s["scale"] * (s["q"][i, u, j * share : (j + 1) * share].double() @ k.T), 1)
                out[i, u, j * share : (j + 1) * share] = w @ v
    return out

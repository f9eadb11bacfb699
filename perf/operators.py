"""The operators of the 16-bit key/value cache, as cases to be measured.

A cache holds the keys and values of B sequences in bf16 or fp16 (head_dim
128), in pages of 32 tokens [n_pages][Hkv][32][128] reached through a block
table, or contiguous [B][Hkv][T][128]; the lengths n_tok[B] live on the
device, and a float32 attention weight per (KV head, token) may go with it.

  write       new tokens of every sequence into the cache, at given positions
  attention   the newest tokens' queries against the cache: causal, with an
              optional sliding window and first tokens that stay visible
  decode      the same for one query per sequence, optionally adding its
              probabilities to the tokens' weights
  accumulate  the probabilities of a prompt's last queries added to the weights
  evict       the first, the newest and the heaviest tokens of each KV head
              into another cache, in order of position

`own` false: the plain forms, elementary torch operations in 32 bits over
padded batches.  `own` true: the framework's calls.
"""
import math
import random

import torch

own = False

D, PAGE = 128, 32
SCALE = 1.0 / math.sqrt(D)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
HEADS = ((32, 8), (32, 4), (8, 8), (12, 4), (14, 2), (16, 1), (1, 1), (24, 2), (10, 2))


def listed():
    return [
        # a decode step's append: one new token for each of 8 sequences, latency-bound
        {"name": "write_step", "op": "write", "B": 8, "Hq": 32, "Hkv": 8, "ctx": 4096, "new": 1, "low": 0.2, "dtype": "bf16", "paged": True},
        # prompts of unequal length stored whole
        {"name": "write_prompts", "op": "write", "B": 6, "Hq": 32, "Hkv": 8, "ctx": 0, "new": 8192, "low": 0.1, "dtype": "fp16", "paged": True},
        # a batch of chat-sized questions: short, ragged, latency-bound
        {"name": "attention_short", "op": "attention", "B": 4, "Hq": 32, "Hkv": 8, "ctx": 0, "new": 96, "low": 0.1, "window": 0, "sink": 0, "dtype": "bf16", "paged": True},
        # a layer with a sliding window and sinks, the next part of each prompt behind what is cached
        {"name": "attention_window", "op": "attention", "B": 4, "Hq": 32, "Hkv": 4, "ctx": 1000, "new": 4096, "low": 0.5, "window": 1000, "sink": 4, "dtype": "fp16", "paged": True},
        # one long prompt, causal, over the raw keys and values that the packing prefill takes
        {"name": "attention_prompt", "op": "attention", "B": 1, "Hq": 32, "Hkv": 8, "ctx": 0, "new": 8192, "low": 1.0, "window": 0, "sink": 0, "dtype": "bf16", "paged": False},
        # the smallest decode: one head, 1024 tokens
        {"name": "decode_tiny", "op": "decode", "B": 1, "Hq": 1, "Hkv": 1, "ctx": 1024, "low": 1.0, "window": 0, "sink": 0, "weights": False, "dtype": "bf16", "paged": True},
        # a large batch on a windowed layer
        {"name": "decode_window", "op": "decode", "B": 48, "Hq": 32, "Hkv": 8, "ctx": 16384, "low": 0.2, "window": 4096, "sink": 4, "weights": False, "dtype": "fp16", "paged": True},
        # long contexts of unequal length, with the weights that a later eviction goes by
        {"name": "decode_ragged", "op": "decode", "B": 16, "Hq": 32, "Hkv": 4, "ctx": 65536, "low": 0.2, "window": 0, "sink": 0, "weights": True, "dtype": "bf16", "paged": True},
        # the weights of long prompts' tokens under their last 128 queries, before an eviction
        {"name": "accumulate_observed", "op": "accumulate", "B": 4, "Hq": 32, "Hkv": 8, "ctx": 16000, "new": 384, "low": 0.4, "window": 0, "sink": 0, "observe": 128, "dtype": "bf16", "paged": True},
        # the weights under all queries of a prompt
        {"name": "accumulate_prompt", "op": "accumulate", "B": 2, "Hq": 32, "Hkv": 4, "ctx": 0, "new": 4096, "low": 0.7, "window": 0, "sink": 0, "observe": 0, "dtype": "bf16", "paged": False},
        # a cache that outgrew its budget by a few pages
        {"name": "evict_step", "op": "evict", "B": 4, "Hq": 32, "Hkv": 4, "ctx": 2176, "low": 0.95, "first": 4, "recent": 512, "top": 1532, "dtype": "fp16", "paged": True},
        # long prompts cut down to a budget
        {"name": "evict_prompts", "op": "evict", "B": 8, "Hq": 32, "Hkv": 8, "ctx": 32768, "low": 0.3, "first": 4, "recent": 512, "top": 1532, "dtype": "bf16", "paged": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        c = {"op": rng.choice(("write", "attention", "attention", "decode", "decode", "accumulate", "evict"))}
        c["B"] = log(1, 48)
        c["Hq"], c["Hkv"] = rng.choice(HEADS)
        c["low"] = round(rng.uniform(0.05, 1.0), 2)
        c["dtype"] = rng.choice(("bf16", "fp16"))
        c["paged"] = rng.random() < 0.7
        if c["op"] == "write":
            c["ctx"], c["new"] = log(1, 8192), log(1, 8192)
            fits = c["B"] * c["Hkv"] * c["new"] <= 8 * 6 * 8192 and c["B"] * c["Hkv"] * (c["ctx"] + c["new"]) <= 1 << 22
        elif c["op"] in ("attention", "accumulate"):
            c["ctx"], c["new"] = rng.choice((0, log(1, 32768))), log(1, 8192)
            c["window"], c["sink"] = rng.choice(((0, 0), (log(1, 4096), 0), (log(16, 4096), log(1, 128))))
            if c["op"] == "accumulate":
                c["observe"] = rng.choice((0, log(1, 256)))
            pairs = c["B"] * c["Hq"] * c["new"] * (c["ctx"] + c["new"] / 2)
            fits = pairs <= (1 << 30) and c["B"] * c["Hkv"] * (c["ctx"] + c["new"]) <= 1 << 22
        elif c["op"] == "decode":
            c["ctx"] = log(1, 131072)
            c["window"], c["sink"] = rng.choice(((0, 0), (0, 0), (log(1, 8192), log(1, 128))))
            c["weights"] = rng.random() < 0.4
            fits = c["B"] * c["Hkv"] * c["ctx"] <= 2400000
        else:
            c["ctx"] = log(64, 65536)
            c["first"], c["recent"] = log(1, 64), log(1, 1024)
            c["top"] = log(1, 4096)
            fits = c["B"] * c["Hkv"] * c["ctx"] <= 1 << 21
        if fits:
            return c


# ---------------------------------------------------------------- the inputs

def _lengths(case, most):
    """A length for each sequence, from low * most to most, the first the longest: the same for every seed."""
    r = random.Random("%d %d %s" % (case["B"], most, case["low"]))
    return [most] + [max(1, int(most * r.uniform(case["low"], 1.0))) for _ in range(case["B"] - 1)]


def _shape(case):
    """(new tokens, cached tokens with them) of every sequence."""
    new = _lengths(case, case["new"]) if "new" in case else [0] * case["B"]
    ctx = _lengths(case, case["ctx"]) if case["ctx"] else [0] * case["B"]
    return new, [a + b for a, b in zip(new, ctx)]


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _make_cache(gen, case, n_tok, weights):
    """A cache's tensors for the lengths n_tok, its pages in random order; keys have a few strong channels."""
    B, Hkv, dtype = case["B"], case["Hkv"], TYPES[case["dtype"]]
    blocks = -(-max(n_tok) // PAGE)
    c = {"n_tok": _int32(n_tok), "most": max(n_tok), "blocks": blocks, "table": None, "weight": None}
    lead = (B * blocks, Hkv, PAGE) if case["paged"] else (B, Hkv, blocks * PAGE)
    if case["paged"]:
        c["table"] = torch.randperm(B * blocks, generator=gen, device="cuda").to(torch.int32).view(B, blocks)
    c["k"] = _normal(gen, lead + (D,), dtype)
    c["k"][..., 5::32] *= 3
    c["v"] = _normal(gen, lead + (D,), dtype)
    if weights:
        u = torch.rand(lead, generator=gen, device="cuda")
        c["weight"] = u.pow(6) * 8 * (u > 0.1)
    return c


def _handle(c):
    from int2_kv_cache_02_gb300 import oscar as L
    return L.KV16Cache(c["k"], c["v"], c["n_tok"], block_table=c["table"], weight=c["weight"])


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, B, Hq, Hkv, dtype = case["op"], case["B"], case["Hq"], case["Hkv"], TYPES[case["dtype"]]
    new, n_tok = _shape(case)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s = {"case": case, "total": start[-1], "start": _int32(start), "max_q": max(new)}
    s["cache"] = c = _make_cache(gen, case, n_tok, op in ("write", "accumulate", "evict") or case.get("weights", False))
    if op == "write":
        s["k_new"], s["v_new"] = (_normal(gen, (s["total"], Hkv, D), dtype) for _ in range(2))
        s["pos0"] = _int32([t - n for t, n in zip(n_tok, new)])
    elif op in ("attention", "accumulate"):
        s["q"] = _normal(gen, (s["total"], Hq, D), dtype)
        s["lse"] = torch.empty((s["total"], Hq), dtype=torch.float32, device="cuda")
        if op == "accumulate":
            s["lse"].copy_(_attention(s, case["observe"])[1])
        s["out"] = torch.empty_like(s["q"])
    elif op == "decode":
        s["q"] = _normal(gen, (B, Hq, D), dtype)
        s["out"] = torch.empty_like(s["q"])
    else:
        keep = case["first"] + case["recent"] + case["top"]
        s["to"] = _make_cache(gen, case, [keep] * B, True)
        s["kept"] = torch.empty((B, Hkv, keep), dtype=torch.int32, device="cuda")
    if own:
        from int2_kv_cache_02_gb300 import oscar as L
        s["handle"] = h = _handle(c)
        if op == "attention":
            s["workspace"] = L.alloc_workspace(L.kv16_attention_workspace_bytes(h, Hq, s["total"], c["most"], case["window"], case["sink"]))
        elif op == "decode":
            s["workspace"] = L.alloc_workspace(L.kv16_decode_workspace_bytes(h, Hq, c["most"], case["window"], case["sink"], case["weights"]))
        elif op == "evict":
            s["to_handle"] = _handle(s["to"])
            s["workspace"] = L.alloc_workspace(L.kv16_evict_workspace_bytes(h, c["most"], case["first"], case["recent"], case["top"]))
    return s


# ------------------------------------------------------------ the plain forms

def _rows(c, x):
    """Keys, values or weights of a cache in token order: [B][Hkv][blocks * 32]..., float32."""
    if c["table"] is not None:
        x = x[c["table"].long()].transpose(1, 2)
        x = x.reshape(x.shape[0], x.shape[1], -1, *x.shape[4:])
    return x.float()


def _put_weight(c, w):
    if c["table"] is None:
        c["weight"].copy_(w)
    else:
        c["weight"][c["table"].long()] = w.unflatten(2, (-1, PAGE)).transpose(1, 2)


def _visible(at, n_keys, window, sink):
    """Whether the query at position `at` sees each of n_keys tokens."""
    j = torch.arange(n_keys, device=at.device)
    at = at[..., None]
    seen = j <= at
    if window:
        seen = seen & ((j > at - window) | (j < sink))
    return seen


def _padded(s, last):
    """Row numbers [B][most] of every sequence's last `last` queries (0: all), which of them exist, and their positions."""
    start = s["start"].long()
    n = start[1:] - start[:-1]
    m = n.clamp(max=last) if last else n
    i = torch.arange(min(last, s["max_q"]) if last else s["max_q"], device=start.device)
    exists = i < m[:, None]
    row = (start[1:] - m)[:, None] + i
    at = (s["cache"]["n_tok"].long() - m)[:, None] + i
    return row.clamp(max=max(s["total"] - 1, 0)), exists, at


def _scores(s, q, at):
    """Scores of padded queries q [B][n][Hq][128]: [B][Hkv][g][n][keys], -inf where a key is not visible."""
    case, c = s["case"], s["cache"]
    B, n, Hkv = q.shape[0], q.shape[1], case["Hkv"]
    q = q.float().unflatten(2, (Hkv, -1)).permute(0, 2, 3, 1, 4)
    k = _rows(c, c["k"])
    x = (q.flatten(2, 3) @ k.transpose(-1, -2)).mul_(SCALE).unflatten(2, (-1, n))
    seen = _visible(at, k.shape[2], case["window"], case["sink"])
    return x.masked_fill_(~seen[:, None, None], -math.inf)


def _attend(s, q, at):
    """(output, log of the sum, probabilities) of padded queries."""
    x = _scores(s, q, at)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    v = _rows(s["cache"], s["cache"]["v"])
    o = (p.flatten(2, 3) @ v).unflatten(2, p.shape[2:4]) / torch.where(l == 0, 1.0, l)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3), (l.log() + m)[..., 0].permute(0, 3, 1, 2).flatten(2, 3), p, l


def _attention(s, last=0):
    row, exists, at = _padded(s, last)
    o, lse, _, _ = _attend(s, s["q"][row], at)
    out, out_lse = s["out"] if "out" in s else torch.empty_like(s["q"]), s["lse"]
    where = row[exists]
    out[where] = o[exists].to(out.dtype)
    out_lse[where] = lse[exists]
    return out, out_lse


def _write(s):
    c = s["cache"]
    row = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["start"][1:].long(), row, right=True)
    at = s["pos0"].long()[b] + row - s["start"].long()[b]
    if c["table"] is None:
        place = (b, slice(None), at)
    else:
        place = (c["table"].long()[b, at // PAGE], slice(None), at % PAGE)
    c["k"][place] = s["k_new"]
    c["v"][place] = s["v_new"]
    c["weight"][place] = 0.0
    c["n_tok"].copy_(s["pos0"] + s["start"][1:] - s["start"][:-1])
    return c["k"], c["v"], c["weight"], c["n_tok"]


def _decode(s):
    c = s["cache"]
    o, _, p, l = _attend(s, s["q"][:, None], c["n_tok"].long()[:, None] - 1)
    s["out"].copy_(o[:, 0].to(s["out"].dtype))
    if not s["case"]["weights"]:
        return s["out"]
    _put_weight(c, _rows(c, c["weight"]) + (p / torch.where(l == 0, 1.0, l)).sum((2, 3)))
    return s["out"], c["weight"]


def _accumulate(s):
    c = s["cache"]
    row, exists, at = _padded(s, s["case"]["observe"])
    x = _scores(s, s["q"][row], at)
    lse = s["lse"][row].unflatten(2, (s["case"]["Hkv"], -1)).permute(0, 2, 3, 1)
    lse = torch.where(exists[:, None, None], lse, math.inf)
    _put_weight(c, _rows(c, c["weight"]) + x.sub_(lse[..., None]).exp_().sum((2, 3)))
    return c["weight"]


def _evict(s):
    case, c, to = s["case"], s["cache"], s["to"]
    keep = case["first"] + case["recent"] + case["top"]
    w = _rows(c, c["weight"])
    j = torch.arange(w.shape[2], device="cuda")
    n = c["n_tok"].long()[:, None, None]
    rank = torch.where((j < case["first"]) | (j >= n - case["recent"]), math.inf, w)
    rank = torch.where(j < n, rank, -math.inf)
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices
    order = order[..., :keep]
    order = torch.nn.functional.pad(order, (0, keep - order.shape[2]))
    i = torch.arange(keep, device="cuda")
    held = (i < n).expand(order.shape)
    order = torch.where(held, order, w.shape[2]).sort(dim=2).values
    s["kept"].copy_(torch.where(held, order, -1))
    b, h = torch.meshgrid(torch.arange(w.shape[0], device="cuda"), torch.arange(w.shape[1], device="cuda"), indexing="ij")
    b, h, i, old = b[..., None].expand_as(order), h[..., None].expand_as(order), i.expand_as(order), order.clamp(max=w.shape[2] - 1)

    def place(x, t):
        return (b, h, t) if x["table"] is None else (x["table"].long()[b, t // PAGE], h, t % PAGE)

    here, there = place(c, old), place(to, i)
    to["k"][there] = torch.where(held[..., None], c["k"][here], to["k"][there])
    to["v"][there] = torch.where(held[..., None], c["v"][here], to["v"][there])
    to["weight"][there] = torch.where(held, c["weight"][here], to["weight"][there])
    to["n_tok"].copy_(c["n_tok"].clamp(max=keep))
    return s["kept"], to["k"], to["v"], to["weight"], to["n_tok"]


PLAIN = {"write": _write, "attention": _attention, "decode": _decode, "accumulate": _accumulate, "evict": _evict}


# -------------------------------------------------------------------- a pass

def run(s):
    case = s["case"]
    if not own:
        return PLAIN[case["op"]](s)
    from int2_kv_cache_02_gb300 import oscar as L
    op, c, h = case["op"], s["cache"], s["handle"]
    if op == "write":
        L.kv16_write(h, s["k_new"], s["v_new"], s["start"], s["pos0"])
        return c["k"], c["v"], c["weight"], c["n_tok"]
    if op == "attention":
        L.kv16_attention(h, s["q"], s["start"], SCALE, c["most"], s["out"], s["workspace"], window=case["window"], n_sink=case["sink"], lse=s["lse"])
        return s["out"], s["lse"]
    if op == "decode":
        L.kv16_decode_attention(h, s["q"], SCALE, c["most"], s["out"], s["workspace"], window=case["window"], n_sink=case["sink"], accumulate=case["weights"])
        return (s["out"], c["weight"]) if case["weights"] else s["out"]
    if op == "accumulate":
        L.kv16_accumulate(h, s["q"], s["lse"], s["start"], SCALE, c["most"], window=case["window"], n_sink=case["sink"], n_obs=case["observe"])
        return c["weight"]
    L.kv16_evict(h, s["to_handle"], c["most"], case["first"], case["recent"], case["top"], s["workspace"], kept=s["kept"])
    to = s["to"]
    return s["kept"], to["k"], to["v"], to["weight"], to["n_tok"]


# ----------------------------------------------------- what a pass has to do

def _seen(at, window, sink):
    """How many tokens the query at position `at` sees."""
    near = min(window, at + 1) if window else at + 1
    return near + min(sink, at + 1 - near)


def work(case):
    op, Hq, Hkv = case["op"], case["Hq"], case["Hkv"]
    new, n_tok = _shape(case)
    row = 2 * D
    if op == "write":
        rows = sum(new) * Hkv
        return {"bytes": rows * (4 * row + 4), "flops": 0}
    if op == "decode":
        seen = sum(_seen(n - 1, case["window"], case["sink"]) for n in n_tok)
        weights = 8 * seen * Hkv if case["weights"] else 0
        return {"bytes": 2 * row * seen * Hkv + 2 * row * Hq * len(n_tok) + weights, "flops": 4 * D * Hq * seen}
    if op == "evict":
        keep = case["first"] + case["recent"] + case["top"]
        kept = sum(min(n, keep) for n in n_tok) * Hkv
        ranked = sum(n for n in n_tok if n > keep) * Hkv
        return {"bytes": kept * (4 * row + 8 + 4) + 4 * ranked, "flops": 0}
    pairs = keys = rows = 0
    for q, n in zip(new, n_tok):
        if case.get("observe"):
            q = min(q, case["observe"])
        rows += q
        pairs += sum(_seen(at, case["window"], case["sink"]) for at in range(n - q, n))
        first = max(0, n - q + 1 - case["window"]) if case["window"] else 0
        keys += n - first + min(case["sink"], first)
    if op == "accumulate":
        return {"bytes": row * (rows * Hq + keys * Hkv) + 4 * rows * Hq + 8 * keys * Hkv, "flops": 2 * D * Hq * pairs}
    return {"bytes": 2 * row * (rows * Hq + keys * Hkv) + 4 * rows * Hq, "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definition, one KV head of one sequence at a time.  A write and an eviction compute no numbers: None."""
    op = case["op"]
    if op in ("write", "evict"):
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, g = s["cache"], case["Hq"] // case["Hkv"]
    new, n_tok = _shape(case)
    if op == "decode":
        new = [1] * case["B"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    log_sum = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    weight = c["weight"].double() if c["weight"] is not None else None
    first = 0
    for b in range(case["B"]):
        n, q = n_tok[b], new[b]
        skip = max(0, q - case["observe"]) if case.get("observe") else 0
        t = torch.arange(n, device="cuda")
        for h in range(case["Hkv"]):
            place = (b, h, t) if c["table"] is None else (c["table"][b].long()[t // PAGE], h, t % PAGE)
            k, v = c["k"][place].double(), c["v"][place].double()
            total = torch.zeros(n, dtype=torch.float64, device="cuda")
            for i in range(skip, q, 1024):
                rows = slice(first + i, first + min(i + 1024, q))
                heads = slice(h * g, h * g + g)
                x = torch.einsum("ijd,td->ijt", s["q"][rows, heads].double(), k) * SCALE
                at = n - q + torch.arange(i, min(i + 1024, q), device="cuda")[:, None, None]
                hidden = t > at
                if case["window"]:
                    hidden = hidden | ((t <= at - case["window"]) & (t >= case["sink"]))
                x = x.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, -1)
                if op == "accumulate":
                    z = s["lse"][rows, heads].double()
                p = torch.exp(x - z[..., None])
                total += p.sum((0, 1))
                if op != "accumulate":
                    out[rows, heads] = torch.einsum("ijt,td->ijd", p, v)
                    log_sum[rows, heads] = z
            if weight is not None:
                weight[place] += total
        first += q
    if op == "accumulate":
        return weight
    if op == "attention":
        return out, log_sum
    return (out, weight) if case["weights"] else out

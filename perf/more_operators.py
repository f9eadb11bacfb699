"""Sequences of the 16-bit key/value cache that have tokens in common, as cases
to be measured: attention that reads a shared prefix once, and the page
operators that make and tidy such sequences.

A cache holds the keys and values of B sequences in bf16 or fp16 (head_dim
128), in pages of 32 tokens [n_pages][Hkv][32][128] reached through a block
table, or contiguous [B][Hkv][T][128]; the lengths n_tok[B] live on the
device, and a float32 attention weight per (KV head, token) may go with it.
Neighbouring sequences group[i] .. group[i + 1] - 1 form group i, whose
members have their first prefix[i] tokens in common.

  shared_decode     attention of one query per sequence, that of its newest
                    token, over the group's prefix and its own tokens
  shared_attention  the same for several new tokens per sequence, causal
  fork              sequences made of others: whole pages taken over by
                    reference or copied, the page in which the tokens end copied
  compact           the pages that tables name moved to the lowest page ids,
                    tables rewritten, for all layers that use the table

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
        # two samples of a short prompt on a small model, just begun: latency-bound
        {"name": "decode_tiny", "op": "shared_decode", "groups": 1, "members": 2, "Hq": 8, "Hkv": 8, "prefix": 512, "own": 20, "low": 0.5, "window": 0, "sink": 0, "dtype": "bf16"},
        # sixteen samples of one prompt
        {"name": "decode_samples", "op": "shared_decode", "groups": 1, "members": 16, "Hq": 32, "Hkv": 8, "prefix": 8192, "own": 512, "low": 0.4, "window": 0, "sink": 0, "dtype": "bf16"},
        # requests under a few system prompts of unequal length, each at a place of its own
        {"name": "decode_system", "op": "shared_decode", "groups": 4, "members": 32, "Hq": 32, "Hkv": 8, "prefix": 16384, "own": 2048, "low": 0.1, "window": 0, "sink": 0, "dtype": "bf16"},
        # many requests about two long documents: as much arithmetic as reading
        {"name": "decode_documents", "op": "shared_decode", "groups": 2, "members": 64, "Hq": 32, "Hkv": 4, "prefix": 65536, "own": 1024, "low": 0.3, "window": 0, "sink": 0, "dtype": "fp16"},
        # a layer with a sliding window and sinks: the window reaches back into the prefix, which ends inside a page
        {"name": "decode_window", "op": "shared_decode", "groups": 4, "members": 12, "Hq": 24, "Hkv": 2, "prefix": 6007, "own": 2500, "low": 0.1, "window": 4096, "sink": 4, "dtype": "fp16"},
        # questions behind a common instruction, read for the first time
        {"name": "attention_questions", "op": "shared_attention", "groups": 2, "members": 8, "Hq": 32, "Hkv": 8, "prefix": 8192, "own": 0, "new": 96, "low": 0.1, "window": 0, "sink": 0, "dtype": "bf16"},
        # a few drafted tokens of every sample to be verified at once
        {"name": "attention_drafts", "op": "shared_attention", "groups": 1, "members": 32, "Hq": 32, "Hkv": 8, "prefix": 32768, "own": 512, "new": 5, "low": 0.6, "window": 0, "sink": 0, "dtype": "bf16"},
        # a prompt's sequence turned into eight samples
        {"name": "fork_samples", "op": "fork", "B": 8, "parents": 1, "Hkv": 8, "ctx": 8190, "low": 1.0, "idle": 0.0, "share": True, "weights": False, "from_paged": True, "to_paged": True, "dtype": "bf16"},
        # a step of a beam search: every beam continues one of the beams before
        {"name": "fork_beams", "op": "fork", "B": 96, "parents": 96, "Hkv": 8, "ctx": 4096, "low": 0.2, "idle": 0.1, "share": True, "weights": False, "from_paged": True, "to_paged": True, "dtype": "fp16"},
        # sequences copied whole with their tokens' weights, since an eviction will go by each copy's own
        {"name": "fork_copies", "op": "fork", "B": 12, "parents": 3, "Hkv": 8, "ctx": 16384, "low": 0.4, "idle": 0.0, "share": False, "weights": True, "from_paged": True, "to_paged": True, "dtype": "bf16"},
        # a small pool, nearly full, after a few requests have ended
        {"name": "compact_small", "op": "compact", "B": 8, "Hkv": 4, "ctx": 2048, "low": 0.3, "live": 0.9, "layers": 1, "weights": False, "dtype": "fp16"},
        # a pool of several layers half of whose requests have ended
        {"name": "compact_layers", "op": "compact", "B": 64, "Hkv": 8, "ctx": 8192, "low": 0.1, "live": 0.5, "layers": 4, "weights": False, "dtype": "bf16"},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        c = {"op": rng.choice(("shared_decode", "shared_decode", "shared_attention", "shared_attention", "fork", "compact"))}
        c["Hq"], c["Hkv"] = rng.choice(HEADS)
        c["low"] = round(rng.uniform(0.05, 1.0), 2)
        c["dtype"] = rng.choice(("bf16", "fp16"))
        if c["op"] in ("shared_decode", "shared_attention"):
            c["groups"], c["members"] = log(1, 8), log(1, 96)
            c["prefix"], c["own"] = log(1, 65536), rng.choice((0, log(1, 4096)))
            c["window"], c["sink"] = rng.choice(((0, 0), (0, 0), (log(1, 8192), log(1, 128))))
            if c["op"] == "shared_attention":
                c["new"] = log(1, 512)
            rows = c["groups"] * c["members"]
            most = c["prefix"] + c["own"] + c.get("new", 1)
            fits = rows * c["Hkv"] * most <= 1 << 24 and rows * c["Hq"] * c.get("new", 1) * most <= 1 << 28
        elif c["op"] == "fork":
            del c["Hq"]
            c["B"], c["parents"], c["ctx"] = log(1, 128), log(1, 128), log(1, 32768)
            c["idle"] = rng.choice((0.0, 0.2))
            c["share"], c["weights"] = rng.random() < 0.5, rng.random() < 0.4
            c["from_paged"], c["to_paged"] = (True, True) if c["share"] else (rng.random() < 0.6, rng.random() < 0.6)
            fits = max(c["parents"], c["B"]) * c["Hkv"] * c["ctx"] <= 12 * 8 * 16384
        else:
            del c["Hq"]
            c["B"], c["ctx"], c["layers"] = log(1, 96), log(32, 32768), log(1, 6)
            c["live"] = round(rng.uniform(0.2, 1.0), 2)
            c["weights"] = rng.random() < 0.4
            fits = c["B"] * c["Hkv"] * c["ctx"] * c["layers"] <= 1 << 23
        if fits:
            return c


# ---------------------------------------------------------------- the inputs

def _lengths(n, most, low):
    """n lengths from low * most to most, the first the longest: the same for every seed."""
    r = random.Random("%d %d %s" % (n, most, low))
    return [most] + [max(min(1, most), int(most * r.uniform(low, 1.0))) for _ in range(n - 1)]


def _shape(case):
    """(prefix of each group, new tokens, all tokens) of every sequence."""
    G, M = case["groups"], case["members"]
    prefix = _lengths(G, case["prefix"], max(case["low"], 0.5))
    new = _lengths(G * M, case["new"], case["low"]) if "new" in case else [1] * (G * M)
    mine = _lengths(G * M, case["own"], case["low"])
    return prefix, new, [prefix[b // M] + mine[b] + new[b] for b in range(G * M)]


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _fill(gen, lead, dtype, weights):
    """Keys (a few strong channels), values and weights of a pool or of contiguous rows."""
    c = {"k": _normal(gen, lead + (D,), dtype), "v": _normal(gen, lead + (D,), dtype), "weight": None, "table": None}
    c["k"][..., 5::32] *= 3
    if weights:
        u = torch.rand(lead, generator=gen, device="cuda")
        c["weight"] = u.pow(6) * 8 * (u > 0.1)
    return c


def _blocks(n):
    return -(-n // PAGE)


def _prepare_shared(case, gen):
    G, M, Hkv, dtype = case["groups"], case["members"], case["Hkv"], TYPES[case["dtype"]]
    prefix, new, n_tok = _shape(case)
    B, wide = G * M, _blocks(max(n_tok))
    # a page for every block, those of a prefix's whole pages taken once a group
    ids, pages = [[-1] * wide for _ in range(B)], 0
    for b in range(B):
        for j in range(_blocks(n_tok[b])):
            if j < prefix[b // M] // PAGE and b % M:
                ids[b][j] = ids[b - b % M][j]
            else:
                ids[b][j], pages = pages, pages + 1
    c = _fill(gen, (pages, Hkv, PAGE), dtype, False)
    place = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    ids = _int32(ids)
    c["table"] = torch.where(ids < 0, -1, place[ids.clamp(min=0).long()])
    c["n_tok"], c["most"] = _int32(n_tok), max(n_tok)
    for i, n in enumerate(prefix):
        if n % PAGE:    # the prefix's last tokens stand in a page of each member's own
            t = c["table"][i * M:(i + 1) * M, n // PAGE].long()
            c["k"][t, :, :n % PAGE] = c["k"][t[0], :, :n % PAGE]
            c["v"][t, :, :n % PAGE] = c["v"][t[0], :, :n % PAGE]
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s = {"cache": c, "total": start[-1], "start": _int32(start), "max_q": max(new),
         "group": _int32(range(0, B + 1, M)), "prefix": _int32(prefix)}
    s["q"] = _normal(gen, (s["total"], case["Hq"], D), dtype)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((s["total"], case["Hq"]), dtype=torch.float32, device="cuda")
    return s


def _prepare_fork(case, gen):
    B, P, Hkv, dtype = case["B"], case["parents"], case["Hkv"], TYPES[case["dtype"]]
    n = _lengths(P, case["ctx"], case["low"])
    wide = _blocks(case["ctx"])
    parent = torch.randint(P, (B,), generator=gen, device="cuda", dtype=torch.int32)
    parent[torch.rand(B, generator=gen, device="cuda") < case["idle"]] = -1
    there = P * wide if case["from_paged"] else 0
    here = (B if case["share"] else B * wide) if case["to_paged"] else 0
    place = torch.randperm(there + here, generator=gen, device="cuda").to(torch.int32)
    pool = _fill(gen, (there + here, Hkv, PAGE), dtype, case["weights"]) if there + here else None
    src = dict(pool) if there else _fill(gen, (P, Hkv, wide * PAGE), dtype, case["weights"])
    dst = dict(pool) if here else _fill(gen, (B, Hkv, wide * PAGE), dtype, case["weights"])
    if there:
        src["table"] = place[:there].view(P, wide).contiguous()
    if here:
        dst["table"] = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
        if case["share"]:
            last = _int32(n)[parent.clamp(min=0).long()].long() // PAGE
            dst["table"].scatter_(1, last.clamp(max=wide - 1)[:, None], place[there:, None])
        else:
            dst["table"].copy_(place[there:].view(B, wide))
    src["n_tok"], dst["n_tok"] = _int32(n), torch.zeros(B, dtype=torch.int32, device="cuda")
    return {"cache": src, "to": dst, "parent": parent, "most": case["ctx"]}


def _pool_shape(case):
    """(pages of every sequence, pages of the pool, pages that have to move)."""
    n = [_blocks(x) for x in _lengths(case["B"], case["ctx"], case["low"])]
    live = sum(n)
    pages = max(live, int(live / case["live"]))
    return n, pages, min(live, round(live * (pages - live) / pages))


def _prepare_compact(case, gen):
    n, pages, moved = _pool_shape(case)
    live = sum(n)
    ids = torch.cat((torch.randperm(pages - live, generator=gen, device="cuda")[:moved] + live,
                     torch.randperm(live, generator=gen, device="cuda")[:live - moved]))
    ids = ids[torch.randperm(live, generator=gen, device="cuda")].to(torch.int32)
    table = torch.full((case["B"], _blocks(case["ctx"])), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, blocks in enumerate(n):
        table[b, :blocks] = ids[at:at + blocks]
        at += blocks
    s = {"table": table, "new_table": torch.empty_like(table), "pages": pages, "layers": []}
    for _ in range(case["layers"]):
        c = _fill(gen, (pages, case["Hkv"], PAGE), TYPES[case["dtype"]], case["weights"])
        c["table"], c["n_tok"] = table, _int32(_lengths(case["B"], case["ctx"], case["low"]))
        s["layers"].append(c)
    s["moves"] = torch.empty((pages // 2, 2), dtype=torch.int32, device="cuda")
    s["counts"] = torch.empty(2, dtype=torch.int32, device="cuda")
    return s


def _handle(c):
    from int2_kv_cache_02_gb300 import oscar as L
    return L.KV16Cache(c["k"], c["v"], c["n_tok"], block_table=c["table"], weight=c["weight"])


PREPARE = {"shared_decode": _prepare_shared, "shared_attention": _prepare_shared, "fork": _prepare_fork, "compact": _prepare_compact}


def prepare(case, seed):
    op = case["op"]
    s = PREPARE[op](case, torch.Generator("cuda").manual_seed(seed))
    s["case"] = case
    if own:
        from int2_kv_cache_02_gb300 import oscar as L
        if op == "fork":
            s["handle"], s["to_handle"] = _handle(s["cache"]), _handle(s["to"])
        elif op == "compact":
            s["handles"] = [_handle(c) for c in s["layers"]]
            s["workspace"] = L.alloc_workspace(L.page_compact_workspace_bytes(s["table"], s["pages"]))
        else:
            s["handle"] = h = _handle(s["cache"])
            shape = (s["cache"]["most"], case["window"], case["sink"])
            if op == "shared_decode":
                need = L.kv16_shared_decode_workspace_bytes(h, case["Hq"], case["groups"], *shape)
            else:
                need = L.kv16_shared_attention_workspace_bytes(h, case["Hq"], case["groups"], s["total"], *shape)
            s["workspace"] = L.alloc_workspace(need)
    return s


# ------------------------------------------------------------ the plain forms

def _rows(c, x):
    """Keys or values of a paged cache in token order: [B][Hkv][blocks * 32][128], float32."""
    x = x[c["table"].clamp(min=0).long()].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, D).float()


def _shared(s):
    """Softmax attention of every sequence's newest tokens over its cached ones."""
    case, c = s["case"], s["cache"]
    start, n = s["start"].long(), c["n_tok"].long()
    m = start[1:] - start[:-1]
    i = torch.arange(s["max_q"], device="cuda")
    exists = i < m[:, None]
    row = (start[:-1, None] + i).clamp(max=s["total"] - 1)
    at = ((n - m)[:, None] + i)[..., None]
    k = _rows(c, c["k"])
    j = torch.arange(k.shape[2], device="cuda")
    seen = j <= at
    if case["window"]:
        seen = seen & ((j > at - case["window"]) | (j < case["sink"]))
    q = s["q"][row].float().unflatten(2, (case["Hkv"], -1)).permute(0, 2, 3, 1, 4)
    x = (q.flatten(2, 3) @ k.transpose(-1, -2)).mul_(SCALE).unflatten(2, (-1, s["max_q"]))
    del k
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ _rows(c, c["v"])).unflatten(2, p.shape[2:4]) / l
    where = row[exists]
    s["out"][where] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[exists].to(s["out"].dtype)
    s["lse"][where] = (l.log() + top)[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[exists]
    return s["out"] if case["op"] == "shared_decode" else (s["out"], s["lse"])


def _place(c, b, t):
    return (b, slice(None), t) if c["table"] is None else (c["table"].long()[b, t // PAGE], slice(None), t % PAGE)


def _fork(s):
    c, to, share = s["cache"], s["to"], s["case"]["share"]
    parent = s["parent"].long()
    n = torch.where(parent >= 0, c["n_tok"].long()[parent.clamp(min=0)], 0)
    first = n // PAGE * PAGE if share else torch.zeros_like(n)
    if share:
        block = torch.arange(to["table"].shape[1], device="cuda")
        to["table"].copy_(torch.where(block < (first // PAGE)[:, None], c["table"][parent.clamp(min=0)], to["table"]))
    t = torch.arange(s["most"], device="cuda")
    b, t = torch.nonzero((t >= first[:, None]) & (t < n[:, None]), as_tuple=True)
    here, there = _place(c, parent[b], t), _place(to, b, t)
    for name in ("k", "v", "weight"):
        if c[name] is not None:
            to[name][there] = c[name][here]
    to["n_tok"].copy_(torch.where(parent >= 0, n, to["n_tok"].long()))
    return _forked(s)


def _forked(s):
    to = s["to"]
    out = [to["n_tok"], to["k"], to["v"]]
    return out + [x for x in (to["table"], to["weight"]) if x is not None]


def _compact(s):
    table, pages = s["table"], s["pages"]
    used = torch.zeros(pages, dtype=torch.bool, device="cuda")
    used[table[table >= 0].long()] = True
    live = used.sum()
    ids = torch.arange(pages, device="cuda")
    old, new = torch.nonzero(used & (ids >= live))[:, 0], torch.nonzero(~used & (ids < live))[:, 0]
    ids[old] = new
    s["new_table"].copy_(torch.where(table >= 0, ids[table.clamp(min=0).long()].to(torch.int32), table))
    s["moves"].fill_(-1)
    s["moves"][:old.shape[0]] = torch.stack((old, new), 1).to(torch.int32)
    s["counts"][0] = old.shape[0]
    s["counts"][1] = live
    for c in s["layers"]:
        for name in ("k", "v", "weight"):
            if c[name] is not None:
                c[name][new] = c[name][old]
    return _compacted(s)


def _compacted(s):
    out = [s["new_table"], s["moves"], s["counts"]]
    return out + [c[name] for c in s["layers"] for name in ("k", "v", "weight") if c[name] is not None]


PLAIN = {"shared_decode": _shared, "shared_attention": _shared, "fork": _fork, "compact": _compact}


# -------------------------------------------------------------------- a pass

def run(s):
    case = s["case"]
    if not own:
        return PLAIN[case["op"]](s)
    from int2_kv_cache_02_gb300 import oscar as L
    op = case["op"]
    if op == "fork":
        L.kv16_fork(s["handle"], s["to_handle"], s["parent"], s["most"], share=case["share"])
        return _forked(s)
    if op == "compact":
        L.page_compact(s["table"], s["new_table"], s["pages"], s["moves"], s["counts"], s["workspace"])
        for h in s["handles"]:
            L.kv16_copy_pages(h, h, s["moves"], s["counts"])
        return _compacted(s)
    c, h = s["cache"], s["handle"]
    if op == "shared_decode":
        L.kv16_shared_decode_attention(h, s["q"], s["group"], s["prefix"], SCALE, c["most"], s["out"], s["workspace"],
                                       window=case["window"], n_sink=case["sink"])
        return s["out"]
    L.kv16_shared_attention(h, s["q"], s["start"], s["group"], s["prefix"], SCALE, c["most"], s["out"], s["workspace"],
                            window=case["window"], n_sink=case["sink"], lse=s["lse"])
    return s["out"], s["lse"]


# ----------------------------------------------------- what a pass has to do

def _seen(at, window, sink):
    """How many tokens the query at position `at` sees."""
    near = min(window, at + 1) if window else at + 1
    return near + min(sink, at + 1 - near)


def work(case):
    op, Hkv, row = case["op"], case["Hkv"], 2 * D
    if op == "fork":
        n = _lengths(case["parents"], case["ctx"], case["low"])
        each = 4 * row + (8 if case["weights"] else 0)
        tokens = sum(x % PAGE if case["share"] else x for x in n) / len(n) * case["B"] * (1 - case["idle"])
        table = sum(x // PAGE for x in n) / len(n) * case["B"] * (1 - case["idle"]) * 8 if case["share"] else 0
        return {"bytes": int(tokens * Hkv * each + table + 12 * case["B"]), "flops": 0}
    if op == "compact":
        _, _, moved = _pool_shape(case)
        each = 4 * row + (8 if case["weights"] else 0)
        return {"bytes": moved * PAGE * Hkv * each * case["layers"] + 8 * case["B"] * _blocks(case["ctx"]), "flops": 0}
    prefix, new, n_tok = _shape(case)
    M, window, sink = case["members"], case["window"], case["sink"]
    pairs = keys = 0
    for i, p in enumerate(prefix):
        common = p      # of the prefix, the first position that a window reaches
        for b in range(i * M, (i + 1) * M):
            n, q = n_tok[b], new[b]
            pairs += sum(_seen(at, window, sink) for at in range(n - q, n))
            first = max(0, n - q + 1 - window) if window else 0
            keys += n - max(first, p) + max(0, min(sink, first) - p)
            common = min(common, first)
        keys += p - common + min(sink, common)
    total = sum(new) * case["Hq"]
    return {"bytes": 2 * row * (keys * Hkv + total) + (4 * total if op == "shared_attention" else 0), "flops": 4 * D * case["Hq"] * pairs}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definition, one KV head of one sequence at a time.  Forks and compactions compute no numbers: None."""
    op = case["op"]
    if op in ("fork", "compact"):
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, g = s["cache"], case["Hq"] // case["Hkv"]
    _, new, n_tok = _shape(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    log_sum = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    first = 0
    for n, q, pages in zip(n_tok, new, c["table"].long()):
        t = torch.arange(n, device="cuda")
        at = n - q + torch.arange(q, device="cuda")[:, None, None]
        hidden = t > at
        if case["window"]:
            hidden = hidden | ((t <= at - case["window"]) & (t >= case["sink"]))
        rows = slice(first, first + q)
        for h in range(case["Hkv"]):
            k, v = (x[pages[t // PAGE], h, t % PAGE].double() for x in (c["k"], c["v"]))
            heads = slice(h * g, h * g + g)
            x = torch.einsum("ijd,td->ijt", s["q"][rows, heads].double(), k) * SCALE
            x = x.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(x, -1)
            out[rows, heads] = torch.einsum("ijt,td->ijd", torch.exp(x - z[..., None]), v)
            log_sum[rows, heads] = z
        first += q
    return out if op == "shared_decode" else (out, log_sum)

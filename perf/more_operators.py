"""What the operators of a serving loop around a verification step are measured on.

A loop that serves a batch hands out the pages of the cache (`pages`), attends
to a prompt that several sequences share without reading it once for each
(`prefix`), draws tokens under temperature, top-k, top-p and min-p (`sample`)
and leaves of the logits only what such a draw may take, for a verification that
stays lossless (`truncate`).  Each case is one call of one of these (for `pages`
a step's two: pages for its tokens, and back those that it did not keep).

`run` computes a case in its plain form (elementary torch operations in 32
bits, whole numbers in 64) or, where `own` is true, by the library's own entry
points; `exact` states the same definitions in 64 bits.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
_ONE = 2.0 ** 44                # the largest weight of a row, as a whole number


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one new token for each sequence of a serving batch: latency-bound
        {"name": "pages decode", "op": "pages", "B": 64, "N": 1, "P": 16, "lo": 1000, "hi": 32000,
         "keep": 1, "tree": 0, "base": False},
        # trees of 16 drafts of 8 behind a shared prompt; a few tokens of each are kept
        {"name": "pages trees", "op": "pages", "B": 48, "N": 129, "P": 16, "lo": 0, "hi": 4000,
         "keep": 4, "tree": 8, "base": True},
        # prompts of many requests enter, and leave again when they are done
        {"name": "pages prompts", "op": "pages", "B": 300, "N": 8191, "P": 16, "lo": 0, "hi": 0,
         "keep": 0, "tree": 0, "base": False},
        # four samples of one short prompt: latency-bound
        {"name": "prefix 4 samples", "op": "prefix", "B": 4, "groups": 1, "N": 1, "Hq": 64, "Hk": 8,
         "D": 128, "P": 16, "plo": 1024, "phi": 1024, "lo": 0, "hi": 63, "tree": 0,
         "dtype": "bf16", "cache": "bf16"},
        # a serving batch of single tokens behind one long instruction
        {"name": "prefix decode", "op": "prefix", "B": 128, "groups": 1, "N": 1, "Hq": 64, "Hk": 8,
         "D": 128, "P": 16, "plo": 8191, "phi": 8191, "lo": 1, "hi": 700, "tree": 0,
         "dtype": "bf16", "cache": "bf16"},
        # several samples of each of eight ragged prompts, quantised cache
        {"name": "prefix groups e4m3", "op": "prefix", "B": 96, "groups": 8, "N": 1, "Hq": 64, "Hk": 8,
         "D": 128, "P": 64, "plo": 1000, "phi": 12000, "lo": 0, "hi": 500, "tree": 0,
         "dtype": "bf16", "cache": "e4m3"},
        # trees of 16 drafts of 16 for sequences that share a document
        {"name": "prefix trees 16x16", "op": "prefix", "B": 16, "groups": 1, "N": 257, "Hq": 64, "Hk": 8,
         "D": 128, "P": 16, "plo": 6001, "phi": 6001, "lo": 10, "hi": 500, "tree": 16,
         "dtype": "bf16", "cache": "bf16"},
        # questions of uneven length behind two documents, an odd group of small heads
        {"name": "prefix chunk fp16", "op": "prefix", "B": 6, "groups": 2, "N": 333, "Hq": 28, "Hk": 4,
         "D": 64, "P": 16, "plo": 2000, "phi": 4001, "lo": 0, "hi": 100, "tree": 0,
         "dtype": "fp16", "cache": "fp16"},
        # a single stream's next token
        {"name": "sample one row", "op": "sample", "B": 1, "per": 1, "V": 152064, "T": True, "k": False,
         "p": True, "m": False, "dtype": "bf16"},
        # a serving batch's next tokens, each request with its own parameters
        {"name": "sample batch", "op": "sample", "B": 256, "per": 1, "V": 152064, "T": True, "k": True,
         "p": True, "m": True, "dtype": "bf16"},
        # rows in 32 bits over an odd vocabulary, several draws a request
        {"name": "sample fp32 odd", "op": "sample", "B": 24, "per": 7, "V": 32001, "T": True, "k": False,
         "p": True, "m": True, "dtype": "fp32"},
        # every draft position of a serving batch, cut before its verification
        {"name": "truncate serving", "op": "truncate", "B": 8, "per": 136, "V": 152064, "T": True,
         "k": True, "p": True, "m": False, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(["pages", "prefix", "prefix", "sample", "sample", "truncate"])
    if op == "pages":
        kind = rng.choice(["token", "tree", "prompt"])
        gamma = rng.choice([4, 8, 15, 16])
        N = 1 if kind == "token" else 1 + gamma * rng.randint(1, 16) if kind == "tree" \
            else _log(rng, 2, 8000)
        lo = 0 if kind == "prompt" else _log(rng, 1, 8000) - 1
        return {"op": op, "B": _log(rng, 1, 2000), "N": N, "P": rng.choice([1, 16, 16, 24, 64, 128]), "lo": lo,
                "hi": lo if kind == "prompt" else lo + _log(rng, 1, 24000),
                "keep": 0 if kind == "prompt" else rng.randint(0, N),
                "tree": gamma if kind == "tree" else 0, "base": rng.random() < 0.5}
    if op == "prefix":
        kind = rng.choice(["token", "token", "tree", "chunk"])
        gamma = rng.choice([4, 8, 15, 16])
        N = 1 if kind == "token" else \
            1 + gamma * rng.randint(1, 16) if kind == "tree" else _log(rng, 2, 500)
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        Hk = rng.choice([1, 2, 4, 8])
        groups = rng.choice([1, 1, 2, 5])
        plo = _log(rng, 1, 8000) - 1
        lo = _log(rng, 1, 500) - 1
        return {"op": op, "B": groups * _log(rng, 1, 100), "groups": groups, "N": N,
                "Hq": Hk * rng.choice([1, 4, 7, 8]), "Hk": Hk, "D": rng.choice([64, 128, 128, 96]),
                "P": rng.choice([16, 32, 64, 128]), "plo": plo, "phi": plo + _log(rng, 1, 8000),
                "lo": lo, "hi": lo + _log(rng, 1, 500), "tree": gamma if kind == "tree" else 0,
                "dtype": dtype, "cache": rng.choice([dtype, "e4m3"])}
    return {"op": op, "B": _log(rng, 1, 256), "per": rng.choice([1, 1, 3, 17, 136]),
            "V": rng.choice([8, 1]) * _log(rng, 500, 19008), "T": rng.random() < 0.8,
            "k": rng.random() < 0.5, "p": rng.random() < 0.6, "m": rng.random() < 0.4,
            "dtype": rng.choice(["bf16", "bf16", "fp32"])}


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        t = top.setdefault(c["op"], [0, 0, 0])
        t[:] = [max(t[0], w["bytes"]), max(t[1], w["flops"]), max(t[2], _scratch(c))]
    while True:
        c = _draw_once(rng)
        w = work(c)
        if w["bytes"] <= top[c["op"]][0] and w["flops"] <= max(top[c["op"]][1], 1) \
                and _scratch(c) <= top[c["op"]][2]:
            return c


def _scratch(c):
    """Values that the plain form holds at once (for `pages`: places of the table;
    for rows: how many logits there are)."""
    if c["op"] == "pages":
        return c["B"] * (c["N"] + _per(c))
    if c["op"] == "prefix":
        return c["B"] * c["Hq"] * c["N"] * (c["phi"] + c["hi"] + c["N"]) + \
            2 * c["B"] * (c["hi"] + c["N"]) * c["Hk"] * c["D"]
    return c["B"] * c["per"] * c["V"]


def _lens(c):
    """Each sequence's tokens in the cache and new tokens, from the case alone."""
    r = random.Random("%d %d %d %d" % (c["B"], c["N"], c["lo"], c["hi"]))
    start = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    whole = c["N"] == 1 or c["tree"]
    count = [c["N"] if whole or b == 0 else r.randint((c["N"] + 1) // 2, c["N"])
             for b in range(c["B"])]
    return start, count


def _prefix_lens(c):
    r = random.Random("%d %d %d" % (c["groups"], c["plo"], c["phi"]))
    return [c["phi"] if g == 0 else r.randint(c["plo"], c["phi"]) for g in range(c["groups"])]


def _ceil(a, b):
    return -(-a // b)


def _per(c):
    """Pages that a sequence's row of the table holds."""
    return _ceil(c["hi"] + c["N"], c["P"])


def _kept(c):
    """Positions of each sequence after the step."""
    start, count = _lens(c)
    return [s + min(n, c["keep"]) for s, n in zip(start, count)]


def _visible(c):
    """Pairs of a new token and a new token that it sees, per full tree."""
    n, g = c["N"], c["tree"]
    return 1 + (n - 1) // g * (g + g * (g + 1) // 2) if g else n * (n + 1) // 2


def work(case):
    c = case
    if c["op"] == "pages":
        start, count = _lens(c)
        kept = [_ceil(k, c["P"]) for k in _kept(c)]
        taken = sum(max(_ceil(s + n, c["P"]) - k, 0) for s, n, k in zip(start, count, kept))
        # pages: read from the list, written to the table, read again, written back, the place marked
        # tokens: their page's entry, position and slot, their depth in a tree
        n = 20 * taken + sum(count) * 12 + 4 * sum(_ceil(n, c["P"]) for n in count)
        n += c["B"] * (20 + 4 * c["base"]) + (4 * sum(count) if c["tree"] else 0)
        return {"bytes": n, "flops": 4 * sum(count) + 8 * c["B"]}
    if c["op"] == "prefix":
        start, count = _lens(c)
        size = _BYTES[c["dtype"]]
        cell = 2 * c["Hk"] * (c["D"] * _BYTES[c["cache"]] + (c["cache"] == "e4m3"))
        prefix = _prefix_lens(c)
        held = sum(s + n for s, n in zip(start, count)) + sum(prefix)
        n = held * cell + 2 * sum(count) * c["Hq"] * c["D"] * size + 4 * sum(count) * c["Hq"]
        n += 4 * held // c["P"] + 8 * c["B"] + (c["N"] * _ceil(c["N"], 32) * 4 if c["tree"] else 0)
        each = c["B"] // c["groups"]
        pairs = sum((s + prefix[b // each]) * k for b, (s, k) in enumerate(zip(start, count)))
        pairs += c["B"] * _visible(c) if c["tree"] else sum(k * (k + 1) // 2 for k in count)
        return {"bytes": n, "flops": 4 * c["Hq"] * c["D"] * pairs}
    rows = c["B"] * c["per"]
    n = rows * c["V"] * _BYTES[c["dtype"]] * (2 if c["op"] == "truncate" else 1) + 16 * c["B"]
    return {"bytes": n + rows * (4 if c["op"] == "truncate" else 16), "flops": 3 * rows * c["V"]}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _fill(cells, exps, g, gain, dt):
    """Every page filled, quantised where there are powers of two."""
    for p0 in range(0, cells.shape[0], 4096):
        p1 = min(p0 + 4096, cells.shape[0])
        part = (_randn(g, (p1 - p0,) + cells.shape[1:]) * gain).to(dt)
        if exps is not None:
            x = part.float()
            m, e = torch.frexp(x.abs().amax(-1))            # 448 = 0.875 * 2^9
            e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 127)
            part = torch.ldexp(x, -e[..., None]).to(cells.dtype)
            exps[p0:p1] = (e + 127).to(torch.uint8)
        cells[p0:p1].view(torch.uint8).copy_(part.view(torch.uint8))


def _tree_words(N, gamma):
    """Who sees whom in a tree of a root and chains of gamma nodes, as bits of
    32-bit words: node i sees the root and its own chain up to itself."""
    i = torch.arange(N, device="cuda")
    chain = (i - 1) // gamma
    see = (chain[:, None] == chain[None, :]) & (i[None, :] <= i[:, None])
    see |= (i[None, :] == 0)
    see[0, 1:] = False
    W = _ceil(N, 32)
    bits = torch.zeros(N, W * 32, dtype=torch.int64, device="cuda")
    bits[:, :N] = see
    w = (bits.view(N, W, 32) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _prepare_pages(c, g):
    """The state before a step: each sequence holds the pages of what it will
    keep, the others are free, in any order."""
    start, count = _lens(c)
    kept = [_ceil(k, c["P"]) for k in _kept(c)]
    need = [max(_ceil(s + n, c["P"]), k) for s, n, k in zip(start, count, kept)]
    pages = sum(need) + 7
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    given = sum(kept)
    per = _per(c)
    held = _ints(kept)
    place = torch.arange(per, device="cuda")
    before = torch.cumsum(held.long(), 0) - held
    mine = place < held[:, None]
    table = torch.where(mine, order[(before[:, None] + place).clamp(max=pages - 1)], -1)
    free = torch.zeros(pages, dtype=torch.int32, device="cuda")
    free[:pages - given] = order[given:]
    s = {"table": table.contiguous(), "held": held, "list": free, "free": _ints([pages - given]),
         "start": _ints(start), "count": _ints(count), "kept": _ints(_kept(c)), "base": None, "depth": None}
    if c["base"]:
        s["base"] = torch.randint(0, 9000, (c["B"],), generator=g, device="cuda", dtype=torch.int32)
    if c["tree"]:
        i = torch.arange(c["N"], device="cuda")
        depth = torch.where(i == 0, 0, (i - 1) % c["tree"] + 1)
        s["depth"] = depth.to(torch.int32).expand(c["B"], -1).contiguous()
    return s


def _prepare_prefix(c, g):
    dt = _TYPES[c["dtype"]]
    per, ppre = _per(c), _ceil(max(c["phi"], 1), c["P"])
    pages = c["B"] * per + c["groups"] * ppre + 1
    order = torch.randperm(pages - 1, generator=g, device="cuda").to(torch.int32)
    start, count = _lens(c)
    s = {"table": order[:c["B"] * per].view(c["B"], per).contiguous(),
         "prefix_table": order[c["B"] * per:].view(c["groups"], ppre).contiguous(),
         "start": _ints(start), "count": _ints(count), "prefix_len": _ints(_prefix_lens(c))}
    # keys have a few channels that are larger than the others, as trained ones do
    gain = 1 + 3 * (torch.rand(c["D"], generator=g, device="cuda") < 0.05).float()
    e4m3 = c["cache"] == "e4m3"
    shape = (pages, c["Hk"], c["P"], c["D"])
    for name, by in (("k", gain), ("v", 1.0)):
        cells = torch.zeros(shape, dtype=torch.float8_e4m3fn if e4m3 else dt, device="cuda")
        exps = torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") if e4m3 else None
        _fill(cells, exps, g, by, dt)
        s[name + "_cache"], s[name + "_exp"] = cells, exps
    # queries are parts of one projection's output
    qkv = _randn(g, (c["B"], c["N"], c["Hq"] + 2 * c["Hk"], c["D"])).to(dt)
    s["q"] = qkv[:, :, :c["Hq"]]
    s["mask"] = _tree_words(c["N"], c["tree"]) if c["tree"] else None
    return s


def _prepare_rows(c, g):
    B, per, V = c["B"], c["per"], c["V"]
    prior = -1.1 * torch.log1p(torch.arange(V, device="cuda", dtype=torch.float32))
    s = {"logits": torch.empty((B, per, V), dtype=_TYPES[c["dtype"]], device="cuda")}
    for b in range(B):
        s["logits"][b] = (_randn(g, (per, V)) * 3 + prior + 8).to(s["logits"].dtype)
    one = lambda lo, hi: torch.rand(B, generator=g, device="cuda") * (hi - lo) + lo  # noqa: E731
    s["temperature"] = s["top_k"] = s["top_p"] = s["min_p"] = None
    if c["T"]:          # now and then a request that wants the best token alone
        s["temperature"] = torch.where(one(0, 1) < 0.05, 0.0, one(0.5, 1.3))
    if c["k"]:          # 0: not cut
        s["top_k"] = torch.where(one(0, 1) < 0.2, 0, torch.exp(one(0, math.log(300))).round()).to(torch.int32)
    if c["p"]:
        s["top_p"] = torch.where(one(0, 1) < 0.2, 1.0, one(0.5, 0.99))
    if c["m"]:
        s["min_p"] = torch.where(one(0, 1) < 0.2, 0.0, one(0.001, 0.2))
    s["u"] = torch.rand((B, per), generator=g, device="cuda")
    return s


def prepare(case, seed):
    g = _gen(seed)
    make = {"pages": _prepare_pages, "prefix": _prepare_prefix}.get(case["op"], _prepare_rows)
    return {"c": case, **make(case, g)}


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

def _pages(s):
    c, P = s["c"], s["c"]["P"]
    table, held, free = s["table"], s["held"].long(), s["free"].long()
    place = torch.arange(table.shape[1], device="cuda")
    # pages for the step's tokens, from the end of the list
    end = s["start"].long() + s["count"]
    need = (end + P - 1) // P
    take = (need - held).clamp(min=0)
    upto = torch.cumsum(take, 0)
    take = torch.where(upto <= free, take, 0)
    mine = (place >= held[:, None]) & (place < (held + take)[:, None])
    at = free - 1 - ((upto - take)[:, None] + place - held[:, None])
    table.copy_(torch.where(mine, s["list"][at.clamp(0, s["list"].numel() - 1)], table))
    held = held + take
    free = free - take.sum()
    n = torch.arange(c["N"], device="cuda")
    live = n < s["count"][:, None]
    pos = s["start"][:, None].long() + n
    page = table.gather(1, (pos // P).clamp(max=table.shape[1] - 1)).long()
    slots = torch.where(live & (page >= 0), page * P + pos % P, -1)
    positions = pos if s["depth"] is None else s["start"][:, None].long() + s["depth"]
    if s["base"] is not None:
        positions = positions + s["base"][:, None]
    positions = torch.where(live, positions, 0).to(torch.int32)
    # back those behind what is kept, so that the list is as it was
    kept = torch.minimum((s["kept"].long() + P - 1) // P, held)
    give = held - kept
    before = torch.cumsum(give, 0) - give
    mine = (place >= kept[:, None]) & (place < held[:, None])
    top = free + give.sum()
    at = top - 1 - (before[:, None] + place - kept[:, None])
    s["list"][at[mine]] = table[mine]
    table.masked_fill_(mine, -1)
    s["held"].copy_(kept)
    s["free"].copy_(top)
    return {"positions": positions, "slots": slots, "table": table, "held": s["held"], "free": s["free"],
            "list": s["list"]}


def _values(s, name, pages):
    """What the cells of pages [..., n] stand for in 32 bits, [..., Hk, n * P, D]."""
    cells, exps = s[name + "_cache"], s[name + "_exp"]
    pages = pages.long()
    if exps is None:
        x = cells[pages].float()
    else:
        x = cells.view(torch.uint8)[pages].view(cells.dtype).float()
        x = x * ((exps[pages].to(torch.int32)) << 23).view(torch.float32)[..., None]
    x = x.transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _prefix(s):
    c = s["c"]
    B, G, N, Hq, Hk, D, P = (c[n] for n in ("B", "groups", "N", "Hq", "Hk", "D", "P"))
    each, g = B // G, Hq // Hk
    scale = 1 / math.sqrt(D)
    q = s["q"].float().view(B, N, Hk, g, D).permute(0, 2, 3, 1, 4)              # [B, Hk, g, N, D]
    qg = q.reshape(G, each, Hk, g * N, D).transpose(1, 2).reshape(G, Hk, -1, D)
    kp, vp = _values(s, "k", s["prefix_table"]), _values(s, "v", s["prefix_table"])
    Lp = kp.shape[2]
    at = torch.arange(Lp, device="cuda")
    far = (qg @ kp.transpose(-1, -2)) * scale
    far.masked_fill_((at >= s["prefix_len"][:, None])[:, None, None], -math.inf)
    far = far.view(G, Hk, each, g, N, Lp).transpose(1, 2).reshape(B, Hk, g, N, Lp)
    ko, vo = _values(s, "k", s["table"]), _values(s, "v", s["table"])
    L = ko.shape[2]
    near = (q.reshape(B, Hk, g * N, D) @ ko.transpose(-1, -2)).view(B, Hk, g, N, L) * scale
    at = torch.arange(L, device="cuda")
    new = at - s["start"][:, None]                               # [B, L]: which new token this is
    i = torch.arange(N, device="cuda")
    if s["mask"] is None:
        see = new[:, None, :] <= i[:, None]
    else:
        w = new.clamp(0, N - 1)
        see = ((s["mask"][:, w // 32] >> (w % 32)) & 1).bool().transpose(0, 1) | (new < 0)[:, None, :]
    see = see & (new < s["count"][:, None])[:, None, :]
    near.masked_fill_(~see[:, None, None], -math.inf)
    dead = (i >= s["count"][:, None])[:, None, None, :, None]                   # [B, 1, 1, N, 1]
    far.masked_fill_(dead, -math.inf)
    near.masked_fill_(dead, -math.inf)
    top = torch.maximum(far.amax(-1, keepdim=True), near.amax(-1, keepdim=True))
    base = torch.where(top == -math.inf, 0, top)
    far.sub_(base).exp_()
    near.sub_(base).exp_()
    total = far.sum(-1, keepdim=True) + near.sum(-1, keepdim=True)
    out = (near.view(B, Hk, g * N, L) @ vo).view(B, Hk, g, N, D)
    x = far.view(G, each, Hk, g * N, Lp).transpose(1, 2).reshape(G, Hk, -1, Lp) @ vp
    out = out + x.view(G, Hk, each, g, N, D).transpose(1, 2).reshape(B, Hk, g, N, D)
    out = out / torch.where(total == 0, 1, total)
    lse = (top + torch.log(total)).squeeze(-1)
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D).to(s["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(B, N, Hq).contiguous()}


def _chosen(s, r0, r1):
    """Rows r0 .. r1 - 1 in falling order (ties by index): values, indices, whole
    weights and how many are kept."""
    c = s["c"]
    V = c["V"]
    who = torch.arange(r0, r1, device="cuda") // c["per"]
    by = lambda name, off: torch.full((r1 - r0, 1), off, dtype=torch.float64, device="cuda") \
        if s[name] is None else s[name][who].double()[:, None]  # noqa: E731
    x, order = torch.sort(s["logits"].view(-1, V)[r0:r1].float(), dim=-1, descending=True, stable=True)
    T = by("temperature", 1.0)
    fall = x.double() - x[:, :1].double()
    w = torch.where(fall == 0, _ONE, torch.round(torch.exp(fall / T) * _ONE))
    w = torch.where(T == 0, torch.where(fall == 0, _ONE, 0.0), w).long()
    floor = x[:, :1].double() + T * torch.log(by("min_p", 0.0))
    n = ((x > -math.inf) & ((x.double() >= floor) | (by("min_p", 0.0) == 0))).sum(-1, keepdim=True)
    k = by("top_k", 0.0).long()
    n = torch.where(k > 0, torch.minimum(n, k), n)
    at = torch.arange(V, device="cuda")
    w = torch.where(at < n, w, 0)
    upto = torch.cumsum(w, -1)
    p = by("top_p", 1.0)
    under = ((upto - w).double() < p * upto[:, -1:].double()) & (at < n)
    n = torch.where(p < 1, torch.minimum(n, under.sum(-1, keepdim=True)), n)
    n = torch.where(T == 0, 1, n)
    return x, order, torch.where(at < n, w, 0), n


_ROWS = 64          # rows that the plain form holds in 64 bits at once


def _sample(s):
    rows = s["u"].numel()
    out = {"token": torch.empty(rows, dtype=torch.int32, device="cuda"),
           "logprob": torch.empty(rows, dtype=torch.float32, device="cuda")}
    for r0 in range(0, rows, _ROWS):
        r1 = min(r0 + _ROWS, rows)
        x, order, w, _ = _chosen(s, r0, r1)
        upto = torch.cumsum(w, -1)
        aim = (s["u"].view(-1)[r0:r1].double()[:, None] * upto[:, -1:].double()).long()
        at = torch.searchsorted(upto, aim, right=True)
        out["token"][r0:r1] = order.gather(-1, at).squeeze(-1).to(torch.int32)
        part = w.gather(-1, at).double() / upto[:, -1:].double()
        out["logprob"][r0:r1] = torch.log(part).squeeze(-1).float()
    return {n: t.view(s["u"].shape) for n, t in out.items()}


def _truncate(s):
    rows, V = s["u"].numel(), s["c"]["V"]
    flat = s["logits"].view(-1, V)
    out = torch.empty_like(flat)
    kept = torch.empty(rows, dtype=torch.int32, device="cuda")
    for r0 in range(0, rows, _ROWS):
        r1 = min(r0 + _ROWS, rows)
        _, order, _, n = _chosen(s, r0, r1)
        keep = torch.zeros_like(order, dtype=torch.bool)
        keep.scatter_(1, order, torch.arange(V, device="cuda") < n)
        out[r0:r1] = flat[r0:r1].masked_fill(~keep, -math.inf)
        kept[r0:r1] = n.squeeze(-1).to(torch.int32)
    return {"out": out.view(s["logits"].shape), "kept": kept.view(s["u"].shape)}


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(state):
    s, op = state, state["c"]["op"]
    if own:
        return _own(s, op)
    return {"pages": _pages, "prefix": _prefix, "sample": _sample, "truncate": _truncate}[op](s)


def _own(s, op):
    from draft_verification_sdv_gb300 import binding as bd
    c = s["c"]
    if op == "pages":
        positions, slots = bd.sdv_pages_extend(s["list"], s["free"], s["table"], s["held"], s["start"],
                                               c["N"], c["P"], count=s["count"], depth=s["depth"],
                                               base=s["base"])
        bd.sdv_pages_release(s["list"], s["free"], s["table"], s["held"], s["kept"], c["P"])
        return {"positions": positions, "slots": slots, "table": s["table"], "held": s["held"],
                "free": s["free"], "list": s["list"]}
    if op == "prefix":
        out, lse = bd.sdv_prefix_attn(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"],
                                      s["prefix_len"], s["table"], s["start"], count=s["count"],
                                      mask=s["mask"], k_exp=s["k_exp"], v_exp=s["v_exp"], lse=True)
        return {"out": out, "lse": lse}
    cut = dict(temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    if op == "sample":
        token, logprob = bd.sdv_sample(s["logits"], s["u"], logprob=True, **cut)
        return {"token": token, "logprob": logprob}
    out, kept = bd.sdv_logits_truncate(s["logits"], kept=True, **cut)
    return {"out": out, "kept": kept}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_pages(c, s):
    """The list as a stack, a sequence after the other."""
    P = c["P"]
    table, held = s["table"].tolist(), s["held"].tolist()
    start, count, kept = s["start"].tolist(), s["count"].tolist(), s["kept"].tolist()
    base = s["base"].tolist() if c["base"] else [0] * c["B"]
    whole, free = s["list"].tolist(), s["free"].item()
    stack = whole[:free]
    wanted = 0
    for b in range(c["B"]):
        more = max(_ceil(start[b] + count[b], P) - held[b], 0)
        wanted += more
        if wanted <= free:
            for _ in range(more):
                table[b][held[b]] = stack.pop()
                held[b] += 1
    n = torch.arange(c["N"])
    positions = torch.zeros((c["B"], c["N"]), dtype=torch.int32)
    slots = torch.full((c["B"], c["N"]), -1, dtype=torch.int64)
    for b in range(c["B"]):
        at = start[b] + n[:count[b]]
        page = torch.tensor(table[b], dtype=torch.int64)[at // P]
        slots[b, :count[b]] = torch.where(page < 0, -1, page * P + at % P)
        step = s["depth"][b, :count[b]].cpu() if c["tree"] else n[:count[b]]
        positions[b, :count[b]] = (base[b] + start[b] + step).to(torch.int32)
    for b in range(c["B"] - 1, -1, -1):
        while held[b] > _ceil(kept[b], P):
            held[b] -= 1
            stack.append(table[b][held[b]])
            table[b][held[b]] = -1
    whole[:len(stack)] = stack
    return {"positions": positions.cuda(), "slots": slots.cuda(), "table": _ints(table), "held": _ints(held),
            "free": _ints([len(stack)]), "list": _ints(whole)}


def _exact_cells(s, name, pages, n):
    """The first n positions on these pages, [n, Hk, D] in 64 bits."""
    cells = s[name + "_cache"]
    pages = pages[:_ceil(n, cells.shape[2])].long()
    x = cells.view(torch.uint8)[pages].view(cells.dtype).double() if cells.element_size() == 1 \
        else cells[pages].double()
    if s[name + "_exp"] is not None:
        x = x * torch.exp2(s[name + "_exp"][pages].double() - 127)[..., None]
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:n]


def _exact_prefix(c, s):
    B, N, Hq, Hk, D = (c[n] for n in ("B", "N", "Hq", "Hk", "D"))
    (start, count), prefix, each = _lens(c), _prefix_lens(c), B // c["groups"]
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n, held, far = count[b], start[b] + count[b], prefix[b // each]
        if b % each == 0:
            kp, vp = (_exact_cells(s, x, s["prefix_table"][b // each], far) for x in ("k", "v"))
        see = torch.ones((n, far + held), dtype=torch.bool, device="cuda")
        i, j = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")
        if c["tree"]:
            same = (i - 1) // c["tree"] == (j - 1) // c["tree"]
            see[:, far + start[b]:] = (j == 0) | (same & (j <= i) & (i > 0))
        else:
            see[:, far + start[b]:] = j <= i
        k = torch.cat((kp, _exact_cells(s, "k", s["table"][b], held)))
        v = torch.cat((vp, _exact_cells(s, "v", s["table"][b], held)))
        for h in range(Hk):
            mine = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            x = torch.einsum("ngd,ld->ngl", s["q"][b, :n, mine].double(), k[:, h]) / math.sqrt(D)
            x.masked_fill_(~see[:, None], -math.inf)
            lse[b, :n, mine] = torch.logsumexp(x, -1)
            out[b, :n, mine] = torch.einsum("ngl,ld->ngd", torch.softmax(x, -1), v[:, h])
    return {"out": out, "lse": lse}


def _exact_rows(c, s):
    """A row's values from the largest down, each with the places where it
    stands, until the kept ones are counted."""
    rows, V = c["B"] * c["per"], c["V"]
    flat = s["logits"].view(-1, V)
    asked = {n: None if s[n] is None else s[n].double().tolist()
             for n in ("temperature", "top_k", "top_p", "min_p")}
    token = torch.zeros(rows, dtype=torch.int32)
    logprob = torch.zeros(rows, dtype=torch.float64)
    kept = torch.zeros(rows, dtype=torch.int32)
    out = torch.full((rows, V), -math.inf, dtype=torch.float64, device="cuda") if c["op"] == "truncate" else None
    u = s["u"].view(-1).double().tolist()
    for r in range(rows):
        T, k, p, m = (None if asked[n] is None else asked[n][r // c["per"]]
                      for n in ("temperature", "top_k", "top_p", "min_p"))
        T = 1.0 if T is None else T
        x = flat[r].double()
        value, count = torch.unique(x, return_counts=True)
        value, count = value.flip(0), count.flip(0)
        best = value[0].item()
        if T == 0:
            limit, weight = 1, torch.full_like(value, _ONE).long()
        else:
            weight = torch.round(torch.exp2((value - best) / (T * math.log(2)) + 44)).long()
            limit = int(count[value >= best + T * math.log(m)].sum()) if m else V
            limit = min(limit, int(k)) if k else limit
        share = (limit - (torch.cumsum(count, 0) - count)).clamp(min=0).minimum(count)
        upto = torch.cumsum(share * weight, 0)
        if p is not None and p < 1 and T != 0:
            bound = math.ceil(p * float(upto[-1].item()))
            left = bound - (upto - share * weight)
            share = ((left + weight.clamp(min=1) - 1) // weight.clamp(min=1)).clamp(min=0).minimum(share)
            upto = torch.cumsum(share * weight, 0)
        kept[r] = int(share.sum())
        if out is not None:
            last = int((share > 0).sum()) - 1
            out[r] = torch.where(x > value[last], x, -math.inf)
            at = torch.nonzero(x == value[last])[:int(share[last]), 0]
            out[r, at] = x[at]
            continue
        total = upto[-1].item()
        aim = int(u[r] * float(total))
        i = int((upto <= aim).sum())
        j = (aim - (upto[i] - share[i] * weight[i]).item()) // weight[i].item()
        token[r] = int(torch.nonzero(x == value[i])[j, 0])
        logprob[r] = math.log(weight[i].item() / total)
    shape = (c["B"], c["per"])
    if out is not None:
        return {"out": out.view(c["B"], c["per"], V), "kept": kept.view(shape).cuda()}
    return {"token": token.view(shape).cuda(), "logprob": logprob.view(shape).cuda()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"pages": _exact_pages, "prefix": _exact_prefix}.get(case["op"], _exact_rows)(case, s)

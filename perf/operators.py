"""What the operators around a verification step are measured on.

A verifier that scores a tree of drafted tokens rotates its queries and keys
(`rope`), writes the new keys and values into a paged cache (`kv_write`), reads
them back (`kv_read`), attends from every node of the tree to the cache
(`attn`) and adjusts the logits of every draft position (`logits`).  Each case
is one call of one of these, at the sizes of a decode loop.

`run` computes a case in its plain form (elementary torch operations in 32
bits) or, where `own` is true, by the library's own entry points; `exact`
states the same definition in 64 bits.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one sequence's next token: both projections of one position
        {"name": "rope one token", "op": "rope", "T": 1, "Hq": 64, "Hk": 8, "D": 128, "R": 128,
         "interleaved": False, "far": 4000, "dtype": "bf16"},
        # the flattened drafts of a large-window batch at far positions
        {"name": "rope large window", "op": "rope", "T": 16416, "Hq": 64, "Hk": 8, "D": 128,
         "R": 128, "interleaved": False, "far": 131000, "dtype": "bf16"},
        # the drafts of a self-selection batch, kept in their own type
        {"name": "kv write drafts", "op": "kv_write", "B": 8, "N": 65, "Hk": 8, "D": 128, "P": 16,
         "lo": 0, "hi": 1000, "dtype": "bf16", "cache": "bf16"},
        # a prompt's keys and values, quantised on the way in
        {"name": "kv write prompt e4m3", "op": "kv_write", "B": 8, "N": 4099, "Hk": 8, "D": 128,
         "P": 64, "lo": 0, "hi": 3, "dtype": "bf16", "cache": "e4m3"},
        # prefixes read back from a quantised cache (to move or to inspect them)
        {"name": "kv read e4m3", "op": "kv_read", "B": 8, "N": 2000, "Hk": 8, "D": 128, "P": 16,
         "lo": 0, "hi": 900, "dtype": "bf16", "cache": "e4m3"},
        # one sequence, one new token: the plain decode step, latency-bound
        {"name": "attn one token", "op": "attn", "B": 1, "N": 1, "Hq": 64, "Hk": 8, "D": 128,
         "P": 16, "lo": 2047, "hi": 2047, "tree": 0, "dtype": "bf16", "cache": "bf16"},
        # a serving batch of single tokens with ragged long prefixes
        {"name": "attn decode ragged e4m3", "op": "attn", "B": 64, "N": 1, "Hq": 64, "Hk": 8,
         "D": 128, "P": 64, "lo": 1000, "hi": 32000, "tree": 0, "dtype": "bf16", "cache": "e4m3"},
        # the trees of a self-selection batch: a root and 4 drafts of 16
        {"name": "attn tree 4x16", "op": "attn", "B": 8, "N": 65, "Hq": 64, "Hk": 8, "D": 128,
         "P": 16, "lo": 500, "hi": 8000, "tree": 16, "dtype": "bf16", "cache": "bf16"},
        # the trees of a large-window batch: a root and 16 drafts of 32
        {"name": "attn tree 16x32", "op": "attn", "B": 16, "N": 513, "Hq": 64, "Hk": 8, "D": 128,
         "P": 32, "lo": 1500, "hi": 3500, "tree": 32, "dtype": "bf16", "cache": "bf16"},
        # a chunk of a prompt: a causal chain of many tokens, small heads
        {"name": "attn chunk fp16", "op": "attn", "B": 3, "N": 1900, "Hq": 32, "Hk": 8, "D": 64,
         "P": 16, "lo": 0, "hi": 4100, "tree": 0, "dtype": "fp16", "cache": "fp16"},
        # a single stream's draft, no grammar
        {"name": "logits single stream", "op": "logits", "B": 1, "K": 1, "G": 8, "V": 152064,
         "M": 20, "allow": False, "tree": False, "dtype": "bf16"},
        # a serving batch under a grammar, rows taken from the tree's logits
        {"name": "logits serving grammar", "op": "logits", "B": 32, "K": 8, "G": 16, "V": 152064,
         "M": 300, "allow": True, "tree": True, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(["rope", "kv_write", "kv_read", "attn", "attn", "attn", "logits"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    D = rng.choice([64, 128, 128, 96])
    Hk = rng.choice([1, 2, 4, 8])
    if op == "rope":
        return {"op": op, "T": _log(rng, 1, 16000), "Hq": Hk * rng.choice([1, 3, 7, 8]), "Hk": Hk,
                "D": D, "R": rng.choice([D, D, D // 2]), "interleaved": rng.random() < 0.4,
                "far": _log(rng, 100, 1000000), "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op in ("kv_write", "kv_read"):
        lo = _log(rng, 1, 500) - 1
        return {"op": op, "B": _log(rng, 1, 32), "N": _log(rng, 1, 4000), "Hk": Hk, "D": D,
                "P": rng.choice([16, 32, 64, 128]), "lo": lo, "hi": lo + _log(rng, 1, 900),
                "dtype": dtype, "cache": rng.choice([dtype, "e4m3"])}
    if op == "attn":
        kind = rng.choice(["token", "tree", "tree", "chunk"])
        gamma = rng.choice([4, 8, 15, 16, 32])
        N = 1 if kind == "token" else \
            1 + gamma * rng.randint(1, 16) if kind == "tree" else _log(rng, 2, 2000)
        lo = _log(rng, 1, 8000) - 1
        return {"op": op, "B": _log(rng, 1, 64), "N": N, "Hq": Hk * rng.choice([1, 4, 7, 8]),
                "Hk": Hk, "D": D, "P": rng.choice([16, 32, 64, 128]), "lo": lo,
                "hi": lo + _log(rng, 1, 24000 if N == 1 else 6000),
                "tree": gamma if kind == "tree" else 0, "dtype": dtype,
                "cache": rng.choice([dtype, "e4m3"])}
    return {"op": op, "B": _log(rng, 1, 48), "K": rng.choice([1, 3, 4, 8, 16]), "G": rng.randint(1, 32),
            "V": 8 * _log(rng, 500, 19008), "M": rng.choice([0, 7, 300]), "allow": rng.random() < 0.5,
            "tree": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "fp32"])}


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
    """Values that the plain form holds at once."""
    if c["op"] == "attn":
        L = c["hi"] + c["N"] + c["P"]
        return c["B"] * L * (2 * c["Hk"] * c["D"] + 2 * c["Hq"] * c["N"])
    if c["op"] == "logits":
        return c["B"] * c["K"] * (c["G"] + 1) * c["V"]
    return 0


def _lens(c):
    """Each sequence's tokens in the cache and new tokens, from the case alone."""
    r = random.Random("%d %d %d %d" % (c["B"], c["N"], c["lo"], c["hi"]))
    start = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    whole = c["N"] == 1 or c["op"] == "attn" and c["tree"]
    count = [c["N"] if whole or b == 0 else r.randint((c["N"] + 1) // 2, c["N"])
             for b in range(c["B"])]
    return start, count


def _pages(c):
    """(pages of the cache, pages a sequence's row of the table holds): the
    last page belongs to no sequence."""
    per = -(-(c["hi"] + c["N"]) // c["P"])
    return c["B"] * per + 1, per


def _visible(c):
    """Pairs of a new token and a new token that it sees, per full tree."""
    n, g = c["N"], c["tree"]
    return 1 + (n - 1) // g * (g + g * (g + 1) // 2) if g else n * (n + 1) // 2


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": 2 * n * _BYTES[c["dtype"]] + 4 * c["T"] + 2 * c["R"],
                "flops": 3 * c["T"] * (c["Hq"] + c["Hk"]) * c["R"]}
    if c["op"] == "logits":
        rows = c["B"] * c["K"] * (c["G"] + 1)
        src = c["B"] * (1 + c["K"] * c["G"]) if c["tree"] else rows
        n = (src + rows) * c["V"] * _BYTES[c["dtype"]] + c["B"] * c["V"] * 4 + c["B"] * c["V"] // 8
        n += rows * (c["V"] // 8) * c["allow"] + c["B"] * (8 * c["M"] + 4 * c["K"] * c["G"] + 12)
        return {"bytes": n, "flops": 4 * rows * c["V"]}
    start, count = _lens(c)
    cell = 2 * c["Hk"] * (c["D"] * _BYTES[c["cache"]] + (c["cache"] == "e4m3"))
    if c["op"] in ("kv_write", "kv_read"):
        rows = sum(count)
        given = rows if c["op"] == "kv_write" else c["B"] * c["N"]
        return {"bytes": rows * cell + 2 * given * c["Hk"] * c["D"] * _BYTES[c["dtype"]] + 8 * c["B"],
                "flops": 2 * rows * c["Hk"] * c["D"]}
    held = sum(s + n for s, n in zip(start, count))
    size = _BYTES[c["dtype"]]
    n = held * cell + 2 * sum(count) * c["Hq"] * c["D"] * size + 4 * sum(count) * c["Hq"]
    n += 4 * held // c["P"] + 8 * c["B"] + (c["N"] * -(-c["N"] // 32) * 4 if c["tree"] else 0)
    pairs = sum(s * k for s, k in zip(start, count))
    pairs += c["B"] * _visible(c) if c["tree"] else sum(k * (k + 1) // 2 for k in count)
    return {"bytes": n, "flops": 4 * c["Hq"] * c["D"] * pairs}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _frequencies(R, far):
    """Rotary frequencies; past 8192 positions the slow ones are slowed down
    further and the fast ones left, with a ramp between them."""
    i = torch.arange(0, R, 2, dtype=torch.float64)
    f = 10000.0 ** (-i / R)
    if far > 8192:
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f = f * keep + f / (far / 8192) * (1 - keep)
    return f.to(torch.float32).cuda()


def _prepare_cells(c, g):
    """Tables, lengths and a cache with every page filled."""
    pages, per = _pages(c)
    dt = _TYPES[c["dtype"]]
    shape = (pages, c["Hk"], c["P"], c["D"])
    s = {}
    order = torch.randperm(pages - 1, generator=g, device="cuda").to(torch.int32)
    s["table"] = order.view(c["B"], per).contiguous()
    start, count = _lens(c)
    s["start"], s["count"] = _ints(start), _ints(count)
    # keys have a few channels that are larger than the others, as trained ones do
    gain = 1 + 3 * (torch.rand(c["D"], generator=g, device="cuda") < 0.05).float()
    e4m3 = c["cache"] == "e4m3"
    for name, by in (("k", gain), ("v", 1.0)):
        cells = torch.zeros(shape, dtype=torch.float8_e4m3fn if e4m3 else dt, device="cuda")
        exps = torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") if e4m3 else None
        for p0 in range(0, pages if c["op"] != "kv_write" else 0, 4096):
            p1 = min(p0 + 4096, pages)
            part = (_randn(g, (p1 - p0,) + shape[1:], torch.float32) * by).to(dt)
            if e4m3:
                part, exps[p0:p1] = _quantise(part)
            cells[p0:p1].view(torch.uint8).copy_(part.view(torch.uint8))
        s[name + "_cache"], s[name + "_exp"] = cells, exps
    return s


def _tree_words(N, gamma):
    """Who sees whom in a tree of a root and chains of gamma nodes, as bits of
    32-bit words: node i sees the root and its own chain up to itself."""
    i = torch.arange(N, device="cuda")
    chain = (i - 1) // gamma
    see = (chain[:, None] == chain[None, :]) & (i[None, :] <= i[:, None])
    see |= (i[None, :] == 0)
    see[0, 1:] = False
    W = -(-N // 32)
    bits = torch.zeros(N, W * 32, dtype=torch.int64, device="cuda")
    bits[:, :N] = see
    w = (bits.view(N, W, 32) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    dt = _TYPES[c["dtype"]]
    if c["op"] == "rope":
        # queries and keys are parts of one projection's output
        qkv = _randn(g, (c["T"], (c["Hq"] + 2 * c["Hk"]) * c["D"]), dt)
        s["q"] = qkv[:, :c["Hq"] * c["D"]].view(c["T"], c["Hq"], c["D"])
        s["k"] = qkv[:, c["Hq"] * c["D"]:-c["Hk"] * c["D"]].view(c["T"], c["Hk"], c["D"])
        s["pos"] = torch.randint(0, c["far"], (c["T"],), generator=g, device="cuda", dtype=torch.int32)
        s["freq"] = _frequencies(c["R"], c["far"])
        s["factor"] = 1.0 if c["far"] <= 8192 else 0.1 * math.log(c["far"] / 8192) + 1.0
        return s
    if c["op"] == "logits":
        B, K, G, V = c["B"], c["K"], c["G"], c["V"]
        src = (B, 1 + K * G, V) if c["tree"] else (B, K, G + 1, V)
        prior = -1.1 * torch.log1p(torch.arange(V, device="cuda", dtype=torch.float32))
        s["logits"] = torch.empty(src, dtype=dt, device="cuda")
        for b in range(B):
            s["logits"][b] = (torch.randn(src[1:], generator=g, device="cuda") * 3 + prior + 8).to(dt)
        s["rows"] = None
        if c["tree"]:       # row j of draft k is the one of its token j - 1; row 0 is the root's
            rows = 1 + torch.arange(K, device="cuda")[:, None] * G + torch.arange(-1, G, device="cuda")
            rows[:, 0] = 0
            s["rows"] = rows.to(torch.int32).expand(B, K, G + 1).contiguous()
        u = torch.rand((B, 400), generator=g, device="cuda")
        said = (torch.exp(u * math.log(V)) - 1).long().clamp(0, V - 1)
        s["counts"] = torch.zeros((B, V), dtype=torch.int32, device="cuda")
        s["counts"].scatter_add_(1, said, torch.ones_like(said, dtype=torch.int32))
        words = -(-V // 32)
        s["prompt"] = _ints([1 << (i % 31) for i in range(words)]).repeat(B, 1)
        s["prompt"] *= (torch.rand((B, words), generator=g, device="cuda") < 0.1).int()
        s["drafts"] = (torch.exp(torch.rand((B, K, G), generator=g, device="cuda") * math.log(V)) - 1
                       ).clamp(0, V - 1).to(torch.int32)
        one = lambda lo, hi: torch.rand(B, generator=g, device="cuda") * (hi - lo) + lo  # noqa: E731
        s["repetition"], s["frequency"], s["presence"] = one(1.0, 1.3), one(0.0, 0.5), one(0.0, 0.5)
        s["ids"] = s["bias"] = s["allow"] = None
        if c["M"]:
            s["ids"] = torch.stack([torch.randperm(V, generator=g, device="cuda")[:c["M"]]
                                    for _ in range(B)]).to(torch.int32)
            s["bias"] = torch.randn((B, c["M"]), generator=g, device="cuda") * 4
        if c["allow"]:
            shape = (B, K, G + 1, words)
            a = torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device="cuda", dtype=torch.int32)
            # a grammar leaves little at most positions and everything at some
            free = torch.rand(shape[:3], generator=g, device="cuda") < 0.3
            few = torch.rand(shape, generator=g, device="cuda") < 0.02
            s["allow"] = torch.where(free[..., None], -1, torch.where(few, a, 0)).to(torch.int32)
        return s
    s.update(_prepare_cells(c, g))
    if c["op"] == "kv_write":
        qkv = _randn(g, (c["B"], c["N"], 3, c["Hk"], c["D"]), dt)
        s["k"], s["v"] = qkv[:, :, 1], qkv[:, :, 2]
    if c["op"] == "attn":
        s["q"] = _randn(g, (c["B"], c["N"], c["Hq"], c["D"]), dt)
        s["mask"] = _tree_words(c["N"], c["tree"]) if c["tree"] else None
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

def _power(e):
    """2^e in fp32 for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """Rows of x in e4m3 with one power of two a row: the smallest one that
    brings the row's largest value to at most 448, no less than 2^-126.  Returns the values and the
    exponents + 127."""
    x = x.float()
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(top == 0, -126, torch.where(m <= 0.875, e - 9, e - 8)).clamp(-126, 127)
    q = (x * _power(-e)[..., None]).to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8)


def _values(cells, exps):
    """What cells stand for, in 32 bits."""
    x = cells.float()
    return x if exps is None else x * _power(exps.to(torch.int32) - 127)[..., None]


def _where(s, n):
    """Page and place of the first n positions from `start` on, [B, n] each."""
    P, table = s["c"]["P"], s["table"]
    at = s["start"][:, None].long() + torch.arange(n, device="cuda")
    return table.long().gather(1, (at // P).clamp(max=table.shape[1] - 1)), at % P


def _rope(s):
    c, half = s["c"], s["c"]["R"] // 2
    angle = s["pos"].double()[:, None] * s["freq"].double()
    cos = (torch.cos(angle) * s["factor"]).float()[:, None]
    sin = (torch.sin(angle) * s["factor"]).float()[:, None]

    def turn(x):
        y = x.float()
        r = y[..., :c["R"]]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
        ra, rb = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((ra, rb), -1).flatten(-2) if c["interleaved"] else torch.cat((ra, rb), -1)
        return torch.cat((r, y[..., c["R"]:]), -1).to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _kv_write(s):
    c = s["c"]
    page, off = _where(s, c["N"])
    spare = s["k_cache"].shape[0] - 1
    dead = torch.arange(c["N"], device="cuda") >= s["count"][:, None]
    page = torch.where(dead, spare, page)
    out = {}
    for name in ("k", "v"):
        cache, exps = s[name + "_cache"], s[name + "_exp"]
        if exps is None:
            cache[page, :, off] = s[name]
        else:
            q, e = _quantise(s[name])
            cache.view(torch.uint8)[page, :, off] = q.view(torch.uint8)
            exps[page, :, off] = e
            out[name + "_exp"] = exps[:-1]
        out[name + "_cache"] = cache[:-1]
    return out


def _kv_read(s):
    c = s["c"]
    page, off = _where(s, c["N"])
    dead = (torch.arange(c["N"], device="cuda") >= s["count"][:, None])[..., None, None]
    out = {}
    for name in ("k", "v"):
        cells, exps = s[name + "_cache"], s[name + "_exp"]
        x = cells[page, :, off] if exps is None else cells.view(torch.uint8)[page, :, off].view(cells.dtype)
        x = _values(x, None if exps is None else exps[page, :, off])
        out[name] = torch.where(dead, 0, x).to(_TYPES[c["dtype"]])
    return out


def _attn(s):
    c, table = s["c"], s["table"]
    B, N, Hq, Hk, D, P = (c[n] for n in ("B", "N", "Hq", "Hk", "D", "P"))
    L = table.shape[1] * P

    def rows(name):
        cells, exps = s[name + "_cache"], s[name + "_exp"]
        x = cells[table.long()] if exps is None else \
            cells.view(torch.uint8)[table.long()].view(cells.dtype)
        x = _values(x, None if exps is None else exps[table.long()])
        return x.transpose(1, 2).reshape(B, Hk, L, D)

    q = s["q"].float().view(B, N, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    score = (q @ rows("k").transpose(-1, -2)).view(B, Hk, Hq // Hk, N, L) * (1 / math.sqrt(D))
    at = torch.arange(L, device="cuda")
    new = at - s["start"][:, None]                               # [B, L]: which new token this is
    i = torch.arange(N, device="cuda")
    if s["mask"] is None:
        see = new[:, None, :] <= i[:, None]
    else:
        near = new.clamp(0, N - 1)
        see = ((s["mask"][:, near // 32] >> (near % 32)) & 1).bool().transpose(0, 1)
        see = see | (new < 0)[:, None, :]
    see = see & (new < s["count"][:, None])[:, None, :] & (i < s["count"][:, None])[..., None]
    score.masked_fill_(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score = torch.exp(score - torch.where(top == -math.inf, 0, top))
    total = score.sum(-1, keepdim=True)
    out = (score.view(B, Hk, -1, L) @ rows("v")).view(B, Hk, Hq // Hk, N, D)
    out = out / torch.where(total == 0, 1, total)
    lse = (top + torch.log(total)).squeeze(-1)
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D).to(s["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(B, N, Hq).contiguous()}


def _bits(words, V):
    v = torch.arange(V, device="cuda")
    return ((words[..., v // 32] >> (v % 32).int()) & 1).bool()


def _logits(s):
    c = s["c"]
    B, K, G, V = (c[n] for n in ("B", "K", "G", "V"))
    x = s["logits"]
    if s["rows"] is not None:
        x = x[torch.arange(B, device="cuda")[:, None, None], s["rows"].long()]
    x = x.float()
    count = s["counts"][:, None, None].expand(B, K, G + 1, V).clone()
    before = torch.arange(G, device="cuda") < torch.arange(G + 1, device="cuda")[:, None]
    count.scatter_add_(-1, s["drafts"].long()[:, :, None].expand(B, K, G + 1, G),
                       before.int().expand(B, K, G + 1, G))
    seen = (count > 0) | _bits(s["prompt"], V)[:, None, None]
    by = lambda name: s[name].view(B, 1, 1, 1)  # noqa: E731
    x = torch.where(seen, torch.where(x > 0, x / by("repetition"), x * by("repetition")), x)
    x = x - by("frequency") * count - by("presence") * (count > 0)
    if s["ids"] is not None:
        x = x + torch.zeros((B, V), device="cuda").scatter_add_(1, s["ids"].long(), s["bias"])[:, None, None]
    if s["allow"] is not None:
        x = x.masked_fill(~_bits(s["allow"], V), -math.inf)
    return x.to(s["logits"].dtype)


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(state):
    s, op = state, state["c"]["op"]
    if own:
        return _own(s, op)
    return {"rope": _rope, "kv_write": _kv_write, "kv_read": _kv_read, "attn": _attn,
            "logits": _logits}[op](s)


def _own(s, op):
    from draft_verification_sdv_gb300 import binding as bd
    c = s["c"]
    if op == "rope":
        q, k = bd.sdv_rope(s["q"], s["k"], s["pos"], s["freq"], factor=s["factor"],
                           interleaved=c["interleaved"])
        return {"q": q, "k": k}
    if op == "kv_write":
        bd.sdv_kv_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["start"],
                        count=s["count"], k_exp=s["k_exp"], v_exp=s["v_exp"])
        out = {"k_cache": s["k_cache"][:-1], "v_cache": s["v_cache"][:-1]}
        if s["k_exp"] is not None:
            out["k_exp"], out["v_exp"] = s["k_exp"][:-1], s["v_exp"][:-1]
        return out
    if op == "kv_read":
        k, v = bd.sdv_kv_read(s["k_cache"], s["v_cache"], s["table"], s["start"], c["N"],
                              count=s["count"], k_exp=s["k_exp"], v_exp=s["v_exp"],
                              dtype=_TYPES[c["dtype"]])
        return {"k": k, "v": v}
    if op == "attn":
        out, lse = bd.sdv_tree_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["start"],
                                    count=s["count"], mask=s["mask"], k_exp=s["k_exp"],
                                    v_exp=s["v_exp"], lse=True)
        return {"out": out, "lse": lse}
    return bd.sdv_logits_process(s["logits"], s["drafts"], counts=s["counts"], prompt=s["prompt"],
                                 repetition=s["repetition"], frequency=s["frequency"],
                                 presence=s["presence"], bias_ids=s["ids"], bias=s["bias"],
                                 allow=s["allow"], rows=s["rows"])


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _grid_values():
    """The finite values of e4m3 from zero up, by its definition."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")


def _exact_cells(x):
    """Rows of x quantised: the values in units of their row's power of two,
    and that power."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 448))
    e = torch.where(top / 448 > torch.exp2(e), e + 1, e)
    e = torch.where(top / 448 <= torch.exp2(e - 1), e - 1, e).clamp(min=-126)
    grid = _grid_values()
    y = x.abs() / torch.exp2(e)
    up = torch.searchsorted(grid, y).clamp(max=126)
    down = (up - 1).clamp(min=0)
    far_up, far_down = grid[up] - y, y - grid[down]
    at = torch.where((far_up < far_down) | ((far_up == far_down) & (up % 2 == 0)), up, down)
    return grid[at] * torch.sign(x), e.squeeze(-1)


def _exact_rows(s, name, b, n):
    """The first n positions of sequence b, [n, Hk, D] in 64 bits."""
    P = s["c"]["P"]
    pages = s["table"][b, :-(-n // P)].long()
    cells = s[name + "_cache"]
    x = cells.view(torch.uint8)[pages].view(cells.dtype).double() if cells.element_size() == 1 \
        else cells[pages].double()
    if s[name + "_exp"] is not None:
        x = x * torch.exp2(s[name + "_exp"][pages].double() - 127)[..., None]
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:n]


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "rope":
        turn = torch.polar(torch.full((), float(s["factor"]), dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None, None] * s["freq"].double())
        out = {}
        for name in ("q", "k"):
            y = s[name].double().clone()
            r = y[..., :c["R"]].clone()
            pair = r.unflatten(-1, (-1, 2)) if c["interleaved"] else r.unflatten(-1, (2, -1)).transpose(-1, -2)
            z = torch.view_as_real(torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous()) * turn)
            y[..., :c["R"]] = (z if c["interleaved"] else z.transpose(-1, -2)).flatten(-2)
            out[name] = y
        return out
    start, count = _lens(c) if op != "logits" else (None, None)
    if op == "kv_write":
        out = {}
        for name in ("k", "v"):
            cells = s[name + "_cache"].double()
            x, e = _exact_cells(s[name]) if c["cache"] == "e4m3" else (s[name].double(), None)
            for b in range(c["B"]):
                at = start[b] + torch.arange(count[b], device="cuda")
                page = s["table"][b].long()[at // c["P"]]
                cells[page, :, at % c["P"]] = x[b, :count[b]]
                if e is not None:
                    s[name + "_exp"][page, :, at % c["P"]] = (e[b, :count[b]] + 127).to(torch.uint8)
            out[name + "_cache"] = cells[:-1]
            if e is not None:
                out[name + "_exp"] = s[name + "_exp"][:-1]
        return out
    if op == "kv_read":
        out = {n: torch.zeros((c["B"], c["N"], c["Hk"], c["D"]), dtype=torch.float64, device="cuda")
               for n in ("k", "v")}
        for name, t in out.items():
            for b in range(c["B"]):
                t[b, :count[b]] = _exact_rows(s, name, b, start[b] + count[b])[start[b]:]
        return out
    if op == "attn":
        B, N, Hq, Hk, D = (c[n] for n in ("B", "N", "Hq", "Hk", "D"))
        out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device="cuda")
        lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            n, held = count[b], start[b] + count[b]
            see = torch.ones((n, held), dtype=torch.bool, device="cuda")
            i, j = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")
            if c["tree"]:
                same = (i - 1) // c["tree"] == (j - 1) // c["tree"]
                see[:, start[b]:] = (j == 0) | (same & (j <= i) & (i > 0))
            else:
                see[:, start[b]:] = j <= i
            k, v = _exact_rows(s, "k", b, held), _exact_rows(s, "v", b, held)
            for h in range(Hk):
                mine = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
                x = torch.einsum("ngd,ld->ngl", s["q"][b, :n, mine].double(), k[:, h]) / math.sqrt(D)
                x.masked_fill_(~see[:, None], -math.inf)
                lse[b, :n, mine] = torch.logsumexp(x, -1)
                out[b, :n, mine] = torch.einsum("ngl,ld->ngd", torch.softmax(x, -1), v[:, h])
        return {"out": out, "lse": lse}
    B, K, G, V = (c[n] for n in ("B", "K", "G", "V"))
    out = torch.empty((B, K, G + 1, V), dtype=torch.float64, device="cuda")
    word = lambda w: ((w[..., None] >> torch.arange(32, device="cuda")) & 1).flatten(-2)[..., :V] != 0  # noqa: E731
    for b in range(B):
        prompt = word(s["prompt"][b])
        bias = torch.zeros(V, dtype=torch.float64, device="cuda")
        if c["M"]:
            bias[s["ids"][b].long()] = s["bias"][b].double()
        rep, freq, pres = (s[n][b].double() for n in ("repetition", "frequency", "presence"))
        for k in range(K):
            count = s["counts"][b].double()
            for j in range(G + 1):
                if j:
                    count[s["drafts"][b, k, j - 1].long()] += 1
                x = (s["logits"][b, s["rows"][b, k, j].long()] if c["tree"] else s["logits"][b, k, j]).double()
                said = count > 0
                x = torch.where(said | prompt, x * torch.where(x > 0, 1 / rep, rep), x)
                x = x - (freq * count + pres * said) + bias
                if c["allow"]:
                    x[~word(s["allow"][b, k, j])] = -math.inf
                out[b, k, j] = x
    return out

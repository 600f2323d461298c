"""Draws from batches of rows and their truncation against the definition
(rows_ref.py): numbers of rows that share a GPU in every way, and places that lie
anywhere in a row."""
import math
import random

import pytest
import torch

import rows_ref as ref
from draft_verification_sdv_gb300 import binding as bd
from test_gpu_layer import _status

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bd.load(build=True)


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _dev(cut):
    names = dict(T="temperature", top_k="top_k", top_p="top_p", min_p="min_p")
    return {names[n]: torch.tensor(v, dtype=torch.int32 if n == "top_k" else F32, device="cuda")
            for n, v in cut.items() if v is not None}


def _check(x, cut, u):
    """Both calls on rows [R, V], each with parameters of its own."""
    R, V = x.shape
    st = _status()
    kept = torch.full((R,), -5, dtype=torch.int32, device="cuda")
    tokens, logs = bd.sdv_sample(x, torch.tensor(u, dtype=F32, device="cuda"), logprob=True, kept=kept, status=st, **_dev(cut))
    out, many = bd.sdv_logits_truncate(x, kept=True, status=st, **_dev(cut))
    assert int(st) == 0
    n, stay, want, wlogs = ref.rows(x, u=u, **cut)
    assert kept.tolist() == n and many.tolist() == n
    assert torch.equal(out, x.masked_fill(~stay, -math.inf))
    assert tokens.tolist() == want
    # the quotient's one rounding, of what the logarithm takes, and the logarithm's own
    for got, lp in zip(logs.tolist(), wlogs):
        assert abs(got - lp) <= 2.0 ** -23 + 2.0 ** -22 * abs(lp)


@pytest.mark.parametrize("many", [100, 130, 255, 256, 257, 400])
def test_draws_of_a_value_that_many_tokens_have(many):
    """A value far down, all of whose tokens lie in the row's first part: their list is
    complete long before the row is."""
    R, V, value = _sms() + 9, 60011, -0.40625
    g = torch.Generator(device="cuda").manual_seed(many)
    x = torch.randn((R, V), generator=g, device="cuda").to(BF)
    x[x == value] = -0.5
    r = random.Random(many)
    u, p = [], []
    for b in range(R):
        first = r.choice([0, 1, 7, 300])             # (rows begin on any 2 bytes: V is odd)
        at = sorted(r.sample(range(first, 16000), many))
        x[b, torch.tensor(at, device="cuda")] = value
    T = [r.choice([0.8, 1.0, 1.3]) for _ in range(R)]
    # where that value's tokens lie in the order of a row that keeps all
    xs = x.double()
    w = ref.weights(torch.cat([xs.amax(1, keepdim=True), xs], 1), torch.tensor([ref.f32(t) for t in T], device="cuda")[:, None].double())[:, 1:]
    before = torch.where(xs > value, w, 0).sum(1).tolist()
    own = torch.where(xs == value, w, 0).sum(1).tolist()
    total = w.sum(1).tolist()
    for b in range(R):
        rank = r.choice([0, 1, many // 2, many - 1, r.randrange(many)])
        u.append((before[b] + own[b] * (rank + 0.5) / many) / total[b])
        p.append((before[b] + own[b] * (rank + 0.5) / many) / total[b])
    _, _, tokens, _ = ref.rows(x, T=T, u=u)
    assert (x.gather(1, torch.tensor(tokens, device="cuda")[:, None]) == value).all()
    _check(x, dict(T=T), u)
    # a truncation that ends among them, and draws from what it leaves
    _check(x, dict(T=T, top_p=p), [r.random() for _ in range(R)])


# ---- batches ----

KINDS = ["model", "flat", "few", "equal", "masked", "peak", "far", "nan", "inf", "none"]
BAD = KINDS[-3:]


def _batch(R, V, dtype, seed):
    """Rows of every kind side by side, and their kinds."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    x = torch.randn((R, V), generator=g, device="cuda")
    at = torch.arange(V, device="cuda")
    kinds = [r.choice(KINDS[:4] if b % 3 else KINDS) for b in range(R)]
    for b, kind in enumerate(kinds):
        y = x[b]
        if kind == "model":
            y = r.choice([1.0, 3.0, 6.0]) * y + 8 - 1.1 * torch.log1p(at)
        elif kind == "flat":
            y = y * r.choice([1e-3, 0.3])
        elif kind == "few":                          # many equal values, and zeros of both signs
            y = (y * 2).round() / 2
            y = torch.where(y == 0, torch.where(at % 2 == 0, 0.0, -0.0), y)
        elif kind == "equal":
            y = torch.full_like(y, -3.25)
        elif kind in ("masked", "none"):
            y = torch.where(torch.rand(V, generator=g, device="cuda") < (0.9 if kind == "masked" else 2), -math.inf, 2 * y)
            if kind == "masked":
                y[V // 2] = 1.0
        elif kind == "far":                          # over all magnitudes that the type has
            y = y * torch.exp2(torch.randint(-120, 120, (V,), generator=g, device="cuda").float())
        elif kind == "nan":
            y[r.randrange(V)] = math.nan
        elif kind == "inf":
            y[r.randrange(V)] = math.inf
        x[b] = y
    return x.to(dtype), kinds


def _ask(R, V, seed, which):
    r = random.Random(seed)
    some = lambda off, f: [off if r.random() < 0.3 else f() for _ in range(R)]  # noqa: E731
    cut = dict(T=some(0.0 if "0" in which else 1.0, lambda: r.uniform(0.3, 3.0)) if "T" in which else None,
               top_k=some(0, lambda: int(math.exp(r.uniform(0, math.log(2 * V))))) if "k" in which else None,
               top_p=some(1.0, lambda: r.choice([r.uniform(0.05, 0.999), 0.95, 0.999])) if "p" in which else None,
               min_p=some(0.0, lambda: math.exp(r.uniform(math.log(1e-5), 0))) if "m" in which else None)
    return cut, [r.choice([r.random(), r.random(), 0.0, 1 - 2.0 ** -24]) for _ in range(R)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("which", ["", "T0p", "p", "Tkp", "m", "T0kpm"])
@pytest.mark.parametrize("V", [2103, 20011])
@pytest.mark.parametrize("batch", range(5))
def test_batches_of_rows(batch, V, which, dtype):
    """The number of rows picks how many CTAs share one (eight to one, and some that
    take several): every answer is the definition's, and the one that a few of the rows
    get by themselves, in place too."""
    m = _sms()
    R = [m // 4, m // 4 + 1, m // 2 + 1, m + 1, 2 * m + 97][batch]
    x, kinds = _batch(R, V, dtype, 100 * batch + V)
    cut, u = _ask(R, V, batch, which)
    dev, us = _dev(cut), torch.tensor(u, dtype=F32, device="cuda")
    st = _status()
    kept = torch.full((R,), -5, dtype=torch.int32, device="cuda")
    tokens, logs = bd.sdv_sample(x, us, logprob=True, kept=kept, status=st, **dev)
    out, many = bd.sdv_logits_truncate(x, kept=True, status=st, **dev)
    bad = torch.tensor([k in BAD for k in kinds], device="cuda")
    good = ~bad
    assert int(st) == (bd.SDV_STATUS_BAD_ROW if bad.any() else 0)
    assert torch.equal(kept, many)
    assert (tokens[bad] == -1).all() and logs[bad].isnan().all() and (kept[bad] == 0).all() and out[bad].isnan().all()
    pick = good.nonzero().flatten().tolist()
    n, stay, want, wlogs = ref.rows(x[good], u=[u[b] for b in pick], **{k: v and [v[b] for b in pick] for k, v in cut.items()})
    assert kept[good].tolist() == n
    assert torch.equal(out[good], x[good].masked_fill(~stay, -math.inf))
    assert tokens[good].tolist() == want
    for got, lp in zip(logs[good].tolist(), wlogs):
        assert abs(got - lp) <= 2.0 ** -23 + 2.0 ** -22 * abs(lp)
    # a few rows at a time, and without the counts that another way may be taken for
    eq = lambda a, b: torch.equal(a.view(torch.int32 if a.element_size() == 4 else torch.int16),  # noqa: E731
                                  b.view(torch.int32 if b.element_size() == 4 else torch.int16))
    for r0 in range(0, R, 30):
        part = slice(r0, r0 + 30)
        few = {name: t[part] for name, t in dev.items()}
        t, lp = bd.sdv_sample(x[part], us[part], logprob=True, **few)
        assert torch.equal(t, tokens[part]) and eq(lp, logs[part])
        assert eq(bd.sdv_logits_truncate(x[part], **few), out[part])
    same = x.clone()
    assert eq(bd.sdv_logits_truncate(same, out=same, **dev), out) and same.data_ptr() != x.data_ptr()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_batches_that_share_parameters(dtype):
    """Several rows a sequence, more than there are places for."""
    m, per, V = _sms(), 7, 5003
    B = 2 * m // per + 5
    x, kinds = _batch(B * per, V, dtype, 5)
    good = [k not in BAD for k in kinds]
    x[torch.tensor([not k for k in good], device="cuda")] = 0.5
    cut, _ = _ask(B, V, 3, "T0kpm")
    _, u = _ask(B * per, V, 4, "")
    n, stay, want, _ = ref.rows(x, u=u, **{k: [a for a in v for _ in range(per)] for k, v in cut.items()})
    x3 = x.view(B, per, V)
    tokens = bd.sdv_sample(x3, torch.tensor(u, dtype=F32, device="cuda").view(B, per), **_dev(cut))
    out, many = bd.sdv_logits_truncate(x3, kept=True, **_dev(cut))
    assert tokens.flatten().tolist() == want and many.flatten().tolist() == n
    assert torch.equal(out.view(-1, V), x.masked_fill(~stay, -math.inf))


# ---- borders ----

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R", [1, 400])
def test_min_p_around_the_head(R, dtype):
    """A row is first looked through for its largest few hundred logits: min-p's reach
    onto, just above and just below logits of every rank from 1 to far behind those."""
    V = 20011
    g = torch.Generator(device="cuda").manual_seed(9)
    row = (3 * torch.randn(V, generator=g, device="cuda") + 8).to(dtype)
    value = torch.unique(row.double()).flip(0).tolist()
    ranks = list(range(min(len(value), 1500))) if dtype == BF else list(range(0, 4000, 7))
    T, mins = [], []
    for i in ranks:
        t = [1.0, 0.7, 2.5][i % 3]
        p = torch.tensor(math.exp((value[i] - value[0]) / t), dtype=F32)
        if not 0 < float(p) <= 1:
            continue
        for q in (p, torch.nextafter(p, torch.tensor(0.0)), torch.nextafter(p, torch.tensor(2.0))):
            if 0 < float(q) <= 1:
                T.append(t), mins.append(float(q))
    # logits on the floor itself: T ln(min_p) is exact in 64 bits only at 1, so the floor lies
    # within 2^-52 of itself from either side of what is asked
    x = row.expand(len(T), V)
    for k in (None, [600] * len(T)):
        for r0 in range(0, len(T), R) if R > 1 else range(0, len(T), 37):
            part = slice(r0, r0 + R)
            cut = dict(T=T[part], min_p=mins[part], top_k=k and k[part])
            kept = torch.empty((len(T[part]),), dtype=torch.int32, device="cuda")
            bd.sdv_sample(x[part], torch.zeros(kept.shape, device="cuda"), kept=kept, **_dev(cut))
            out, many = bd.sdv_logits_truncate(x[part], kept=True, **_dev(cut))
            n, stay, _, _ = ref.rows(x[part], **cut)
            assert kept.tolist() == n and many.tolist() == n
            assert torch.equal(out, x[part].masked_fill(~stay, -math.inf))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1024, 1 << 17])
@pytest.mark.parametrize("R", [1, 400])
def test_products_with_the_sum_are_exact(R, N, dtype):
    """Sums beyond 2^53, which 64-bit floating point would round, at a border."""
    # N equal logits and one that weighs 1: half of N 2^44 + 1 lies just behind N / 2 of them
    x = torch.zeros((R, N + 1), dtype=dtype, device="cuda")
    x[:, 77] = -30.5                                 # 2^44 e^-30.5 = 0.9986
    assert ref.weights(torch.tensor([[0.0, -30.5]], dtype=torch.float64), torch.ones((1, 1), dtype=torch.float64))[0, 1] == 1
    assert 0.5 * float(N * 2 ** 44 + 1) == N // 2 * 2 ** 44
    out, kept = bd.sdv_logits_truncate(x, top_p=torch.full((R,), 0.5, device="cuda"), kept=True)
    assert (kept == N // 2 + 1).all()
    keep = torch.arange(N + 1, device="cuda") < N // 2 + 2
    keep[77] = False
    assert torch.equal(out > -math.inf, keep.expand(R, -1))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R", [1, 400])
def test_draws_at_a_border_that_rounding_moves(R, dtype):
    """u W for a W beyond 2^53 whose rounding passes a border between two tokens."""
    N, fall, u = 2048, 18.5, 1 - 2.0 ** -24          # u W = W - 2^-24 W lies among the light tokens
    found = []
    for i in range(400000):
        T = 1.0 + i * 2.0 ** -22
        real = math.exp(-fall / T) * 2.0 ** 44
        w = math.floor(real + 0.5)
        # one that fp32 gives exactly: an exponent below 32 is off by 2^-20 at most, and so the
        # weight by less than 0.7 * 2^-20 of itself
        if abs(real - w) + 0.7 * 2.0 ** -20 * w > 0.4:
            continue
        for m in (2 ** 31 // w + 2, 2 ** 31 // w + 300):
            W = N * 2 ** 44 + m * w
            exact, rounded = W - -(-W >> 24), int(u * float(W))
            a, b = (exact - N * 2 ** 44) // w, (rounded - N * 2 ** 44) // w
            if a != b and 0 <= a < m and 0 <= b < m:
                found.append((T, m, a))
        if len(found) >= 4:
            break
    assert found
    for T, m, rank in found:
        x = torch.zeros((R, N + m), dtype=dtype, device="cuda")
        x[:, N // 2:N // 2 + m] = -fall
        kept = torch.empty((R,), dtype=torch.int32, device="cuda")
        tokens = bd.sdv_sample(x, torch.full((R,), u, device="cuda"), temperature=torch.full((R,), T, device="cuda"), kept=kept)
        assert (kept == N + m).all() and (tokens == N // 2 + rank).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R", [30, 700])
@pytest.mark.parametrize("V", [1500, 12000, 100000])
def test_log_probabilities_of_light_tokens(V, R, dtype):
    """Five heavy tokens and many of 1 to 2^21 units, of which one of the last is drawn."""
    falls = torch.linspace(15.5, 29.5, R).to(BF)
    x = torch.full((R, V), 1.0, dtype=BF)
    x[:, 5:] = 1.0 - falls[:, None]
    x = x.to(dtype).cuda()
    r = random.Random(V)
    T = [r.uniform(0.98, 1.0) for _ in range(R)]
    u = torch.full((R,), 1 - 2.0 ** -24, device="cuda")
    tokens, logs = (t.tolist() for t in bd.sdv_sample(x, u, logprob=True, **_dev(dict(T=T))))
    last = x[:, -1].double().tolist()
    for b, (token, got) in enumerate(zip(tokens, logs)):
        if token >= 5:                               # (what u passes in the rows with the lightest is the heavy ones)
            w = math.floor(math.exp((last[b] - 1.0) / ref.f32(T[b])) * 2.0 ** 44 + 0.5)
            # the sum may be off by a unit a token (2^-29 of itself), and is rounded to fp32
            lp = math.log(w / (5 * 2 ** 44 + (V - 5) * w))
            assert abs(got - lp) <= 2.0 ** -23 + 2.0 ** -22 * abs(lp), (b, w)
    assert sum(t >= 5 for t in tokens) > R // 5


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_leave_the_cache_to_others(dtype):
    """A kernel that reads what fits the L2 cache over and over is as fast after draws and
    truncations as before them."""
    y, out = torch.ones(25 << 20, device="cuda"), torch.empty((), device="cuda")

    def best():
        times = []
        for _ in range(40):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            torch.sum(y, dim=0, out=out)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times[10:])
    before = best()
    x, _ = _batch(256, 152064, dtype, 1)
    u = torch.full((256,), 0.5, device="cuda")
    for cut in (dict(), dict(top_k=[50] * 256), dict(top_p=[0.95] * 256)):
        bd.sdv_sample(x, u, **_dev(cut))
        bd.sdv_logits_truncate(x, **_dev(cut))
    assert best() <= 1.15 * before


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R", [1, 50, 330])
def test_the_longest_rows(R, dtype):
    """2^19 logits, all equal: their weights add up to 2^63."""
    V = 1 << 19
    x = torch.full((R, V), 2.5, dtype=dtype, device="cuda")
    r = random.Random(R)
    u = [r.choice([0.0, 1 - 2.0 ** -24, r.random()]) for _ in range(R)]
    p = [r.choice([1 - 2.0 ** -24, 0.5, r.random()]) for _ in range(R)]
    tokens, logs = bd.sdv_sample(x, torch.tensor(u, dtype=F32, device="cuda"), logprob=True)
    assert tokens.tolist() == [int(ref.f32(v) * V) for v in u]   # (43 bits: exact)
    assert ((logs + 19 * math.log(2)).abs() <= 2.0 ** -20).all()           # (13.2, rounded to 2^-20, and its logarithm's own)
    out, kept = bd.sdv_logits_truncate(x, top_p=torch.tensor(p, dtype=F32, device="cuda"), kept=True)
    want = torch.tensor([math.ceil(ref.f32(v) * V) for v in p], device="cuda")
    assert torch.equal(kept.long(), want)
    assert torch.equal(out > -math.inf, torch.arange(V, device="cuda") < want[:, None])

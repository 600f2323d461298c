"""The serving loop's operators on the GPU against plain host implementations:
pages from request lengths, attention behind shared prefixes, draws from rows
of logits and their truncation."""
import math
import random

import pytest
import torch

import serve_ref as sref
from draft_verification_sdv_gb300 import binding as bd
from test_gpu_layer import TYPES, _cache, _i32, _status, _tables

pytestmark = pytest.mark.gpu
BF, HF, F8, F32 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bd.load(build=True)


# ---- pages ----

class _Pages:
    """The same state on the host and on the GPU."""

    def __init__(self, r, B, P, most, spare, held=None):
        held = [r.randint(0, most) for _ in range(B)] if held is None else held
        pages = sum(held) + spare
        ids = list(range(pages))
        r.shuffle(ids)
        table, at = [], 0
        for h in held:
            table.append(ids[at:at + h] + [-1] * (most - h))
            at += h
        self.host = sref.Pages(ids[at:], table, held, P, pages)
        self.P, self.pages = P, pages
        self.list = torch.full((pages,), -7, dtype=torch.int32, device="cuda")
        self.list[:spare] = _i32(ids[at:]) if spare else self.list[:0]
        self.free, self.table, self.held = _i32([spare]), _i32(table), _i32(held)
        self.status = _status()

    def check(self):
        assert int(self.status) == self.host.status
        assert self.free.tolist() == [len(self.host.stack)]
        assert self.held.tolist() == self.host.held
        assert self.table.tolist() == self.host.table
        assert self.list[:len(self.host.stack)].tolist() == self.host.stack

    def extend(self, start, N, count=None, depth=None, base=None):
        want = self.host.extend(start, N, count, depth, base)
        give = lambda x: None if x is None else _i32(x)  # noqa: E731
        got = bd.sdv_pages_extend(self.list, self.free, self.table, self.held, _i32(start), N, self.P,
                                  count=give(count), depth=give(depth), base=give(base), status=self.status)
        assert torch.equal(got[0].cpu(), want[0])
        assert torch.equal(got[1].cpu(), want[1])
        self.check()

    def release(self, keep):
        self.host.release(keep)
        bd.sdv_pages_release(self.list, self.free, self.table, self.held, _i32(keep), self.P, status=self.status)
        self.check()


@pytest.mark.parametrize("B,N,P,most", [(1, 1, 1, 3), (3, 7, 16, 40), (64, 1, 16, 100), (48, 129, 16, 20), (5, 3000, 24, 200),
                                        (700, 3, 4, 9), (1500, 1, 128, 4), (2, 513, 1, 1200), (600, 40, 8, 12)])
def test_pages_through_a_step(B, N, P, most):
    r = random.Random(B + N)
    room = most * P
    start = [r.randint(0, max(room - N, 0)) for _ in range(B)]
    count = [r.randint(0, min(N, room)) for _ in range(B)]
    held = [min(sref.ceil_div(s, P) + r.randint(0, 1), most) for s in start]
    s = _Pages(r, B, P, most, B * (sref.ceil_div(N, P) + 1) + 2, held)
    depth = [[r.randint(0, 50) for _ in range(N)] for _ in range(B)]
    before = s.list.clone(), s.table.clone()
    s.extend(start, N, count, depth, [r.randint(0, 9000) for _ in range(B)])
    assert s.host.status == 0
    s.release([h * P for h in held])                 # back to what was held: the list as it was
    assert torch.equal(s.list, before[0]) and torch.equal(s.table, before[1])
    s.extend(start, N, count)
    s.release([x + r.randint(0, n) for x, n in zip(start, count)])
    s.release([0 if r.random() < 0.5 else 10 ** 6 for _ in range(B)])
    s.release([0] * B)
    assert not any(s.host.held)
    if max(N, 1) <= room:
        s.extend([0] * B, N, [min(n, P) for n in count])


@pytest.mark.parametrize("P", [1, 3, 127, 128, 129, 511, 512, 513, 1000, 2600])
@pytest.mark.parametrize("B,N", [(3, 2500), (70, 129), (40, 65)])
def test_pages_of_any_size_for_any_number_of_tokens(B, N, P):
    """A thread's tokens are a number of pages and a rest apart."""
    r = random.Random(P + N)
    most = sref.ceil_div(2 * N, P) + 1
    start = [r.choice([0, 1, N, r.randint(0, most * P - N)]) for _ in range(B)]
    held = [min(sref.ceil_div(x, P) + r.randint(0, 1), most) for x in start]
    s = _Pages(r, B, P, most, B * (sref.ceil_div(N, P) + 1), held)
    s.extend(start, N, [r.choice([0, 1, N - 1, N, r.randint(0, N)]) for _ in range(B)])
    assert s.host.status == 0
    s.release(start)


@pytest.mark.parametrize("B,N", [(9, 40), (90, 33), (700, 16)])
def test_pages_that_run_out(B, N):
    """Sequences are served in order until one no longer is; those after it that
    lack a page are not, those that lack none are."""
    r = random.Random(B)
    P, most = 8, 30
    held = [r.randint(0, 8) for _ in range(B)]
    s = _Pages(r, B, P, most, B // 2, held)
    start = [h * P - (r.randint(0, P - 1) if h else 0) for h in held]
    s.extend(start, N, [r.randint(0, N) for _ in range(B)])
    assert s.host.status == 128 and any(s.host.held[b] > held[b] for b in range(B))
    assert s.host.stack or sum(s.host.held) == s.pages


def test_pages_of_bad_numbers():
    r = random.Random(4)
    B, P, most, N = 8, 4, 6, 9
    s = _Pages(r, B, P, most, 30, [2] * B)
    s.extend([5, -1, 8, 16, 2 ** 31 - 1, 0, 3, 4], N, [3, 2, 10, 9, 1, -1, 0, 9])
    assert s.host.status == 16
    # what a sequence holds is out of range
    s = _Pages(r, B, P, most, 30, [2] * B)
    s.held[1], s.host.held[1], s.held[4], s.host.held[4] = -1, -1, 7, 7
    s.extend([8] * B, N, [1] * B)
    s.release([4] * B)
    assert s.host.status == 16
    # the stack's height is
    for height in (-1, 1000):
        s = _Pages(r, B, P, most, 30, [2] * B)
        before = s.list.clone(), s.table.clone()
        s.free.fill_(height)
        pos, slots = bd.sdv_pages_extend(s.list, s.free, s.table, s.held, _i32([7] * B), 3, P, status=s.status)
        assert int(s.status) == 16 and int(s.free) == height and s.held.tolist() == [2] * B
        want = [[int(row[1]) * P + 3, -1, -1] for row in before[1].tolist()]
        assert slots.tolist() == want and pos.tolist() == [[7, 8, 9]] * B
        bd.sdv_pages_release(s.list, s.free, s.table, s.held, _i32([0] * B), P, status=s.status)
        assert torch.equal(s.list, before[0]) and torch.equal(s.table, before[1]) and s.held.tolist() == [2] * B
    # more comes back than the list holds
    s = _Pages(r, B, P, most, 30, [2] * B)
    s.free.fill_(s.pages - 3)
    bd.sdv_pages_release(s.list, s.free, s.table, s.held, _i32([0] * B), P, status=s.status)
    assert int(s.status) == 16 and s.held.tolist() == [2] * B and int(s.free) == s.pages - 3
    # entries of the list that are no pages
    s = _Pages(r, B, P, most, 30, [2] * B)
    s.list[29], s.host.stack[29] = 46, 46
    s.list[20], s.host.stack[20] = -2, -2
    s.extend([8] * B, N, [8] * B)
    assert s.host.status == 64
    s.release([8] * B)


# ---- attention behind shared prefixes ----

def _prefix_case(B, G, N, Hq, Hk, D, P, far, ctx, dtype, cdtype, seed, strided=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    per, ppre = -(-(max(ctx) + N) // P) + 1, -(-max(max(far), 1) // P) + 1
    pages = B * per + G * ppre + 2
    kc, vc, ke, ve = _cache(pages, Hk, P, D, cdtype, False)
    order = _tables(1, B * per + G * ppre, pages, seed)[0]
    table, ptable = order[:B * per].view(B, per).contiguous(), order[B * per:].view(G, ppre).contiguous()
    for t, n, L in ((table, B, max(ctx) + N), (ptable, G, max(far))):
        if L:
            k, v = (torch.randn((n, L, Hk, D), generator=g, device="cuda").to(dtype) for _ in range(2))
            bd.sdv_kv_write(k, v, kc, vc, t, _i32([0] * n), k_exp=ke, v_exp=ve)
    if strided:                                      # sequences further apart than their nodes need
        q = torch.randn((B, N + 2, Hq + 1, D), generator=g, device="cuda").to(dtype)[:, :N, :Hq]
    else:
        q = torch.randn((B, N, Hq + 1, D), generator=g, device="cuda").to(dtype)[:, :, :Hq]
    return q, kc, vc, ke, ve, ptable, table


def _check_prefix(case, far, ctx, count=None, mask=None, scale=None):
    q, kc, vc, ke, ve, ptable, table = case
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    st = _status()
    out, lse = bd.sdv_prefix_attn(q, kc, vc, ptable, _i32(far), table, _i32(ctx),
                                  count=None if count is None else _i32(count), mask=mask, scale=scale, k_exp=ke,
                                  v_exp=ve, lse=True, status=st)
    assert int(st) == 0
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    want, wl, tol, tl = sref.prefix_attn(q.cpu(), cpu(kc), cpu(vc), ptable.cpu(), far, table.cpu(), ctx, count, cpu(mask),
                                         scale, cpu(ke), cpu(ve))
    # the join of the two parts adds five fp32 roundings and two 2^x: far below what
    # the reference allows for the parts' own (2^-20 in a probability)
    assert not out.isnan().any()
    err = (out.double().cpu() - want).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())
    lse = lse.double().cpu()
    assert torch.equal(lse == -math.inf, wl == -math.inf)
    fin = wl > -math.inf
    assert ((lse - wl).abs()[fin] <= tl[fin]).all(), float(((lse - wl).abs()[fin] / tl[fin]).max())
    return out


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("B,G,N,Hq,Hk,D,P,far,ctx", [
    (1, 1, 1, 1, 1, 64, 16, [0], [0]), (2, 1, 1, 8, 1, 128, 16, [1], [0, 5]), (6, 2, 1, 8, 2, 128, 16, [129, 300], [0, 1, 15, 16, 17, 90]),
    (3, 3, 1, 7, 7, 96, 5, [300, 0, 63], [40, 0, 7]), (4, 1, 1, 4, 2, 16, 1, [40], [0, 3, 2, 9]), (2, 2, 2, 8, 1, 256, 32, [333, 32], [1, 64]),
    (4, 2, 9, 8, 2, 128, 16, [0, 250], [0, 250, 3, 16]), (2, 1, 70, 3, 1, 64, 8, [100], [0, 31]), (3, 1, 33, 5, 1, 80, 64, [127], [0, 128, 64]),
    (40, 1, 1, 8, 1, 128, 16, [500], list(range(40))), (12, 2, 1, 16, 2, 64, 32, [77, 640], [7 * i for i in range(12)])])
def test_prefix_attn(B, G, N, Hq, Hk, D, P, far, ctx, dtype, cdtype):
    case = _prefix_case(B, G, N, Hq, Hk, D, P, far, ctx, dtype, cdtype, seed=B + N + D)
    _check_prefix(case, far, ctx)


@pytest.mark.parametrize("dtype,cdtype", [(BF, BF), (HF, F8)])
@pytest.mark.parametrize("B,G,K,gamma,Hq,Hk,D,far,ctx,P", [
    (4, 2, 3, 5, 4, 1, 64, [77, 200], [0, 3, 0, 40], 16), (3, 1, 4, 16, 8, 1, 128, [400], [1, 0, 129], 16),
    (2, 1, 5, 7, 2, 2, 96, [33], [0, 126], 12)])
def test_prefix_attn_trees(B, G, K, gamma, Hq, Hk, D, far, ctx, P, dtype, cdtype):
    g = torch.Generator(device="cuda").manual_seed(K)
    drafts = torch.randint(0, 3, (B, K, gamma), generator=g, device="cuda", dtype=torch.int32)
    t = bd.sdv_tree_build(_i32([0] * B), drafts)
    count = t["count"].tolist()
    count[0] = 0                                     # a sequence that has nothing this step
    case = _prefix_case(B, G, 1 + K * gamma, Hq, Hk, D, P, far, ctx, dtype, cdtype, seed=gamma)
    out = _check_prefix(case, far, ctx, count=count, mask=t["mask"])
    for b in range(B):
        assert not out[b, count[b]:].any()


@pytest.mark.parametrize("dtype,cdtype", [(BF, BF), (BF, F8), (HF, HF)])
@pytest.mark.parametrize("N,Hq,D,P", [(1, 4, 64, 16), (5, 6, 128, 16), (40, 3, 128, 12), (40, 8, 64, 64)])
def test_prefix_attn_strides_scale_and_unseen_cells(N, Hq, D, P, dtype, cdtype):
    """Sequences that are not evenly apart, a negative scale, and NaN in every
    cell that no node sees."""
    B, G, far, ctx = 4, 2, [90, 35], [0, 20, 3, 17]
    count = [N, N - N // 2, N, 0]
    case = _prefix_case(B, G, N, Hq, 1, D, P, far, ctx, dtype, cdtype, seed=N, strided=True)
    q, kc, vc, ke, ve, ptable, table = case
    seen = torch.zeros(kc.shape[:3], dtype=torch.bool, device="cuda")
    for g in range(G):
        for t in range(far[g]):
            seen[ptable[g, t // P], :, t % P] = True
    for b in range(B):
        for t in range(ctx[b] + count[b]):
            seen[table[b, t // P], :, t % P] = True
    for t in (kc, vc):
        if cdtype == F8:
            t.view(torch.uint8)[~seen] = 0x7f
        else:
            t[~seen] = math.nan
    _check_prefix(case, far, ctx, count=count, scale=-0.2)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("N,Hq,Hk,D", [(1, 8, 1, 128), (1, 5, 1, 80), (3, 8, 2, 64), (40, 8, 1, 128), (70, 7, 1, 64)])
def test_prefix_attn_of_padded_queries_that_are_no_numbers(N, Hq, Hk, D, dtype, cdtype):
    """The prefix's pass knows no count: rows behind it come out as nothing, and leave
    the others as they are."""
    B, G, far, ctx = 6, 2, [70, 300], [0, 20, 3, 0, 140, 9]
    count = [0, N, N - N // 2, N, max(N - 1, 1), 0]
    q, *rest = _prefix_case(B, G, N, Hq, Hk, D, 16, far, ctx, dtype, cdtype, seed=N + D)
    kc, vc, ke, ve, ptable, table = rest
    want, wl, tol, tl = sref.prefix_attn(q.cpu(), kc.cpu(), vc.cpu(), ptable.cpu(), far, table.cpu(), ctx, count, None,
                                         D ** -0.5, None if ke is None else ke.cpu(), None if ve is None else ve.cpu())
    for bad in (math.nan, math.inf, -math.inf):
        for b in range(B):
            q[b, count[b]:] = bad
        st = _status()
        out, lse = bd.sdv_prefix_attn(q, kc, vc, ptable, _i32(far), table, _i32(ctx), count=_i32(count), k_exp=ke, v_exp=ve,
                                      lse=True, status=st)
        assert int(st) == 0 and not out.isnan().any() and not lse.isnan().any()
        assert ((out.double().cpu() - want).abs() <= tol).all()
        assert torch.equal(lse.cpu() == -math.inf, wl == -math.inf)
        fin = wl > -math.inf
        assert ((lse.double().cpu() - wl).abs()[fin] <= tl[fin]).all()
        for b in range(B):
            assert not out[b, count[b]:].any()


def test_prefix_attn_without_a_prefix_and_bad_numbers():
    B, G, N, Hq, Hk, D, P = 4, 2, 3, 8, 2, 64, 16
    far, ctx = [40, 50], [5, 0, 31, 2]
    q, kc, vc, ke, ve, ptable, table = _prefix_case(B, G, N, Hq, Hk, D, P, far, ctx, BF, BF, seed=1)
    st = _status()
    good = bd.sdv_prefix_attn(q, kc, vc, ptable, _i32(far), table, _i32(ctx))
    got, lse = bd.sdv_prefix_attn(q, kc, vc, ptable, _i32([0, 0]), table, _i32(ctx), lse=True, status=st)
    alone, alse = bd.sdv_tree_attn(q, kc, vc, table, _i32(ctx), lse=True)
    assert torch.equal(got, alone) and torch.allclose(lse, alse, rtol=2.0 ** -22, atol=2.0 ** -22) and int(st) == 0
    for bad in (-1, ptable.shape[1] * P + 1):
        st.zero_()
        got, lse = bd.sdv_prefix_attn(q, kc, vc, ptable, _i32([40, bad]), table, _i32(ctx), count=_i32([3, 1, 2, 3]), lse=True,
                                      status=st)
        assert int(st) == bd.SDV_STATUS_BAD_LENGTH
        assert torch.equal(got[0], good[0]) and torch.equal(got[1, :1], good[1, :1]) and not got[1, 1:].any()
        assert got[2, :2].isnan().all() and got[3].isnan().all() and lse[3].isnan().all()
        assert not got[2, 2:].any() and (lse[2, 2:] == -math.inf).all()
    # one sequence's own length
    st.zero_()
    got = bd.sdv_prefix_attn(q, kc, vc, ptable, _i32(far), table, _i32([5, -1, 31, 2]), status=st)
    assert int(st) == bd.SDV_STATUS_BAD_LENGTH and got[1].isnan().all() and torch.equal(got[[0, 2, 3]], good[[0, 2, 3]])
    # a page of one prefix
    st.zero_()
    other = ptable.clone()
    other[1, 1] = kc.shape[0]
    got = bd.sdv_prefix_attn(q, kc, vc, other, _i32(far), table, _i32(ctx), status=st)
    assert int(st) == bd.SDV_STATUS_BAD_PAGE and torch.equal(got[:2], good[:2]) and got[2:].isnan().all()


# ---- draws and truncation ----

def _rows(shape, V, dtype, seed, kind="model"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape + (V,), generator=g, device="cuda")
    if kind == "model":
        x = 3 * x + 8 - 1.1 * torch.log1p(torch.arange(V, device="cuda"))
    elif kind == "flat":
        x = x * 1e-3
    elif kind == "few":                              # many equal values, and zeros of both signs
        x = (x * 2).round() / 2 * torch.where(x > 0, 1.0, -1.0)
        x = torch.where(x == 0, torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0), x)
    elif kind == "equal":
        x = torch.full_like(x, -3.25)
    elif kind == "masked":                           # a grammar leaves little
        x = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.9, -math.inf, 2 * x)
        x[..., V // 2] = 1.0
    elif kind == "peak":
        x[..., V // 3] = 60.0
    elif kind == "far":                              # over all magnitudes that the type has
        x = x * torch.exp2(torch.randint(-120, 120, x.shape, generator=g, device="cuda").float())
    return x.to(dtype)


def _params(B, seed, T=True, k=True, p=True, m=True, V=1000):
    r = random.Random(seed)
    f = lambda lo, hi, off: [off if r.random() < 0.2 else r.uniform(lo, hi) for _ in range(B)]  # noqa: E731
    return dict(temperature=f(0.3, 2.0, 0.0) if T else None,
                top_k=[0 if r.random() < 0.2 else int(math.exp(r.uniform(0, math.log(2 * V)))) for _ in range(B)] if k else None,
                top_p=f(0.05, 0.999, 1.0) if p else None, min_p=f(0.0005, 0.5, 0.0) if m else None)


def _on(cut):
    return {n: None if v is None else torch.tensor(v, dtype=torch.int32 if n == "top_k" else F32, device="cuda")
            for n, v in cut.items()}


def _check_rows(x, cut, seed=0, us=None):
    """Both calls on x [B, n, V] against the definition, row by row."""
    B, n, V = x.shape
    g = torch.Generator().manual_seed(seed)
    u = torch.rand((B, n), generator=g) if us is None else us
    st = _status()
    kept = torch.full((B, n), -5, dtype=torch.int32, device="cuda")
    tokens, logs = bd.sdv_sample(x, u.cuda(), logprob=True, kept=kept, status=st, **_on(cut))
    out, many = bd.sdv_logits_truncate(x, kept=True, status=st, **_on(cut))
    assert int(st) == 0
    assert torch.equal(kept, many)
    host, out, many = x.float().cpu(), out.float().cpu(), many.cpu()
    for b in range(B):
        args = dict(T=1.0 if cut["temperature"] is None else cut["temperature"][b],
                    **{n: v[b] for n, v in cut.items() if n != "temperature" and v is not None})
        for j in range(n):
            row = host[b, j].double().tolist()
            idx, w = sref.choose(row, **args)
            assert int(many[b, j]) == len(idx), (b, j, args)
            want = torch.full((V,), -math.inf)
            want[idx] = host[b, j, idx]
            assert torch.equal(out[b, j], want), (b, j, args)
            token, lp = sref.drawn(idx, w, float(u[b, j]))
            assert int(tokens[b, j]) == token, (b, j, args, float(u[b, j]))
            # the quotient's one rounding, of what the logarithm takes, and the logarithm's own
            assert abs(float(logs[b, j]) - lp) <= 2.0 ** -23 + 2.0 ** -22 * abs(lp)


KINDS = ["model", "flat", "few", "equal", "masked", "peak", "far"]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [1, 7, 64, 1000, 4099])
def test_rows_of_all_kinds(V, kind, dtype):
    if kind == "far" and dtype == BF and V == 1:
        pytest.skip("the same as fp32")
    for seed, which in enumerate([dict(), dict(k=False), dict(p=False, m=False), dict(k=False, p=False), dict(T=False, m=False),
                                  dict(T=False, k=False, p=False, m=False)]):
        _check_rows(_rows((6, 2), V, dtype, seed + V, kind), _params(6, seed, V=V, **which), seed)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [32001, 152064])
def test_rows_of_a_vocabulary(V, dtype):
    x = _rows((4, 2), V, dtype, V)
    _check_rows(x, dict(temperature=[0.7, 1.0, 1.3, 0.0], top_k=[0, 50, 0, 5], top_p=[0.9, 1.0, 0.99, 0.5], min_p=[0.0, 0.0, 0.01, 0.0]))
    _check_rows(x, dict(temperature=None, top_k=None, top_p=None, min_p=None), 1)
    _check_rows(_rows((2, 1), V, dtype, V, "equal"), dict(temperature=None, top_k=[0, 100000], top_p=[0.5, 0.9], min_p=None), 2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [2056, 7000, 16400, 30008, 30011])
def test_rows_that_keep_many(V, dtype):
    """Nuclei of thousands of tokens, and draws from far down."""
    cut = dict(temperature=[3.0, 1.5, 5.0, 1.0], top_k=[0, 0, 3000, 0], top_p=[0.97, 0.9, 0.9, 1.0], min_p=[0.0, 0.0, 0.0, 1e-6])
    us = torch.tensor([0.02, 0.6, 0.999]).repeat(4, 1)
    _check_rows(_rows((4, 3), V, dtype, V), cut, us=us)
    _check_rows(_rows((4, 3), V, dtype, V)[:, :, 3:], {**cut, "min_p": None, "top_k": None}, us=us)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_with_very_many_of_one_value(dtype):
    """More equal logits than 16 bits count: of either sign, zeros of both, and
    places that a grammar masks."""
    V = 140000
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((6, 1, V), generator=g, device="cuda")
    many = torch.rand(V, generator=g, device="cuda") < 0.6
    x[0, 0, many], x[1, 0, many], x[2, 0, many] = 1.5, -1.5, -math.inf
    x[3, 0, many] = 0.0
    x[3, 0, ::2] *= -1.0                             # half of the zeros are negative
    x[4, 0] = torch.where(many, 2.0, -math.inf)
    x[5, 0, many], x[5, 0, ~many] = -math.inf, 0.25
    cut = dict(temperature=[1.0, 0.7, 1.0, 2.0, 1.0, 0.0], top_k=[0, 100000, 0, 90000, 70001, 0],
               top_p=[0.5, 1.0, 0.9, 0.7, 1.0, 1.0], min_p=[0.0, 0.0, 0.1, 0.0, 0.0, 0.0])
    _check_rows(x.to(dtype), cut, 3)
    x[0, 0, 5], x[1, 0, 77], x[2, 0, :70000] = math.nan, math.inf, math.inf
    st = _status()
    got = bd.sdv_sample(x[:3].to(dtype), torch.zeros((3, 1), device="cuda"), status=st)
    assert int(st) == bd.SDV_STATUS_BAD_ROW and (got == -1).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_row_strides_alignment_and_places(dtype):
    """Rows that begin anywhere, apart by more than their length, in place, and
    several draws of one row; nothing beside the rows is written."""
    V = 1003
    cut = _params(3, 5, V=V)
    wide = _rows((3, 5), V + 14, dtype, 3)
    for off in (0, 1, 3, 8):
        x = wide[:, :, off:off + V]
        want = bd.sdv_logits_truncate(x.contiguous(), **_on(cut))
        assert torch.equal(bd.sdv_logits_truncate(x, **_on(cut)), want)
        room = torch.full_like(wide, 7.0)
        bd.sdv_logits_truncate(x, out=room[:, :, 5:5 + V], **_on(cut))
        assert torch.equal(room[:, :, 5:5 + V], want) and (room[:, :, :5] == 7).all() and (room[:, :, 5 + V:] == 7).all()
        same = wide.clone()
        bd.sdv_logits_truncate(same[:, :, off:off + V], out=same[:, :, off:off + V], **_on(cut))
        assert torch.equal(same[:, :, off:off + V], want)
        assert torch.equal(same[:, :, :off], wide[:, :, :off]) and torch.equal(same[:, :, off + V:], wide[:, :, off + V:])
        _check_rows(x, cut, off)
    last = wide[:, -1, :V]                           # [B, V], rows far apart
    u = torch.rand((3,), generator=torch.Generator().manual_seed(1)).cuda()
    assert torch.equal(bd.sdv_sample(last, u, **_on(cut)), bd.sdv_sample(last.contiguous(), u, **_on(cut)))
    one = wide[:1, 0, :V]
    u = torch.linspace(0, 0.999, 40, device="cuda").view(1, 40)
    got = bd.sdv_sample(one[:, None].expand(1, 40, V), u, **_on(_params(1, 5, V=V)))
    assert torch.equal(got, bd.sdv_sample(one[:, None].repeat(1, 40, 1), u, **_on(_params(1, 5, V=V))))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_draws_at_the_ends(dtype):
    x = _rows((3, 4), 700, dtype, 8)
    us = torch.tensor([0.0, 1 - 2.0 ** -24, 2.0 ** -24, 0.5]).repeat(3, 1)
    _check_rows(x, dict(temperature=[0.5, 2.0 ** -64, 2.0 ** 64], top_k=None, top_p=[1.0, 1.0, 1 - 2.0 ** -24], min_p=None), us=us)
    _check_rows(x, dict(temperature=[1.0, 1.0, 100.0], top_k=[1, 0, 700], top_p=[1.0, 1e-30, 1.0], min_p=[0.0, 0.0, 1.0]), us=us)
    _check_rows(x, dict(temperature=[1.0, 1.0, 1.0], top_k=[2 ** 31 - 1, 699, 0], top_p=None, min_p=[1.0, 0.0, 1e-40]), us=us)


def test_bad_rows_and_parameters():
    x = _rows((9, 1), 300, BF, 2)
    x[1, 0, 17], x[2, 0, 299], x[3] = math.nan, math.inf, -math.inf
    x[4, 0, 0] = -math.inf
    base = dict(temperature=[1.0] * 9, top_k=[0] * 9, top_p=[0.9] * 9, min_p=[0.0] * 9)
    u = torch.full((9, 1), 0.3, device="cuda")

    def both(cut, u, want, bad):
        st = _status()
        kept = torch.full((9, 1), -5, dtype=torch.int32, device="cuda")
        tokens, logs = bd.sdv_sample(x, u, logprob=True, kept=kept, status=st, **_on(cut))
        assert int(st) == want
        good = [b for b in range(9) if b not in bad]
        assert (tokens[bad] == -1).all() and logs[bad].isnan().all() and (kept[bad] == 0).all()
        assert (tokens[good] >= 0).all() and not logs[good].isnan().any() and (kept[good] > 0).all()
        return good

    both(base, u, bd.SDV_STATUS_BAD_ROW, [1, 2, 3])
    st = _status()
    out, many = bd.sdv_logits_truncate(x, kept=True, status=st, **_on(base))
    assert int(st) == bd.SDV_STATUS_BAD_ROW and out[1:4].isnan().all() and not out[0].isnan().any() and not out[4:].isnan().any()
    assert (many[1:4] == 0).all()
    x[1, 0, 17], x[2, 0, 299], x[3] = 0.0, 0.0, 0.0
    for name, values in (("temperature", [-1.0, math.nan, math.inf, 2.0 ** -65]), ("top_p", [0.0, 1.5, math.nan, -0.1]),
                         ("min_p", [-0.1, 1.01, math.nan, math.inf])):
        both({**base, name: values + base[name][4:]}, u, bd.SDV_STATUS_BAD_PARAM, [0, 1, 2, 3])
    both({**base, "top_k": [-1, -2 ** 31] + [0] * 7}, u, bd.SDV_STATUS_BAD_PARAM, [0, 1])
    v = u.clone()
    v[:4, 0] = torch.tensor([1.0, -0.1, math.nan, math.inf])
    both(base, v, bd.SDV_STATUS_BAD_PARAM, [0, 1, 2, 3])


def test_truncated_rows_verify():
    """A Verifier takes truncated rows: accepted and next tokens are kept ones."""
    B, K, G, V = 3, 2, 4, 1024
    p, q = _rows((B, K, G + 1), V, F32, 1), _rows((B, K, G), V, F32, 2)
    cut = _on(dict(temperature=[0.8, 1.0, 1.2], top_k=[20, 0, 5], top_p=[1.0, 0.7, 0.95], min_p=None))
    pt, qt = bd.sdv_logits_truncate(p, **cut), bd.sdv_logits_truncate(q, **cut)
    u = torch.rand((B, K, G), generator=torch.Generator().manual_seed(3)).cuda()
    drafts = bd.sdv_sample(q, u, **cut)
    assert (qt.gather(-1, drafts.long()[..., None]) > -math.inf).all()
    ver = bd.Verifier(B, K, G, V, F32)
    for seed in range(20):
        out = ver(pt, qt, drafts, temps=cut["temperature"], seed=seed)
        ver.sync()
        for b in range(B):
            s, a, t = (int(out[n][b]) for n in ("sel", "accept_len", "next_token"))
            assert pt[b, s, a, t] > -math.inf
            for j in range(a):
                assert pt[b, s, j, drafts[b, s, j]] > -math.inf

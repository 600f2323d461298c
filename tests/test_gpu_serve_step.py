"""The serving loop's operators as a program uses them: a whole loop against a 64-bit
model, calls on other streams and in captured graphs, queries that lie anywhere,
and refusals."""
import math
import os
import sys

import pytest
import torch

from draft_verification_sdv_gb300 import binding as bd
from test_gpu_layer import _cache, _i32, _status, _tables
from test_gpu_layer_step import _model64
from test_gpu_serve import _on, _params, _prefix_case, _rows

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
BF, HF, F8, F32 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bd.load(build=True)


# ---- the loop ----

# (the slack in a logit is that of the decoding loop's test: 27 roundings to bf16 of values of
# spread 2, and e4m3 cells on top)
@pytest.mark.parametrize("e4m3,slack", [(False, 0.25), (True, 1.0)])
@pytest.mark.parametrize("length", [1, 16, 75])
def test_samples_of_one_prompt(e4m3, slack, length):
    import shared_prompt as ex
    prompt = torch.randint(0, 512, (length,), generator=torch.Generator().manual_seed(length)).tolist()
    model = ex.Model()
    cut = dict(temperature=torch.tensor([0.0, 0.7, 1.0, 1.3], device="cuda"), top_k=_i32([0, 5, 20, 1]),
               top_p=torch.tensor([1.0, 0.9, 1.0, 0.5], device="cuda"))
    s = ex.Server(model, prompt, 4, room=40, page=8, e4m3=e4m3, seed=5, **cut)
    for _ in range(21):
        s.step()
    assert s.held.tolist() == [3] * 4 and s.length.tolist() == [21] * 4
    for b, k in enumerate((1, 5, 20, 1)):
        text = s.text[b]
        assert len(text) == 22
        want = _model64(model, prompt + text[:-1])[length - 1:]
        for row, token in zip(want, text):
            assert row[token] >= row.topk(k).values[-1] - slack, (b, token)
    # sample 0 and 3 keep one token each step, whatever their temperature
    assert abs(float(s.logprob[0])) == 0 and float(s.logprob[3]) == 0


def test_samples_that_end_give_their_pages_back():
    import shared_prompt as ex
    model = ex.Model()
    prompt = list(range(40))
    free = ex.Server(model, prompt, 3, room=40, page=4, seed=9)
    for _ in range(12):
        free.step()
    end = free.text[1][5]                            # a token that the second sample draws on its way
    s = ex.Server(model, prompt, 3, room=40, page=4, seed=9, end=end)
    for _ in range(12):
        s.step()
    for b in range(3):
        n = free.text[b].index(end) + 1 if end in free.text[b] else 13
        assert s.text[b] == free.text[b][:n]
        used = 0 if n < 13 else 3
        assert s.held[b] == used and (s.table[b] >= 0).sum() == used
    assert s.free.item() + int(s.held.sum()) + 10 == s.pages
    whole = torch.cat([s.pool[:s.free.item()], s.table[s.table >= 0], s.prefix_table[0]])
    assert sorted(whole.tolist()) == list(range(s.pages))


# ---- streams and graphs ----

def _serve_state(seed, cdtype=BF, N=1):
    B, G, Hq, Hk, D, V, P = 6, 2, 8, 2, 64, 3001, 16
    far, ctx = [100, 37], [0, 15, 31, 4, 40, 9]
    q, kc, vc, ke, ve, ptable, table = _prefix_case(B, G, N, Hq, Hk, D, P, far, ctx, BF, cdtype, seed)
    st = dict(q=q, kc=kc, vc=vc, ke=ke, ve=ve, ptable=ptable, table=table, far=_i32(far), ctx=_i32(ctx))
    st["logits"] = _rows((B, 3), V, BF, seed)
    st["u"] = torch.rand((B, 3), generator=torch.Generator().manual_seed(seed)).cuda()
    st["cut"] = _on(_params(B, 3, V=V))
    st["pool"], st["free"] = torch.arange(50, 0, -1, dtype=torch.int32, device="cuda"), _i32([50])
    st["rows"] = torch.full((B, 20), -1, dtype=torch.int32, device="cuda")
    st["held"], st["len"] = _i32([0] * B), _i32([0, 3, 16, 17, 5, 1])
    return st


def _serve(st, **kw):
    pos, slots = bd.sdv_pages_extend(st["pool"], st["free"], st["rows"], st["held"], st["len"], 9, 16, **kw)
    bd.sdv_pages_release(st["pool"], st["free"], st["rows"], st["held"], st["len"], 16, **kw)
    out, lse = bd.sdv_prefix_attn(st["q"], st["kc"], st["vc"], st["ptable"], st["far"], st["table"], st["ctx"], k_exp=st["ke"],
                                  v_exp=st["ve"], lse=True, **kw)
    cut, kept = bd.sdv_logits_truncate(st["logits"], kept=True, **st["cut"], **kw)
    tokens, logs = bd.sdv_sample(st["logits"], st["u"], logprob=True, **st["cut"], **kw)
    wide, wkept = bd.sdv_logits_truncate(st["logits"].float(), kept=True, **st["cut"], **kw)
    return [pos, slots, out, lse, cut, kept, tokens, logs, wide, wkept]


@pytest.mark.parametrize("cdtype", [BF, F8])
@pytest.mark.parametrize("N", [1, 40])
def test_calls_on_another_stream(cdtype, N):
    want = [t.clone() for t in _serve(_serve_state(1, cdtype, N))]
    st = _serve_state(1, cdtype, N)
    wide = st["logits"].float()
    st["logits"].float = lambda: wide                # (a conversion on this stream would not be ordered)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                    # the current stream is busy: nothing may wait for it
    got = _serve(st, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    with torch.cuda.stream(side):
        got = _serve(_serve_state(1, cdtype, N))
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("cdtype", [BF, F8])
@pytest.mark.parametrize("N", [1, 40])
def test_calls_in_a_graph(cdtype, N):
    """Captured once, replayed on other inputs; two graphs with workspaces of their own."""
    graphs = []
    for seed in (1, 2):
        st = _serve_state(seed, cdtype, N)
        _serve(st)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _serve(st)
        graphs.append((g, st, out))
    for seed in (3, 4):
        for g, st, out in graphs:
            fresh = _serve_state(seed, cdtype, N)
            for name, t in fresh.items():
                if torch.is_tensor(t):
                    dst, src = st[name], t
                    if dst.dtype == F8:
                        dst, src = dst.view(torch.uint8), src.view(torch.uint8)
                    dst.copy_(src)
            g.replay()
            torch.cuda.synchronize()
            for x, y in zip(out, _serve(_serve_state(seed, cdtype, N))):
                assert torch.equal(x, y)


def test_two_calls_at_once():
    """Calls on two streams, each with outputs and workspace of its own."""
    a, b = _serve_state(5), _serve_state(6, F8)
    want = [[t.clone() for t in _serve(_serve_state(5))], [t.clone() for t in _serve(_serve_state(6, F8))]]
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(one):
            x = _serve(a)
        with torch.cuda.stream(two):
            y = _serve(b)
    torch.cuda.synchronize()
    for got, ref in zip((x, y), want):
        for s, t in zip(got, ref):
            assert torch.equal(s, t)


# ---- queries that lie anywhere, workspaces, refusals ----

@pytest.mark.parametrize("cdtype", [BF, F8])
@pytest.mark.parametrize("N,Hq,D", [(1, 8, 128), (1, 4, 64), (1, 16, 128), (3, 6, 64), (40, 8, 128)])
def test_prefix_attn_of_unaligned_queries(N, Hq, D, cdtype):
    far, ctx = [200, 33], [0, 70, 3, 18]
    q, kc, vc, ke, ve, ptable, table = _prefix_case(4, 2, N, Hq, 1, D, 16, far, ctx, BF, cdtype, seed=D)
    args = (kc, vc, ptable, _i32(far), table, _i32(ctx))
    want = bd.sdv_prefix_attn(q.contiguous(), *args, k_exp=ke, v_exp=ve)
    room = torch.empty(q.numel() + 3, dtype=BF, device="cuda")
    for off in (1, 3):
        odd = room[off:off + q.numel()].view(q.shape)
        odd.copy_(q)
        assert torch.equal(bd.sdv_prefix_attn(odd, *args, k_exp=ke, v_exp=ve), want)


@pytest.mark.parametrize("Hq", [1, 8, 16])
@pytest.mark.parametrize("B", [2, 160])
def test_prefix_attn_single_tokens_in_parts_and_whole(B, Hq):
    """Few sequences are cut into parts, many are not: the same numbers within fp32
    roundings of the join."""
    far, ctx = [64], [7 * b % 300 for b in range(B)]
    case = _prefix_case(B, 1, 1, Hq, 1, 128, 16, far, ctx, HF, HF, seed=B)
    from test_gpu_serve import _check_prefix
    _check_prefix(case, far, ctx)
    q, kc, vc, ke, ve, ptable, table = case
    mask = torch.zeros((1, 1), dtype=torch.int32, device="cuda")           # the token does not see itself
    _check_prefix(case, far, ctx, mask=mask)
    _check_prefix(case, far, ctx, mask=mask, count=[b % 2 for b in range(B)])


def test_prefix_attn_refusals():
    q, kc, vc, ke, ve, ptable, table = _prefix_case(4, 2, 2, 4, 2, 64, 16, [50, 20], [9] * 4, BF, BF, seed=6)
    far, ctx = _i32([50, 20]), _i32([9] * 4)
    need = bd.load().sdv_prefix_attn_workspace(4, 2, 4, 64)
    for workspace in (64, need - 1):
        with pytest.raises(bd.SdvError) as e:
            bd.sdv_prefix_attn(q, kc, vc, ptable, far, table, ctx, workspace=torch.empty(workspace, dtype=torch.uint8, device="cuda"))
        assert e.value.status == bd.SDV_ERR_SCRATCH
    room = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(bd.sdv_prefix_attn(q, kc, vc, ptable, far, table, ctx, workspace=room),
                       bd.sdv_prefix_attn(q, kc, vc, ptable, far, table, ctx))
    with pytest.raises(ValueError):
        bd.sdv_prefix_attn(q, kc, vc, ptable, _i32([50, 20, 5]), table, ctx)   # groups do not divide the batch
    with pytest.raises(ValueError):
        bd.sdv_prefix_attn(q, kc, vc, ptable[:1], far, table, ctx)
    with pytest.raises(TypeError):
        bd.sdv_prefix_attn(q, kc, vc, ptable.long(), far, table, ctx)
    with pytest.raises(TypeError):
        bd.sdv_prefix_attn(q.float(), kc, vc, ptable, far, table, ctx)
    with pytest.raises(bd.SdvError):
        bd.sdv_prefix_attn(q[:, :, :3], kc, vc, ptable, far, table, ctx)
    with pytest.raises(bd.SdvError):
        bd.sdv_prefix_attn(q, kc, vc, ptable, far, table, ctx, scale=math.nan)
    with pytest.raises(ValueError):
        bd.sdv_prefix_attn(q, kc, vc, ptable, far, table, ctx, mask=torch.zeros((3, 1), dtype=torch.int32, device="cuda"))


def test_rows_and_pages_refusals():
    x = _rows((2, 3), 100, BF, 1)
    u = torch.zeros((2, 3), device="cuda")
    with pytest.raises(ValueError):
        bd.sdv_sample(x, u[:, :2])
    with pytest.raises(TypeError):
        bd.sdv_sample(x, u.double())
    with pytest.raises(TypeError):
        bd.sdv_sample(x.half(), u)
    with pytest.raises(ValueError):
        bd.sdv_sample(x, u, temperature=torch.ones(3, device="cuda"))
    with pytest.raises(TypeError):
        bd.sdv_sample(x, u, top_k=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        bd.sdv_logits_truncate(x, out=x[:, :2])
    with pytest.raises(ValueError):
        bd.sdv_logits_truncate(x.transpose(0, 1)[:, :, :50])
    with pytest.raises(bd.SdvError):
        bd.sdv_logits_truncate(x[:, :1], out=x.view(-1)[:200].view(2, 1, 100))          # the same rows with other strides
    pool, free, rows, held = _i32(list(range(9))), _i32([9]), torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), _i32([0, 0])
    with pytest.raises(ValueError):
        bd.sdv_pages_extend(pool, free, rows[:1], held, held, 3, 16)
    with pytest.raises(TypeError):
        bd.sdv_pages_extend(pool.long(), free, rows, held, held, 3, 16)
    with pytest.raises(ValueError):
        bd.sdv_pages_extend(pool, free, rows, held, held, 3, 16, depth=_i32([0, 0]))
    with pytest.raises(bd.SdvError):
        bd.sdv_pages_extend(pool, free, rows, held, held, 3, 0)
    with pytest.raises(ValueError):
        bd.sdv_pages_release(pool, _i32([9, 9]), rows, held, held, 16)
    assert bd.sdv_sample(x[:0], u[:0]).shape == (0, 3) and bd.sdv_logits_truncate(x[:, :0]).shape == (2, 0, 100)


def test_rows_beyond_2_31_bytes():
    """Offsets of rows pass 32 bits."""
    V, rows = 152064, 16000
    x = torch.zeros((rows, V), dtype=BF, device="cuda")
    x[:, 5] = 1.0
    x[-1, 150000] = 9.0
    x[rows // 2, 7] = 8.0
    cut = dict(top_k=_i32([1] * rows))
    got = bd.sdv_sample(x, torch.full((rows,), 0.5, device="cuda"), **cut)
    want = torch.full((rows,), 5, dtype=torch.int32, device="cuda")
    want[-1], want[rows // 2] = 150000, 7
    assert torch.equal(got, want)
    out, kept = bd.sdv_logits_truncate(x, kept=True, out=x, **cut)
    assert (kept == 1).all() and torch.equal((out[-2:] > -math.inf).nonzero()[:, 1].int().cpu(), torch.tensor([5, 150000], dtype=torch.int32))
    assert int((out[rows // 2] > -math.inf).nonzero()) == 7

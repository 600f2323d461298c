"""The verifier's-layer operators as a program uses them: a whole decoding loop
against a 64-bit model, calls on other streams and in a captured graph, the row
counts where another attention kernel takes over, and buffers beyond 2^31
elements."""
import os
import sys

import pytest
import torch

import layer_ref as ref
from draft_verification_sdv_gb300 import binding as bd
from test_gpu_layer import _attn_case, _cache, _check_attn, _i32, _status

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bd.load(build=True)


# ---- the decoding loop ----

def _model64(model, text):
    """Logits [len(text), V] in 64 bits, without a cache."""
    n, D, g = len(text), model.D, model.Hq // model.Hk
    x = model.embed.double().cpu()[torch.tensor(text)]
    norm = lambda y: y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    pos, freq = torch.arange(n), model.freq.cpu()
    for w_qkv, w_out, w_up, w_down in model.layers:
        q, k, v = (norm(x) @ w_qkv.double().cpu()).view(n, -1, D).split([model.Hq, model.Hk, model.Hk], dim=1)
        q, k = (ref.rope(t, pos, freq, model.factor, False)[0] for t in (q, k))
        k, v = k.repeat_interleave(g, dim=1), v.repeat_interleave(g, dim=1)
        s = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), -torch.inf)
        x = x + torch.einsum("hij,jhd->ihd", s.softmax(-1), v).reshape(n, -1) @ w_out.double().cpu()
        x = x + torch.nn.functional.silu(norm(x) @ w_up.double().cpu()) @ w_down.double().cpu()
    return norm(x) @ model.head.double().cpu()


# A logit has a spread of 2 and the best of 512 is some 6 above the mean.  About 27
# roundings to bf16 stand between the tokens and a logit, 2^-8 / sqrt(3) of a
# value each: 0.012 of the spread, and six times that is 0.15.  e4m3 cells are off
# by 2^-4 / sqrt(3) of their values: 0.05 of an attention output, at most 0.07
# of the spread after two layers, six times of which is 0.85.
@pytest.mark.parametrize("e4m3,slack", [(False, 0.25), (True, 1.0)])
@pytest.mark.parametrize("repetition,presence", [(1.0, 0.0), (1.25, 0.5)])
def test_decoding_loop(e4m3, slack, repetition, presence):
    import tree_decode as ex
    gen = torch.Generator().manual_seed(11)
    prompts = [torch.randint(0, 512, (n,), generator=gen).tolist() for n in (5, 40, 1)]
    model = ex.Model()
    d = ex.Decoder(model, prompts, room=200, page=16, e4m3=e4m3, repetition=repetition, presence=presence)
    steps = 24
    total = sum(sum(d.step()) for _ in range(steps))
    assert repetition > 1.0 or total > steps * len(prompts)          # drafts are accepted
    for b, prompt in enumerate(prompts):
        text = d.text[b]
        assert d.start[b].item() == len(text) - 1
        want = _model64(model, text[:-1])
        for i in range(len(prompt), len(text)):
            row = want[i - 1].clone()
            for t in set(text[:i]):
                row[t] = row[t] / repetition if row[t] > 0 else row[t] * repetition
            for t in set(text[len(prompt):i]):
                row[t] -= presence
            assert row[text[i]] >= row.max() - slack, (b, i)


def test_drafts_change_nothing_but_the_steps():
    """Drafts that repeat what an undrafted run gave are accepted whole wherever
    that run's choices were clear, and cells that were moved are those of a
    sequence written in one go."""
    import tree_decode as ex
    prompts = [[7, 300, 11], [500, 2, 2, 9]]
    model = ex.Model()
    none = torch.zeros((2, 2, 4), dtype=torch.int32, device="cuda"), _i32([0, 0])
    plain = ex.Decoder(model, prompts, K=2, G=4)
    for _ in range(12):
        assert plain.step(*none) == [1, 1]
    d = ex.Decoder(model, prompts, K=2, G=4)
    done = [0, 0]
    while min(done) < 8:
        drafts = torch.zeros((2, 2, 4), dtype=torch.int32)
        for b, p in enumerate(prompts):
            future = plain.text[b][len(p) + done[b]:][:4]
            drafts[b, 1, :len(future)] = torch.tensor(future, dtype=torch.int32)
            drafts[b, 0, :len(future)] = drafts[b, 1, :len(future)]
            drafts[b, 0, 1] = (drafts[b, 1, 1] + 1) % 512               # the other draft branches off
        got = d.step(drafts.cuda(), _i32([4, 4]))
        done = [a + n for a, n in zip(done, got)]
    for b, p in enumerate(prompts):
        n = min(len(d.text[b]), len(plain.text[b]))
        want = _model64(model, plain.text[b][:n]).topk(2).values
        clear = (want[:, 0] - want[:, 1] > 0.5).tolist()
        same = [x == y for x, y in zip(d.text[b][:n], plain.text[b][:n])]
        first = same.index(False) if False in same else n
        assert first == n or not clear[first - 1]
    for layer in range(len(model.layers)):
        rows = []
        for run in (d, plain):
            (kc, vc), _ = run.cache[layer]
            rows.append(bd.sdv_kv_read(kc, vc, run.table, _i32([0, 0]), 6))
        for x, y in zip(*rows):
            # the same tokens through products of other shapes: bf16 values, some 12
            # roundings of 2^-8 in, whose vectors have entries of about 1
            assert (x.float() - y.float()).abs().max() <= 12 * 2.0 ** -8 * 4


# ---- streams and graphs ----

def _layer_state(seed, cdtype=BF):
    B, K, G, Hq, Hk, D, V, P = 3, 2, 6, 8, 2, 64, 1000, 16
    g = torch.Generator(device="cuda").manual_seed(seed)
    drafts = torch.randint(0, 4, (B, K, G), generator=g, device="cuda", dtype=torch.int32)
    kc, vc, ke, ve = _cache(40, Hk, P, D, cdtype)
    qkv = torch.randn((B * (1 + K * G), Hq + 2 * Hk, D), generator=g, device="cuda").to(BF)
    return dict(drafts=drafts, root=_i32([1, 2, 3]), kc=kc, vc=vc, ke=ke, ve=ve,
                table=torch.arange(39, device="cuda", dtype=torch.int32).view(3, 13), start=_i32([0, 50, 130]), qkv=qkv,
                logits=torch.randn((B, 1 + K * G, V), generator=g, device="cuda"),
                counts=torch.zeros((B, V), dtype=torch.int32, device="cuda"),
                sel=_i32([0, 1, 0]), acc=_i32([2, 0, 6]), nxt=_i32([5, 6, 7]),
                freq=bd.sdv_rope_freqs(D), rep=torch.full((B,), 1.5, device="cuda"),
                ws=torch.empty(bd.load().sdv_tree_attn_workspace(), dtype=torch.uint8, device="cuda"), shape=(B, K, G, Hq, Hk, D))


def _layer_step(s, stream=None):
    B, K, G, Hq, Hk, D = s["shape"]
    N = 1 + K * G
    kw = dict(k_exp=s["ke"], v_exp=s["ve"], stream=stream)
    t = bd.sdv_tree_build(s["root"], s["drafts"], stream=stream)
    q, k, v = s["qkv"].split([Hq, Hk, Hk], dim=1)
    pos = (s["start"][:, None] + t["depth"]).reshape(-1)
    q, k = bd.sdv_rope(q, k, pos, *s["freq"], stream=stream)
    q, k, v = (x.unflatten(0, (B, N)) for x in (q, k, v))
    bd.sdv_kv_write(k, v, s["kc"], s["vc"], s["table"], s["start"], count=t["count"], **kw)
    o, lse = bd.sdv_tree_attn(q, s["kc"], s["vc"], s["table"], s["start"], count=t["count"], mask=t["mask"], lse=True,
                              workspace=s["ws"], **kw)
    rows = bd.sdv_logits_process(s["logits"], s["drafts"], counts=s["counts"], repetition=s["rep"], rows=t["rows"], stream=stream)
    new = bd.sdv_kv_commit(s["kc"], s["vc"], s["table"], s["start"], t["nodes"], s["sel"], s["acc"], **kw)
    bd.sdv_counts_commit(s["counts"], s["drafts"], s["sel"], s["acc"], s["nxt"], stream=stream)
    live = torch.arange(N, device="cuda") < t["count"][:, None]
    return [o, lse, rows, new, live]


def _state_of(s):
    return [x.clone() for x in (s["kc"], s["vc"], s["counts"])]


def _same(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8) if x.dtype == F8 else x, y.view(torch.uint8) if y.dtype == F8 else y)


@pytest.mark.parametrize("cdtype", [BF, F8])
def test_layer_on_another_stream(cdtype):
    s = _layer_state(5, cdtype)
    want = _layer_step(s) + _state_of(s)
    s = _layer_state(5, cdtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _layer_step(s)                                    # the current stream
    torch.cuda.current_stream().wait_stream(side)
    _same(want, got + _state_of(s))
    s = _layer_state(5, cdtype)
    B, K, G, Hq, Hk, D = s["shape"]
    t = bd.sdv_tree_build(s["root"], s["drafts"])
    q = torch.randn((B, 1 + K * G, Hq, D), device="cuda").to(BF)
    torch.cuda.synchronize()
    one = bd.sdv_tree_attn(q, s["kc"], s["vc"], s["table"], s["start"], mask=t["mask"], k_exp=s["ke"], v_exp=s["ve"])
    two = bd.sdv_tree_attn(q, s["kc"], s["vc"], s["table"], s["start"], mask=t["mask"], k_exp=s["ke"], v_exp=s["ve"], stream=side)
    side.synchronize()
    _same([one], [two])                                         # one that is named


@pytest.mark.parametrize("cdtype", [BF, F8])
def test_layer_in_a_graph(cdtype):
    s = _layer_state(6, cdtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _layer_step(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _layer_step(s)
    for seed in (7, 8):
        new = _layer_state(seed, cdtype)
        for n, x in s.items():
            if torch.is_tensor(x) and n != "ws":
                x.copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        _same(_layer_step(new) + _state_of(new), got + _state_of(s))


# ---- row counts where another kernel takes over; queries and scales of every kind ----

@pytest.mark.parametrize("dtype,cdtype", [(BF, BF), (HF, HF), (BF, F8), (HF, F8)])
@pytest.mark.parametrize("D,P", [(128, 16), (64, 8), (128, 12), (160, 16)])
@pytest.mark.parametrize("N,g", [(16, 1), (17, 1), (11, 3), (33, 1), (7, 7), (10, 5), (13, 5), (65, 1), (16, 5), (27, 3)])
def test_attn_row_counts(N, g, D, P, dtype, cdtype):
    case = _attn_case(2, N, 2 * g, 2, D, P, [150, 3], dtype, cdtype, seed=N * g)
    _check_attn(*case, [150, 3], count=[N, N - 1])


@pytest.mark.parametrize("N", [3, 40])
@pytest.mark.parametrize("cdtype", [BF, F8])
def test_attn_queries_anywhere_and_negative_scales(N, cdtype):
    q, *cache = _attn_case(2, N, 8, 1, 64, 16, [90, 200], BF, cdtype, seed=N)
    room = torch.zeros(q.numel() * 2 + 9, dtype=BF, device="cuda")
    for first, stride in ((1, 64), (8, 68), (3, 128)):          # two bytes off; odd strides
        view = room[first:].as_strided((2, N, 8, 64), (N * 8 * stride, 8 * stride, stride, 1))
        view.copy_(q)
        _check_attn(view, *cache, [90, 200])
        _check_attn(view, *cache, [90, 200], scale=-0.125)
    _check_attn(q, *cache, [90, 200], scale=0.0)


# ---- offsets beyond 2^31 elements ----

@pytest.mark.parametrize("N", [1, 20])
@pytest.mark.parametrize("cdtype", [BF, F8])
def test_cache_beyond_32_bits(N, cdtype):
    pages, H, P, D = 4, 2, 16, 64
    stride = (5 << 28) + 64                                       # elements of a page: page 2 begins past 2^31
    big = [torch.zeros(3 * stride + H * P * D, dtype=torch.uint8 if cdtype == F8 else cdtype, device="cuda").view(cdtype)
           for _ in range(2)]
    kc, vc = (x.as_strided((pages, H, P, D), (stride, P * D, D, 1)) for x in big)
    ke, ve = (torch.zeros((pages, H, P), dtype=torch.uint8, device="cuda") if cdtype == F8 else None for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn((1, 60, H, D), generator=g, device="cuda").to(BF)
    small = _cache(pages, H, P, D, cdtype)
    table, st = _i32([[3, 0, 2, 1]]), _status()
    out = []
    for k_, v_, ke_, ve_ in ((kc, vc, ke, ve), small):
        bd.sdv_kv_write(x, -x, k_, v_, table, _i32([0]), k_exp=ke_, v_exp=ve_, status=st)
        out.append(bd.sdv_kv_read(k_, v_, table, _i32([0]), 60, k_exp=ke_, v_exp=ve_, status=st) +
                   (bd.sdv_tree_attn(x[:, :N], k_, v_, table, _i32([60 - N]), k_exp=ke_, v_exp=ve_, status=st),))
    assert int(st) == 0
    _same(*out)


def test_logits_beyond_32_bits():
    B, K, G, V = 2, 64, 128, 132000                               # 2.18e9 logits a side
    lg = torch.zeros((B, K, G + 1, V), dtype=BF, device="cuda")
    lg[-1, -1, -1] = 3.0
    drafts = torch.zeros((B, K, G), dtype=torch.int32, device="cuda")
    counts = torch.zeros((B, V), dtype=torch.int32, device="cuda")
    counts[1, V - 1] = 2
    out = bd.sdv_logits_process(lg, drafts, counts=counts, frequency=torch.ones(B, device="cuda"))
    want = torch.full((V,), 3.0)
    want[V - 1], want[0] = 1.0, 3.0 - G                           # counted twice; the draft's tokens
    assert torch.equal(out[-1, -1, -1].float().cpu(), want)
    assert out[0, 0, 0].eq(0).all() and out[-1, -1, 0, V - 1] == -2

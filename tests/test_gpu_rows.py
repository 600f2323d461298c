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

"""Attention behind shared prefixes at its edges: block tables far wider than what the
sequences hold, as a server's are that has room for its longest request, waits that run
out, infinities."""
import math

import pytest
import torch

from draft_verification_sdv_gb300 import binding as bd
from test_gpu_layer import TYPES, _i32, _status
from test_gpu_serve import _check_prefix, _prefix_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bd.load(build=True)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("B,N,Hq,Hk,D,ctx", [(4, 1, 8, 1, 128, [0, 63, 64, 500]), (3, 1, 8, 2, 128, [1000, 255, 700]), (2, 1, 16, 2, 64, [1, 200]), (160, 1, 4, 1, 128, list(range(160))),
                                             (3, 4, 8, 2, 128, [0, 70, 300]), (2, 40, 8, 1, 64, [9, 128])])
def test_wide_tables(B, N, Hq, Hk, D, ctx, dtype, cdtype):
    far = [300]
    q, kc, vc, ke, ve, ptable, table = _prefix_case(B, 1, N, Hq, Hk, D, 16, far, ctx, dtype, cdtype, seed=B)
    # (entries that nothing is held in are no pages: they are not looked at)
    wide = torch.full((B, 2000), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    wptable = torch.full((1, 4000), 1 << 30, dtype=torch.int32, device="cuda")
    wptable[:, :ptable.shape[1]] = ptable
    _check_prefix((q, kc, vc, ke, ve, wptable, wide), far, ctx)
    st = _status()
    args = dict(k_exp=ke, v_exp=ve, lse=True, status=st)
    one = bd.sdv_prefix_attn(q, kc, vc, wptable, _i32(far), wide, _i32(ctx), **args)
    two = bd.sdv_prefix_attn(q, kc, vc, wptable, _i32(far), wide, _i32(ctx), **args)
    assert int(st) == 0 and all(torch.equal(a, b) for a, b in zip(one, two))
    # the same work is shared out the same way whatever the tables' width
    tight = bd.sdv_prefix_attn(q, kc, vc, ptable, _i32(far), table, _i32(ctx), **args)
    assert all(torch.equal(a, b) for a, b in zip(one, tight))


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("B,N,g,D,far,ctx", [(8, 1, 8, 128, 20000, 50), (6, 40, 4, 128, 20000, 300), (6, 40, 3, 64, 20000, 300), (4, 2, 2, 64, 20000, 300)])
def test_waits_that_run_out(B, N, g, D, far, ctx, dtype, cdtype):
    """A tile of the first block never comes, in the prefix's pass and in the own
    positions': what goes on from that block's rows is no number, the rest is right, and
    so is the next call."""
    # (20000 positions of four heads are 628 tiles of 128 or more: the first block has a second one)
    Hk, lens = 4, [ctx - b for b in range(B)]
    q, kc, vc, ke, ve, ptable, table = _prefix_case(B, 1, N, Hk * g, Hk, D, 16, [far], lens, dtype, cdtype, seed=N)
    call = lambda st: bd.sdv_prefix_attn(q, kc, vc, ptable, _i32([far]), table, _i32(lens), k_exp=ke, v_exp=ve, lse=True, status=st)  # noqa: E731
    good, good_lse = call(_status())
    st = _status()
    torch.cuda.synchronize()
    assert bd.sdv_set_attn_test_hooks(bd.SDV_HOOK_ATTN_NO_COPY) == bd.SDV_OK
    try:
        out, lse = call(st)
        torch.cuda.synchronize()
    finally:
        assert bd.sdv_set_attn_test_hooks(0) == bd.SDV_OK
    assert int(st) == bd.SDV_STATUS_TIMEOUT
    bad = out.isnan().all(-1)
    assert torch.equal(bad, lse.isnan()) and torch.equal(bad, out.isnan().any(-1))
    assert torch.equal(out[~bad], good[~bad]) and torch.equal(lse[~bad], good_lse[~bad])
    assert bad[0, 0, :g].all() and not bad.all()                # (the first block has the first head's first rows, 16 or more)
    again, again_lse = call(_status())
    assert torch.equal(again, good) and torch.equal(again_lse, good_lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,N,g,D,P", [(3, 1, 8, 128, 16), (60, 1, 16, 64, 16), (3, 1, 2, 96, 16), (3, 1, 8, 64, 12), (3, 9, 1, 64, 16), (3, 40, 4, 128, 16),
                                       (2, 30, 1, 192, 16)])
def test_infinities(B, N, g, D, P, dtype):
    """A score of -infinity has weight 0 on either side, and nodes that have no other have
    nothing; +infinity, an infinite value and NaN that a node sees make it not finite."""
    Hk, far, ctx = 2, [150], [7 + 31 * b % 120 for b in range(B)]
    q, kc, vc, ke, ve, ptable, table = _prefix_case(B, 1, N, Hk * g, Hk, D, P, far, ctx, dtype, dtype, seed=N)
    q = q.clone()
    q[..., 0] = 2.0
    gen = torch.Generator(device="cuda").manual_seed(N)
    kp = torch.randn((1, far[0], Hk, D), generator=gen, device="cuda").to(dtype)
    ko = torch.randn((B, max(ctx) + N, Hk, D), generator=gen, device="cuda").to(dtype)

    def run(fill, prefix=None, own=None, value=None):
        for k, where, t in ((kp, prefix, ptable), (ko, own, table)):
            kk, v = k.clone(), k.flip(1).clone()
            if where is not None:
                (kk if value is None else v)[:, where, :, 0] = fill if value is None else value
            bd.sdv_kv_write(kk, v, kc, vc, t, _i32([0] * k.shape[0]))
        st = _status()
        got = bd.sdv_prefix_attn(q, kc, vc, ptable, _i32(far), table, _i32(ctx), lse=True, status=st)
        assert int(st) == 0
        return got
    some, every = slice(3, None, 17), slice(None)
    for prefix, own in ((some, None), (None, some), (some, some), (every, None), (None, every), (every, some)):
        want, got = run(-6.0e4, prefix, own), run(-math.inf, prefix, own)
        assert want[0].isfinite().all() and torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    out, lse = run(-math.inf, every, every)
    assert not out.any() and (lse == -math.inf).all()
    for prefix, own in ((some, None), (None, slice(3, 4))):
        for fill in (math.inf, math.nan):
            assert not run(fill, prefix, own)[0].isfinite().all(-1).any()
        assert not run(0.0, prefix, own, value=math.inf)[0].isfinite().all(-1).any()

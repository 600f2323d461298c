"""The verifier's-layer operators where they can go wrong unseen: slots of
shared memory that are used again, waits that run out, powers of two that 16 bits
do not hold, streams, infinities, far positions, schedules of many units."""
import math
from fractions import Fraction

import pytest
import torch

import layer_ref as ref
from draft_verification_sdv_gb300 import binding as bd
from test_gpu_layer import _attn_case, _cache, _check_attn, _i32, _status, _tables

pytestmark = pytest.mark.gpu
BF, HF, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bd.load(build=True)


def _words(see):
    """Rows of truth values [N, N] as int32 words on the device."""
    N = see.shape[0]
    w = torch.zeros((N, (N + 31) // 32), dtype=torch.int64)
    for m in range(see.shape[1]):
        w[:, m // 32] |= see[:, m].long() << (m % 32)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32).cuda()


# ---- shared memory that is used again ----

@pytest.mark.parametrize("dtype,cdtype", [(BF, BF), (HF, HF), (BF, F8), (HF, F8)])
@pytest.mark.parametrize("B,N,g,D", [(96, 12, 1, 128), (96, 8, 2, 64), (96, 100, 2, 64), (40, 70, 4, 128)])
def test_attn_values_kept_out_do_not_reach_later_tiles(B, N, g, D, dtype, cdtype):
    """Values that are not numbers are zeroed in the slots of the ring, which later
    tiles of the same CTA use: with them, the outputs are those without."""
    Hk, ctx = 4, [130 + 37 * (b % 9) for b in range(B)]
    q, kc, vc, ke, ve, table = _attn_case(B, N, Hk * g, Hk, D, 16, ctx, dtype, cdtype, seed=N)
    see = torch.ones((N, N), dtype=torch.bool).tril()
    see[:, [2, N - 3]] = False
    mask = _words(see)
    out = []
    for val in (0.0, math.nan, math.inf):
        x = torch.full((B, 1, Hk, D), val, device="cuda", dtype=dtype)
        for node in (2, N - 3):
            bd.sdv_kv_write(x, x, kc, vc, table, _i32([c + node for c in ctx]), k_exp=ke, v_exp=ve)
        out.append(bd.sdv_tree_attn(q, kc, vc, table, _i32(ctx), mask=mask, k_exp=ke, v_exp=ve, lse=True))
    for o, lse in out[1:]:
        assert o.isfinite().all() and torch.equal(o, out[0][0]) and torch.equal(lse, out[0][1])


# ---- waits that run out ----

@pytest.mark.parametrize("dtype,cdtype", [(BF, BF), (HF, HF), (BF, F8), (HF, F8)])
@pytest.mark.parametrize("B,N,g,D,ctx", [
    (8, 1, 8, 128, 6000), (100, 2, 8, 64, 300), (8, 40, 4, 128, 6000), (8, 40, 3, 64, 6000), (100, 40, 4, 64, 300),
    (40, 80, 8, 128, 200), (400, 2, 8, 64, 300), (400, 40, 4, 64, 300)])
def test_attn_waits_that_run_out(B, N, g, D, ctx, dtype, cdtype):
    """A tile of the first block never comes: nothing of what the block writes after
    that is taken for a result, and the next call is right again."""
    Hk, lens = 4, [ctx - b % 7 for b in range(B)]
    case = _attn_case(B, N, Hk * g, Hk, D, 16, lens, dtype, cdtype, seed=N)
    q, kc, vc, ke, ve, table = case
    kw = dict(k_exp=ke, v_exp=ve, lse=True)
    good, good_lse = bd.sdv_tree_attn(q, kc, vc, table, _i32(lens), **kw)
    st = _status()
    torch.cuda.synchronize()
    assert bd.sdv_set_attn_test_hooks(bd.SDV_HOOK_ATTN_NO_COPY) == bd.SDV_OK
    try:
        out, lse = bd.sdv_tree_attn(q, kc, vc, table, _i32(lens), status=st, **kw)
        torch.cuda.synchronize()
    finally:
        assert bd.sdv_set_attn_test_hooks(0) == bd.SDV_OK
    assert int(st) == bd.SDV_STATUS_TIMEOUT
    bad = out.isnan().all(-1)
    assert torch.equal(bad, lse.isnan()) and torch.equal(bad, out.isnan().any(-1))
    assert torch.equal(out[~bad], good[~bad]) and torch.equal(lse[~bad], good_lse[~bad])
    rows = bad.view(B, N, Hk, g).transpose(1, 2).reshape(B * Hk, N * g)     # of each (sequence, head)
    assert rows[0, :256].all() and not rows.all()
    if N * g <= 256:                                            # a head's rows share their fate; later units too
        units = rows.all(1)
        assert torch.equal(rows.any(1), units)
        n = int(units.sum())
        assert units[:n].all() and (n > 1 or B < 300)
    again, again_lse = bd.sdv_tree_attn(q, kc, vc, table, _i32(lens), status=_status(), **kw)
    assert torch.equal(again, good) and torch.equal(again_lse, good_lse)


def test_attn_hooks_refused():
    assert bd.sdv_set_attn_test_hooks(1) == bd.SDV_ERR_ARG
    assert bd.sdv_set_attn_test_hooks(4) == bd.SDV_ERR_ARG


# ---- values of one channel that are far larger than the others ----

@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("N,g,D,P", [(12, 1, 64, 16), (1, 8, 128, 16), (60, 1, 96, 8), (12, 1, 128, 12), (60, 1, 64, 4),
                                     (9, 2, 192, 16)])
def test_attn_channels_beside_a_large_one(N, g, D, P, dtype):
    """Rows of e4m3 values in units of very different powers of two: what the small
    ones add keeps its digits."""
    B, Hk, ctx = 2, 2, [300, 40]
    q, kc, vc, ke, ve, table = _attn_case(B, N, Hk * g, Hk, D, P, ctx, dtype, F8, seed=N + D)
    gen = torch.Generator(device="cuda").manual_seed(N)
    k, v = (torch.randn((B, max(ctx) + N, Hk, D), generator=gen, device="cuda") for _ in range(2))
    v[:, 9::50, :, 3] = -65000.0
    bd.sdv_kv_write(k.to(dtype), v.to(dtype), kc, vc, table, _i32([0] * B), k_exp=ke, v_exp=ve)
    _check_attn(q, kc, vc, ke, ve, table, ctx)


# ---- powers of two of e4m3 rows that fp16 does not hold ----

@pytest.mark.parametrize("kind", ["large keys", "large values", "tiny keys", "top of fp16"])
@pytest.mark.parametrize("N,g,D,P", [(12, 1, 64, 16), (100, 1, 128, 16), (34, 3, 64, 8), (100, 1, 96, 12), (150, 2, 128, 32)])
def test_attn_fp16_queries_on_rows_beyond_fp16(N, g, D, P, kind):
    """An e4m3 row stands for more than fp16 holds: whatever the number of query
    rows, and so the kernel, finite rows give the finite answer."""
    B, Hk, ctx = 2, 2, [300, 40]
    write = HF if kind == "top of fp16" else BF
    q, kc, vc, ke, ve, table = _attn_case(B, N, Hk * g, Hk, D, P, ctx, write, F8, seed=N + D)
    gen = torch.Generator(device="cuda").manual_seed(N)
    k, v = (torch.randn((B, max(ctx) + N, Hk, D), generator=gen, device="cuda") for _ in range(2))
    q, scale = q.to(HF), D ** -0.5
    if kind == "large keys":                     # in a channel that the queries leave alone
        k[:, 7::31, :, 0] = 3.0e5
        q[..., 0] = 0.0
    elif kind == "large values":
        v[:, 5::61] *= 1.0e5
        v[:, 41] *= 1.0e30
        k[:, 41, :, 0], q[..., 0] = -1000.0, 16.0    # ... of a probability that is 0 even against that
    elif kind == "tiny keys":
        k *= 2.0 ** -18
        q, scale = q * 2.0 ** 12, 16.0 * 8 / D ** 0.5
    else:
        k[:, 7::31, :, 0] = 65000.0
        q[..., 0] = 0.0
        v[:, 9::50, :, 3] = -65000.0
    bd.sdv_kv_write(k.to(write), v.to(write), kc, vc, table, _i32([0] * B), k_exp=ke, v_exp=ve)
    st = _status()
    out, lse = bd.sdv_tree_attn(q, kc, vc, table, _i32(ctx), scale=scale, k_exp=ke, v_exp=ve, lse=True, status=st)
    assert int(st) == 0
    v0 = vc.cpu()
    if kind == "large values":                   # the reference without what has no weight
        for row in table.cpu():
            v0.view(torch.uint8)[row[41 // P], :, 41 % P] = 0
    want, wl, tol, tl = ref.attn(q.cpu(), kc.cpu(), v0, table.cpu(), ctx, None, None, scale, ke.cpu(), ve.cpu())
    got, top = out.double().cpu(), 65504.0
    over = want.abs() > top + tol                # more than fp16 holds: infinite, of its sign
    assert torch.equal(got[over], want[over].sign() * math.inf) and not got.isnan().any()
    fin = want.abs() < top - tol
    assert ((got - want).abs()[fin] <= tol[fin]).all(), float(((got - want).abs()[fin] / tol[fin]).max())
    assert fin.sum() > 0.9 * fin.numel() and ((lse.double().cpu() - wl).abs() <= tl).all()
    # and from one call to the next: rows that fp16 holds again
    one = torch.randn(k.shape, generator=gen, device="cuda").to(write)
    bd.sdv_kv_write(one, one, kc, vc, table, _i32([0] * B), k_exp=ke, v_exp=ve)
    _check_attn(q if kind != "tiny keys" else q * 2.0 ** -12, kc, vc, ke, ve, table, ctx)


# ---- outputs of calls on a named stream ----

def _calls():
    """Each call that makes its own outputs, as a function of the stream."""
    B, K, G, Hq, Hk, D, V, P = 3, 2, 6, 8, 2, 64, 1000, 16
    drafts, root = _i32([[[1] * G, [2] * G]] * B), _i32([1, 2, 3])
    kc, vc, _, _ = _cache(40, Hk, P, D, BF)
    table, start = _tables(B, 12, 40, 1), _i32([0, 50, 130])
    q, k = torch.randn((30, Hq, D), device="cuda").to(BF), torch.randn((30, Hk, D), device="cuda").to(BF)
    pos, (freq, factor) = torch.arange(30, dtype=torch.int32, device="cuda"), bd.sdv_rope_freqs(D)
    tree = bd.sdv_tree_build(root, drafts)
    logits = torch.randn((B, K, G + 1, V), device="cuda")
    qt = torch.randn((B, 1 + K * G, Hq, D), device="cuda").to(BF)
    sel = _i32([0, 1, 0])
    torch.cuda.synchronize()
    return {
        "tree": lambda s: list(bd.sdv_tree_build(root, drafts, stream=s).values()),
        "rope": lambda s: list(bd.sdv_rope(q, k, pos, freq, factor, stream=s)),
        "read": lambda s: list(bd.sdv_kv_read(kc, vc, table, start, 20, stream=s)),
        "commit": lambda s: [bd.sdv_kv_commit(kc, vc, table, start, tree["nodes"], sel, sel, stream=s)],
        "attn": lambda s: list(bd.sdv_tree_attn(qt, kc, vc, table, start, mask=tree["mask"], lse=True, stream=s)),
        "logits": lambda s: [bd.sdv_logits_process(logits, drafts, stream=s)],
    }


def _wait():
    torch.cuda._sleep(200_000_000)          # about 0.1 s on the current stream


@pytest.mark.parametrize("named", ["object", "handle", "default"])
@pytest.mark.parametrize("name", ["tree", "rope", "read", "commit", "attn", "logits"])
def test_outputs_on_a_named_stream(name, named):
    """Neither is a block that the current stream still uses written by the call's
    stream, nor one of the call's handed out again while the current stream reads it."""
    call = _calls()[name]
    side = torch.cuda.Stream()
    stream = {"object": side, "handle": side.cuda_stream, "default": 0}[named]
    here = torch.cuda.current_stream() if named != "default" else torch.cuda.Stream()
    want = [x.clone() for x in call(None)]
    torch.cuda.synchronize()
    with torch.cuda.stream(here):
        blocks = [torch.full_like(x, 7) for x in want for _ in range(3)]
        _wait()
        copies = [x.clone() for x in blocks]        # still to come when the blocks go
        used = {x.untyped_storage().data_ptr() for x in blocks}
        del blocks
        out = call(stream)
        assert not used & {x.untyped_storage().data_ptr() for x in out}
        torch.cuda.synchronize()
        assert all((x == 7).all() for x in copies)
        for x, y in zip(out, want):
            assert torch.equal(x, y)
        _wait()
        reads = [x.clone() for x in out]            # the caller's reads, on its stream
        used = {x.untyped_storage().data_ptr() for x in out}
        x = y = None
        del out
        again = call(stream)
        assert not used & {x.untyped_storage().data_ptr() for x in again}
        torch.cuda.synchronize()
        for x, y in zip(reads, want):
            assert torch.equal(x, y)


# ---- infinite keys ----

@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("N,g,D,P", [(1, 8, 128, 16), (12, 1, 64, 16), (40, 4, 64, 16), (60, 3, 128, 16), (12, 1, 64, 12),
                                     (60, 1, 192, 16)])
def test_attn_infinite_keys(N, g, D, P, dtype):
    """A score of -infinity has weight 0, +infinity is not a number, and nodes whose
    scores are all -infinity have nothing."""
    Hk, ctx = 2, [200]
    q, kc, vc, ke, ve, table = _attn_case(1, N, Hk * g, Hk, D, P, ctx, dtype, dtype, seed=N)
    q = q.clone()
    q[..., 0] = 2.0
    gen = torch.Generator(device="cuda").manual_seed(N)
    k = torch.randn((1, ctx[0] + N, Hk, D), generator=gen, device="cuda").to(dtype)
    at = torch.zeros(ctx[0] + N, dtype=torch.bool)
    at[3::17] = True
    at[ctx[0]] = False                          # (the first node sees itself)

    def run(fill, where):
        kk = k.clone()
        kk[0, where, :, 0] = fill
        bd.sdv_kv_write(kk, k.flip(1), kc, vc, table, _i32([0]))
        return bd.sdv_tree_attn(q, kc, vc, table, _i32(ctx), lse=True)

    want, got = run(-6.0e4, at), run(-math.inf, at)
    assert want[0].isfinite().all() and torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    out, lse = run(math.inf, at)
    assert not out.isfinite().all(-1).any()
    none, lse = run(-math.inf, torch.ones_like(at))
    assert not none.any() and (lse == -math.inf).all()


# ---- sampling parameters ----

@pytest.mark.parametrize("dtype", [F32, BF])
def test_logits_repetition_is_a_quotient(dtype):
    """x / repetition, rounded once (bf16: from a quotient two roundings of fp32 off at
    most), for factors whose reciprocal is rounded, infinite or next to zero too."""
    reps = [1.3, 3.0, 0.7, 1.0e-39, 3.0e38, 49.0]
    B, V = len(reps), 4096
    gen = torch.Generator().manual_seed(2)
    x = torch.randn((B, 1, 2, V), generator=gen) * torch.exp2(torch.randint(-60, 20, (B, 1, 2, V), generator=gen).float())
    x, rep = x.to(dtype), torch.tensor(reps)
    counts = torch.ones((B, V), dtype=torch.int32, device="cuda")
    drafts = torch.zeros((B, 1, 1), dtype=torch.int32, device="cuda")
    out = bd.sdv_logits_process(x.cuda(), drafts, counts=counts, repetition=rep.cuda()).cpu()
    r = rep.view(B, 1, 1, 1).double()
    want = torch.where(x > 0, x.double() / r, x.double() * r)
    if dtype == F32:
        assert torch.equal(out, want.float())
        return
    over = want.abs() > 3.395e38                                # past bf16's largest by half a step
    assert torch.equal(out[over], (want[over].sign() * math.inf).to(BF))
    fin = want.abs() < 3.38e38
    tol = (2.0 ** -8 + 2.0 ** -22) * want.abs() + 2.0 ** -133
    assert ((out.double() - want).abs()[fin] <= tol[fin]).all()


# ---- rotary positions far away ----

def test_rope_angles_at_any_position():
    """Angles to 2^-26 of a turn, by whole-number arithmetic on frequency and position
    with 1 / (2 pi) to 50 digits."""
    turn = Fraction(10 ** 50, 2 * 314159265358979323846264338327950288419716939937511)
    freq = torch.tensor([1.0, 0.7598, 100.3, 1.0e-4, 0.1, 6.0e5, -3.7, 0.0], dtype=torch.float32)
    pos = [2 ** 31 - 1, -2 ** 31, 1234567891, 16777217, -7, 0]
    half = len(freq)
    q = torch.zeros((len(pos), 1, 2 * half), device="cuda")
    q[..., :half] = 1.0                                  # (1, 0) turns to (cos, sin)
    out = bd.sdv_rope(q, None, _i32(pos), freq.cuda())[0].double().cpu()[:, 0]
    # the angle, and sine and cosine to two units of fp32
    tol = 2 * math.pi * (2.0 ** -26 + 2.0 ** -32) + 2 * 2.0 ** -24
    for i, p in enumerate(pos):
        for j, f in enumerate(freq.tolist()):
            part = p * Fraction(f) * turn
            angle = 2 * math.pi * float(part - round(part))
            assert abs(float(out[i, j]) - math.cos(angle)) <= tol, (p, f)
            assert abs(float(out[i, half + j]) - math.sin(angle)) <= tol, (p, f)


# ---- schedules: more units than blocks, in rounds and a line of unequal parts ----

def _definition(q, kc, vc, ke, ve, table, ctx, count, mask, scale):
    """ref.attn's results and tolerances for whole sequences at once, in 64 bits on
    the device, sequence by sequence: (out, lse, tol_out, tol_lse)."""
    B, N, Hq, D = q.shape
    Hk, half = kc.shape[1], ref.HALF_STEP[q.dtype]
    g = Hq // Hk
    for b in range(B):
        c, n = ctx[b], count[b]
        see = torch.ones((n, c + n), dtype=torch.bool, device="cuda")
        i = torch.arange(n, device="cuda")
        if mask is None:
            see[:, c:] = i[None, :] <= i[:, None]
        else:
            see[:, c:] = (mask[b, :n][:, i // 32] >> (i % 32).int() & 1).bool()
        out = torch.zeros((N, Hq, D), dtype=torch.float64, device="cuda")
        lse = torch.full((N, Hq), -math.inf, dtype=torch.float64, device="cuda")
        tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
        k, v = (ref.sequence(t, e, table[b], c + n) for t, e in ((kc, ke), (vc, ve)))
        for h in range(Hq):
            x, kh, vh = q[b, :n, h].double(), k[:, h // g], v[:, h // g]
            s = (x @ kh.T * scale).masked_fill(~see, -math.inf)
            size = (x.abs() @ kh.abs().T).masked_fill(~see, 0.0).amax(1) * abs(scale)
            ds = (D + 8) * 2.0 ** -24 * size + 4 * 2.0 ** -24 * s.masked_fill(~see, 0.0).abs().amax(1) + 2.0 ** -20
            p = s.softmax(1)
            out[:n, h], lse[:n, h] = p @ vh, s.logsumexp(1)
            tol[:n, h] = half * out[:n, h].abs() + (half + 2 * ds)[:, None] * (p @ vh.abs()) * 1.01 + 2 * ref.FLOOR[q.dtype]
            if q.dtype == HF:
                tol[:n, h] += 2.0 ** -24 * (see.double() @ vh.abs())
            tol_l[:n, h] = ds + 2.0 ** -23 * lse[:n, h].abs()
        yield out, lse, tol, tol_l


@pytest.mark.parametrize("dtype,cdtype", [(BF, BF), (HF, HF), (BF, F8), (HF, F8)])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,K,G,Hq,Hk,D", [(24, 10, 32, 16, 8, 64), (13, 20, 30, 12, 6, 128)])
def test_attn_in_rounds(B, K, G, Hq, Hk, D, tree, dtype, cdtype):
    gen = torch.Generator(device="cuda").manual_seed(B)
    N, ctx = 1 + K * G, [(b * 977) % 1900 if b % 5 else 3 * b for b in range(B)]
    drafts = torch.randint(0, 9, (B, K, G), generator=gen, device="cuda", dtype=torch.int32)
    t = bd.sdv_tree_build(_i32([0] * B), drafts, _i32([G - b % 3 for b in range(B)]))
    count = t["count"].tolist()
    tiles = -(-N * (Hq // Hk) // 256)
    assert tiles > 1 and B * Hk * tiles >= 2 * torch.cuda.get_device_properties(0).multi_processor_count
    q, kc, vc, ke, ve, table = _attn_case(B, N, Hq, Hk, D, 16, ctx, dtype, cdtype, seed=B)
    mask, st = (t["mask"] if tree else None), _status()
    out, lse = bd.sdv_tree_attn(q, kc, vc, table, _i32(ctx), count=t["count"], mask=mask, k_exp=ke, v_exp=ve, lse=True,
                                status=st)
    assert int(st) == 0
    for b, (want, wl, tol, tl) in enumerate(_definition(q, kc, vc, ke, ve, table, ctx, count, mask, D ** -0.5)):
        assert ((out[b].double() - want).abs() <= tol).all(), b
        fin = wl > -math.inf
        assert torch.equal(lse[b] > -math.inf, fin) and ((lse[b].double() - wl).abs()[fin] <= tl[fin]).all(), b


# ---- rows that are not written ----

@pytest.mark.parametrize("cdtype", [BF, F8])
@pytest.mark.parametrize("N", [3, 40])
def test_kv_rows_that_are_refused_leave_the_cells(N, cdtype):
    """Every byte of a cache after writes of which some are refused is that of the
    cache with the others alone."""
    H, D, P, per = 2, 32, 4, 12
    gen = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn((2, N, H, D), generator=gen, device="cuda").to(BF)
    y = -2.0 * x
    table = _tables(2, per, 2 * per, 1)
    off = table.clone()
    off[1, 0], off[0, 1] = 2 * per, -1
    places = per * P
    bits = bd.SDV_STATUS_BAD_LENGTH
    for start, count, pages, want in (([-1, 0], [N, N], table, bits), ([places - 2, 0], [N, 2], table, bits),
                                      ([0, 0], [N + 1, 2], table, bits), ([0, 5], [-1, N], table, bits),
                                      ([-2 ** 31, 2 ** 31 - 1], [N, N], table, bits),
                                      ([2, 2], [N, N], off, bd.SDV_STATUS_BAD_PAGE)):
        caches = []
        for alone in (False, True):
            kc, vc, ke, ve = _cache(2 * per, H, P, D, cdtype)
            for t in (kc, vc):
                t.view(torch.uint8).fill_(0x11)
            for t in (ke, ve):
                if t is not None:
                    t.fill_(99)
            if not alone:
                st = _status()
                bd.sdv_kv_write(x, y, kc, vc, pages, _i32(start), count=_i32(count), k_exp=ke, v_exp=ve, status=st)
                assert int(st) == want
            else:                                # the good rows one by one
                for b in range(2):
                    for n in range(N):
                        pos = start[b] + n
                        if not 0 <= count[b] <= N or n >= count[b] or not 0 <= pos < places:
                            continue
                        if 0 <= int(pages[b, pos // P]) < 2 * per:
                            bd.sdv_kv_write(x[b:b + 1, n:n + 1], y[b:b + 1, n:n + 1], kc, vc, pages[b:b + 1].contiguous(),
                                            _i32([pos]), k_exp=ke, v_exp=ve)
            caches.append([t.contiguous().view(torch.uint8) for t in (kc, vc, ke, ve) if t is not None])
        for a, b in zip(*caches):
            assert torch.equal(a, b), (start, count)


# ---- caches whose strides are those of dimensions of one entry ----

@pytest.mark.parametrize("cdtype", [BF, F8])
@pytest.mark.parametrize("pages,H,P", [(9, 1, 16), (60, 2, 1), (60, 1, 1), (1, 2, 64), (1, 1, 64)])
def test_cache_strides_that_mean_nothing(pages, H, P, cdtype):
    D, N, ctx = 64, 9, 40
    views = [t if t is None else t.as_strided(t.shape, [7 if n == 1 else x for n, x in zip(t.shape, t.stride())])
             for t in _cache(pages, H, P, D, cdtype)]
    plain = _cache(pages, H, P, D, cdtype)
    assert any(a is not None and a.stride() != b.stride() for a, b in zip(views, plain))
    x = torch.randn((1, ctx + N, H, D), device="cuda").to(BF)
    q = torch.randn((1, N, 3 * H, D), device="cuda").to(BF)
    table = torch.arange(-(-(ctx + N) // P), dtype=torch.int32, device="cuda")[None]
    res = []
    for kc, vc, ke, ve in (views, plain):
        kw = dict(k_exp=ke, v_exp=ve)
        bd.sdv_kv_write(x, -x, kc, vc, table, _i32([0]), **kw)
        bd.sdv_kv_commit(kc, vc, table, _i32([ctx]), _i32([[[3, 5]]]), _i32([0]), _i32([2]), **kw)
        res.append(bd.sdv_kv_read(kc, vc, table, _i32([0]), ctx + N, **kw) +
                   (bd.sdv_tree_attn(q, kc, vc, table, _i32([ctx]), **kw),))
    for a, b in zip(*res):
        assert torch.equal(a, b)
    good = _cache(4, 2, 8, D, cdtype)
    for i in (0, 1) if cdtype == BF else (0, 1, 2, 3):       # what is not contiguous is refused
        bad = list(good)
        bad[i] = bad[i].transpose(1, 2).contiguous().transpose(1, 2)
        with pytest.raises(ValueError):
            bd.sdv_kv_read(bad[0], bad[1], _i32([[0]]), _i32([0]), 1, k_exp=bad[2], v_exp=bad[3])


# ---- biases that would be passed over ----

def test_logits_biases_of_the_wrong_size_are_refused():
    x = torch.randn((2, 1, 3, 64), device="cuda").to(BF)
    d = _i32([[[1, 2]], [[3, 4]]])
    one, f = _i32([5]), torch.ones(1, device="cuda")
    for ids, bias in ((one, f), (None, f), (one, None), (_i32([1, 2, 3]), torch.ones(3, device="cuda")),
                      (_i32([[1], [2]]), torch.ones((2, 2), device="cuda"))):
        with pytest.raises(ValueError):
            bd.sdv_logits_process(x, d, bias_ids=ids, bias=bias)
    none = torch.empty((2, 0), device="cuda")
    assert torch.equal(bd.sdv_logits_process(x, d, bias_ids=none.int(), bias=none), x)


# ---- captured calls ----

@pytest.mark.parametrize("large", [False, True])
def test_attn_redo_in_a_graph(large):
    """fp16 queries on an e4m3 cache: what a replay finds in the cache decides, not
    what was there when the call was captured."""
    B, N, Hk, g, D, ctx = 2, 50, 2, 3, 64, [100, 170]
    q, kc, vc, ke, ve, table = _attn_case(B, N, Hk * g, Hk, D, 16, ctx, HF, F8, seed=4)
    lens = _i32(ctx)
    kw = dict(k_exp=ke, v_exp=ve, lse=True)

    def fill(big):
        gen = torch.Generator(device="cuda").manual_seed(5 + big)
        v = torch.randn((B, max(ctx) + N, Hk, D), generator=gen, device="cuda").to(BF)
        if big:
            v[:, 20] *= 1.0e5
        bd.sdv_kv_write(v / 4, v, kc, vc, table, _i32([0] * B), k_exp=ke, v_exp=ve)

    fill(large)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bd.sdv_tree_attn(q, kc, vc, table, lens, **kw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = bd.sdv_tree_attn(q, kc, vc, table, lens, **kw)
    for big in (not large, large, not large):
        fill(big)
        graph.replay()
        want, wl = bd.sdv_tree_attn(q, kc, vc, table, lens, **kw)
        # (a key of 25000 has all the weight of some rows, whose value of 1e5 fp16 does not hold)
        assert torch.equal(out, want) and torch.equal(lse, wl) and not out.isnan().any()
        assert big or out.isfinite().all()

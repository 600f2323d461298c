"""The verifier's-layer operators on the GPU against plain 64-bit
implementations (tests/layer_ref.py), at the sizes, types, strides and masks
where each can go wrong, with the tolerances that their roundings give."""
import math

import pytest
import torch

import layer_ref as ref
from draft_verification_sdv_gb300 import binding as bd

pytestmark = pytest.mark.gpu
BF, HF, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bd.load(build=True)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- draft tree ----

@pytest.mark.parametrize("B,K,G,words,ragged", [(1, 1, 1, 5, False), (3, 4, 7, 2, False), (2, 16, 32, 2, True),
                                                (2, 5, 1, 2, False), (1, 64, 128, 2, False), (4, 3, 6, 50, True)])
def test_tree_build(B, K, G, words, ragged):
    gen = torch.Generator().manual_seed(B * 100 + K + G)
    drafts = torch.randint(0, words, (B, K, G), generator=gen, dtype=torch.int32)
    root = torch.randint(0, 99, (B,), generator=gen, dtype=torch.int32)
    lens = torch.randint(0, G + 1, (B,), generator=gen, dtype=torch.int32) if ragged else None
    st = _status()
    out = bd.sdv_tree_build(root.cuda(), drafts.cuda(), None if lens is None else lens.cuda(), status=st)
    got = {k: t.cpu() for k, t in out.items()}
    assert int(st) == 0
    N = 1 + K * G
    for b in range(B):
        L = G if lens is None else int(lens[b])
        tokens, depth, parent, nodes = ref.tree(int(root[b]), drafts[b].tolist(), L)
        n = len(tokens)
        assert int(got["count"][b]) == n
        assert got["tokens"][b].tolist() == tokens + [-1] * (N - n)
        assert got["depth"][b].tolist() == depth + [0] * (N - n)
        for k in range(K):
            assert got["nodes"][b, k].tolist() == nodes[k] + [-1] * (G - L)
            assert got["rows"][b, k].tolist() == [0] + nodes[k] + [0] * (G - L)
        want = torch.zeros((N, N), dtype=torch.bool)
        for i in range(n):
            m = i
            while m >= 0:
                want[i, m] = True
                m = parent[m]
        bits = (got["mask"][b][:, :, None] >> torch.arange(32)) & 1
        bits = bits.view(N, -1).bool()
        assert torch.equal(bits[:, :N], want) and not bits[:, N:].any()


def test_tree_build_bad_length():
    st = _status()
    out = bd.sdv_tree_build(_i32([1, 2]), _i32([[[1, 2]], [[3, 4]]]), _i32([3, 2]), status=st)
    assert int(st) == bd.SDV_STATUS_BAD_LENGTH
    assert out["count"].tolist() == [1, 3] and out["tokens"][0].tolist() == [1, -1, -1]


# ---- rotary positions ----

@pytest.mark.parametrize("T,Hq,Hk,D,R,inter,dtype,far", [
    (1, 8, 1, 128, 128, False, BF, 100), (5, 7, 2, 64, 64, True, HF, 5000), (9, 3, 3, 96, 96, False, F32, 1 << 20),
    (3, 2, 1, 80, 32, False, BF, 900), (4, 1, 1, 128, 64, True, F32, 2 ** 31 - 1), (6, 2, 1, 10, 6, False, BF, 50),
    (6, 2, 1, 9, 2, True, HF, 50), (67, 28, 4, 128, 128, False, BF, 30000), (2, 3, 0, 256, 256, False, HF, 77),
    (1300, 2, 1, 64, 64, False, BF, 4000)])
def test_rope(T, Hq, Hk, D, R, inter, dtype, far):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    pad = 3 if D in (10, 9) else 8
    buf = torch.randn((T, (Hq + Hk) * D + pad), generator=g, device="cuda").to(dtype)
    q = buf[:, :Hq * D].view(T, Hq, D)
    k = buf[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D) if Hk else None
    pos = torch.randint(-far if far < 1000 else 0, far, (T,), generator=g, device="cuda").to(torch.int32)
    pos[-1] = far
    freq, _ = bd.sdv_rope_freqs(R)
    oq, ok = bd.sdv_rope(q, k, pos, freq, factor=1.25, interleaved=inter)
    # the angle is off by at most 2^-32 of a turn and the rounding of its last
    # 32 bits to fp32, sine and cosine by two units, then the pair's products
    for x, y in ((q, oq), (k, ok)) if Hk else ((q, oq),):
        want, mag = ref.rope(x, pos, freq, 1.25, inter)
        turn = 2.0 ** -24 * (2 * math.pi) + 8 * 2.0 ** -24
        tol = ref.HALF_STEP[dtype] * want.abs() + turn * mag * 1.01 + ref.FLOOR[dtype]
        assert ((y.double().cpu() - want).abs() <= tol).all()
        assert torch.equal(y[..., R:], x[..., R:])
    if k is not None:                              # in place, the same bits
        q2, k2 = q.clone(), k.clone()
        bd.sdv_rope(q2, k2, pos, freq, factor=1.25, interleaved=inter, out_q=q2, out_k=k2)
        assert torch.equal(q2, oq) and torch.equal(k2, ok)


def test_rope_edges():
    freq, _ = bd.sdv_rope_freqs(64)
    q = torch.randn((0, 2, 64), device="cuda").to(BF)
    assert bd.sdv_rope(q, None, _i32([]), freq)[0].shape == (0, 2, 64)
    q = torch.randn((2, 2, 64), device="cuda")
    assert torch.equal(bd.sdv_rope(q, None, _i32([0, 0]), freq)[0], q)
    bad = freq.clone()
    bad[3] = math.inf
    y = bd.sdv_rope(q, None, _i32([1, 2]), bad)[0]
    assert y[..., 3].isnan().all() and y[..., 35].isnan().all() and int(y.isnan().sum()) == 8
    with pytest.raises(ValueError):
        bd.sdv_rope(q, None, _i32([1]), freq)
    with pytest.raises(bd.SdvError):
        bd.sdv_rope(q, None, _i32([1, 2]), torch.ones(40, device="cuda"))        # R > D
    with pytest.raises(bd.SdvError):                                             # in place, other strides
        big = torch.zeros((2, 4, 64), device="cuda")
        bd.sdv_rope(big[:, :2], None, _i32([1, 2]), freq, out_q=big.view(-1)[:256].view(2, 2, 64))


# ---- paged cache ----

def _cache(pages, H, P, D, dtype, split=False):
    if split:                                      # k and v as the halves of one buffer
        buf = torch.zeros((pages, 2, H, P, D), dtype=torch.uint8 if dtype == F8 else dtype, device="cuda")
        kc, vc = buf[:, 0], buf[:, 1]
        if dtype == F8:
            kc, vc = kc.view(F8), vc.view(F8)
    else:
        kc, vc = (torch.zeros((pages, H, P, D), dtype=dtype, device="cuda") for _ in range(2))
    if dtype != F8:
        return kc, vc, None, None
    e = torch.zeros((pages, 2, H, P), dtype=torch.uint8, device="cuda")
    return kc, vc, e[:, 0], e[:, 1]


def _tables(B, per, pages, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(pages, generator=g)[:B * per].view(B, per).to(torch.int32).cuda()


@pytest.mark.parametrize("B,N,H,D,P,dtype,cdtype,split", [
    (1, 1, 1, 64, 16, BF, BF, False), (3, 5, 2, 128, 16, BF, F8, False), (2, 33, 4, 96, 8, HF, F8, True),
    (2, 7, 3, 16, 1, HF, HF, False), (2, 9, 1, 256, 5, BF, F8, True), (1, 40, 8, 80, 64, BF, BF, True),
    (4, 3, 5, 48, 7, BF, F8, False)])
def test_kv_write_and_read(B, N, H, D, P, dtype, cdtype, split):
    g = torch.Generator(device="cuda").manual_seed(N + D)
    per = -(-(N + 13) // P)
    pages = B * per + 3
    kc, vc, ke, ve = _cache(pages, H, P, D, cdtype, split)
    table = _tables(B, per, pages, D)
    start = _i32([(5 * b) % 13 for b in range(B)])
    count = _i32([N - (b % 2) * (N // 2) for b in range(B)])
    qkv = torch.randn((B, N, 3, H, D), generator=g, device="cuda")
    qkv *= torch.exp2(torch.randint(-20, 8, (B, N, 3, H, 1), generator=g, device="cuda").float())
    qkv[0, 0, 1, 0] = 0.0
    qkv = qkv.to(dtype)
    qkv[:, 0, 2, 0, 0] = 448.0 if dtype == BF else 447.0
    k, v = qkv[:, :, 1], qkv[:, :, 2]
    st = _status()
    bd.sdv_kv_write(k, v, kc, vc, table, start, count=count, k_exp=ke, v_exp=ve, status=st)
    assert int(st) == 0
    written = torch.zeros((pages, P), dtype=torch.bool)
    for b in range(B):
        for n in range(int(count[b])):
            pos = int(start[b]) + n
            page, off = int(table[b, pos // P]), pos % P
            written[page, off] = True
            for x, cells, exps in ((k, kc, ke), (v, vc, ve)):
                row = cells[page, :, off].float().cpu()
                if cdtype != F8:
                    assert torch.equal(row, x[b, n].float().cpu())
                    continue
                for h in range(H):
                    q, e = ref.quantise_row(x[b, n, h].tolist())
                    assert e == int(exps[page, h, off])
                    assert row[h].tolist() == q
    for cells in (kc, vc):                          # nothing else was touched
        left = cells.float().cpu().transpose(1, 2)[~written]
        assert not left.any()
    rk, rv = bd.sdv_kv_read(kc, vc, table, start, N, count=count, k_exp=ke, v_exp=ve, dtype=dtype, status=st)
    assert int(st) == 0
    for b in range(B):
        c = int(count[b])
        for got, cells, exps in ((rk, kc, ke), (rv, vc, ve)):
            want = torch.stack([ref.cells(cells.cpu().float() if cdtype == F8 else cells.cpu(),
                                          None if exps is None else exps.cpu(), table[b].cpu(),
                                          int(start[b]) + n, P) for n in range(c)])
            assert torch.equal(got[b, :c].cpu(), want.to(dtype))
            assert not got[b, c:].any()


def test_kv_write_not_numbers_and_bad_places():
    H, D, P = 2, 32, 4
    kc, vc, ke, ve = _cache(4, H, P, D, F8)
    x = torch.randn((2, 3, H, D), device="cuda").to(BF)
    x[0, 1, 1, 5] = math.nan
    x[0, 2, 0, 7] = -math.inf
    st = _status()
    table = _i32([[0, 1], [2, 9]])
    bd.sdv_kv_write(x, x, kc, vc, table, _i32([0, 2]), k_exp=ke, v_exp=ve, status=st)
    assert int(st) == bd.SDV_STATUS_BAD_PAGE            # sequence 1's third row is on page 9
    rk, _ = bd.sdv_kv_read(kc, vc, table, _i32([0, 2]), 3, k_exp=ke, v_exp=ve)
    assert rk[0, 1, 1].isnan().all() and rk[0, 2, 0].isnan().all() and rk[1, 2].isnan().all()
    assert int(rk.isnan().any(-1).sum()) == 4
    for start, count in (([-1, 0], [3, 3]), ([6, 0], [3, 2]), ([0, 0], [4, 2]), ([0, 0], [-1, 2])):
        st.zero_()
        before = kc.float().clone()
        bd.sdv_kv_write(x, x, kc, vc, _i32([[0, 1], [2, 3]]), _i32(start), count=_i32(count), k_exp=ke, v_exp=ve,
                        status=st)
        assert int(st) == bd.SDV_STATUS_BAD_LENGTH
        del before
    torch.cuda.synchronize()


@pytest.mark.parametrize("cdtype,P", [(BF, 4), (F8, 16)])
def test_kv_commit_moves_the_accepted_path(cdtype, P):
    B, K, G, H, D = 5, 3, 6, 2, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    drafts = torch.randint(0, 3, (B, K, G), generator=g, device="cuda", dtype=torch.int32)
    t = bd.sdv_tree_build(_i32([7] * B), drafts)
    N = 1 + K * G
    per = -(-(N + 11) // P)
    kc, vc, ke, ve = _cache(B * per, H, P, D, cdtype)
    table = _tables(B, per, B * per, 1)
    start = _i32([0, 3, 11, 5, 2])
    k, v = (torch.randn((B, N, H, D), generator=g, device="cuda").to(BF) for _ in range(2))
    bd.sdv_kv_write(k, v, kc, vc, table, start, count=t["count"], k_exp=ke, v_exp=ve)
    whole = lambda: bd.sdv_kv_read(kc, vc, table, _i32([0] * B), per * P, k_exp=ke, v_exp=ve)  # noqa: E731
    bk, bv = whole()
    sel, acc = [0, 2, 1, -1, 2], [6, 4, 0, -1, 6]
    st = _status()
    new = bd.sdv_kv_commit(kc, vc, table, start, t["nodes"], _i32(sel), _i32(acc), k_exp=ke, v_exp=ve, status=st)
    assert int(st) == 0
    assert new.tolist() == [7, 8, 12, 5, 9]
    ak, av = whole()
    for b in range(B):
        path = [] if sel[b] < 0 else t["nodes"][b, sel[b], :acc[b]].tolist()
        s = int(start[b])
        for old, got in ((bk, ak), (bv, av)):
            want = old[b].clone()
            for j, n in enumerate(path):
                want[s + 1 + j] = old[b, s + n]
            assert torch.equal(got[b], want)
    # a path that does not grow, a length that is too long: reported, the length stays
    for nodes, acc in ((_i32([[[2, 2]]]), 2), (_i32([[[1, 2]]]), 3), (_i32([[[0, 1]]]), 1)):
        st.zero_()
        new = bd.sdv_kv_commit(kc, vc, table[:1].contiguous(), _i32([1]), nodes, _i32([0]), _i32([acc]), k_exp=ke,
                               v_exp=ve, status=st)
        assert int(st) == bd.SDV_STATUS_BAD_LENGTH and new.tolist() == [1]


# ---- tree attention ----

def _attn_case(B, N, Hq, Hk, D, P, ctx, dtype, cdtype, seed, count=None, split=False, spread=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = -(-(max(ctx) + N) // P) + 1
    pages = B * per + 2
    kc, vc, ke, ve = _cache(pages, Hk, P, D, cdtype, split)
    table = _tables(B, per, pages, seed)
    L = max(ctx) + N
    k, v = (torch.randn((B, L, Hk, D), generator=g, device="cuda") for _ in range(2))
    if spread:                                     # rows of very different magnitudes
        v *= torch.exp2(torch.randint(-spread, spread, (B, L, Hk, 1), generator=g, device="cuda").float())
    bd.sdv_kv_write(k.to(dtype), v.to(dtype), kc, vc, table, _i32([0] * B), k_exp=ke, v_exp=ve)
    q = torch.randn((B, N, Hq + 1, D), generator=g, device="cuda").to(dtype)[:, :, :Hq]   # strided
    return q, kc, vc, ke, ve, table


def _check_attn(q, kc, vc, ke, ve, table, ctx, count=None, mask=None, scale=None):
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    st = _status()
    out, lse = bd.sdv_tree_attn(q, kc, vc, table, _i32(ctx), count=None if count is None else _i32(count),
                                mask=mask, scale=scale, k_exp=ke, v_exp=ve, lse=True, status=st)
    assert int(st) == 0
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    want, wl, tol, tl = ref.attn(q.cpu(), cpu(kc), cpu(vc), table.cpu(), ctx, count, cpu(mask), scale, cpu(ke), cpu(ve))
    err = (out.double().cpu() - want).abs()
    assert not out.isnan().any()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())
    lse = lse.double().cpu()
    assert torch.equal(lse == -math.inf, wl == -math.inf)
    fin = wl > -math.inf
    assert ((lse - wl).abs()[fin] <= tl[fin]).all(), float(((lse - wl).abs()[fin] / tl[fin]).max())
    return out


TYPES = [(BF, BF), (HF, HF), (BF, F8), (HF, F8)]


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("B,N,Hq,Hk,D,P,ctx", [
    (1, 1, 1, 1, 64, 16, [0]), (1, 1, 8, 1, 128, 16, [1]), (3, 1, 8, 2, 128, 16, [0, 129, 700]),
    (2, 1, 7, 7, 96, 5, [300, 63]), (2, 1, 4, 2, 16, 1, [40, 17]), (1, 2, 8, 1, 256, 32, [333]),
    (2, 9, 8, 2, 128, 16, [0, 250]), (1, 70, 3, 1, 64, 8, [100]), (2, 33, 5, 1, 80, 64, [127, 128]),
    (1, 40, 2, 1, 192, 16, [65])])
def test_attn_chain(B, N, Hq, Hk, D, P, ctx, dtype, cdtype):
    case = _attn_case(B, N, Hq, Hk, D, P, ctx, dtype, cdtype, seed=B + N + D, split=P == 16)
    _check_attn(*case, ctx)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("B,K,G,Hq,Hk,D,ctx", [(2, 3, 5, 4, 1, 64, [0, 77]), (1, 4, 16, 8, 1, 128, [130]),
                                               (2, 5, 7, 2, 2, 96, [33, 126])])
def test_attn_tree(B, K, G, Hq, Hk, D, ctx, dtype, cdtype):
    g = torch.Generator(device="cuda").manual_seed(K)
    drafts = torch.randint(0, 3, (B, K, G), generator=g, device="cuda", dtype=torch.int32)
    t = bd.sdv_tree_build(_i32([0] * B), drafts)
    N = 1 + K * G
    case = _attn_case(B, N, Hq, Hk, D, 16, ctx, dtype, cdtype, seed=G)
    count = t["count"].tolist()
    out = _check_attn(*case, ctx, count=count, mask=t["mask"])
    for b in range(B):
        assert not out[b, count[b]:].any()


# many query rows: row tiles of 256 in streams of 128, cut and whole units
@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("B,N,Hq,Hk,D,P,ctx", [
    (1, 65, 1, 1, 128, 16, [0]), (1, 17, 8, 1, 64, 16, [5]), (2, 30, 8, 1, 128, 16, [200, 0]),
    (1, 129, 1, 1, 128, 7, [300]), (1, 257, 2, 1, 16, 16, [127]), (2, 100, 6, 2, 96, 32, [129, 1]),
    (1, 300, 3, 1, 48, 1, [513]), (3, 40, 10, 2, 80, 64, [0, 1000, 31]), (1, 70, 7, 1, 112, 16, [64])])
def test_attn_many_rows(B, N, Hq, Hk, D, P, ctx, dtype, cdtype):
    case = _attn_case(B, N, Hq, Hk, D, P, ctx, dtype, cdtype, seed=B + N + D, split=P == 16)
    count = [N - 3 * b for b in range(B)]
    _check_attn(*case, ctx, count=count)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("B,K,G,Hq,Hk,D,ctx", [(2, 8, 16, 4, 1, 128, [1, 250]), (1, 16, 16, 2, 1, 64, [0]),
                                               (3, 4, 31, 6, 2, 96, [97, 3, 128])])
def test_attn_large_tree(B, K, G, Hq, Hk, D, ctx, dtype, cdtype):
    g = torch.Generator(device="cuda").manual_seed(K)
    drafts = torch.randint(0, 4, (B, K, G), generator=g, device="cuda", dtype=torch.int32)
    t = bd.sdv_tree_build(_i32([0] * B), drafts)
    case = _attn_case(B, 1 + K * G, Hq, Hk, D, 16, ctx, dtype, cdtype, seed=G)
    _check_attn(*case, ctx, count=t["count"].tolist(), mask=t["mask"])


@pytest.mark.parametrize("dtype,cdtype", [(BF, BF), (HF, F8)])
@pytest.mark.parametrize("tree", [False, True])
def test_attn_more_units_than_the_machine_holds(dtype, cdtype, tree):
    """Row tiles enough for whole rounds and a line cut into unequal parts; the
    reference is each sequence by itself (which few CTAs share)."""
    B, K, G, Hq, Hk, D, P = 9, 10, 32, 16, 8, 64, 16
    N = 1 + K * G
    ctx = [700, 3, 0, 1500, 130, 90, 2100, 40, 513]
    g = torch.Generator(device="cuda").manual_seed(3)
    drafts = torch.randint(0, 9, (B, K, G), generator=g, device="cuda", dtype=torch.int32)
    t = bd.sdv_tree_build(_i32([0] * B), drafts)
    mask = t["mask"] if tree else None
    q, kc, vc, ke, ve, table = _attn_case(B, N, Hq, Hk, D, P, ctx, dtype, cdtype, seed=31)
    st = _status()
    out, lse = bd.sdv_tree_attn(q, kc, vc, table, _i32(ctx), count=t["count"], mask=mask, k_exp=ke, v_exp=ve, lse=True,
                                status=st)
    assert int(st) == 0
    half = ref.HALF_STEP[dtype]
    for b in range(B):
        o, x = bd.sdv_tree_attn(q[b:b + 1], kc, vc, table[b:b + 1].contiguous(), _i32(ctx[b:b + 1]),
                                count=t["count"][b:b + 1].contiguous(), k_exp=ke, v_exp=ve, lse=True,
                                mask=None if mask is None else mask[b:b + 1].contiguous())
        # the same probabilities, their references and their order of summing apart
        err = (out[b].double() - o[0].double()).abs()
        assert (err <= 2 * half * o[0].double().abs() + 2 * half * 4).all()
        assert float(err.square().mean().sqrt()) <= half * float(o[0].double().square().mean().sqrt())
        fin = x[0] > -math.inf
        assert torch.equal(fin, lse[b] > -math.inf) and (lse[b] - x[0])[fin].abs().max() <= 2.0 ** -16
    # and one sequence against the definition
    few = [2, 40, 77]
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    want, wl, tol, tl = ref.attn(q[1:2].cpu(), cpu(kc), cpu(vc), table[1:2].cpu(), ctx[1:2], [78], cpu(mask[1:2]) if tree else None,
                                 D ** -0.5, cpu(ke), cpu(ve))
    got = out[1:2, few].double().cpu()
    assert ((got - want[:, few]).abs() <= tol[:, few]).all()


@pytest.mark.parametrize("dtype,cdtype", TYPES)
def test_attn_growing_scores(dtype, cdtype):
    """Scores that grow along the positions, so that the running maximum moves
    at every tile, by little and by much."""
    ctx, N, Hq, D = [700], 40, 4, 64
    for slope in (0.01, 0.2):
        q, kc, vc, ke, ve, table = _attn_case(1, N, Hq, 1, D, 16, ctx, dtype, cdtype, seed=12)
        k, v = (torch.randn((1, 740, 1, D), device="cuda") for _ in range(2))
        k[..., 0] = torch.arange(740, device="cuda").view(1, 740, 1) * slope
        bd.sdv_kv_write(k.to(dtype), v.to(dtype), kc, vc, table, _i32([0]), k_exp=ke, v_exp=ve)
        q = q.clone()
        q[..., 0] = 8.0
        _check_attn(q, kc, vc, ke, ve, table, ctx)


@pytest.mark.parametrize("heads", [4, 12])
@pytest.mark.parametrize("cdtype", [BF, F8])
def test_attn_rows_that_see_nothing_and_what_is_not_seen(cdtype, heads):
    B, N, Hq, Hk, D, P = 3, 40, heads, 2, 64, 16
    ctx = [0, 0, 90]
    q, kc, vc, ke, ve, table = _attn_case(B, N, Hq, Hk, D, P, ctx, BF, cdtype, seed=9)
    count = [40, 0, 37]
    gen = torch.Generator().manual_seed(5)
    see = torch.rand((N, N), generator=gen) < 0.3
    see[3] = False
    see[:, [7, 21]] = False                                       # nodes that nobody sees
    see[11, 7] = True                                             # ... but one
    words = torch.zeros((N, 2), dtype=torch.int64)
    for m in range(N):
        words[:, m // 32] |= see[:, m].long() << (m % 32)
    mask = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32).cuda()
    ref_out = _check_attn(q, kc, vc, ke, ve, table, ctx, count, mask)
    assert not ref_out[0, 3].any() and not ref_out[1].any() and not ref_out[2, 37:].any()
    # not-a-numbers where nobody looks: past the nodes, on unseen nodes, on pages of nobody
    x = torch.full((B, 1, Hk, D), math.nan, device="cuda", dtype=BF)
    inf = torch.full((B, 1, Hk, D), math.inf, device="cuda", dtype=BF)
    for b in range(B):
        for node, val in ((21, x), (7, inf)):
            bd.sdv_kv_write(val[:1], val[:1], kc, vc, table[b:b + 1].contiguous(), _i32([ctx[b] + node]),
                            k_exp=ke, v_exp=ve)
    # (position 37 of sequence 2 is past its nodes, position 0 of sequence 1 too)
    bd.sdv_kv_write(x[:1], inf[:1], kc, vc, table[2:].contiguous(), _i32([90 + 37]), k_exp=ke, v_exp=ve)
    bd.sdv_kv_write(x[:1], inf[:1], kc, vc, table[1:2].contiguous(), _i32([0]), k_exp=ke, v_exp=ve)
    out, lse = bd.sdv_tree_attn(q, kc, vc, table, _i32(ctx), count=_i32(count), mask=mask, k_exp=ke, v_exp=ve, lse=True)
    bad = torch.zeros((B, N), dtype=torch.bool)
    bad[0, 11] = bad[2, 11] = True                                # sees node 7's infinities
    assert torch.equal(out.isfinite().all(-1).all(-1).cpu(), ~bad)
    assert torch.equal(out.cpu()[~bad], ref_out.cpu()[~bad])


@pytest.mark.parametrize("dtype,cdtype", TYPES)
def test_attn_values_of_very_different_magnitudes(dtype, cdtype):
    ctx = [200]
    case = _attn_case(1, 3, 4, 1, 64, 16, ctx, dtype, cdtype, seed=2, spread=9)
    _check_attn(*case, ctx)


def test_attn_zero_values_and_tiny_ones_in_e4m3():
    q, kc, vc, ke, ve, table = _attn_case(1, 1, 2, 1, 64, 16, [300], BF, F8, seed=3)
    z = torch.zeros((1, 301, 1, 64), device="cuda", dtype=BF)
    bd.sdv_kv_write(z, z, kc, vc, table, _i32([0]), k_exp=ke, v_exp=ve)
    out, lse = bd.sdv_tree_attn(q, kc, vc, table, _i32([300]), k_exp=ke, v_exp=ve, lse=True)
    assert not out.any() and (lse - math.log(301)).abs().max() < 1e-5
    t = torch.full((1, 301, 1, 64), 2.0 ** -100, device="cuda", dtype=BF)
    bd.sdv_kv_write(z, t, kc, vc, table, _i32([0]), k_exp=ke, v_exp=ve)
    out = bd.sdv_tree_attn(q, kc, vc, table, _i32([300]), k_exp=ke, v_exp=ve)
    assert ((out.double() * 2.0 ** 100 - 1).abs() <= 2.0 ** -8).all()


def test_attn_bad_page_does_not_spread():
    """A bad page after tiles with flagged values: only rows that see one of the two are not numbers."""
    N, ctx = 300, [600]
    q, kc, vc, ke, ve, table = _attn_case(1, N, 2, 1, 64, 16, ctx, BF, BF, seed=16)
    x = torch.full((1, 1, 1, 64), math.nan, device="cuda", dtype=BF)
    bd.sdv_kv_write(x, x, kc, vc, table, _i32([600 + 40]))
    bad = table.clone()
    bad[0, 53] = 10 ** 6                                      # positions 848 .. 863: nodes 248 .. 263
    out = bd.sdv_tree_attn(q, kc, vc, bad, _i32(ctx))
    fin = out.isfinite().all(-1).all(-1)[0].cpu()
    assert fin[:40].all() and not fin[40:].any()
    st = _status()
    bd.sdv_kv_write(torch.zeros_like(x), torch.zeros_like(x), kc, vc, table, _i32([600 + 40]))
    good = bd.sdv_tree_attn(q, kc, vc, table, _i32(ctx))
    out = bd.sdv_tree_attn(q, kc, vc, bad, _i32(ctx), status=st)
    assert int(st) == bd.SDV_STATUS_BAD_PAGE
    fin = out.isfinite().all(-1).all(-1)[0].cpu()
    assert fin[:248].all() and not fin[248:].any()
    assert torch.equal(out[0, :248], good[0, :248])


@pytest.mark.parametrize("N", [5, 50])
def test_attn_large_scores(N):
    q, kc, vc, ke, ve, table = _attn_case(1, N, 4, 2, 64, 16, [150], BF, BF, seed=8)
    _check_attn(q * 30, kc, vc, ke, ve, table, [150], scale=4.0)
    _check_attn(q, kc, vc, ke, ve, table, [150], scale=0.0)
    _check_attn(q, kc, vc, ke, ve, table, [150], scale=-0.3)


@pytest.mark.parametrize("N", [2, 60])
@pytest.mark.parametrize("cdtype", [BF, F8])
def test_attn_bad_lengths_and_pages(N, cdtype):
    q, kc, vc, ke, ve, table = _attn_case(4, N, 4, 2, 64, 16, [50] * 4, BF, cdtype, seed=6)
    st = _status()
    kw = {"k_exp": ke, "v_exp": ve}
    good = bd.sdv_tree_attn(q, kc, vc, table, _i32([50] * 4), **kw)
    out, lse = bd.sdv_tree_attn(q, kc, vc, table, _i32([50, -1, 50, 10 ** 6]), count=_i32([N, N, N + 1, N]),
                                lse=True, status=st, **kw)
    assert int(st) == bd.SDV_STATUS_BAD_LENGTH
    assert out[1:].isnan().all() and lse[1:].isnan().all() and torch.equal(out[0], good[0])
    st.zero_()
    bad = table.clone()
    bad[2, 1] = 10 ** 6
    bad[3, 0] = -5
    out = bd.sdv_tree_attn(q, kc, vc, bad, _i32([50] * 4), status=st, **kw)
    assert int(st) == bd.SDV_STATUS_BAD_PAGE
    assert out[2:].isnan().all() and torch.equal(out[:2], good[:2])


def test_attn_refusals():
    q, kc, vc, ke, ve, table = _attn_case(2, 2, 4, 2, 64, 16, [50] * 2, BF, BF, seed=6)
    ctx = _i32([50, 50])
    with pytest.raises(ValueError):
        bd.sdv_tree_attn(q, kc, vc, table, ctx, mask=torch.zeros((2, 3, 1), dtype=torch.int32, device="cuda"))
    with pytest.raises(bd.SdvError):
        bd.sdv_tree_attn(q[:, :, :3], kc, vc, table, ctx)                       # heads do not divide
    with pytest.raises(bd.SdvError):
        bd.sdv_tree_attn(q.to(HF), kc, vc, table, ctx)                          # another type than the cells
    with pytest.raises(TypeError):
        bd.sdv_tree_attn(q.float(), kc, vc, table, ctx)
    with pytest.raises(bd.SdvError):
        bd.sdv_tree_attn(q, kc, vc, table, ctx, scale=math.inf)
    with pytest.raises(bd.SdvError) as e:
        bd.sdv_tree_attn(q, kc, vc, table, ctx, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == bd.SDV_ERR_SCRATCH
    with pytest.raises(ValueError):
        bd.sdv_tree_attn(q, kc, vc, table[:1], ctx)
    with pytest.raises(TypeError):
        bd.sdv_tree_attn(q, kc, vc, table.long(), ctx)
    with pytest.raises(ValueError):
        bd.sdv_tree_attn(q, kc.cpu(), vc, table, ctx)
    with pytest.raises(ValueError):
        bd.sdv_tree_attn(q, kc.transpose(1, 2), vc.transpose(1, 2), table, ctx)


# ---- sampling parameters ----

@pytest.mark.parametrize("B,K,G,V,dtype,M,tree,allow,some", [
    (1, 1, 1, 8, BF, 0, False, False, True), (2, 3, 4, 2056, BF, 5, False, True, True),
    (2, 2, 9, 1028, F32, 40, True, True, True), (1, 4, 6, 4104, F32, 0, True, False, False),
    (1, 2, 33, 264, BF, 1500, True, True, True), (3, 1, 2, 40, BF, 3, False, False, False)])
def test_logits_process(B, K, G, V, dtype, M, tree, allow, some):
    g = torch.Generator(device="cuda").manual_seed(V)
    rnd = lambda *s: torch.randint(0, V, s, generator=g, device="cuda").to(torch.int32)  # noqa: E731
    W = -(-V // 32)
    src = (B, 1 + K * G, V) if tree else (B, K, G + 1, V)
    x = (torch.randn(src, generator=g, device="cuda") * 4).to(dtype)
    x.view(-1)[3] = -math.inf
    x.view(-1)[5] = math.inf
    drafts = rnd(B, K, G) % max(2, V // 3)
    drafts[0, 0, 0] = V + 5                                  # an id of nothing
    if G > 1:
        drafts[0, 0, 1] = -3
    rows = torch.randint(0, 1 + K * G, (B, K, G + 1), generator=g, device="cuda").to(torch.int32) if tree else None
    kw = {"rows": rows}
    if some:
        kw["counts"] = (rnd(B, V) % 4 - 1).clamp(min=0).to(torch.int32)
        kw["prompt"] = torch.randint(-2 ** 31, 2 ** 31, (B, W), generator=g, device="cuda").to(torch.int32)
        kw["repetition"] = torch.rand(B, generator=g, device="cuda") + 0.7
        kw["frequency"] = torch.randn(B, generator=g, device="cuda")
        kw["presence"] = torch.randn(B, generator=g, device="cuda")
    if M:
        kw["bias_ids"] = rnd(B, M)
        kw["bias_ids"][0, 0] = V
        kw["bias_ids"][0, 1:3] = 4                           # one id twice
        kw["bias"] = torch.randn((B, M), generator=g, device="cuda")
    if allow:
        kw["allow"] = torch.randint(-2 ** 31, 2 ** 31, (B, K, G + 1, W), generator=g, device="cuda").to(torch.int32)
        kw["allow"][0, 0, 0] = 0                             # nothing at all
    st = _status()
    out = bd.sdv_logits_process(x, drafts, status=st, **kw)
    assert int(st) == 0 and out.dtype == dtype
    c = lambda n: kw[n].cpu() if kw.get(n) is not None else None  # noqa: E731
    want, mag = ref.logits(x.cpu(), c("rows"), drafts.cpu(), c("counts"), c("prompt"), c("repetition"),
                           c("frequency"), c("presence"), c("bias_ids"), c("bias"), c("allow"))
    got = out.double().cpu()
    fin = want.isfinite()
    assert torch.equal(got[~fin], want[~fin])
    # a quotient, the products and sums of at most M / 8 + 4 terms in fp32, then one rounding
    tol = ref.HALF_STEP[dtype] * want.abs() + (M + 8) * 2.0 ** -24 * mag + ref.FLOOR[dtype]
    assert ((got - want).abs()[fin] <= tol[fin]).all()
    if not tree:                                             # in place, the same bits
        y = x.clone()
        bd.sdv_logits_process(y, drafts, out=y, **kw)
        assert torch.equal(y, out)


def test_logits_process_neutral_is_a_copy_and_refusals():
    x = torch.randn((2, 1, 3, 64), device="cuda").to(BF)
    d = _i32([[[1, 2]], [[3, 4]]])
    assert torch.equal(bd.sdv_logits_process(x, d), x)
    st = _status()
    y = bd.sdv_logits_process(x[:, 0], d, rows=_i32([[[0, 3, 1]], [[2, -1, 0]]]), status=st)
    assert int(st) == bd.SDV_STATUS_BAD_LENGTH
    assert y[0, 0, 1].isnan().all() and y[1, 0, 1].isnan().all() and torch.equal(y[0, 0, 2], x[0, 0, 1])
    with pytest.raises(ValueError):
        bd.sdv_logits_process(x[:, :, :2], d)
    with pytest.raises(TypeError):
        bd.sdv_logits_process(x.half(), d)
    with pytest.raises(bd.SdvError):
        bd.sdv_logits_process(torch.zeros((2, 1, 3, 12), device="cuda", dtype=BF), d)
    with pytest.raises(ValueError):
        bd.sdv_logits_process(x, d, counts=_i32([[0] * 63] * 2))
    with pytest.raises(ValueError):
        bd.sdv_logits_process(x, d, bias_ids=_i32([[1], [2]]), bias=torch.zeros((2, 2), device="cuda"))


def test_counts_commit():
    B, K, G, V = 6, 3, 5, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    d = torch.randint(0, V, (B, K, G), generator=g, device="cuda").to(torch.int32)
    d[4, 1, 0] = V
    counts = torch.randint(0, 3, (B, V), generator=g, device="cuda").to(torch.int32)
    want = counts.clone()
    sel, acc, nxt = [0, 2, 1, -1, 1, 0], [5, 0, 3, -1, 2, 6], [3, 9, 31, -1, 2, 2]
    for b in (0, 1, 2, 4):
        for tok in d[b, sel[b], :acc[b]].tolist() + [nxt[b]]:
            if 0 <= tok < V:
                want[b, tok] += 1
    st = _status()
    bd.sdv_counts_commit(counts, d, _i32(sel), _i32(acc), _i32(nxt), status=st)
    assert torch.equal(counts, want)
    assert int(st) == bd.SDV_STATUS_BAD_TOKEN | bd.SDV_STATUS_BAD_LENGTH

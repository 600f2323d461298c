"""The serving loop's operators without a GPU: the host references against small
cases worked by hand, and refusals."""
import math

import pytest
import torch

import serve_ref as sref
from draft_verification_sdv_gb300 import binding as bd


@pytest.fixture(scope="module")
def lib():
    return bd.load(build=True)


def test_reference_pages_by_hand():
    s = sref.Pages([4, 9, 2, 7], [[0, -1, -1], [1, 3, -1]], [1, 2], 4, 10)
    positions, slots = s.extend([3, 8], 3, base=[100, 0])
    assert positions.tolist() == [[103, 104, 105], [8, 9, 10]]
    assert slots.tolist() == [[3, 28, 29], [8, 9, 10]]           # page 7 for the first, 2 for the second
    assert s.table == [[0, 7, -1], [1, 3, 2]] and s.held == [2, 3] and s.stack == [4, 9] and s.status == 0
    s.release([3, 8])
    assert s.stack == [4, 9, 2, 7] and s.held == [1, 2] and s.table == [[0, -1, -1], [1, 3, -1]]
    s.release([0, 5])
    assert s.stack == [4, 9, 2, 7, 0] and s.held == [0, 2]
    s = sref.Pages([5], [[0, -1, -1], [1, -1, -1], [2, 3, -1]], [1, 1, 2], 4, 10)
    _, slots = s.extend([4, 4, 7], 5, count=[5, 1, 1])
    assert s.status == 128 and s.held == [1, 1, 2] and slots[2].tolist() == [15, -1, -1, -1, -1]


def test_reference_draws_by_hand():
    x = [1.0, 2.0, 2.0, 0.5, -math.inf]
    one = 2 ** 44
    assert sref.choose(x, top_k=1) == ([1], [one])
    assert sref.choose(x, top_p=0.5)[0] == [1, 2]               # 1 / (2 + e^-1 + e^-1.5) = 0.39
    assert sref.choose(x, top_p=0.25)[0] == [1]
    assert sref.choose(x, min_p=0.3)[0] == [1, 2, 0]
    assert sref.choose(x, T=0.0) == ([1], [one])
    idx, w = sref.choose(x)
    assert idx == [1, 2, 0, 3] and abs(w[2] / one - math.exp(-1)) < 1e-12
    assert [sref.drawn(idx, w, u)[0] for u in (0.0, 0.5, 0.9, 0.999)] == [1, 2, 0, 3]
    assert abs(sref.drawn(idx, w, 0.5)[1] + math.log(2 + math.exp(-1) + math.exp(-1.5))) < 1e-9


def test_reference_prefix_by_hand():
    # one prefix position and one of the sequence's own: two keys on pages apart
    q = torch.zeros((1, 1, 1, 16), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    k = torch.zeros((3, 1, 2, 16), dtype=torch.bfloat16)
    v = torch.full((3, 1, 2, 16), math.nan, dtype=torch.bfloat16)
    k[2, 0, 0, 0], k[1, 0, 0, 0] = 1.0, 2.0
    v[2, 0, 0], v[1, 0, 0] = 1.0, 0.0
    out, lse, _, _ = sref.prefix_attn(q, k, v, torch.tensor([[2]]), [1], torch.tensor([[1]]), [0], None, None, 1.0)
    e = math.exp
    assert abs(float(out[0, 0, 0, 3]) - e(1) / (e(1) + e(2))) < 1e-12
    assert abs(float(lse[0, 0, 0]) - math.log(e(1) + e(2))) < 1e-12


def test_entry_points_refuse_null_and_host_pointers(lib):
    host = torch.zeros(4096, dtype=torch.int32)
    p = host.data_ptr()
    cache = bd._KVCache(p, p, None, None, 16 * 64, 0, 1, 16, 1, 64, bd.SDV_BF16)
    E = bd.SDV_ERR_ARG
    assert lib.sdv_pages_extend(1, 1, 8, 16, 8, None, *[None] * 11) == E
    assert lib.sdv_pages_extend(1, 1, 8, 16, 8, None, *[p] * 11) == E
    assert lib.sdv_pages_release(1, 8, 16, 8, None, *[None] * 6) == E
    assert lib.sdv_pages_release(1, 8, 16, 8, None, *[p] * 6) == E
    assert lib.sdv_prefix_attn(None, 1, 1, 1, 1, 0, None, p, 64, 64, 64, p, 1, p, p, 1, p, None, None, 0, 1.0, p,
                               None, p, 1 << 30, None) == E
    assert lib.sdv_prefix_attn(cache, 1, 1, 1, 1, 0, None, p, 64, 64, 64, p, 1, p, p, 1, p, None, None, 0, 1.0, p,
                               None, p, 1 << 30, None) == E
    assert lib.sdv_sample(1, 1, 64, 0, None, None, 64, *[None] * 9) == E
    assert lib.sdv_sample(1, 1, 64, 0, None, p, 64, None, None, None, None, p, p, None, None, None) == E
    assert lib.sdv_logits_truncate(1, 1, 64, 0, None, p, 64, None, None, None, None, p, 64, None, None) == E


@pytest.mark.parametrize("rows,per,V,dtype,step", [
    (-1, 1, 64, 0, 64), (3, 2, 64, 0, 64), (2, 0, 64, 0, 64), (2, 1, 0, 0, 64), (2, 1, (1 << 19) + 1, 0, 1 << 20),
    (2, 1, 64, bd.SDV_F16, 64), (2, 1, 64, bd.SDV_E4M3, 64), (2, 1, 64, 9, 64), (2, 1, 64, 0, -64), ((1 << 31) + 1, 1, 64, 0, 64)])
def test_rows_refusals(lib, rows, per, V, dtype, step):
    p = torch.zeros(4096, dtype=torch.int32).data_ptr()
    assert lib.sdv_sample(rows, per, V, dtype, None, p, step, None, None, None, None, p, p, None, None, None) == bd.SDV_ERR_ARG
    assert lib.sdv_logits_truncate(rows, per, V, dtype, None, p, step, None, None, None, None, p, 64, None, None) == bd.SDV_ERR_ARG


def test_no_rows_are_no_work(lib):
    assert lib.sdv_sample(0, 1, 64, 0, None, None, 64, *[None] * 9) == bd.SDV_OK
    assert lib.sdv_logits_truncate(0, 1, 64, 0, None, None, 64, None, None, None, None, None, 64, None, None) == bd.SDV_OK


@pytest.mark.parametrize("B,N,pages,P,most", [(0, 1, 8, 16, 8), (1, 0, 8, 16, 8), (1, 1, 0, 16, 8), (1, 1, 8, 0, 8), (1, 1, 8, 16, 0),
                                              (1, (1 << 20) + 1, 8, 16, 8), ((1 << 20) + 1, 1, 8, 16, 8), (1, 1, 8, 1 << 20, 1 << 11)])
def test_pages_refusals(lib, B, N, pages, P, most):
    p = torch.zeros(64, dtype=torch.int32).data_ptr()
    assert lib.sdv_pages_extend(B, N, pages, P, most, None, *[p] * 11) == bd.SDV_ERR_ARG
    if N == 1:
        assert lib.sdv_pages_release(B, pages, P, most, None, *[p] * 6) == bd.SDV_ERR_ARG


@pytest.mark.parametrize("B,N,Hq,D", [(0, 1, 1, 64), (1, 0, 1, 64), (1, 1, 0, 64), (1, 1, 1, 24), (1, 1, 1, 272), (1 << 16, 1 << 10, 64, 64)])
def test_prefix_workspace_of_bad_shapes(lib, B, N, Hq, D):
    assert lib.sdv_prefix_attn_workspace(B, N, Hq, D) == 0


def test_python_checks_refuse_host_tensors_and_shapes():
    i = torch.zeros((1, 4), dtype=torch.int32)
    x = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    c = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bd.sdv_prefix_attn(x[None], c, c, i, i[:, 0], i, i[:, 0])
    with pytest.raises(ValueError):
        bd.sdv_sample(x, torch.zeros((1, 4)))
    with pytest.raises(ValueError):
        bd.sdv_logits_truncate(x)
    with pytest.raises(ValueError):
        bd.sdv_pages_release(i[0], i[0, :1], i, i[0, :1], i[0, :1], 16)


def test_rows_of_uneven_strides_are_refused():
    even = torch.empty((3, 5, 64), device="meta")
    rows = bd._logit_rows
    for t in (even, even[:, :, :60], even[:, :1], even[:, 2], even[:1], even[:, :0]):
        with pytest.raises(ValueError, match="CUDA"):            # (meta is no CUDA tensor: what comes first)
            rows(t, "logits")

    class Fake:
        is_cuda = True

        def __init__(self, shape, stride):
            self.shape, self._stride = shape, stride

        def stride(self):
            return self._stride
    assert rows(Fake((3, 5, 64), (320, 64, 1)), "x") == (3, 5, 64, 64)
    assert rows(Fake((3, 5, 60), (320, 64, 1)), "x") == (3, 5, 60, 64)
    assert rows(Fake((3, 64), (320, 1)), "x") == (3, 1, 64, 320)
    assert rows(Fake((3, 1, 64), (320, 7, 1)), "x") == (3, 1, 64, 320)
    assert rows(Fake((1, 1, 64), (5, 7, 1)), "x") == (1, 1, 64, 64)
    assert rows(Fake((1, 9, 64), (0, 0, 1)), "x") == (1, 9, 64, 0)
    with pytest.raises(ValueError):
        rows(Fake((3, 4, 64), (320, 64, 1)), "x")
    with pytest.raises(ValueError):
        rows(Fake((3, 5, 64), (64, 192, 1)), "x")
    with pytest.raises(ValueError):
        rows(Fake((64,), (1,)), "x")
    with pytest.raises(ValueError):
        rows(Fake((3, 64), (1, 3)), "x")

"""The verifier's-layer operators without a GPU: the 64-bit references against
small cases worked by hand, the rotary tables, and refusals."""
import ctypes
import math

import pytest
import torch

import layer_ref as ref
from draft_verification_sdv_gb300 import binding as bd


@pytest.fixture(scope="module")
def lib():
    return bd.load(build=True)


def test_reference_attention_by_hand():
    # one head, one cached position and two nodes that do not see each other
    q = torch.tensor([[[[1.0] + [0.0] * 15], [[0.0, 2.0] + [0.0] * 14]]], dtype=torch.bfloat16)
    k = torch.zeros((1, 1, 4, 16), dtype=torch.bfloat16)
    v = torch.zeros((1, 1, 4, 16), dtype=torch.bfloat16)
    k[0, 0, 0, 0], k[0, 0, 1, 0], k[0, 0, 2, 1] = 1.0, 2.0, 3.0
    v[0, 0, 0, 0], v[0, 0, 1, 1], v[0, 0, 2, 2] = 1.0, 1.0, math.nan
    v[0, 0, 2] = 1.0
    mask = torch.tensor([[1], [2]], dtype=torch.int32)
    out, lse, _, _ = ref.attn(q, k, v, torch.tensor([[0]]), [1], None, mask, 1.0)
    e = math.exp
    assert abs(float(out[0, 0, 0, 0]) - e(1) / (e(1) + e(2))) < 1e-12
    assert abs(float(out[0, 0, 0, 1]) - e(2) / (e(1) + e(2))) < 1e-12
    assert float(out[0, 0, 0, 2]) == 0.0
    assert abs(float(lse[0, 1, 0]) - math.log(e(0) + e(6))) < 1e-12
    assert abs(float(out[0, 1, 0, 5]) - e(6) / (1 + e(6))) < 1e-12


def test_reference_quantiser_agrees_with_the_type():
    assert len([x for x in ref.E4M3 if x >= 0]) == 127 and max(ref.E4M3) == 448.0
    g = torch.Generator().manual_seed(3)
    x = torch.cat([torch.randn(400, generator=g) * 60, torch.tensor(ref.E4M3, dtype=torch.float32)]).clamp(-448, 448)
    x[0] = 448.0
    got, e = ref.quantise_row(x.tolist())
    assert e == 127
    assert torch.equal(torch.tensor(got, dtype=torch.float32), x.to(torch.float8_e4m3fn).float())
    assert ref.quantise_row([0.0] * 4) == ([0.0] * 4, 1)
    assert ref.quantise_row([449.0, 1.0])[1] == 128
    assert ref.quantise_row([1.0, math.inf])[1] == 255


def test_rope_frequencies(lib):
    f, at = bd.sdv_rope_freqs(64, base=10000.0, device="cpu")
    want = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert at == 1.0 and max(abs(a - b) / b for a, b in zip(f.tolist(), want)) <= 2.0 ** -24
    f, _ = bd.sdv_rope_freqs(64, scaling=bd.SDV_ROPE_LINEAR, factor=4.0, device="cpu")
    assert max(abs(a - b / 4) / b for a, b in zip(f.tolist(), want)) <= 2.0 ** -24
    f, _ = bd.sdv_rope_freqs(64, scaling=bd.SDV_ROPE_BASE, factor=8.0, device="cpu")
    # the first frequency stays, the last one is that of positions shrunk by the factor
    assert f[0] == 1.0 and abs(float(f[-1]) * 8.0 / want[-1] - 1) < 1e-6
    f, at = bd.sdv_rope_freqs(64, scaling=bd.SDV_ROPE_PARTS, factor=8.0, original=4096, device="cpu")
    for a, b in zip(f.tolist(), want):
        turns = 4096 * b / (2 * math.pi)
        if turns >= 32:
            assert abs(a / b - 1) <= 2.0 ** -24
        elif turns <= 1:
            assert abs(a * 8 / b - 1) <= 2.0 ** -23
        else:
            assert b / 8 < a < b
    assert abs(at - (0.1 * math.log(8.0) + 1)) < 1e-6


@pytest.mark.parametrize("args", [
    (0, 1e4, 0, 1.0, 1.0, 32.0, 1.0), (3, 1e4, 0, 1.0, 1.0, 32.0, 1.0), (514, 1e4, 0, 1.0, 1.0, 32.0, 1.0),
    (64, 0.0, 0, 1.0, 1.0, 32.0, 1.0), (64, math.nan, 0, 1.0, 1.0, 32.0, 1.0), (64, 1e4, 4, 1.0, 1.0, 32.0, 1.0),
    (64, 1e4, 1, 0.5, 1.0, 32.0, 1.0), (2, 1e4, 2, 2.0, 1.0, 32.0, 1.0), (64, 1e4, 3, 2.0, 0.0, 32.0, 1.0),
    (64, 1e4, 3, 2.0, 4096.0, 1.0, 1.0), (64, 1e4, 3, 2.0, 4096.0, 2.0, -1.0)])
def test_rope_frequencies_refusals(lib, args):
    buf = (ctypes.c_float * 512)()
    assert lib.sdv_rope_freqs(*args, buf, None) == bd.SDV_ERR_ARG
    assert lib.sdv_rope_freqs(64, 1e4, 0, 1.0, 1.0, 32.0, 1.0, None, None) == bd.SDV_ERR_ARG


def test_entry_points_refuse_null_and_host_pointers(lib):
    host = torch.zeros(4096, dtype=torch.int32)
    p = host.data_ptr()
    cache = bd._KVCache(p, p, None, None, 16 * 64, 0, 1, 16, 1, 64, bd.SDV_BF16)
    E = bd.SDV_ERR_ARG
    assert lib.sdv_tree_build(1, 1, 4, None, *[None] * 10) == E
    assert lib.sdv_tree_build(1, 1, 4, None, *[p] * 10) == E
    assert lib.sdv_rope(1, 1, 0, 64, 64, 0, 0, None, p, 64, 64, None, 0, 0, p, p, 1.0, p, 64, 64, None, 0, 0) == E
    assert lib.sdv_kv_write(None, 1, 1, 0, None, p, 0, 0, 0, p, 0, 0, 0, p, 1, p, None, None) == E
    assert lib.sdv_kv_write(cache, 1, 1, 0, None, p, 0, 0, 0, p, 0, 0, 0, p, 1, p, None, None) == E
    assert lib.sdv_kv_read(cache, 1, 1, 0, None, p, p, p, 1, p, None, None) == E
    assert lib.sdv_kv_commit(cache, 1, 1, 4, None, p, 1, p, p, p, p, None, None) == E
    assert lib.sdv_tree_attn(cache, 1, 1, 1, 0, None, p, 64, 64, 64, p, 1, p, None, None, 0, 1.0, p, None, p,
                             1 << 30, None) == E
    assert lib.sdv_logits_process(1, 1, 1, 64, 0, None, p, 0, None, p, None, None, None, None, None, 0, None,
                                  None, None, p, None) == E
    assert lib.sdv_counts_commit(1, 1, 1, 64, None, p, p, p, p, p, None) == E


def test_python_checks_refuse_host_tensors():
    i = torch.zeros((1, 4), dtype=torch.int32)
    x = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bd.sdv_rope(x, None, i[0, :1], torch.ones(32))
    c = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bd.sdv_kv_write(x[None], x[None], c, c, i, i[:, 0])
    with pytest.raises(ValueError):
        bd.sdv_tree_attn(x[None], c, c, i, i[:, 0])


def test_reference_tree_by_hand():
    tokens, depth, parent, nodes = ref.tree(9, [[1, 2], [1, 3], [1, 2]], 2)
    assert tokens == [9, 1, 2, 3] and depth == [0, 1, 2, 2] and parent == [-1, 0, 1, 1]
    assert nodes == [[1, 2], [1, 3], [1, 2]]

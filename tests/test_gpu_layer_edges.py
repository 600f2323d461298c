"""The verifier's-layer operators where they can go wrong unseen: slots of
shared memory that are used again, waits that run out, powers of two that 16 bits
do not hold, streams, infinities, far positions, schedules of many units."""
import math

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

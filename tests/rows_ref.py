"""Draws and truncations of whole batches of rows from their definition: weights as
whole numbers in 64 bits, their products with u and top_p exact (Fractions).  Rows
are handled together where 64-bit arithmetic allows it, so that batches that fill a
GPU can be checked; shares no code with the library."""
import math
from fractions import Fraction

import torch

ONE = 2.0 ** 44


def f32(v):
    """A number as the device has it."""
    return float(torch.tensor(v, dtype=torch.float32))


def weights(x, T):
    """Whole weights of rows [R, V] in falling order; T [R, 1], all in 64 bits."""
    fall = x - x[:, :1]
    w = torch.floor(torch.exp(fall / T) * ONE + 0.5)
    w = torch.where(fall == 0, ONE, w)
    return torch.where(x > -math.inf, w, 0.0).long()


def rows(x, T=None, top_k=None, top_p=None, min_p=None, u=None):
    """(kept [R], which logits stay [R, V], the drawn tokens [R] and their
    log-probabilities) of good rows x [R, V]; parameters are lists of R numbers.
    Without u the last two are None."""
    R, V = x.shape
    off = dict(T=1.0, top_k=0, top_p=1.0, min_p=0.0)
    T, top_k, top_p, min_p = ([off[n]] * R if v is None else v
                              for n, v in (("T", T), ("top_k", top_k), ("top_p", top_p), ("min_p", min_p)))
    T, top_p, min_p = ([f32(v) for v in p] for p in (T, top_p, min_p))
    col = lambda v: torch.tensor(v, dtype=torch.float64, device=x.device)[:, None]  # noqa: E731
    x = x.double() + 0.0                             # both zeros are one value
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = weights(x, col([t if t else 1.0 for t in T]))
    upto = torch.cumsum(w, 1)
    floor = [top + t * math.log(m) if m else -math.inf for top, t, m in zip(x[:, 0].tolist(), T, min_p)]
    n = ((x >= col(floor)) & (x > -math.inf)).sum(1).tolist()
    n = [min(a, k) if k else a for a, k in zip(n, top_k)]
    n = [1 if t == 0 else a for a, t in zip(n, T)]
    at = lambda i: upto.gather(1, torch.tensor(i, device=x.device)[:, None] - 1).squeeze(1).tolist()  # noqa: E731
    # tokens while what lies before them weighs less than top_p of all: before < ceil(top_p W)
    need = [math.ceil(Fraction(p) * total) for p, total in zip(top_p, at(n))]
    under = ((upto - w) < torch.tensor(need, device=x.device)[:, None]).sum(1).tolist()
    n = [min(a, b) if p < 1 and t else a for a, b, p, t in zip(n, under, top_p, T)]
    total = at(n)
    stay = torch.zeros((R, V), dtype=torch.bool, device=x.device)
    stay.scatter_(1, order, torch.arange(V, device=x.device) < torch.tensor(n, device=x.device)[:, None])
    if u is None:
        return n, stay, None, None
    aim = [math.floor(Fraction(f32(v)) * s) if t else 0 for v, s, t in zip(u, total, T)]
    place = (upto <= torch.tensor(aim, device=x.device)[:, None]).sum(1, keepdim=True)
    token = order.gather(1, place).squeeze(1)
    mine = w.gather(1, place).squeeze(1).tolist()
    logs = [math.log(a / b) if t else 0.0 for a, b, t in zip(mine, total, T)]
    return n, stay, token.tolist(), logs

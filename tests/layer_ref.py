"""Plain 64-bit implementations of the verifier's-layer operators on the host,
from their definitions, and the tolerances that their arithmetic gives.  Slow
and simple; they share no code with the library."""
import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# smallest absolute spacing of the type, where relative rounding ends
FLOOR = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def rope(x, pos, freq, factor, interleaved):
    """x [T, H, D] double; returns the turned heads and, per element, |a| + |b|
    of its pair (what its rounding is relative to)."""
    x = x.double().cpu()
    R = 2 * freq.numel()
    ang = pos.double().cpu()[:, None] * freq.double().cpu()
    c, s = (torch.cos(ang) * factor)[:, None], (torch.sin(ang) * factor)[:, None]
    r = x[..., :R]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :R // 2], r[..., R // 2:])
    out, mag = x.clone(), x.abs()
    ya, yb, m = a * c - b * s, b * c + a * s, (a.abs() + b.abs()) * abs(factor)
    if interleaved:
        out[..., 0:R:2], out[..., 1:R:2] = ya, yb
        mag[..., 0:R:2], mag[..., 1:R:2] = m, m
    else:
        out[..., :R // 2], out[..., R // 2:R] = ya, yb
        mag[..., :R // 2], mag[..., R // 2:R] = m, m
    return out, mag


E4M3 = sorted({s * v for s in (1, -1) for v in
               [m * 2.0 ** -9 for m in range(8)] +
               [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]})


def quantise_row(row):
    """(values in units of the row's power of two, exponent + 127)."""
    row = [float(v) for v in row]
    if any(math.isnan(v) or math.isinf(v) for v in row):
        return [math.nan] * len(row), 255
    top = max(abs(v) for v in row)
    e = -126
    while top > 448.0 * 2.0 ** e:
        e += 1
    grid = np.array(E4M3)
    out = []
    for v in row:
        y = abs(v) / 2.0 ** e
        d = np.abs(grid[grid >= 0] - y)
        near = np.flatnonzero(d == d.min())
        i = near[0] if len(near) == 1 or near[0] % 2 == 0 else near[1]    # ties to the even code
        out.append(math.copysign(grid[grid >= 0][i], v))
    return out, e + 127


def cells(cache, exp, table_row, pos, P):
    """Row [H, D] (double) of one position of one sequence."""
    page, off = int(table_row[pos // P]), pos % P
    x = cache[page, :, off].double()
    if exp is not None:
        x = x * torch.exp2(exp[page, :, off].double() - 127)[:, None]
    return x


def sequence(cache, exp, table_row, n):
    """Rows [n, H, D] (double) of positions 0 .. n - 1."""
    P = cache.shape[2]
    if n == 0:
        return torch.zeros((0, cache.shape[1], cache.shape[3]), dtype=torch.float64)
    pages = table_row[:-(-n // P)].long()
    x = cache[pages].double() if cache.dtype != torch.float8_e4m3fn else cache.float()[pages].double()
    if exp is not None:
        x = x * torch.exp2(exp[pages].double() - 127)[..., None]
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:n]


def visible(mask, b, i, n):
    """Nodes m < n that node i sees (mask None: a chain)."""
    if mask is None:
        return torch.arange(n) <= i
    row = (mask[b] if mask.dim() == 3 else mask)[i]
    return torch.tensor([(int(row[m // 32]) >> (m % 32)) & 1 for m in range(n)], dtype=torch.bool)


def attn(q, k_cache, v_cache, table, ctx, count, mask, scale, k_exp=None, v_exp=None):
    """(out, lse, tol_out, tol_lse) in double; host tensors in.  What is not
    seen is left out before anything is multiplied."""
    B, N, Hq, D = q.shape
    Hk = k_cache.shape[1]
    g = Hq // Hk
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64)
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    half = HALF_STEP[q.dtype]
    for b in range(B):
        c, n = int(ctx[b]), int(count[b]) if count is not None else N
        ks, vs = (sequence(t, e, table[b], c + n) for t, e in ((k_cache, k_exp), (v_cache, v_exp)))
        for i in range(n):
            see = torch.cat([torch.ones(c, dtype=torch.bool), visible(mask, b, i, n)])
            if not see.any():
                continue
            k, v = ks[see], vs[see]
            for h in range(Hq):
                x = q[b, i, h].double()
                s = (k[:, h // g] @ x) * scale
                lse[b, i, h] = torch.logsumexp(s, 0)
                p = torch.softmax(s, 0)
                out[b, i, h] = p @ v[:, h // g]
                # a score's fp32 sum of D products is off by at most D roundings of
                # their magnitudes; that and a few more roundings (scale, 2^x of
                # relative 2^-22, rescalings) make a probability's relative error
                ds = (D + 8) * 2.0 ** -24 * float((k[:, h // g].abs() @ x.abs()).max()) * abs(scale)
                top = float(s.abs().max())
                ds += 4 * 2.0 ** -24 * top + 2.0 ** -20
                # each probability is rounded to 16 bits, and the output once
                mag = p @ v[:, h // g].abs()
                tol[b, i, h] = half * out[b, i, h].abs() + (half + 2 * ds) * mag * 1.01 + 2 * FLOOR[q.dtype]
                if q.dtype == torch.float16:    # probabilities below fp16's range vanish
                    tol[b, i, h] += 2.0 ** -24 * v[:, h // g].abs().sum(0)
                tol_l[b, i, h] = ds + 2.0 ** -23 * abs(float(lse[b, i, h]))
    return out, lse, tol, tol_l


def tree(root, drafts, lens):
    """The tree of drafts as plain dictionaries: tokens, depth, parent, nodes."""
    tokens, depth, parent, nodes = [root], [0], [-1], []
    index = {(): 0}
    for k in range(len(drafts)):
        path, mine = (), []
        for j in range(lens):
            up = index[path]
            path += (int(drafts[k][j]),)
            if path not in index:
                index[path] = len(tokens)
                tokens.append(int(drafts[k][j]))
                depth.append(j + 1)
                parent.append(up)
            mine.append(index[path])
        nodes.append(mine)
    return tokens, depth, parent, nodes


def logits(x, rows, drafts, counts, prompt, rep, freq, pres, ids, bias, allow):
    """[B, K, gamma + 1, V] double and the magnitude its rounding is relative to."""
    B, K, G = drafts.shape
    V = x.shape[-1]
    out = torch.zeros((B, K, G + 1, V), dtype=torch.float64)
    mag = torch.zeros_like(out)
    bit = lambda w: torch.tensor([(int(w[v // 32]) >> (v % 32)) & 1 for v in range(V)], dtype=torch.bool)  # noqa: E731
    for b in range(B):
        inp = bit(prompt[b]) if prompt is not None else torch.zeros(V, dtype=torch.bool)
        add = torch.zeros(V, dtype=torch.float64)
        amag = torch.zeros(V, dtype=torch.float64)
        if ids is not None:
            for i, w in zip(ids[b].tolist(), bias[b].double().tolist()):
                if 0 <= i < V:
                    add[i] += w
                    amag[i] += abs(w)
        r = float(rep[b]) if rep is not None else 1.0
        f = float(freq[b]) if freq is not None else 0.0
        p = float(pres[b]) if pres is not None else 0.0
        for k in range(K):
            c = counts[b].double().clone() if counts is not None else torch.zeros(V, dtype=torch.float64)
            for j in range(G + 1):
                if j and 0 <= int(drafts[b, k, j - 1]) < V:
                    c[int(drafts[b, k, j - 1])] += 1
                y = (x[b, k, j] if rows is None else x[b, int(rows[b, k, j])]).double()
                y = torch.where((c > 0) | inp, torch.where(y > 0, y / r, y * r), y)
                mag[b, k, j] = torch.where(y.isinf(), 0.0, y.abs()) + (f * c).abs() + abs(p) * (c > 0) + amag
                y = y - f * c - p * (c > 0) + add
                if allow is not None:
                    y = torch.where(bit(allow[b, k, j]), y, -math.inf)
                out[b, k, j] = y
    return out, mag

"""Plain host implementations of the serving loop's operators, from their
definitions: pages as a stack, attention behind a shared prefix as attention over
both, draws in 64 bits.  Slow and simple; they share no code with the library."""
import math
from fractions import Fraction

import torch

import layer_ref as ref

ONE = 2.0 ** 44


def ceil_div(a, b):
    return -(-a // b)


class Pages:
    """The state of a page table on the host."""

    def __init__(self, stack, table, held, P, pages):
        self.stack, self.table, self.held = list(stack), [list(r) for r in table], list(held)
        self.P, self.pages = P, pages
        self.status = 0

    def room(self):
        return len(self.table[0]) * self.P

    def extend(self, start, N, count=None, depth=None, base=None):
        B, most = len(self.held), len(self.table[0])
        count = [N] * B if count is None else count
        free, wanted = len(self.stack), 0
        positions = torch.zeros((B, N), dtype=torch.int32)
        slots = torch.full((B, N), -1, dtype=torch.int64)
        for b in range(B):
            if not (0 <= self.held[b] <= most) or start[b] < 0 or not 0 <= count[b] <= N \
                    or start[b] + count[b] > self.room():
                self.status |= 16
                continue
            more = max(ceil_div(start[b] + count[b], self.P) - self.held[b], 0)
            wanted += more
            if more and wanted > free:
                self.status |= 128
            elif more:
                for _ in range(more):
                    page = self.stack.pop()
                    self.status |= 64 * (not 0 <= page < self.pages)
                    self.table[b][self.held[b]] = page
                    self.held[b] += 1
            for n in range(count[b]):
                place = (start[b] + n) // self.P
                page = self.table[b][place] if place < self.held[b] else None
                if page is not None and 0 <= page < self.pages:
                    slots[b, n] = page * self.P + (start[b] + n) % self.P
                elif page is not None:
                    self.status |= 64
                positions[b, n] = start[b] + (n if depth is None else depth[b][n]) + (base[b] if base else 0)
        return positions, slots

    def release(self, keep):
        most = len(self.table[0])
        give = [0] * len(self.held)
        for b, h in enumerate(self.held):
            if not 0 <= h <= most or keep[b] < 0:
                self.status |= 16
                continue
            give[b] = max(h - ceil_div(keep[b], self.P), 0)
        if len(self.stack) + sum(give) > self.pages:
            self.status |= 16
            return
        for b in reversed(range(len(self.held))):
            for _ in range(give[b]):
                self.held[b] -= 1
                page = self.table[b][self.held[b]]
                self.status |= 64 * (not 0 <= page < self.pages)
                self.stack.append(page)
                self.table[b][self.held[b]] = -1


def prefix_attn(q, k_cache, v_cache, prefix_table, prefix_len, table, ctx, count, mask, scale, k_exp=None, v_exp=None):
    """layer_ref.attn over a cache with pages of one position, where each
    sequence's prefix and its own positions follow one another."""
    B, N = q.shape[:2]
    G, P = len(prefix_len), k_cache.shape[2]
    rows, lens = [], []
    for b in range(B):
        n = N if count is None else count[b]
        far = prefix_len[b // (B // G)]
        at = [(int(prefix_table[b // (B // G)][t // P]), t % P) for t in range(far)]
        at += [(int(table[b][t // P]), t % P) for t in range(ctx[b] + n)]
        rows.append(at)
        lens.append(far + ctx[b])
    most = max(len(r) for r in rows)
    one = [[], [], [], []]
    flat = torch.zeros((B, max(most, 1)), dtype=torch.int64)
    done = 0
    for b, at in enumerate(rows):
        pages, offs = (torch.tensor([x[i] for x in at], dtype=torch.int64) for i in (0, 1))
        for into, t in zip(one, (k_cache, v_cache, k_exp, v_exp)):
            if t is not None:
                raw = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
                into.append(raw[pages, :, offs].view(t.dtype))
        flat[b, :len(at)] = done + torch.arange(len(at))
        done += len(at)
    def join(parts, like):
        if like is None:
            return None
        if like.dtype == torch.float8_e4m3fn:
            return torch.cat([p.view(torch.uint8) for p in parts])[:, :, None].view(like.dtype)
        return torch.cat(parts)[:, :, None]
    k, v, ke, ve = (join(p, t) for p, t in zip(one, (k_cache, v_cache, k_exp, v_exp)))
    return ref.attn(q, k, v, flat, lens, count, mask, scale, ke, ve)


def order(x):
    """Indices by falling value, equal ones by index (-inf last)."""
    return sorted(range(len(x)), key=lambda i: (-x[i], i))


def weight(fall, T):
    """round(2^44 e^(-fall / T)) from 64-bit numbers."""
    return int(math.floor(math.exp(-fall / T) * ONE + 0.5))


def choose(x, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(indices that a row keeps, in order; their weights) for a list of floats;
    the parameters as the device has them (rounded to 32 bits)."""
    f = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    T, top_p, min_p = f(T), f(top_p), f(min_p)
    idx = [i for i in order(x) if x[i] > -math.inf]
    top = x[idx[0]]
    if T == 0:
        return idx[:1], [1 << 44]
    n = len(idx)
    if min_p:
        floor = top + T * math.log(min_p)
        n = sum(x[i] >= floor for i in idx)
    if top_k:
        n = min(n, top_k)
    idx = idx[:n]
    w = [weight(top - x[i], T) for i in idx]
    if top_p < 1:
        need = top_p * float(sum(w))
        before, n = 0, 0
        for v in w:
            if Fraction(before) >= Fraction(need):
                break
            before += v
            n += 1
        idx, w = idx[:n], w[:n]
    return idx, w


def drawn(idx, w, u):
    """(token, its log-probability) of a row's choice."""
    total = sum(w)
    aim = int(float(torch.tensor(u, dtype=torch.float32)) * float(total))
    upto = 0
    for i, v in zip(idx, w):
        upto += v
        if upto > aim:
            return i, math.log(v / total)
    raise AssertionError("the weights end before the draw")

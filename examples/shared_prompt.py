"""Several samples of one prompt: the operators of a serving loop together.

A small transformer with random weights continues a prompt a few times at once.  The
prompt's keys and values are written once, on pages of their own, and every sample
attends to them; what a sample adds goes to pages that it takes from one pool as it
grows and gives back when it ends.  Each step draws one token a sample under its
own temperature, top-k, top-p and min-p:

  sdv_pages_extend -> per layer: sdv_rope, sdv_kv_write, sdv_prefix_attn
  -> sdv_sample; sdv_pages_release for samples that are done

    python examples/shared_prompt.py [--steps 24] [--samples 6] [--e4m3]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from draft_verification_sdv_gb300 import binding as bd  # noqa: E402
from tree_decode import Model, norm  # noqa: E402


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Server:
    """One prompt, its samples, and the pool of pages that all of them live on."""

    def __init__(self, model, prompt, samples, room=64, page=16, e4m3=False, end=None, seed=0, **cut):
        m, B = model, samples
        self.model, self.B, self.page, self.end, self.cut = m, B, page, end, cut
        self.text = [[] for _ in range(B)]
        self.random = torch.Generator(device="cuda").manual_seed(seed)
        per, first = -(-room // page), -(-len(prompt) // page)
        self.pages = B * per + first
        shape = (self.pages, m.Hk, page, m.D)
        cells = torch.float8_e4m3fn if e4m3 else m.dtype
        self.cache = []
        for _ in m.layers:
            kv = [torch.zeros(shape, dtype=m.dtype, device="cuda").to(cells) for _ in range(2)]
            exp = [torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") if e4m3 else None for _ in range(2)]
            self.cache.append((kv, dict(k_exp=exp[0], v_exp=exp[1])))
        self.status = _ints([0])
        self.pool = torch.randperm(self.pages, generator=torch.Generator().manual_seed(1)).int().cuda()
        self.free = _ints([self.pages])
        self.table = torch.full((B, per), -1, dtype=torch.int32, device="cuda")
        self.held, self.length = _ints([0] * B), _ints([0] * B)
        self.live = torch.ones(B, dtype=torch.int32, device="cuda")

        # the prompt, once: a causal chain on pages of its own
        n = len(prompt)
        self.prefix_table = torch.full((1, first), -1, dtype=torch.int32, device="cuda")
        self.prefix_len = _ints([n])
        positions, _ = bd.sdv_pages_extend(self.pool, self.free, self.prefix_table, _ints([0]), _ints([0]), n,
                                           page, status=self.status)
        logits = self._forward(_ints([prompt]), positions, self.prefix_table, _ints([0]), None, False)
        # its last row gives every sample's first token: one row, drawn from B times
        self.last = self._draw(logits[0, -1:].expand(B, -1))

    def _forward(self, tokens, positions, table, start, count, shared):
        """Logits [B, N, V] of new tokens, whose keys and values go into the cache."""
        m = self.model
        B, N = tokens.shape
        x = m.embed[tokens.clamp(min=0).long()]
        for (w_qkv, w_out, w_up, w_down), ((k_cache, v_cache), exps) in zip(m.layers, self.cache):
            q, k, v = (norm(x) @ w_qkv).view(B * N, -1, m.D).split([m.Hq, m.Hk, m.Hk], dim=1)
            bd.sdv_rope(q, k, positions.view(-1), m.freq, m.factor, out_q=q, out_k=k)      # in place
            q, k, v = (t.unflatten(0, (B, N)) for t in (q, k, v))
            bd.sdv_kv_write(k, v, k_cache, v_cache, table, start, count=count, status=self.status, **exps)
            if shared:
                o = bd.sdv_prefix_attn(q, k_cache, v_cache, self.prefix_table, self.prefix_len, table, start,
                                       count=count, status=self.status, **exps)
            else:
                o = bd.sdv_tree_attn(q, k_cache, v_cache, table, start, count=count, status=self.status, **exps)
            x = x + o.reshape(B, N, -1) @ w_out
            x = x + torch.nn.functional.silu(norm(x) @ w_up) @ w_down
        return norm(x) @ m.head

    def _draw(self, logits):
        u = torch.rand((self.B,), generator=self.random, device="cuda")
        tokens, self.logprob = bd.sdv_sample(logits, u, logprob=True, status=self.status, **self.cut)
        for b, (t, live) in enumerate(zip(tokens.tolist(), self.live.tolist())):
            if live:
                self.text[b].append(t)
        if self.end is not None:                     # samples that are done give their pages back
            self.live *= tokens != self.end
            self.length *= self.live
            bd.sdv_pages_release(self.pool, self.free, self.table, self.held,
                                 torch.where(self.live > 0, self.length + self.page, 0).int(), self.page,
                                 status=self.status)
        return tokens

    def step(self):
        """One token for each sample that goes on."""
        positions, _ = bd.sdv_pages_extend(self.pool, self.free, self.table, self.held, self.length, 1, self.page,
                                           count=self.live, base=self.prefix_len.expand(self.B).contiguous(),
                                           status=self.status)
        logits = self._forward(self.last[:, None], positions, self.table, self.length, self.live, True)
        self.length = self.length + self.live
        self.last = self._draw(logits[:, 0])
        if self.status.item():
            raise RuntimeError("device status %d" % self.status.item())


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--samples", type=int, default=6)
    ap.add_argument("--e4m3", action="store_true", help="quantised cache")
    args = ap.parse_args()
    prompt = torch.randint(0, 512, (75,), generator=torch.Generator().manual_seed(3)).tolist()
    B = args.samples
    cut = dict(temperature=torch.linspace(0.0, 1.2, B, device="cuda"), top_k=_ints([50] * B),
               top_p=torch.full((B,), 0.95, device="cuda"))
    s = Server(Model(), prompt, B, room=args.steps + 16, e4m3=args.e4m3, end=7, **cut)
    for _ in range(args.steps):
        s.step()
    for b, text in enumerate(s.text):
        print("sample %d (temperature %.2f): %s" % (b, cut["temperature"][b], " ".join(map(str, text[:16]))))
    print("%d of %d pages in use" % (s.pages - s.free.item(), s.pages))


if __name__ == "__main__":
    main()

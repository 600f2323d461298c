"""Decoding with draft trees: the verifier's layer operators together, as a
serving loop uses them.

A small transformer with random weights generates text.  Each step drafts K
continuations per sequence (the latest places where its last token occurred
before, and what followed there), flattens them into one tree, scores the whole
tree in one forward pass over the paged cache, applies the sampling parameters to
every draft position, verifies (against the target's probabilities alone, at a low
temperature), and keeps the accepted path's keys and values:

  sdv_tree_build -> per layer: sdv_rope, sdv_kv_write, sdv_tree_attn
  -> sdv_logits_process -> Verifier -> sdv_kv_commit (per layer), sdv_counts_commit

    python examples/tree_decode.py [--steps 32] [--e4m3]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from draft_verification_sdv_gb300 import binding as bd  # noqa: E402


class Model:
    """Random weights; grouped queries, rotary positions, a two-layer MLP."""

    def __init__(self, V=512, width=256, layers=2, Hq=8, Hk=2, D=64, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.V, self.width, self.Hq, self.Hk, self.D, self.dtype = V, width, Hq, Hk, D, dtype

        def weight(rows, cols, gain=1.0):
            return (torch.randn((rows, cols), generator=gen) * gain * rows ** -0.5).to(dtype).cuda()

        self.embed = (torch.randn((V, width), generator=gen) * 0.5).to(dtype).cuda()
        self.head = weight(width, V, 2.0)
        self.layers = [(weight(width, (Hq + 2 * Hk) * D), weight(Hq * D, width),
                        weight(width, 2 * width), weight(2 * width, width)) for _ in range(layers)]
        self.freq, self.factor = bd.sdv_rope_freqs(D)


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Decoder:
    """Sequences of one batch, their paged cache and their token counts."""

    def __init__(self, model, prompts, K=3, G=4, room=256, page=16, e4m3=False, repetition=1.0,
                 presence=0.0, temperature=0.01, seed=0):
        B, m = len(prompts), model
        self.model, self.K, self.G, self.B = model, K, G, B
        self.text = [list(p) for p in prompts]
        self.temperature, self.seed = temperature, seed
        per = -(-room // page)
        self.table = torch.randperm(B * per, generator=torch.Generator().manual_seed(1)) \
            .view(B, per).int().cuda()
        shape = (B * per, m.Hk, page, m.D)
        cells = torch.float8_e4m3fn if e4m3 else m.dtype
        self.cache = []
        for _ in m.layers:
            kv = [torch.zeros(shape, dtype=m.dtype, device="cuda").to(cells) for _ in range(2)]
            exp = [torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") if e4m3 else None for _ in range(2)]
            self.cache.append((kv, dict(k_exp=exp[0], v_exp=exp[1])))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.workspace = torch.empty(bd.load().sdv_tree_attn_workspace(), dtype=torch.uint8, device="cuda")
        self.verify = bd.Verifier(B, K, G, m.V, m.dtype, greedy=True)

        # what the prompt holds, for the repetition penalty; generated tokens are counted
        bits = torch.zeros((B, (m.V + 31) // 32), dtype=torch.int64)
        for b, p in enumerate(prompts):
            for t in set(p):
                bits[b, t // 32] |= 1 << (t % 32)
        bits = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits)
        self.sampling = dict(counts=torch.zeros((B, m.V), dtype=torch.int32, device="cuda"),
                             prompt=bits.int().cuda(),
                             repetition=torch.full((B,), float(repetition), device="cuda"),
                             presence=torch.full((B,), float(presence), device="cuda"))

        # all of the prompt but its last token, as a causal chain
        longest = max(len(p) for p in prompts) - 1
        tokens = torch.zeros((B, max(longest, 1)), dtype=torch.int32)
        for b, p in enumerate(prompts):
            tokens[b, :len(p) - 1] = torch.tensor(p[:-1], dtype=torch.int32)
        count = torch.tensor([len(p) - 1 for p in prompts], dtype=torch.int32, device="cuda")
        self.start = torch.zeros(B, dtype=torch.int32, device="cuda")
        depth = torch.arange(tokens.shape[1], dtype=torch.int32, device="cuda").expand(B, -1)
        self.forward(tokens.cuda(), depth, count, None)
        self.start = count
        self.last = torch.tensor([p[-1] for p in prompts], dtype=torch.int32, device="cuda")

    def forward(self, tokens, depth, count, mask):
        """Logits [B, N, V] of nodes behind the committed positions; their keys
        and values go into the cache."""
        m = self.model
        B, N = tokens.shape
        positions = (self.start[:, None] + depth).reshape(-1).contiguous()
        x = m.embed[tokens.clamp(min=0).long()]
        for (w_qkv, w_out, w_up, w_down), ((k_cache, v_cache), exps) in zip(m.layers, self.cache):
            q, k, v = (norm(x) @ w_qkv).view(B * N, -1, m.D).split([m.Hq, m.Hk, m.Hk], dim=1)
            bd.sdv_rope(q, k, positions, m.freq, m.factor, out_q=q, out_k=k)      # in place
            q, k, v = (t.unflatten(0, (B, N)) for t in (q, k, v))
            bd.sdv_kv_write(k, v, k_cache, v_cache, self.table, self.start, count=count,
                            status=self.status, **exps)
            o = bd.sdv_tree_attn(q, k_cache, v_cache, self.table, self.start, count=count, mask=mask,
                                 workspace=self.workspace, status=self.status, **exps)
            x = x + o.reshape(B, N, -1) @ w_out
            x = x + torch.nn.functional.silu(norm(x) @ w_up) @ w_down
        return norm(x) @ m.head

    def draft(self):
        """K guesses of G tokens per sequence: what followed its last token before
        (no draft where it is new)."""
        drafts = torch.zeros((self.B, self.K, self.G), dtype=torch.int32)
        length = torch.zeros(self.B, dtype=torch.int32)
        for b, text in enumerate(self.text):
            places = [i for i in range(len(text) - 2, -1, -1) if text[i] == text[-1]][:self.K]
            for k in range(self.K if places else 0):
                after = text[places[min(k, len(places) - 1)] + 1:][:self.G]
                drafts[b, k, :len(after)] = torch.tensor(after, dtype=torch.int32)
                length[b] = self.G
        return drafts.cuda(), length.cuda()

    def step(self, drafts=None, draft_len=None):
        """One decoding step; returns the number of tokens it gave each sequence."""
        if drafts is None:
            drafts, draft_len = self.draft()
        tree = bd.sdv_tree_build(self.last, drafts, draft_len, status=self.status)
        logits = self.forward(tree["tokens"], tree["depth"], tree["count"], tree["mask"])
        rows = bd.sdv_logits_process(logits, drafts, rows=tree["rows"], status=self.status, **self.sampling)
        out = self.verify(rows, None, drafts, temperature=self.temperature, seed=self.seed, draft_len=draft_len)
        self.seed += 1                       # other random numbers for the next step
        now = None
        for (k_cache, v_cache), exps in self.cache:
            now = bd.sdv_kv_commit(k_cache, v_cache, self.table, self.start, tree["nodes"], out["sel"],
                                   out["accept_len"], status=self.status, **exps)
        bd.sdv_counts_commit(self.sampling["counts"], drafts, out["sel"], out["accept_len"],
                             out["next_token"], status=self.status)
        self.start, self.last = now, out["next_token"]
        self.verify.sync()
        if self.status.item():
            raise RuntimeError("device status %d" % self.status.item())
        sel, acc, nxt = (out[n].tolist() for n in ("sel", "accept_len", "next_token"))
        for b in range(self.B):
            self.text[b] += drafts[b, sel[b], :acc[b]].tolist() + [nxt[b]]
        return [a + 1 for a in acc]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--e4m3", action="store_true", help="quantised cache")
    args = ap.parse_args()
    gen = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, 512, (n,), generator=gen).tolist() for n in (5, 40, 1, 23)]
    room = max(map(len, prompts)) + 5 * (args.steps + 3)
    d = Decoder(Model(), prompts, room=room, e4m3=args.e4m3)
    total = sum(sum(d.step()) for _ in range(args.steps))
    for b, p in enumerate(prompts):
        print("sequence %d: %s ..." % (b, " ".join(map(str, d.text[b][len(p):][:16]))))
    print("%.2f tokens per sequence and step" % (total / args.steps / len(prompts)))


if __name__ == "__main__":
    main()

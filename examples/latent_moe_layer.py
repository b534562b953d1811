"""One layer end to end: latent attention, then the routed experts.

    python examples/latent_moe_layer.py [--heads 16] [--hidden 512] [--prompt 300]

Serves one request with random weights, as a serving program would:
  1. prompt: queries and latents are projected, normalized, rotated and put
     into the paged cache (latent_cache_append), keys and values expanded
     (LatentExpand), attention over them (LatentAttention), output projection,
     routed experts (MoEForward);
  2. decode: single tokens over the cache in absorbed form (LatentDecode);
  3. a tree of drafted tokens checked in one call.
Prints how far the absorbed form is from the expanded one on the same tokens
and the tree's branches from the single-token steps, then a training step's
gradients of the attention. The dense projections are plain torch products.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mixture_experts_layer_sigmoid_amd as moe  # noqa: E402

PAGE = 64


class Layer:
    """Weights of one layer and its serving state for one request."""

    def __init__(self, heads, hidden, max_len, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g, device=device) / s[-1] ** 0.5).to(torch.bfloat16)
        self.h, self.H, self.dev = heads, hidden, device
        self.w_q, self.w_a, self.w_o = w(heads * 192, hidden), w(576, hidden), w(hidden, heads * 128)
        self.w_kvb = w(heads, 256, 512)
        self.norm = torch.ones(512, dtype=torch.bfloat16, device=device)
        freq = 10000.0 ** (-torch.arange(32, device=device) / 32)
        ang = torch.arange(max_len, device=device)[:, None] * freq
        self.cos, self.sin = ang.cos().float(), ang.sin().float()
        self.E, self.F = 16, 256
        self.w_r, self.bias = w(self.E, hidden), torch.zeros(self.E, device=device)
        self.experts = moe.ExpertWeights.from_dense(w(self.E, 2 * self.F, hidden), w(self.E, hidden, self.F), "bf16")
        pages = -(-max_len // PAGE)
        self.cache = torch.zeros((pages, PAGE, 576), dtype=torch.bfloat16, device=device)
        self.table = torch.randperm(pages, generator=g, device=device).to(torch.int32)[None]
        self.decode = moe.LatentDecode(self.w_kvb, max_tokens=64, max_seqs=1)

    def slots(self, first, n):
        pos = torch.arange(first, first + n, device=self.dev)
        return self.table[0, pos // PAGE].long() * PAGE + pos % PAGE

    def append(self, x, positions, slots):
        """Rotated queries of the tokens x; their rows go to the cache."""
        q = (x @ self.w_q.t()).view(-1, self.h, 192)
        moe.latent_cache_append(x @ self.w_a.t(), self.cache, slots, norm_weight=self.norm, cos=self.cos,
                                sin=self.sin, positions=positions.to(torch.int32), q=q)
        return q

    def mlp(self, x, att):
        x = x + att.flatten(1) @ self.w_o.t()
        f = moe.MoEForward(T=x.shape[0], H=self.H, F=self.F, E=self.E, n_group=4, topk_group=2, k=4, routed_scale=1.0,
                           fmt="bf16", device=self.dev)
        return x + f(x, self.w_r, self.bias, self.experts)

    def _cu(self, n):
        return torch.tensor([0, n], dtype=torch.int32, device=self.dev)

    def expanded(self, q, first, n, backward=False):
        """Attention of the queries of the tokens first .. first + n - 1 over
        everything cached up to there, keys and values expanded."""
        rows = self.cache.view(-1, 576)[self.slots(0, first + n)]
        kv = moe.LatentExpand(self.w_kvb, max_tokens=first + n)(rows[:, :512].contiguous())
        a = moe.LatentAttention(Tq=n, Tk=first + n, n_heads=self.h, n_seqs=1, backward=backward)
        ins = (q, kv, rows[:, 512:], self._cu(n), self._cu(first + n))
        out, _ = a(*ins)
        if not backward:
            return out
        return out, a.backward(torch.ones_like(out), *ins)

    def absorbed(self, q, length, tree=None):
        lens = torch.tensor([length], dtype=torch.int32, device=self.dev)
        return self.decode(q, self.cache, self.table, lens, self._cu(q.shape[0]), tree).clone()


def far(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def main(heads=16, hidden=512, prompt=300, steps=4):
    dev = "cuda"
    layer = Layer(heads, hidden, prompt + 64)
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    x = torch.randn(prompt + steps, hidden, generator=g, device=dev).to(torch.bfloat16)
    pos = torch.arange(prompt + steps, device=dev)

    q = layer.append(x[:prompt], pos[:prompt], layer.slots(0, prompt))
    out, (dq, dkv, dk_rope) = layer.expanded(q, 0, prompt, backward=True)
    y = layer.mlp(x[:prompt], out)
    print(f"prompt of {prompt}: layer output {tuple(y.shape)}, attention gradients "
          f"{tuple(dq.shape)} {tuple(dkv.shape)} {tuple(dk_rope.shape)}")

    single, worst = [], 0.0
    for i in range(steps):
        n = prompt + i
        q = layer.append(x[n:n + 1], pos[n:n + 1], layer.slots(n, 1))
        out = layer.absorbed(q, n + 1)
        worst = max(worst, far(out, layer.expanded(q, n, 1)))
        layer.mlp(x[n:n + 1], out)
        single.append(out)
    print(f"{steps} decode steps: absorbed form within {worst:.1e} of the expanded form")

    # a tree of 2 * steps drafted tokens: the chain above, with a sibling
    # beside each of its tokens; all rows go behind the prompt
    chain, words, mask, at = [], [], 0, []
    for i in range(steps):
        chain.append(len(words))
        words.append(mask | 1 << len(words))                 # the chain's token
        at.append(i)
        words.append(mask | 1 << len(words))                 # its sibling
        at.append(i)
        mask |= 1 << chain[-1]
    at = torch.tensor(at, device=dev)
    xt = x[prompt + at].clone()
    xt[1::2] += 1                                            # the siblings are other tokens
    q = layer.append(xt, pos[prompt + at], layer.slots(prompt, 2 * steps))
    out = layer.absorbed(q, prompt + 2 * steps, torch.tensor(words, dtype=torch.int64, device=dev))
    tree = max(far(out[c:c + 1], s) for c, s in zip(chain, single))
    print(f"tree of {2 * steps} drafted tokens: its chain within {tree:.1e} of the single steps")
    return worst, tree, (dq, dkv, dk_rope), y


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--prompt", type=int, default=300)
    a = ap.parse_args()
    main(a.heads, a.hidden, a.prompt)

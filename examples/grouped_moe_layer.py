"""One layer end to end: grouped-query attention, then the routed experts.

    python examples/grouped_moe_layer.py [--heads 16] [--kv-heads 2] [--hidden 512] [--prompt 300]

Serves one request with random weights, as a serving program would:
  1. prompt: queries, keys and values come from one projection, every head's
     query and key is normalized and rotated (QKNormRope), attention over them
     (GroupedAttention), keys and values go to the 8-bit paged cache
     (grouped_cache_append), output projection, routed experts (MoEForward);
  2. decode: single tokens over the cache (GroupedDecode);
  3. a tree of drafted tokens checked in one call.
Prints how far decoding over the 8-bit cache is from attention over the bf16
keys and values of the same tokens and the tree's branches from the single-
token steps, then the gradients of a training step of the attention, back to
the projection's rows and the norm's weights. The dense projections are plain
torch products.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mixture_experts_layer_sigmoid_amd as moe  # noqa: E402

PAGE, DIM = 64, 128


class Layer:
    """Weights of one layer and its serving state for one request."""

    def __init__(self, heads, kv_heads, hidden, max_len, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g, device=device) / s[-1] ** 0.5).to(torch.bfloat16)
        self.h, self.kv, self.dev = heads, kv_heads, device
        self.w_qkv, self.w_o = w((heads + 2 * kv_heads) * DIM, hidden), w(hidden, heads * DIM)
        self.norm_q = torch.ones(DIM, dtype=torch.bfloat16, device=device)
        self.norm_k = torch.ones(DIM, dtype=torch.bfloat16, device=device)
        freq = 10000.0 ** (-torch.arange(DIM // 2, device=device) / (DIM // 2))
        ang = torch.arange(max_len, device=device)[:, None] * freq
        self.cos, self.sin = ang.cos().float(), ang.sin().float()
        self.E, self.F = 16, 256
        self.w_r, self.bias = w(self.E, hidden), torch.zeros(self.E, device=device)
        self.experts = moe.ExpertWeights.from_dense(w(self.E, 2 * self.F, hidden), w(self.E, hidden, self.F), "bf16")
        pages = -(-max_len // PAGE)
        self.cache = moe.GroupedCache.empty(pages, PAGE, kv_heads, DIM, device=device)
        self.table = torch.randperm(pages, generator=g, device=device).to(torch.int32)[None]
        size = dict(n_heads=heads, n_kv_heads=kv_heads, head_dim=DIM, device=device)
        self.norm = moe.QKNormRope(T=max_len, backward=True, **size)
        self.attention = moe.GroupedAttention(Tq=max_len, Tk=max_len, n_seqs=1, backward=True, **size)
        self.decode = moe.GroupedDecode(max_tokens=64, max_seqs=1, **size)

    def project(self, x):
        """Query, key and value of the tokens x, slices of one product's rows."""
        rows = (x @ self.w_qkv.t()).view(-1, self.h + 2 * self.kv, DIM)
        return rows.split([self.h, self.kv, self.kv], 1)

    def turn(self, q, k, positions):
        """Normalized and rotated queries and keys."""
        q, k = self.norm(q, k, self.norm_q, self.norm_k, self.cos, self.sin, positions)
        return q.clone(), k.clone()

    def append(self, k, v, length):
        """k and v become the cache's last tokens, length with them."""
        moe.grouped_cache_append(k, v, self.cache, self.table, self._lens(length), self._cu(k.shape[0]))

    def mlp(self, x, att):
        x = x + att.flatten(1) @ self.w_o.t()
        f = moe.MoEForward(T=x.shape[0], H=x.shape[1], F=self.F, E=self.E, n_group=4, topk_group=2, k=4,
                           routed_scale=1.0, fmt="bf16", device=self.dev)
        return x + f(x, self.w_r, self.bias, self.experts)

    def _cu(self, n):
        return torch.tensor([0, n], dtype=torch.int32, device=self.dev)

    def _lens(self, n):
        return torch.tensor([n], dtype=torch.int32, device=self.dev)

    def attend(self, q, k, v):
        out, _ = self.attention(q, k, v, self._cu(q.shape[0]), self._cu(k.shape[0]))
        return out.clone()

    def gradients(self, dout, x, positions):
        """Gradients of attention, rotation and norm from that of the output:
        of the projection's rows and of the norm's weights."""
        q0, k0, v = self.project(x)
        q, k = self.turn(q0, k0, positions)
        self.attend(q, k, v)
        dq, dk, dv = self.attention.backward(dout, q, k, v, self._cu(x.shape[0]), self._cu(x.shape[0]))
        dq, dk, dw_q, dw_k = self.norm.backward(dq, dk, q0, k0, self.norm_q, self.norm_k, self.cos, self.sin, positions)
        return torch.cat([dq, dk, dv], 1), dw_q, dw_k

    def cached(self, q, length, tree=None):
        return self.decode(q, self.cache, self.table, self._lens(length), self._cu(q.shape[0]), tree).clone()


def far(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def main(heads=16, kv_heads=2, hidden=512, prompt=300, steps=4):
    dev = "cuda"
    layer = Layer(heads, kv_heads, hidden, prompt + 64)
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    x = torch.randn(prompt + steps, hidden, generator=g, device=dev).to(torch.bfloat16)
    pos = torch.arange(prompt + steps, device=dev, dtype=torch.int32)

    q0, k0, v = layer.project(x[:prompt])
    q, k = layer.turn(q0, k0, pos[:prompt])
    layer.append(k, v, prompt)
    out = layer.attend(q, k, v)
    y = layer.mlp(x[:prompt], out)
    print(f"prompt of {prompt}: layer output {tuple(y.shape)}")

    keys, values = [k], [v]
    single, worst = [], 0.0
    for i in range(steps):
        n = prompt + i
        q0, k0, v = layer.project(x[n:n + 1])
        q, k = layer.turn(q0, k0, pos[n:n + 1])
        layer.append(k, v, n + 1)
        out = layer.cached(q, n + 1)
        keys.append(k), values.append(v)
        worst = max(worst, far(out, layer.attend(q, torch.cat(keys), torch.cat(values))))
        layer.mlp(x[n:n + 1], out)
        single.append(out)
    print(f"{steps} decode steps: 8-bit cache within {worst:.1e} of bf16 keys and values")

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
    q0, k0, v = layer.project(xt)
    q, k = layer.turn(q0, k0, pos[prompt + at])
    layer.append(k, v, prompt + 2 * steps)
    out = layer.cached(q, prompt + 2 * steps, torch.tensor(words, dtype=torch.int64, device=dev))
    tree = max(far(out[c:c + 1], s) for c, s in zip(chain, single))
    print(f"tree of {2 * steps} drafted tokens: its chain within {tree:.1e} of the single steps")

    grads = layer.gradients(torch.ones_like(layer.attention.out[:prompt]), x[:prompt], pos[:prompt])
    print(f"gradients of the projection's rows {tuple(grads[0].shape)} and of the norm's weights "
          f"{tuple(grads[1].shape)} {tuple(grads[2].shape)}")
    return worst, tree, grads, y


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv-heads", type=int, default=2)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--prompt", type=int, default=300)
    a = ap.parse_args()
    main(a.heads, a.kv_heads, a.hidden, a.prompt)

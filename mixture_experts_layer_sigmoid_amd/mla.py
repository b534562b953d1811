"""Latent attention beside the experts, as sequences of C-ABI calls.

LatentAttention  expanded form: packed sequences of queries over expanded
                 keys and values (prompts, training), forward and backward.
LatentDecode     absorbed form over a paged cache (serving): the last tokens
                 of each request, or a tree of drafted ones.
LatentExpand     keys and values of all heads from latents, for the expanded
                 form (one dense expert GEMM).
latent_cache_append
                 RMS norm of new latents, rotary embedding of their keys and
                 of the queries, rows into the cache.

Sizes: latent 512, rotary 64, per head 128 key and 128 value values, bf16.
As in layer.py only marshalling happens here: shapes and types are checked,
buffers are allocated once, every step runs in the HIP library on the given
stream (default: torch's current one).
"""
from __future__ import annotations

import torch

from . import _lib as L
from .layer import pack_weights

LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128
QK, CACHE_ROW = NOPE + ROPE, LATENT + ROPE
SCALE = QK ** -0.5


def _rows(t: torch.Tensor, name: str, inner: tuple) -> int:
    """Row stride of a bf16 tensor [tokens, *inner] whose tokens are dense
    inside (the tensor may be a slice of wider rows)."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not torch.bfloat16 or not t.is_cuda:
        raise ValueError(f"{name} must be a bfloat16 tensor on the GPU")
    if shape[1:] != inner:
        raise ValueError(f"{name} must have shape [tokens, {', '.join(map(str, inner))}], got {tuple(shape)}")
    last = inner[-1]
    if shape[0] > 0 and (stride[-1] != 1 or (len(inner) == 2 and stride[1] != last and inner[0] > 1)):
        raise ValueError(f"{name}: a token's values must be consecutive")
    # a lone token's stride is never used, and may be anything
    return stride[0] if shape[0] > 1 else last * (inner[0] if len(inner) == 2 else 1)


def _vec(t: torch.Tensor, name: str, dtype, shape: tuple) -> torch.Tensor:
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on the GPU, got "
                         f"{t.dtype} {tuple(t.shape)}")
    return t


def _cache(t: torch.Tensor, what: str) -> None:
    if t.dtype is not torch.bfloat16 or t.shape[-1] != CACHE_ROW or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"cache must be a contiguous bfloat16 tensor {what} on the GPU, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _weights(t: torch.Tensor) -> None:
    if t.dtype is not torch.bfloat16 or t.dim() != 3 or t.shape[1:] != (NOPE + VALUE, LATENT) or not t.is_cuda:
        raise ValueError(f"w_kvb must be a bfloat16 tensor [n_heads, {NOPE + VALUE}, {LATENT}] on the GPU, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _first(t: torch.Tensor, n: int) -> torch.Tensor:
    """The first n rows of a buffer."""
    return t if t.shape[0] == n else t[:n]


class LatentAttention:
    """Attention of up to Tq queries over up to Tk expanded keys in up to
    n_seqs packed sequences (cu_q, cu_k [n_seqs + 1] int32, row offsets).
    With causal, a sequence's last query sees all its keys, each earlier one
    a key less. Outputs are views of the object's buffers, as many rows as the
    call's inputs have; backward=True adds the gradients' buffers and
    workspace."""

    def __init__(self, *, Tq, Tk, n_heads, n_seqs, causal=True, scale=SCALE, backward=False, device="cuda"):
        self.Tq, self.Tk, self.n_heads, self.n_seqs = Tq, Tk, n_heads, n_seqs
        self.causal, self.scale = int(causal), scale
        bf = dict(dtype=torch.bfloat16, device=device)
        self.out = torch.empty((Tq, n_heads, VALUE), **bf)
        self.lse = torch.empty((Tq, n_heads), dtype=torch.float32, device=device)
        self.has_backward = backward
        if backward:
            self.dq = torch.empty((Tq, n_heads, QK), **bf)
            self.dkv = torch.empty((Tk, n_heads, NOPE + VALUE), **bf)
            self.dk_rope = torch.empty((Tk, ROPE), **bf)
            self.ws = torch.empty((max(1, L.moe_mla_attn_bwd_workspace(Tq, Tk, n_heads)),), dtype=torch.uint8,
                                  device=device)

    def _inputs(self, q, kv, k_rope, cu_q, cu_k):
        h = self.n_heads
        B, Tq, Tk = cu_q.shape[0] - 1, q.shape[0], kv.shape[0]
        if Tq > self.Tq or Tk > self.Tk or k_rope.shape[0] != Tk:
            raise ValueError(f"at most {self.Tq} queries and {self.Tk} keys, as many rows of k_rope as of kv")
        if not 0 <= B <= self.n_seqs:
            raise ValueError(f"cu_q must describe at most {self.n_seqs} sequences")
        _vec(cu_q, "cu_q", torch.int32, (B + 1,))
        _vec(cu_k, "cu_k", torch.int32, (B + 1,))
        return (q, _rows(q, "q", (h, QK)), kv, _rows(kv, "kv", (h, NOPE + VALUE)), k_rope,
                _rows(k_rope, "k_rope", (ROPE,))), B, Tq, Tk

    def forward(self, q, kv, k_rope, cu_q, cu_k, stream=None):
        """out [q's rows, n_heads, 128] bf16 and lse [q's rows, n_heads] fp32."""
        ins, B, Tq, Tk = self._inputs(q, kv, k_rope, cu_q, cu_k)
        L.moe_mla_attn_fwd(*ins, L.MOE_BF16, cu_q, cu_k, B, Tq, Tk, self.n_heads, self.causal, self.scale, self.out,
                           self.n_heads * VALUE, self.lse, stream)
        return _first(self.out, Tq), _first(self.lse, Tq)

    __call__ = forward

    def backward(self, dout, q, kv, k_rope, cu_q, cu_k, stream=None):
        """Gradients (dq, dkv, dk_rope) of the last forward, on its inputs."""
        if not self.has_backward:
            raise ValueError("built without backward=True")
        h = self.n_heads
        ins, B, Tq, Tk = self._inputs(q, kv, k_rope, cu_q, cu_k)
        if dout.shape[0] != Tq:
            raise ValueError(f"expected {Tq} rows of dout")
        L.moe_mla_attn_bwd(dout, _rows(dout, "dout", (h, VALUE)), *ins, L.MOE_BF16, self.out, h * VALUE, self.lse,
                           cu_q, cu_k, B, Tq, Tk, h, self.causal, self.scale, self.dq, h * QK, self.dkv,
                           h * (NOPE + VALUE), self.dk_rope, ROPE, self.ws, stream)
        return _first(self.dq, Tq), _first(self.dkv, Tk), _first(self.dk_rope, Tk)


class LatentExpand:
    """kv = latents W_kvb^T for up to max_tokens latents: [T, 512] ->
    [T, n_heads, 256] (each head's key part, then its value), as one
    moe_grouped_fc2 call with a single expert. w_kvb [n_heads, 256, 512] bf16
    is packed once here."""

    def __init__(self, w_kvb, *, max_tokens):
        _weights(w_kvb)
        self.n_heads, self.max_tokens = w_kvb.shape[0], max_tokens
        self.w, _ = pack_weights(w_kvb.reshape(1, -1, LATENT).contiguous(), None, "bf16")
        self.out = torch.empty((max_tokens, self.n_heads, NOPE + VALUE), dtype=torch.bfloat16, device=w_kvb.device)
        # the one expert's segment [0, T) of every T: a call of any size reads
        # its row and writes nothing on the device
        ends = torch.arange(max_tokens + 1, dtype=torch.int32)
        self.offsets = torch.stack((torch.zeros_like(ends), ends), 1).to(w_kvb.device)

    def __call__(self, latents, stream=None):
        """latents [T, 512] bf16, contiguous, T at most max_tokens. Returns
        [T, n_heads, 256], a view of the object's buffer."""
        T = latents.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"at most {self.max_tokens} latents")
        _vec(latents, "latents", torch.bfloat16, (T, LATENT))
        H = self.n_heads * (NOPE + VALUE)
        L.moe_grouped_fc2(latents, None, L.MOE_BF16, self.w, None, L.MOE_BF16, self.offsets[T], 1, H, LATENT, T,
                          self.out, L.MOE_BF16, stream)
        return _first(self.out, T)


class LatentDecode:
    """Attention over a paged latent cache for up to max_tokens new tokens of
    up to max_seqs requests a call. w_kvb [n_heads, 128 + 128, 512]: each
    head's W_UK rows, then its W_UV rows (bf16); packed once here."""

    def __init__(self, w_kvb, *, max_tokens, max_seqs, scale=SCALE):
        _weights(w_kvb)
        h = w_kvb.shape[0]
        self.n_heads, self.max_tokens, self.max_seqs, self.scale = h, max_tokens, max_seqs, scale
        self.w_uk, _ = pack_weights(w_kvb[:, :NOPE].transpose(1, 2).contiguous(), None, "bf16")
        self.w_uv, _ = pack_weights(w_kvb[:, NOPE:].contiguous(), None, "bf16")
        dev = w_kvb.device
        self.out = torch.empty((max_tokens, h, VALUE), dtype=torch.bfloat16, device=dev)
        nws = L.moe_mla_decode_workspace(max_tokens, h)
        if nws == 0:
            raise ValueError("moe_mla_decode does not support these sizes")
        self.ws = torch.empty((nws,), dtype=torch.uint8, device=dev)

    def __call__(self, q, cache, page_table, lens, cu_q, tree_mask=None, lse=None, stream=None):
        """q [T, n_heads, 192] (rotated), cache [n_pages, page_size, 576],
        page_table [B, max_pages] int32, lens [B] int32 (new tokens
        included), cu_q [B + 1] int32, tree_mask optional [T] int64, lse
        optional [T, n_heads] fp32 (filled). Returns out [T, n_heads, 128], a
        view of the object's buffer."""
        T, B, h = q.shape[0], lens.shape[0], self.n_heads
        if T > self.max_tokens or B > self.max_seqs:
            raise ValueError(f"at most {self.max_tokens} tokens of {self.max_seqs} requests")
        if cache.dim() != 3:
            raise ValueError("cache must have three dimensions [n_pages, page_size, 576]")
        _cache(cache, "[n_pages, page_size, 576]")
        _vec(page_table, "page_table", torch.int32, (B, page_table.shape[-1]))
        _vec(lens, "lens", torch.int32, (B,))
        _vec(cu_q, "cu_q", torch.int32, (B + 1,))
        if tree_mask is not None:
            _vec(tree_mask, "tree_mask", torch.int64, (T,))
        if lse is not None:
            _vec(lse, "lse", torch.float32, (T, h))
        L.moe_mla_decode(q, _rows(q, "q", (h, QK)), self.w_uk, self.w_uv, L.MOE_BF16, cache, cache.shape[1],
                         cache.shape[0], page_table, page_table.shape[1], lens, cu_q, tree_mask, B, T, h, self.scale,
                         self.out, h * VALUE, lse, self.ws, stream)
        return self.out[:T]


def latent_cache_append(kv_a, cache, slots, *, norm_weight=None, eps=1e-6, cos=None, sin=None, positions=None,
                        q=None, q_out=None, interleaved=True, stream=None):
    """Normalize and rotate the T rows kv_a [T, 576] (512 latent | 64 rotary)
    and write them to the cache rows slots [T] int64 (page * page_size +
    place; negative: not written). With q [T, n_heads, 192], also its rotary
    part, into q_out (in place without q_out). cos, sin [max_pos, 32] fp32,
    positions [T] int32. Returns q_out."""
    T = kv_a.shape[0]
    _cache(cache, "[..., 576]")
    kv_ld = _rows(kv_a, "kv_a", (CACHE_ROW,))
    _vec(slots, "slots", torch.int64, (T,))
    if norm_weight is not None:
        _vec(norm_weight, "norm_weight", torch.bfloat16, (LATENT,))
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    max_pos = 1
    if cos is not None:
        max_pos = cos.shape[0]
        _vec(cos, "cos", torch.float32, (max_pos, ROPE // 2))
        _vec(sin, "sin", torch.float32, (max_pos, ROPE // 2))
        if positions is None:
            raise ValueError("a rotation needs positions")
        _vec(positions, "positions", torch.int32, (T,))
    h = q_ld = qo_ld = 0
    if q is not None:
        q_out = q if q_out is None else q_out
        if q.shape[0] != T or q_out.shape != q.shape:
            raise ValueError("q and q_out must hold one row per token")
        h = q.shape[1]
        q_ld, qo_ld = _rows(q, "q", (h, QK)), _rows(q_out, "q_out", (h, QK))
    L.moe_mla_append(kv_a, kv_ld, L.MOE_BF16, norm_weight, eps, cos, sin, max_pos, positions, int(interleaved),
                     slots, cache, cache.numel() // CACHE_ROW, q, q_ld, q_out, qo_ld, T, h, stream)
    return q_out

"""Grouped-query attention beside the experts, as sequences of C-ABI calls.

n_heads query heads share n_kv_heads key and value heads of 64 or 128 values.

QKNormRope        RMS norm of every head's query and key and the rotation of
                  their first values by position, in one pass, and backward.
GroupedAttention  packed sequences (prompts, training), forward and backward.
GroupedCache      a paged cache of 8-bit codes with a scale for every 16
                  tokens of a key head; grouped_cache_append fills it.
GroupedDecode     attention over that cache (serving): the last tokens of
                  each request, or a tree of drafted ones.

As in layer.py only marshalling happens here: shapes and types are checked,
buffers are allocated once, every step runs in the HIP library on the given
stream (default: torch's current one). Tensors have to be on the current
device, and an object's buffers too.
"""
from __future__ import annotations

import torch

from . import _lib as L

BLOCK = 16                 # cached tokens that share a scale
DIMS = (64, 128)
_BF, _I32 = torch.bfloat16, torch.int32


def _heads(n_heads, n_kv_heads, head_dim):
    if head_dim not in DIMS:
        raise ValueError(f"head_dim must be 64 or 128, got {head_dim}")
    if not 1 <= n_kv_heads <= n_heads <= 1024 or n_heads % n_kv_heads:
        raise ValueError(f"n_heads must be a multiple of n_kv_heads and at most 1024, got {n_heads}, {n_kv_heads}")


# the checks below run on every call, beside kernels of a few microseconds: they
# ask for plain numbers (torch's device objects and shape slices cost a third
# of a microsecond each)
_current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _here(t: torch.Tensor, name: str) -> int:
    """The current device's number, which has to be t's."""
    dev = t.get_device()
    if dev < 0 or dev != _current():
        raise ValueError(f"{name} must be on the current GPU, got {t.device}")
    return dev


def _beside(t: torch.Tensor, name: str, buffers: int) -> int:
    """The same, which has to be that of the object's buffers too: the kernels
    write to them."""
    dev = _here(t, name)
    if dev != buffers:
        where = f"cuda:{buffers}" if buffers >= 0 else "the host"
        raise ValueError(f"the object's buffers are on {where}, {name} on {t.device}")
    return dev


def _rows(t: torch.Tensor, name: str, heads: int, dim: int, dev: int) -> int:
    """Row stride of a bf16 tensor [tokens, heads, dim] on device dev whose
    tokens are dense inside (the tensor may be a slice of wider rows)."""
    shape = t.shape
    if t.dtype is not _BF or len(shape) != 3 or shape[1] != heads or shape[2] != dim or t.get_device() != dev:
        raise ValueError(f"{name} must be a bfloat16 tensor [tokens, {heads}, {dim}] on the current GPU, got {t.dtype} "
                         f"{tuple(shape)} on {t.device}")
    row, head, one = t.stride()
    if shape[0] > 0 and (one != 1 or (head != dim and heads > 1)):
        raise ValueError(f"{name}: a token's values must be consecutive")
    # a lone token's stride is never used, and may be anything
    return row if shape[0] > 1 else heads * dim


def _vec(t: torch.Tensor, name: str, dtype, shape: tuple, dev: int) -> None:
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on the current GPU, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")


def _first(t: torch.Tensor, n: int) -> torch.Tensor:
    """The first n rows of a buffer."""
    return t if t.shape[0] == n else t[:n]


class QKNormRope:
    """Norm and rotation of the queries and keys of up to T tokens. rotary: how
    many of a head's first values are turned (a multiple of 16; default: all);
    interleaved: pairs (2 i, 2 i + 1) instead of (i, i + rotary / 2). Outputs
    are views of the object's buffers, as many rows as the call's inputs have;
    backward=True adds the gradients' buffers and workspace. One object's calls
    must not overlap."""

    def __init__(self, *, T, n_heads, n_kv_heads, head_dim=128, rotary=None, interleaved=False, eps=1e-6,
                 backward=False, device="cuda"):
        _heads(n_heads, n_kv_heads, head_dim)
        self.T, self.n_heads, self.n_kv_heads, self.head_dim = T, n_heads, n_kv_heads, head_dim
        self.rotary, self.interleaved, self.eps = head_dim if rotary is None else rotary, int(interleaved), eps
        bf = dict(dtype=torch.bfloat16, device=device)
        self.q = torch.empty((T, n_heads, head_dim), **bf)
        self.device = self.q.get_device()
        self.k = torch.empty((T, n_kv_heads, head_dim), **bf)
        self.has_backward = backward
        if backward:
            self.dq, self.dk = torch.empty_like(self.q), torch.empty_like(self.k)
            self.dw_q = torch.empty((head_dim,), dtype=torch.float32, device=device)
            self.dw_k = torch.empty_like(self.dw_q)
            self.ws = torch.empty((L.moe_qk_norm_rope_bwd_workspace(head_dim),), dtype=torch.uint8, device=device)

    def _inputs(self, q, k, w_q, w_k, cos, sin, positions):
        T, h, kv, d = q.shape[0], self.n_heads, self.n_kv_heads, self.head_dim
        if T > self.T or k.shape[0] != T:
            raise ValueError(f"at most {self.T} tokens, as many rows of k as of q")
        dev = _beside(q, "q", self.device)
        if w_q is not None:
            _vec(w_q, "w_q", _BF, (d,), dev)
        if w_k is not None:
            _vec(w_k, "w_k", _BF, (d,), dev)
        if (cos is None) != (sin is None):
            raise ValueError("cos and sin come together")
        max_pos = 1
        if cos is not None:
            max_pos = cos.shape[0]
            table = (max_pos, self.rotary // 2)
            _vec(cos, "cos", torch.float32, table, dev)
            _vec(sin, "sin", torch.float32, table, dev)
            if positions is None:
                raise ValueError("a rotation needs positions")
            _vec(positions, "positions", _I32, (T,), dev)
        head = (q, _rows(q, "q", h, d, dev), k, _rows(k, "k", kv, d, dev), L.MOE_BF16, w_q, w_k, self.eps, cos, sin,
                max_pos, positions, self.rotary, self.interleaved, T, h, kv, d)
        return head, T, dev

    def forward(self, q, k, w_q=None, w_k=None, cos=None, sin=None, positions=None, stream=None):
        """q [T, n_heads, head_dim] and k [T, n_kv_heads, head_dim] bf16 (may be
        slices of a projection's rows), w_q and w_k [head_dim] bf16 (without one:
        not normalized), cos and sin [max_pos, rotary / 2] fp32, positions [T]
        int32. Returns the new q and k."""
        head, T, _ = self._inputs(q, k, w_q, w_k, cos, sin, positions)
        d = self.head_dim
        L.moe_qk_norm_rope(*head, self.q, self.n_heads * d, self.k, self.n_kv_heads * d, stream)
        return _first(self.q, T), _first(self.k, T)

    __call__ = forward

    def backward(self, dq_out, dk_out, q, k, w_q=None, w_k=None, cos=None, sin=None, positions=None, stream=None):
        """Gradients (dq, dk, dw_q, dw_k) from those of the outputs and the
        forward's inputs; dw_q and dw_k are fp32 sums over tokens and heads, None
        for a side without weight."""
        if not self.has_backward:
            raise ValueError("built without backward=True")
        head, T, dev = self._inputs(q, k, w_q, w_k, cos, sin, positions)
        h, kv, d = self.n_heads, self.n_kv_heads, self.head_dim
        if dq_out.shape[0] != T or dk_out.shape[0] != T:
            raise ValueError(f"expected {T} rows of dq_out and dk_out")
        L.moe_qk_norm_rope_bwd(dq_out, _rows(dq_out, "dq_out", h, d, dev), dk_out,
                               _rows(dk_out, "dk_out", kv, d, dev), *head, self.dq, h * d, self.dk, kv * d, self.dw_q,
                               self.dw_k, self.ws, stream)
        return (_first(self.dq, T), _first(self.dk, T), None if w_q is None else self.dw_q,
                None if w_k is None else self.dw_k)


class GroupedAttention:
    """Attention of up to Tq queries over up to Tk keys in up to n_seqs packed
    sequences (cu_q, cu_k [n_seqs + 1] int32, row offsets). With causal, a
    sequence's last query sees all its keys, each earlier one a key less.
    scale defaults to head_dim ** -0.5. Outputs are views of the object's
    buffers, as many rows as the call's inputs have; backward=True adds the
    gradients' buffers and workspace. One object's calls must not overlap."""

    def __init__(self, *, Tq, Tk, n_heads, n_kv_heads, head_dim=128, n_seqs, causal=True, scale=None, backward=False,
                 device="cuda"):
        _heads(n_heads, n_kv_heads, head_dim)
        self.Tq, self.Tk, self.n_seqs = Tq, Tk, n_seqs
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, n_kv_heads, head_dim
        self.causal, self.scale = int(causal), head_dim ** -0.5 if scale is None else scale
        bf = dict(dtype=torch.bfloat16, device=device)
        self.out = torch.empty((Tq, n_heads, head_dim), **bf)
        self.device = self.out.get_device()
        self.lse = torch.empty((Tq, n_heads), dtype=torch.float32, device=device)
        need = L.moe_gqa_attn_fwd_workspace(Tq, n_heads, head_dim)
        self.has_backward = backward
        if backward:
            self.dq = torch.empty_like(self.out)
            self.dk = torch.empty((Tk, n_kv_heads, head_dim), **bf)
            self.dv = torch.empty_like(self.dk)
            need = max(need, L.moe_gqa_attn_bwd_workspace(Tq, Tk, n_heads, n_kv_heads, head_dim))
        self.ws = torch.empty((max(1, need),), dtype=torch.uint8, device=device)

    def _inputs(self, q, k, v, cu_q, cu_k):
        h, kv, d = self.n_heads, self.n_kv_heads, self.head_dim
        B, Tq, Tk = cu_q.shape[0] - 1, q.shape[0], k.shape[0]
        if Tq > self.Tq or Tk > self.Tk or v.shape[0] != Tk:
            raise ValueError(f"at most {self.Tq} queries and {self.Tk} keys, as many rows of v as of k")
        if not 0 <= B <= self.n_seqs:
            raise ValueError(f"cu_q must describe at most {self.n_seqs} sequences")
        dev = _beside(q, "q", self.device)
        _vec(cu_q, "cu_q", _I32, (B + 1,), dev)
        _vec(cu_k, "cu_k", _I32, (B + 1,), dev)
        return (q, _rows(q, "q", h, d, dev), k, _rows(k, "k", kv, d, dev), v, _rows(v, "v", kv, d, dev),
                L.MOE_BF16), B, Tq, Tk, dev

    def forward(self, q, k, v, cu_q, cu_k, stream=None):
        """out [q's rows, n_heads, head_dim] bf16 and lse [q's rows, n_heads]
        fp32; k and v [Tk, n_kv_heads, head_dim]."""
        ins, B, Tq, Tk, _ = self._inputs(q, k, v, cu_q, cu_k)
        h, d = self.n_heads, self.head_dim
        L.moe_gqa_attn_fwd(*ins, cu_q, cu_k, B, Tq, Tk, h, self.n_kv_heads, d, self.causal, self.scale, self.out,
                           h * d, self.lse, self.ws, stream)
        return _first(self.out, Tq), _first(self.lse, Tq)

    __call__ = forward

    def backward(self, dout, q, k, v, cu_q, cu_k, stream=None):
        """Gradients (dq, dk, dv) of the last forward, on its inputs."""
        if not self.has_backward:
            raise ValueError("built without backward=True")
        ins, B, Tq, Tk, dev = self._inputs(q, k, v, cu_q, cu_k)
        h, kv, d = self.n_heads, self.n_kv_heads, self.head_dim
        if dout.shape[0] != Tq:
            raise ValueError(f"expected {Tq} rows of dout")
        L.moe_gqa_attn_bwd(dout, _rows(dout, "dout", h, d, dev), *ins, self.out, h * d, self.lse, cu_q, cu_k, B, Tq,
                           Tk, h, kv, d, self.causal, self.scale, self.dq, h * d, self.dk, kv * d, self.dv, kv * d,
                           self.ws, stream)
        return _first(self.dq, Tq), _first(self.dk, Tk), _first(self.dv, Tk)


class GroupedCache:
    """The 8-bit paged cache: E4M3 codes and scale exponents (bytes e + 127)
    of n_pages pages of page_size tokens. k [n_pages, n_kv_heads, page_size /
    16, head_dim / 16, 16, 16] holds value d of a block's token t at [d / 16, t,
    d % 16], v [n_pages, n_kv_heads, page_size / 16, head_dim / 2, 2, 2, 2, 4] at
    [d / 2, (t / 4) % 2, d % 2, t / 8, t % 4]; k_scales, v_scales [n_pages,
    n_kv_heads, page_size / 16]. Pages are the caller's to hand out; a page's
    content may be copied with these tensors' rows."""

    def __init__(self, k, v, k_scales, v_scales):
        if k.dim() != 6 or k.shape[4:] != (BLOCK, 16) or k.shape[3] * 16 not in DIMS:
            raise ValueError(f"k must have shape [n_pages, n_kv_heads, page_size / 16, head_dim / 16, 16, 16], "
                             f"got {tuple(k.shape)}")
        self.n_pages, self.n_kv_heads, blocks = k.shape[:3]
        self.head_dim, self.page_size = k.shape[3] * 16, blocks * BLOCK
        self.device, u8, head = _here(k, "k"), torch.uint8, (self.n_pages, self.n_kv_heads, blocks)
        _vec(k, "k", u8, tuple(k.shape), self.device)
        _vec(v, "v", u8, (*head, self.head_dim // 2, 2, 2, 2, 4), self.device)
        _vec(k_scales, "k_scales", u8, head, self.device)
        _vec(v_scales, "v_scales", u8, head, self.device)
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales

    @classmethod
    def empty(cls, n_pages, page_size, n_kv_heads, head_dim=128, device="cuda"):
        """A new cache (its memory is not cleared: what lies behind a request's
        length is never used)."""
        if page_size < BLOCK or page_size % BLOCK:
            raise ValueError(f"page_size must be a multiple of 16, got {page_size}")
        if head_dim not in DIMS:
            raise ValueError(f"head_dim must be 64 or 128, got {head_dim}")
        head = (n_pages, n_kv_heads, page_size // BLOCK)
        new = lambda *s: torch.empty((*head, *s), dtype=torch.uint8, device=device)  # noqa: E731
        return cls(new(head_dim // 16, BLOCK, 16), new(head_dim // 2, 2, 2, 2, 4), new(), new())

    def _tensors(self):
        return self.k, self.v, self.k_scales, self.v_scales, self.page_size, self.n_pages


def _requests(cache, page_table, lens, cu, dev):
    B = lens.shape[0]
    if cache.device != dev:
        raise ValueError(f"the cache must be on the current GPU, got cuda:{cache.device}")
    _vec(page_table, "page_table", _I32, (B, page_table.shape[-1]), dev)
    _vec(lens, "lens", _I32, (B,), dev)
    _vec(cu, "cu", _I32, (B + 1,), dev)
    return B


def grouped_cache_append(k, v, cache, page_table, lens, cu, stream=None):
    """New keys and values (rotated already) [T, n_kv_heads, head_dim] bf16
    into the cache: request b's rows cu[b] .. cu[b + 1] become its last tokens,
    lens[b] (new ones included) counts them. The pages written are distinct. page_table [B, max_pages] int32,
    lens [B] and cu [B + 1] int32. A request that goes back (a smaller lens, to
    write over rejected drafts) leaves the scale of the 16 tokens it goes back
    into as large as they had made it."""
    T, kv, d = k.shape[0], cache.n_kv_heads, cache.head_dim
    if v.shape[0] != T:
        raise ValueError("as many rows of v as of k")
    dev = _here(k, "k")
    B = _requests(cache, page_table, lens, cu, dev)
    L.moe_gqa_append(k, _rows(k, "k", kv, d, dev), v, _rows(v, "v", kv, d, dev), L.MOE_BF16, *cache._tensors(),
                     page_table, page_table.shape[1], lens, cu, B, T, kv, d, stream)


class GroupedDecode:
    """Attention over a GroupedCache for up to max_tokens new tokens of up to
    max_seqs requests a call. scale defaults to head_dim ** -0.5. One object's
    calls must not overlap; it is built outside of a graph's capture."""

    def __init__(self, *, n_heads, n_kv_heads, head_dim=128, max_tokens, max_seqs, scale=None, device="cuda"):
        _heads(n_heads, n_kv_heads, head_dim)
        if not (1 <= max_seqs <= 65536 and max_seqs * n_kv_heads <= 1 << 19 and 1 <= max_tokens and
                max_tokens * n_heads <= 1 << 24):
            raise ValueError("moe_gqa_decode does not support these sizes")
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise ValueError("GroupedDecode clears its workspace once, so it cannot be built during a capture")
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, n_kv_heads, head_dim
        self.max_tokens, self.max_seqs = max_tokens, max_seqs
        self.scale = head_dim ** -0.5 if scale is None else scale
        self.out = torch.empty((max_tokens, n_heads, head_dim), dtype=torch.bfloat16, device=device)
        self.device = self.out.get_device()
        # zeros once: where a call counts the pieces of its work, and leaves zeros
        self.ws = torch.zeros((L.moe_gqa_decode_workspace(head_dim),), dtype=torch.uint8, device=device)
        if self.ws.is_cuda:                # the first call may be on another stream
            torch.cuda.current_stream(self.ws.device).synchronize()

    def __call__(self, q, cache, page_table, lens, cu_q, tree_mask=None, lse=None, stream=None):
        """q [T, n_heads, head_dim] bf16 (normalized and rotated), the new
        tokens of all requests, in the cache already; page_table [B, max_pages]
        int32, lens [B] int32 (new tokens included), cu_q [B + 1] int32,
        tree_mask optional [T] int64, lse optional [T, n_heads] fp32 (filled).
        Returns out [T, n_heads, head_dim], a view of the object's buffer."""
        T, h, kv, d = q.shape[0], self.n_heads, self.n_kv_heads, self.head_dim
        dev = _beside(q, "q", self.device)
        B = _requests(cache, page_table, lens, cu_q, dev)
        if T > self.max_tokens or B > self.max_seqs:
            raise ValueError(f"at most {self.max_tokens} tokens of {self.max_seqs} requests")
        if (cache.n_kv_heads, cache.head_dim) != (kv, d):
            raise ValueError(f"the cache holds {cache.n_kv_heads} heads of {cache.head_dim}, expected {kv} of {d}")
        if tree_mask is not None:
            _vec(tree_mask, "tree_mask", torch.int64, (T,), dev)
        if lse is not None:
            _vec(lse, "lse", torch.float32, (T, h), dev)
        L.moe_gqa_decode(q, _rows(q, "q", h, d, dev), L.MOE_BF16, *cache._tensors(), page_table, page_table.shape[1], lens,
                         cu_q, tree_mask, B, T, h, kv, d, self.scale, self.out, h * d, lse, self.ws, stream)
        return _first(self.out, T)

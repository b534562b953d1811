"""Grouped-query attention's classes: their own buffers have to be where the
call's tensors are (no call here reaches the library)."""
import pytest
import torch

from mixture_experts_layer_sigmoid_amd import gqa


class OnGpu(torch.Tensor):
    """A host tensor that says it is on the first GPU."""

    def get_device(self):
        return 0


def _on_gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def no_calls(monkeypatch):
    def reached(*a, **k):
        raise AssertionError("reached the library")
    for name in ("moe_qk_norm_rope", "moe_qk_norm_rope_bwd", "moe_gqa_attn_fwd", "moe_gqa_attn_bwd", "moe_gqa_append",
                 "moe_gqa_decode"):
        monkeypatch.setattr(gqa.L, name, reached)
    monkeypatch.setattr(gqa, "_current", lambda: 0)


def test_buffers_elsewhere_are_refused(no_calls):
    """Objects built in host memory (or for another GPU) take no tensors of the
    current one: the kernels would write to their buffers."""
    size = dict(n_heads=4, n_kv_heads=2, head_dim=64, device="cpu")
    q, k, v = _on_gpu(3, 4, 64), _on_gpu(3, 2, 64), _on_gpu(3, 2, 64)
    i32 = lambda *s: _on_gpu(*s, dtype=torch.int32)
    norm = gqa.QKNormRope(T=3, backward=True, **size)
    att = gqa.GroupedAttention(Tq=3, Tk=3, n_seqs=1, backward=True, **size)
    dec = gqa.GroupedDecode(max_tokens=3, max_seqs=1, **size)
    u8 = lambda *s: _on_gpu(2, 2, 1, *s, dtype=torch.uint8)
    cache = gqa.GroupedCache(u8(4, 16, 16), u8(32, 2, 2, 2, 4), u8(), u8())
    calls = [lambda: norm(q, k), lambda: norm.backward(q, k, q, k), lambda: att(q, k, v, i32(2), i32(2)),
             lambda: att.backward(q, q, k, v, i32(2), i32(2)), lambda: dec(q, cache, i32(1, 1), i32(1), i32(2))]
    for call in calls:
        with pytest.raises(ValueError, match="buffers are on"):
            call()


def test_buffers_beside_the_tensors_pass(no_calls):
    """The same calls reach the library where the buffers are on that GPU too."""
    size = dict(n_heads=4, n_kv_heads=2, head_dim=64, device="cpu")
    q, k = _on_gpu(3, 4, 64), _on_gpu(3, 2, 64)
    norm = gqa.QKNormRope(T=3, **size)
    norm.device = 0
    with pytest.raises(AssertionError, match="reached the library"):
        norm(q, k)

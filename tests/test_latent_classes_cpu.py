"""Refusals of the latent-attention classes that come before any call of the
library (a tensor in host memory must never reach a kernel)."""
import pytest
import torch

from mixture_experts_layer_sigmoid_amd import mla

BF = torch.bfloat16


@pytest.fixture
def no_calls(monkeypatch):
    """The library's entry points fail the test when they are reached."""
    def reached(*a, **k):
        raise AssertionError("reached the library")
    for name in ("moe_mla_decode", "moe_mla_append", "moe_pack_weights", "moe_grouped_fc2"):
        monkeypatch.setattr(mla.L, name, reached)


def _plan(h=2):
    """A LatentDecode without its buffers, which need the GPU."""
    p = object.__new__(mla.LatentDecode)
    p.n_heads, p.max_tokens, p.max_seqs, p.scale = h, 4, 2, mla.SCALE
    return p


def test_decode_refuses_a_cache_in_host_memory(no_calls):
    cache = torch.zeros((3, 16, 576), dtype=BF)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    with pytest.raises(ValueError, match="cache"):
        _plan()(torch.zeros((1, 2, 192), dtype=BF), cache, i32(0)[None], i32(4), i32(0, 1))


def test_append_refuses_a_cache_in_host_memory(no_calls):
    cache = torch.zeros((3, 16, 576), dtype=BF)
    with pytest.raises(ValueError, match="cache"):
        mla.latent_cache_append(torch.zeros((1, 576), dtype=BF), cache, torch.zeros(1, dtype=torch.int64))


@pytest.mark.parametrize("shape,dtype", [((2, 128, 512), BF), ((2, 256, 512), torch.float32),
                                         ((2, 256, 512), torch.float16), ((2, 256, 576), BF), ((256, 512), BF),
                                         ((2, 256, 512), BF)])
def test_weights_are_refused_before_packing(no_calls, shape, dtype):
    """Another shape or type, and the right ones in host memory."""
    w = torch.zeros(shape, dtype=dtype)
    with pytest.raises(ValueError, match="w_kvb"):
        mla.LatentExpand(w, max_tokens=4)
    with pytest.raises(ValueError, match="w_kvb"):
        mla.LatentDecode(w, max_tokens=4, max_seqs=1)


def test_rows_of_no_tokens_have_no_strides_to_check():
    """numpy gives empty arrays strides of their own; there are no values."""
    class Empty:
        dtype, is_cuda = BF, True
        shape = torch.Size((0, 3, 192))

        def stride(self):
            return (0, 0, 0)

    assert mla._rows(Empty(), "q", (3, 192)) == 3 * 192
    Empty.shape = torch.Size((1, 3, 192))
    with pytest.raises(ValueError, match="consecutive"):
        mla._rows(Empty(), "q", (3, 192))

"""The scale of the latent-attention entries (no call here reaches the device)."""
import pytest

from mixture_experts_layer_sigmoid_amd import _lib as L
from tests.test_capi_latent_cpu import INVALID, _bwd, _dec, _fwd


@pytest.mark.parametrize("call", [_fwd, _bwd, _dec])
def test_scales_whose_product_with_log2_e_overflows_are_refused(call):
    lib = L.load()
    for scale in (2.4e38, 2.99e38, 3.3e38):
        assert call(lib, scale=scale) == INVALID, scale
        assert b"scale" in lib.moe_last_error()
    for scale in (2.3e38, 1e-38):                       # (a null pointer is refused after the scale)
        assert call(lib, scale=scale, q=None) == INVALID and b"null pointer" in lib.moe_last_error(), scale

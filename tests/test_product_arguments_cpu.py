"""Refusals of the grouped products that depend on more than one argument, before any HIP call."""
import pytest

import mixture_experts_layer_35_amd as moe
from test_product_cpu import BAD, FAKE, dw, dx, int8, lib, product  # noqa: F401


@pytest.mark.parametrize("call", [product, dx, dw, int8], ids=lambda f: f.__name__)
def test_bounds_and_tokens_lie_at_multiples_of_4(lib, call):  # noqa: F811
    """They are read by 4-byte scalar loads, which drop an address's last two bits."""
    for off in (1, 2, 3):
        assert call(lib, offsets=FAKE + off) == BAD and "offsets must be 4-byte aligned" in moe.moe_last_error()
        if call is not dx:
            assert call(lib, gather=FAKE + off) == BAD and "gather must be 4-byte aligned" in moe.moe_last_error()

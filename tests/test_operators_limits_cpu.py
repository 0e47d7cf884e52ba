"""Extreme but well-formed arguments of the decode-step operators, refused before any CUDA call."""
import pytest

import weight_streaming_megakernel_b200 as wsm
from test_operators_cpu import INVALID, attention, cache

from weight_streaming_megakernel_b200 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    yield


@pytest.mark.parametrize("scale,k_scale", [(2.0 ** 127, 2.0), (-2.0 ** 127, 1.5), (3e38, 1e30)])
def test_a_factor_past_fp32_is_refused(scale, k_scale):
    eight = cache(dtype=3, k_scale=k_scale)
    assert wsm.lib().wsm_paged_attention(eight, attention(scale=scale), None) == INVALID
    assert "past fp32" in wsm.last_error()

"""Scales of the attention operators (include/spec_kv.h) whose product in base 2 is no float32 are refused, on the
host, before any CUDA call."""
import numpy as np
import pytest

from speculative_decoding_verification_33_gb300 import _lib
from tests.test_abi_kv8 import attention, prompt

MOST = float(np.finfo(np.float32).max)


def kv4(**kw):
    a = dict(B=2, T=3, hq=4, hk=2, D=64, ps=16, pages=5, blocks=4, q=1 << 20, qs=256, cache=1 << 20, table=1 << 20,
             lens=1 << 20, cu=1 << 20, scale=0.125, ks=1.0, vs=1.0, most=1, out=1 << 20, lse=1 << 20)
    a.update(kw)
    return _lib.load().spec_kv4_attention(*a.values(), 0)


@pytest.mark.parametrize("scale", [MOST, -MOST, 0.7 * MOST])
def test_scale_too_large(scale):
    for call in (attention, prompt, kv4):
        assert call(scale=scale) == _lib.SV_ERR_INVALID_ARG


def test_product_of_scales_too_large():
    assert kv4(scale=1e20, ks=1e20) == _lib.SV_ERR_INVALID_ARG
    assert kv4(scale=-1e20, ks=1e20) == _lib.SV_ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [0.69 * MOST, -0.69 * MOST, 0.0, 1e-45])
def test_scales_at_the_limits(scale):
    for call in (attention, prompt, kv4):
        assert call(scale=scale, T=0) == _lib.SV_OK

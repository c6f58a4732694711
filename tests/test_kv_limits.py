"""Limits of the block tables' 32-bit sums: refused on the host before any CUDA call."""
import pytest

from speculative_decoding_verification_33_gb300 import _lib
from tests.test_abi_kv import tables


@pytest.mark.parametrize("kw", [dict(max_tokens=2 ** 31 - 1), dict(ring_size=2 ** 31 - 1)])
def test_tables_limits_that_sums_do_not_pass(kw):
    """Sums of pages and tokens are held at 2^31 - 1, so that is no limit they could be seen to pass."""
    assert tables(**kw) == _lib.SV_ERR_UNSUPPORTED

"""Refusals of the verification that are decided before any CUDA call."""
import pytest

from tests.test_cache_host import call
from tests.test_tree_host import VERIFY


@pytest.mark.parametrize("scale", [2.0 ** 127 * (1 + 2.0 ** -23), 3.4e38, -1e-45])
def test_scales_beyond_what_a_product_with_log2_e_holds_are_refused(scale):
    from lossless_kv_cache_bf16_gb300 import splitzip as S

    assert call(S.LIB, "sz_verify_tree", VERIFY, scale=scale) == S.SZ_ERR_INVALID_ARG

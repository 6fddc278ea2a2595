"""The serving operators on a host without a GPU: what their binding and the
library refuse before anything is launched."""
import pytest

from tests.test_attend_host import ATTEND
from tests.test_cache_host import POOL, call


@pytest.fixture(scope="module")
def S():
    from lossless_kv_cache_bf16_gb300 import splitzip

    return splitzip


@pytest.mark.parametrize("change", POOL + [dict(status=None), dict(q=None), dict(ws=None), dict(hq=9)], ids=str)
def test_the_stalled_attention_refuses_what_the_attention_does(S, change):
    stalled = {**ATTEND, "status": ATTEND["lens"]}
    assert call(S.LIB, "sz_debug_attend_stalled", stalled, **change) == S.SZ_ERR_INVALID_ARG

"""CPU checks of the caps that scored attention takes."""
import pytest

from paged_kv_cache_wf_gb300 import binding as wf
from paged_kv_cache_wf_gb300 import build

FAKE = 0x10000   # 16-byte aligned, never dereferenced: a call without requests


@pytest.fixture(scope="module")
def lib():
    build.build()
    return wf.load()


@pytest.mark.parametrize("cap, scale, ok", [(2.0 ** 100, 0.1, True), (2.1e30, 0.1, False), (3e38, 0.1, False), (1e30, 1e-7, True),
                                            (1e30, 1e-9, False), (1e30, -1e-9, False), (1e30, 0.0, True), (1e-20, 0.1, True)])
def test_caps(lib, cap, scale, ok):
    d = wf.wf_pool_desc(10, 16, 2, 64, wf.WF_DTYPE_BF16, 0.0, 0.0)
    rc = lib.wf_paged_scored_attention(FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, FAKE, 0, 0, 0, 64, 8, scale, cap, 0, None, None, d,
                                       FAKE, 0, None, None)
    assert rc == (wf.WF_OK if ok else wf.WF_ERR_INVALID_ARG)

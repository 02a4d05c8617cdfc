"""CPU check: a scale whose exponent factor, scale * log2(e), leaves float32 is refused."""
import math

import pytest

from paged_kv_cache_wf_gb300 import binding as wf
from paged_kv_cache_wf_gb300 import build

FAKE = 0x10000   # 16-byte aligned, never dereferenced by calls that are refused


@pytest.mark.parametrize("pool", [wf.WF_DTYPE_F32, wf.WF_DTYPE_BF16, wf.WF_DTYPE_FP8_E4M3])
def test_scales_past_the_exponents_range(pool):
    build.build()
    d = wf.wf_pool_desc(10, 16, 2, 64, pool, 1.0, 1.0)

    def call(scale):
        # a workspace of no bytes: the call ends there at the latest
        return wf.load().wf_paged_tree_decode(FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, FAKE, FAKE, 1, 2, 10, 7, 64, 8, scale,
                                              d, FAKE, 0, None, None)

    for scale in (2.4e38, -2.4e38, 3.4e38, math.inf, -math.inf, math.nan):
        assert call(scale) == wf.WF_ERR_INVALID_ARG, scale
    for scale in (0.0, -0.0, 1e-45, 0.125, -2.0, 2.3e38, -2.3e38):
        assert call(scale) == wf.WF_ERR_WORKSPACE, scale

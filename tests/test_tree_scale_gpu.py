"""Softmax scales of wf_paged_tree_decode at the ends of what it takes, over every pool type."""
import numpy as np
import pytest
import torch

from paged_kv_cache_wf_gb300 import binding as wf
from tests import _draft as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_wf_gb300 import build
    build.build()


@pytest.mark.parametrize("D,P", [(128, 16), (64, 16), (64, 7)])
@pytest.mark.parametrize("q_size,k_scale", [(2.0, 1 / 64), (2.0 ** -13, 1 / 64), (2.0 ** -6, 1e-4), (1e-30, 1.0)])
@pytest.mark.parametrize("scale", [0.0, 1e-38, -1e-38, -0.2, 0.3])
def test_fp8_scales_and_small_queries(D, P, q_size, k_scale, scale):
    """Scale, K scale and the query rows' size meet in one factor of the scores: however small it gets, a masked
    position has no weight and the others theirs (for a scale next to 0, equal ones)."""
    t = R.Tree([40, 0, 130], [6, 9, 33], 8, 2, D, P, "fp8", seed=90, k_scale=k_scale, v_scale=1 / 96, q_size=q_size)
    t.scale = scale
    d = t.device()
    R.check(t, t.run(d, t.workspace()))
    assert wf.wf_device_status_fetch(d["status"]) == 0


@pytest.mark.parametrize("pool,D,P", [("bf16", 128, 16), ("bf16", 64, 16), ("bf16", 64, 7), ("f32", 128, 16), ("f32", 64, 16)])
@pytest.mark.parametrize("scale", [0.0, 1e-38, -1e-38, -0.2])
def test_other_pools(pool, D, P, scale):
    t = R.Tree([40, 0, 130], [6, 9, 33], 8, 2, D, P, pool, seed=91)
    t.scale = scale
    d = t.device()
    R.check(t, t.run(d, t.workspace()))


@pytest.mark.parametrize("pool,P", [("bf16", 16), ("fp8", 16), ("f32", 16), ("bf16", 7)])
@pytest.mark.parametrize("scale", [2.35e38, -2.35e38])
def test_the_largest_scales_of_scores_of_zero(pool, P, scale):
    """Queries of 0: every score is 0 whatever the scale, the weights are equal."""
    t = R.Tree([40, 0, 130], [6, 9, 33], 8, 2, 64, P, pool, seed=92, **({"k_scale": 1 / 64} if pool == "fp8" else {}))
    t.q[:] = 0
    t.scale = scale
    d = t.device()
    R.check(t, t.run(d, t.workspace()))

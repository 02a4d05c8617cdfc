"""CPU check that scored attention's GPU cases meet each of its kernels' forms: on the tensor cores blocks of at most 32 rows
(spread over the tile), of one query tile and of two."""
import pytest

from paged_kv_cache_wf_gb300 import binding as wf
from paged_kv_cache_wf_gb300 import build
from tests import test_scored_caps_gpu as caps
from tests import test_scored_gpu as cases


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def form(shape):
    """(pool, D, form) of a case on the tensor cores, None on the others."""
    cached, new, H_q, H_kv, D, P, pool = shape
    d = wf.wf_pool_desc(1000, P, H_kv, D, {"f32": 0, "bf16": 1, "fp8": 2}[pool], 1.0, 1.0)
    if wf.wf_paged_tree_decode_kernel(d, H_q) != wf.WF_KERNEL_TENSOR_CORES:
        return None
    group = H_q // H_kv
    return pool, D, "spread" if max(new) <= 32 // group else "one tile" if pool == "fp8" or max(new) <= 128 // group else "two tiles"


WANT = {("bf16", D, f) for D in (64, 128) for f in ("spread", "one tile", "two tiles")} | \
       {("fp8", D, f) for D in (64, 128) for f in ("spread", "one tile")}


def test_every_form_meets_the_softmax():
    assert {form(s) for s in cases.SHAPES.values()} - {None} == WANT


def test_every_form_meets_caps_above_its_scores():
    assert {form(s) for s in caps.SHAPES.values()} - {None} == WANT

"""Tree attention over fp8 pools: the outputs carry no more than fp16 weights' rounding."""
import numpy as np
import pytest
import torch

from paged_kv_cache_wf_gb300 import binding as wf
from paged_kv_cache_wf_gb300 import build
from tests import _draft_tight as X


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    wf.load()


def to(dtype, x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).double().numpy()


@pytest.mark.parametrize("name", list(X.CASES))
def test_the_bound_tells_fp16_weights_from_bf16(name):
    """On the CPU: fp16 weights keep it, and bf16 weights break it where a row sees few positions."""
    t = X.CASES[name]()
    assert t.kernel() == wf.WF_KERNEL_TENSOR_CORES
    ref, lim = t.tight()
    fine, _ = t.tight(lambda w: to(torch.float16, w * 2.0 ** 7) / 2.0 ** 7)
    assert (np.abs(to(torch.bfloat16, fine) - ref) <= lim).all()
    if not name.startswith("ragged"):
        coarse, _ = t.tight(lambda w: to(torch.bfloat16, w))
        assert (np.abs(to(torch.bfloat16, coarse) - ref) > lim).any()


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(X.CASES))
def test_outputs(name):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    t = X.CASES[name]()
    d = t.device()
    got = t.run(d, t.workspace()).double().cpu().numpy()
    ref, lim = t.tight()
    off = np.abs(got - ref)
    assert np.isfinite(got).all()
    assert (off <= lim).all(), f"off by {off.max():.3e}, {(off / lim).max():.2f} of what is allowed"

"""Offsets of drafts that are out of order or out of range: their requests are skipped, the others are right."""
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


LOW = -2 ** 31


# offsets of five requests with 6, 9, 5, 0 and 7 drafts (rows 0, 6, 15, 20, 20 .. 27), and the requests that stay valid
@pytest.mark.parametrize("cu,valid", [
    ([0, 6, 3, 20, 20, 27], (0, 3, 4)),           # 1 runs backwards, 2 has more than the most drafts
    ([0, 6, 100, 20, 20, 27], (0, 3, 4)),         # 1 ends past the rows, 2 runs backwards
    ([0, 6, 15, 20, 20, 28], (0, 1, 2, 3)),       # the last ends past the rows
    ([-6, 6, 15, 20, 20, 27], (1, 2, 3, 4)),      # the first starts before them
    ([0, LOW, 15, 20, 20, 27], (2, 3, 4)),
    ([0, 6, 15, 20, 2 ** 31 - 1, 27], (0, 1, 2)),
])
@pytest.mark.parametrize("pool,P,D", [("bf16", 16, 128), ("bf16", 16, 64), ("fp8", 16, 128), ("fp8", 16, 64),
                                      ("f32", 16, 64), ("bf16", 7, 64), ("fp8", 7, 128)])
def test_bad_offsets_skip_their_requests_only(pool, P, D, cu, valid):
    fp8 = dict(k_scale=1 / 64, v_scale=1 / 96) if pool == "fp8" else {}
    t = R.Tree([40, 50, 130, 10, 0], [6, 9, 5, 0, 7], 8, 2, D, P, pool, seed=93, **fp8)
    ref = t.reference()
    rows = [r for b in valid for r in range(t.cu[b], t.cu[b + 1])]
    d = t.device()
    d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = t.run(d, t.workspace())
    rest = [r for r in range(t.T) if r not in rows]
    assert (got[rest] == 7.0).all(), "rows of a skipped request were written"
    off = np.abs(got.double().cpu().numpy()[rows] - ref[0][rows])
    assert (off <= t.bound(*ref)[rows]).all()
    assert wf.wf_device_status_fetch(d["status"]) == wf.WF_DEV_BAD_SEQLEN

"""wf_paged_scored_attention over V rows that are not finite."""
import numpy as np
import pytest
import torch

from paged_kv_cache_wf_gb300 import binding as wf
from tests._scored import Scored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_wf_gb300 import build
    build.build()


FP8 = dict(k_scale=1 / 64, v_scale=1 / 96)
# new rows, heads, pool: blocks of two query tiles, of one, and of few rows; the CUDA cores
LONG = {"two tiles": (70, 8, 2, 128, 16, "bf16"), "two tiles d64": (70, 4, 1, 64, 16, "bf16"), "one tile": (20, 8, 2, 128, 16, "bf16"),
        "few": (5, 8, 2, 128, 16, "bf16"), "fp8": (40, 8, 2, 128, 16, "fp8"), "fp8 few d64": (3, 4, 1, 64, 16, "fp8"),
        "fp32": (9, 4, 1, 64, 16, "f32")}


@pytest.mark.parametrize("where", ["one", "all"])
@pytest.mark.parametrize("shape", list(LONG))
def test_a_long_context_without_a_position_that_all_rows_see(shape, where):
    """Two documents of 30000 and 12000 tokens whose rows share a block, so that each of its tiles is looked at: elements
    that are no numbers reach the rows that see them, and the call ends in time."""
    new, H_q, H_kv, D, P, pool = LONG[shape]
    first, cached = 30000, 42000
    t = Scored([cached], [new], H_q, H_kv, D, P, pool, seed=3, **(FP8 if pool == "fp8" else {}))
    r = np.zeros((new, 2), np.int32)
    r[::2] = (0, first)
    r[1::2, 0], r[1::2, 1] = first, cached + 1 + np.arange(new)[1::2]
    t.ranges = r
    clean = t.device()
    t.run(clean, t.workspace())
    assert wf.wf_device_status_fetch(clean["status"]) == 0
    d = t.device()
    at = np.array([first // 3]) if where == "one" else np.arange(first)
    blk, off = (torch.from_numpy(np.asarray(x)).cuda().long() for x in (t.table[0, at // P], at % P))
    nan = 0x7F if pool == "fp8" else float("nan")
    d["v"][blk, off, H_kv - 1, 5] = nan
    t.run(d, t.workspace())
    assert wf.wf_device_status_fetch(d["status"]) == 0
    got, want = d["out"].double().cpu().numpy(), clean["out"].double().cpu().numpy()
    want[::2, H_q - H_q // H_kv:, 5] = np.nan
    assert np.array_equal(got, want, equal_nan=True)

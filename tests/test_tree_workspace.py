"""wf_paged_tree_decode_workspace_size: a workspace for the largest call serves every smaller one."""
import itertools

import pytest

from paged_kv_cache_wf_gb300 import binding as wf
from paged_kv_cache_wf_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    wf.load()


def size(pool, D, P, H_kv, group, B, q, length):
    n = wf.wf_paged_tree_decode_workspace_size(B, H_kv * group, q, length, wf.wf_pool_desc(4096, P, H_kv, D, pool, 1.0, 1.0))
    assert n > 0
    return n


POOLS = [wf.WF_DTYPE_F32, wf.WF_DTYPE_BF16, wf.WF_DTYPE_FP8_E4M3]
NUMBER = {"f32": wf.WF_DTYPE_F32, "bf16": wf.WF_DTYPE_BF16, "fp8": wf.WF_DTYPE_FP8_E4M3}
# both sides of every change of form: 8, 16 and 32 rows, 128 and 256
DRAFTS = sorted({q + e for g in range(1, 9) for q in (8 // g, 16 // g, 32 // g, 128 // g, 256 // g) for e in (-1, 0, 1)
                 if q + e >= 1} | {1, 400})


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 7])
def test_more_drafts_need_no_less(pool, D, P):
    for H_kv, group, B, length in itertools.product((1, 2, 8), range(1, 9), (1, 3, 32, 231), (400, 4096)):
        sizes = [size(pool, D, P, H_kv, group, B, q, length) for q in DRAFTS]
        assert sizes == sorted(sizes), (H_kv, group, B, length)


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 7])
def test_more_requests_or_positions_need_no_less(pool, D, P):
    for H_kv, group, q in itertools.product((1, 8), (1, 3, 4, 8), (1, 4, 5, 16, 17, 64)):
        for B in (1, 3, 40):
            by_length = [size(pool, D, P, H_kv, group, B, q, n) for n in (64, 65, 128, 129, 1000, 4096, 1 << 20)]
            assert by_length == sorted(by_length), (H_kv, group, q, B)
        for n in (64, 1000, 1 << 20):
            by_batch = [size(pool, D, P, H_kv, group, b, q, n) for b in (1, 2, 3, 19, 20, 40, 160, 161, 231, 4000)]
            assert by_batch == sorted(by_batch), (H_kv, group, q, n)


@pytest.mark.gpu
@pytest.mark.parametrize("pool,P", [("f32", 16), ("bf16", 16), ("fp8", 16), ("bf16", 7)])
def test_one_workspace_for_every_step(pool, P):
    """Allocated for the largest step, used by steps of fewer drafts, requests and positions."""
    import torch

    from tests import _draft as R
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8 = dict(k_scale=1 / 64, v_scale=1 / 64) if pool == "fp8" else {}
    n = wf.wf_paged_tree_decode_workspace_size(32, 8, 64, 4096, wf.wf_pool_desc(4096, P, 8, 128, NUMBER[pool], 1.0, 1.0))
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    for B, drafts in ((32, 16), (9, 40), (1, 4), (32, 8)):
        t = R.Tree([60] * B, [drafts] * B, 8, 8, 128, P, pool, seed=B + drafts, **fp8)
        t.max_len = 4096
        d = t.device()
        d["table"] = torch.cat([d["table"], torch.full((B, -(-4096 // P) - t.table.shape[1]), -1, dtype=torch.int32,
                                                       device="cuda")], 1)
        R.check(t, t.run(d, ws))
        assert wf.wf_device_status_fetch(d["status"]) == 0

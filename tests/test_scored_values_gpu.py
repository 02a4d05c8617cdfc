"""wf_paged_scored_attention over V rows that are not finite."""
import numpy as np
import pytest
import torch

from paged_kv_cache_wf_gb300 import binding as wf
from tests import _draft as R
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


# cached, new, H_q, H_kv, D, P: few rows a request (one to eight), and more
SEEN = {"decode": ([700, 130, 257], [1, 1, 1], 8, 2, 128, 16), "decode d64": ([700, 130, 257], [1, 1, 1], 4, 4, 64, 16),
        "decode group of 8": ([4000, 17], [1, 1], 16, 2, 128, 32), "few": ([600, 300], [8, 5], 8, 2, 128, 16),
        "one tile": ([600, 300], [20, 9], 8, 2, 128, 16), "two tiles": ([600, 300], [70, 40], 8, 2, 64, 16),
        "blocks of 7": ([300, 100], [1, 4], 8, 2, 128, 7)}
SEEN_RULES = {"plain": dict(), "cap": dict(cap=5.0), "window": dict(window=200), "documents": dict(view="documents"),
              "any": dict(view="any", cap=5.0)}


@pytest.mark.parametrize("rule", list(SEEN_RULES))
@pytest.mark.parametrize("shape", list(SEEN))
def test_an_infinity_that_a_row_sees_makes_it_infinite(shape, rule):
    """Whatever its weight, and whether all rows of a block see it or some: one of either sign in two columns, both signs
    in a third, in the middle of the context."""
    t = Scored(*SEEN[shape], "bf16", seed=7, **SEEN_RULES[rule])
    clean = t.device()
    t.run(clean, t.workspace())
    d = t.device()
    G = t.H_q // t.H_kv
    want = clean["out"].double().cpu().numpy()
    for b in range(t.B):
        at = int(t.lens[b]) - int(t.drafted[b])
        for p, col, value in ((at // 2, 3, np.inf), (max(at - 70, 0), 33, -np.inf), (at // 3, 40, np.inf), (at - 1, 40, -np.inf)):
            if not t.seen(b)[p]:
                continue
            d["v"][int(t.table[b, p // t.P]), p % t.P, t.H_kv - 1, col] = float(value)
            for i in range(int(t.drafted[b])):
                lo, hi = t.range(b, i)
                if lo <= p < hi:
                    with np.errstate(invalid="ignore"):
                        want[t.cu[b] + i, t.H_q - G:, col] += value
    t.run(d, t.workspace())
    assert wf.wf_device_status_fetch(d["status"]) == 0
    assert np.array_equal(d["out"].double().cpu().numpy(), want, equal_nan=True)
    assert np.isinf(want).any() or rule == "any"        # (single tokens see nothing in this view)


@pytest.mark.parametrize("rule", ["plain", "cap", "window"])
@pytest.mark.parametrize("shape", ["decode", "decode d64", "few", "one tile", "two tiles", "blocks of 7"])
def test_values_at_the_end_of_their_range(shape, rule):
    """Normal values times 2^90 and scores far apart: sums over 700 positions stay below 2^104."""
    t = Scored(*SEEN[shape], "bf16", seed=8, q_size=8.0, **SEEN_RULES[rule])
    t.v *= 2.0 ** 90
    t.v[torch.isnan(t.v)] = 0                            # (rows that nobody sees)
    assert float(t.v.abs().max()) < 2.0 ** 94
    d = t.device()
    t.run(d, t.workspace())
    R.check(t, d["out"])
    assert wf.wf_device_status_fetch(d["status"]) == 0

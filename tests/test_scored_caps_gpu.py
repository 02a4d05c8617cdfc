"""wf_paged_scored_attention with caps far above the scores: a capped score is off by a part of itself, not of its cap."""
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
SHAPES = {
    "decode": ([1, 130, 127, 5, 260, 0], [1] * 6, 8, 2, 128, 16, "bf16"),
    "few": ([200, 90, 0], [5, 31, 9], 8, 2, 128, 16, "bf16"),
    "prompts": ([150, 0, 301], [133, 270, 64], 8, 2, 128, 16, "bf16"),
    "prompts d64": ([0, 40], [400, 90], 4, 4, 64, 16, "bf16"),
    "fp8 decode": ([64, 300, 1, 127], [1, 1, 1, 1], 8, 2, 128, 16, "fp8"),
    "fp8 prompts": ([64, 0], [140, 33], 8, 2, 128, 32, "fp8"),
    "decode d64": ([1, 130, 127, 260], [1] * 4, 4, 4, 64, 16, "bf16"),
    "few d64": ([30, 0, 20], [4, 16, 6], 10, 2, 64, 48, "bf16"),
    "fp8 decode d64": ([64, 300, 1, 127], [1, 1, 1, 1], 8, 2, 64, 16, "fp8"),
    "fp8 prompts d64": ([64, 0], [140, 33], 6, 2, 64, 16, "fp8"),
    "fp32 prompts": ([64, 0], [70, 101], 4, 2, 64, 16, "f32"),
}


def check(t):
    """A capped score is below its uncapped one, so an error of a part of its row's largest is below that part of `S`, which
    R.Tree's bound multiplies by (D + 4) 2^-24.  The polynomial: 2^-17.2 of a score and six roundings of 2^-24 at most, below
    2^-17 of it.  The other form, 2^-20 of the cap: for caps above 256 only of scores above 0.36 of it, so below 2^-18 of
    one.  tanhf: 2^-21 of a score."""
    out, W, _ = t.reference()
    cap, t.cap = t.cap, 0.0
    _, _, S = t.reference()
    t.cap, unit = cap, (t.D + 4) * 2.0 ** -24
    S = S * (1 + 2.0 ** -17 / unit) + (2.0 ** -20 * cap / unit if cap <= 256 else 0.0)
    d = t.device()
    t.run(d, t.workspace())
    R.check(t, d["out"], (out, W, S))
    assert wf.wf_device_status_fetch(d["status"]) == 0
    return d["out"]


@pytest.mark.parametrize("cap", [50.0, 256.0, 257.0, 1e3, 1e4, 5e4, 1e6, 1e7, 1e12, 1e30])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_a_cap_above_the_scores(shape, cap):
    for seed, rule in enumerate((dict(), dict(window=70), dict(view="any"), dict(slopes=True), dict(slopes=True, view="prefix"))):
        check(Scored(*SHAPES[shape], seed=seed, cap=cap, q_size=6.0, **rule, **(FP8 if "fp8" in shape else {})))


@pytest.mark.parametrize("shape", list(SHAPES))
def test_a_negative_scale_and_rows_of_other_sizes(shape):
    """Scores beyond the cap's line beside rows of scores a thousand times smaller, which stay as exact as alone."""
    for scale in (0.09, -0.09):
        t = Scored(*SHAPES[shape], seed=5, cap=4e3, q_size=4.0, **(FP8 if "fp8" in shape else {}))
        t.scale = scale
        t.q[::2] *= 512.0
        check(t)


def test_the_largest_cap_and_no_scale():
    for shape in SHAPES:
        t = Scored(*SHAPES[shape], seed=6, cap=2.0 ** 100, **(FP8 if "fp8" in shape else {}))
        check(t)
        t.scale = 0.0
        check(t)

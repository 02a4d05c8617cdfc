"""The kernels' bounded waits, by themselves: a wait that runs out ends, and ends alike in all lanes of a warp."""
import ctypes
import os
import subprocess

import pytest
import torch

from paged_kv_cache_wf_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    so = str(tmp_path_factory.mktemp("waits") / "waits.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_waits.cu")
    subprocess.run([build._nvcc(), *build._flags(), "-I", build.CSRC, "-shared", "-cudart", "static", "-o", so, src],
                   check=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("split", [0, 1, 16, 31, 32])
def test_a_warp_gives_up_together(waits, split):
    out = torch.full((32,), -1, dtype=torch.int32, device="cuda")
    assert waits.part_ways(split, ctypes.c_void_p(out.data_ptr())) == 0
    torch.cuda.synchronize()
    assert out.tolist() == [1 if split == 32 else 0] * 32


@pytest.mark.parametrize("slots", [1, 2, 5, 6])
@pytest.mark.parametrize("uses", [0, 1, 2, 3, 4, 6, 7, 11, 12, 13])
def test_a_drain_waits_for_the_last_phases(waits, slots, uses):
    out = torch.full((32,), -1, dtype=torch.int32, device="cuda")
    for missing in range(min(uses, slots) + 1):
        assert waits.drain(slots, uses, missing, ctypes.c_void_p(out.data_ptr())) == 0
        torch.cuda.synchronize()
        assert out.tolist() == [1 if missing == 0 else 0] * 32

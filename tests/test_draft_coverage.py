"""The GPU cases of the tree attention reach every instance of its kernels (checked without a GPU)."""
from paged_kv_cache_wf_gb300 import binding as wf
from paged_kv_cache_wf_gb300 import build
from tests import test_tree_gpu as gpu_cases


def instance(t):
    """(kernel, pool, D, form): query tiles of the tensor-core kernel, rows of a warp of the other."""
    group = t.H_q // t.H_kv
    if t.kernel() == wf.WF_KERNEL_TENSOR_CORES:
        return "tensor cores", t.pool, t.D, 1 if t.pool == "fp8" or t.max_q <= 128 // group else 2
    rows = t.max_q * group
    return "CUDA cores", t.pool, t.D, 1 if rows <= 8 else 2 if rows <= 16 else 4


def test_every_instance_meets_the_softmax():
    build.build()
    met = {instance(make()) for make in gpu_cases.CASES.values()}
    want = {("tensor cores", "bf16", D, tiles) for D in (64, 128) for tiles in (1, 2)}
    want |= {("tensor cores", "fp8", D, 1) for D in (64, 128)}
    want |= {("CUDA cores", pool, D, rows) for pool in ("f32", "bf16", "fp8") for D in (64, 128) for rows in (1, 2, 4)}
    assert met == want, (sorted(want - met), sorted(met - want))

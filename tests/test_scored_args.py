"""CPU checks of scored attention: what it refuses before any launch, its workspace, and that its cases meet every kernel."""
import math

import pytest
import torch

from paged_kv_cache_wf_gb300 import binding as wf
from paged_kv_cache_wf_gb300 import build
from tests import test_scored_gpu as gpu_cases

FAKE = 0x10000   # 16-byte aligned, never dereferenced by calls that are refused


@pytest.fixture(scope="module")
def lib():
    build.build()
    return wf.load()


def _desc(N=10, P=16, H=2, D=64, dt=wf.WF_DTYPE_BF16, ks=0.0, vs=0.0):
    return wf.wf_pool_desc(N, P, H, D, dt, ks, vs)


def test_refusals(lib):
    f = lib.wf_paged_scored_attention
    d = _desc()
    need = wf.wf_paged_scored_attention_workspace_size(2, 8, 10, 7, 64, d)
    ok = dict(out=FAKE + (1 << 30), q=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, M=4, sl=FAKE, cu=FAKE, B=2, T=10, mq=7, msl=64, Hq=8,
              scale=0.1, cap=0.0, window=0, slopes=None, ranges=None, d=d, ws=FAKE, wsb=need)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["out"], a["q"], a["kp"], a["vp"], a["bt"], a["M"], a["sl"], a["cu"], a["B"], a["T"], a["mq"], a["msl"],
                 a["Hq"], a["scale"], a["cap"], a["window"], a["slopes"], a["ranges"], a["d"], a["ws"], a["wsb"], None, None)

    for none in (dict(B=0), dict(T=0), dict(mq=0)):
        assert call(**none) == wf.WF_OK
    for bad in (dict(B=-1), dict(T=-1), dict(mq=-1), dict(msl=-1), dict(Hq=0), dict(Hq=7), dict(M=0), dict(msl=65),
                dict(mq=65), dict(scale=math.inf), dict(scale=math.nan), dict(scale=3.0e38), dict(cap=-1.0), dict(cap=math.nan),
                dict(cap=math.inf), dict(cap=3.0e38), dict(cap=1e-38, scale=1e6), dict(window=-1), dict(out=None), dict(q=None),
                dict(kp=None), dict(vp=None), dict(bt=None), dict(sl=None), dict(cu=None), dict(out=FAKE + (1 << 30) + 8),
                dict(q=FAKE + 2), dict(kp=FAKE + 4), dict(vp=FAKE + 8), dict(bt=FAKE + 2), dict(sl=FAKE + 1), dict(cu=FAKE + 2),
                dict(slopes=FAKE + 2), dict(ranges=FAKE + 4), dict(out=FAKE), dict(out=FAKE + 10 * 8 * 64 * 2 - 16),
                dict(msl=2 ** 31 - 1024, M=2 ** 27)):
        assert call(**bad) == wf.WF_ERR_INVALID_ARG, bad
    assert call(Hq=18) == wf.WF_ERR_UNSUPPORTED          # G = 9
    assert call(d=_desc(D=80)) == wf.WF_ERR_UNSUPPORTED
    for bad in (dict(ws=None), dict(ws=FAKE + 8), dict(wsb=need - 1), dict(wsb=0)):
        assert call(**bad) == wf.WF_ERR_WORKSPACE, bad


def test_larger_calls_never_need_less_workspace(lib):
    for d in (_desc(), _desc(D=128, dt=wf.WF_DTYPE_FP8_E4M3, ks=1.0, vs=1.0), _desc(dt=wf.WF_DTYPE_F32), _desc(P=7)):
        for heads in (2, 6, 16):
            sizes = [1, 2, 3, 7, 15, 16, 17, 32, 33, 64, 65, 100, 128, 129, 200, 1000, 4096]
            size = lambda B, T, q, n: wf.wf_paged_scored_attention_workspace_size(B, heads, T, q, n, d)   # noqa: E731
            for kind in (lambda x: size(x, 5000, 64, 8192), lambda x: size(9, x, 4096, 8192), lambda x: size(9, 9000, x, 8192),
                         lambda x: size(9, 9000, 64, x)):
                got = [kind(x) for x in sizes]
                assert all(got) and got == sorted(got), (heads, got)
    assert wf.wf_paged_scored_attention_workspace_size(-1, 8, 1, 1, 1, _desc()) == 0
    assert wf.wf_paged_scored_attention_workspace_size(1, 7, 1, 1, 1, _desc()) == 0


def test_tensors_of_other_types_or_shapes_are_refused(lib):
    i = lambda *n: torch.zeros(n, dtype=torch.int32)   # noqa: E731
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16)   # noqa: E731
    ok = dict(out=bf(6, 8, 64), q=bf(6, 8, 64), k_pool=bf(5, 16, 2, 64), v_pool=bf(5, 16, 2, 64), block_tables=i(2, 4),
              seq_lens=i(2), cu_q_lens=i(3), max_q_len=3, max_seq_len=64, scale=0.1, workspace=torch.zeros(64, dtype=torch.uint8))
    for bad in (dict(out=bf(5, 8, 64)), dict(q=torch.zeros(6, 8, 64)), dict(q=bf(6, 8, 128)), dict(v_pool=bf(5, 16, 4, 64)),
                dict(v_pool=torch.zeros(5, 16, 2, 64)), dict(seq_lens=i(3)), dict(cu_q_lens=i(2)), dict(slopes=torch.zeros(7)),
                dict(slopes=torch.zeros(8).double()), dict(row_ranges=i(6)), dict(row_ranges=i(5, 2)),
                dict(row_ranges=torch.zeros(6, 2)), dict(block_tables=i(4, 2).t())):
        with pytest.raises(ValueError):
            wf.wf_paged_scored_attention(**dict(ok, **bad))


def instance(shape):
    """(kernel, pool, D, form) of a case: query tiles of the tensor-core kernel, rows of a warp of the other."""
    cached, new, H_q, H_kv, D, P, pool = shape
    d = _desc(1000, P, H_kv, D, {"f32": 0, "bf16": 1, "fp8": 2}[pool], 1.0, 1.0)
    group = H_q // H_kv
    if wf.wf_paged_tree_decode_kernel(d, H_q) == wf.WF_KERNEL_TENSOR_CORES:
        return "tensor cores", pool, D, 1 if pool == "fp8" or max(new) <= 128 // group else 2
    rows = max(new) * group
    return "CUDA cores", pool, D, 1 if rows <= 8 else 2 if rows <= 16 else 4


def test_every_instance_meets_the_softmax(lib):
    met = {instance(s) for s in gpu_cases.SHAPES.values()}
    want = {("tensor cores", "bf16", D, tiles) for D in (64, 128) for tiles in (1, 2)}
    want |= {("tensor cores", "fp8", D, 1) for D in (64, 128)}
    want |= {("CUDA cores", pool, D, rows) for pool in ("f32", "bf16", "fp8") for D in (64, 128) for rows in (1, 2, 4)}
    assert met == want, (sorted(want - met), sorted(met - want))

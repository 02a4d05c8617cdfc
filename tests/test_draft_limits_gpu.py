"""The draft-verification calls at the ends of their ranges: pools past 32 bits of offset, a scale a
KV head, workspaces and graphs shared one after another, the first call of a process captured."""
import subprocess
import sys

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


@pytest.mark.parametrize("pool,H_kv,D,P", [("bf16", 8, 128, 16), ("bf16", 8, 64, 7), ("f32", 12, 64, 16), ("fp8", 8, 128, 16)])
def test_blocks_past_32_bits_of_elements(pool, H_kv, D, P):
    """The same calls on a small pool and on the last blocks of one with more than 2^32 elements: the same bytes."""
    r = np.random.default_rng(70)
    B, n, per = 3, 5, -(-40 // P)
    small = B * per
    big = (1 << 32) // (P * H_kv * D) + 2 * small
    shift = big - small
    fp8 = dict(k_scale=1 / 64, v_scale=1 / 64) if pool == "fp8" else {}
    pools = [R.to_pool(r.standard_normal((small, P, H_kv, D)), pool).cuda() for _ in range(2)]
    wide = [torch.empty((big, P, H_kv, D), dtype=R.DT[pool], device="cuda") for _ in range(2)]
    for w, s in zip(wide, pools):
        w[shift:] = s
    dt = R.act(pool)
    x = torch.from_numpy(r.standard_normal((B * n, 3 * H_kv, D))).float().to(dt).cuda()
    q, k, v = x.split([H_kv] * 3, 1)
    table = torch.arange(small, dtype=torch.int32, device="cuda").view(B, per)
    lens = torch.full((B,), 31 + n, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    pos = torch.arange(31, 31 + n, dtype=torch.int64, device="cuda")
    slots = (table.long()[:, pos // P] * P + pos % P).view(-1)
    mask = torch.full((B * n, 1), 0b10111, dtype=torch.int32, device="cuda")
    path = torch.tensor([[0, 2, 4]] * B, dtype=torch.int32, device="cuda")
    count = torch.tensor([3, 2, 1], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(wf.wf_paged_tree_decode_workspace_size(B, H_kv, n, 40, wf.pool_desc(pools[0], **fp8)),
                     dtype=torch.uint8, device="cuda")
    outs = []
    for (kp, vp), off in ((pools, 0), (wide, shift)):
        qr, out = torch.zeros_like(q, memory_format=torch.contiguous_format), torch.zeros(B * n, H_kv, D, dtype=dt, device="cuda")
        wf.wf_qk_norm_rope_and_cache(qr, q, k, v, None, None, 1e-6, None, None, kp, vp, slots + off * P, dev_status=status, **fp8)
        wf.wf_paged_tree_decode(out, qr, kp, vp, table + off, lens, cu, mask, n, 40, 0.1, ws, dev_status=status, **fp8)
        wf.wf_keep_accepted(kp, vp, table + off, lens, cu, path, count, dev_status=status)
        outs.append(out)
    assert wf.wf_device_status_fetch(status) == 0
    assert torch.equal(*outs) and float(outs[0].abs().sum()) > 0
    for s, w in zip(pools, wide):
        assert torch.equal(s.view(torch.uint8), w[shift:].view(torch.uint8))


@pytest.mark.parametrize("D,P", [(128, 16), (64, 32), (64, 7)])
def test_a_scale_a_head(D, P):
    t = R.Tree([100, 0, 300], [9, 20, 33], 12, 3, D, P, "fp8", seed=71)
    t.ks, t.vs = np.array([[1 / 64], [1 / 16], [1 / 100]]), np.array([[1 / 96], [1 / 8], [1 / 33]])
    # as the call takes them: fp32
    t.ks, t.vs = t.ks.astype(np.float32).astype(np.float64), t.vs.astype(np.float32).astype(np.float64)
    d = t.device()
    R.check(t, t.run(d, t.workspace()))


@pytest.mark.parametrize("pool", ["bf16", "fp8", "f32"])
def test_two_graphs_share_a_workspace(pool):
    """Replayed one after the other on one stream, in any order, each gives the bytes of its own call."""
    fp8 = dict(k_scale=1 / 64, v_scale=1 / 64) if pool == "fp8" else {}
    a = R.Tree([900, 40, 300], [9, 12, 5], 8, 2, 64, 16, pool, seed=72, **fp8)
    b = R.Tree([20, 1500], [30, 3], 8, 2, 64, 16, pool, seed=73, **fp8)
    both = []
    wa, wb = a.workspace(), b.workspace()
    ws = wa if wa.numel() >= wb.numel() else wb
    for t in (a, b):
        d = t.device()
        first = t.run(d, ws).clone()
        R.check(t, first)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            t.run(d, ws)
        both.append((g, d, first))
    for i in (0, 1, 1, 0, 0, 1):
        g, d, first = both[i]
        d["out"].fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        n = int((a, b)[i].cu[-1])
        assert torch.equal(d["out"][:n], first[:n])


FIRST = """
import torch, numpy as np
from tests import _draft as R
t = R.Tree([100, 0, 300], [9, 20, 5], 8, 2, 64, 16, "%s", seed=74%s)
d, ws = t.device(), t.workspace()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    t.run(d, ws)
g.replay()
torch.cuda.synchronize()
R.check(t, d["out"])
"""


@pytest.mark.parametrize("pool", ["bf16", "fp8", "f32"])
def test_the_first_call_of_a_process_is_captured(pool):
    r = subprocess.run([sys.executable, "-c", FIRST % (pool, ", k_scale=1/64, v_scale=1/64" if pool == "fp8" else "")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("pool,D", [("bf16", 128), ("bf16", 64), ("fp8", 64)])
def test_beside_a_prefill_and_a_decode(pool, D):
    """Tree attention on one stream while prefills and decodes, tensor memory users too, run on two others."""
    fp8 = dict(k_scale=1 / 64, v_scale=1 / 64) if pool == "fp8" else {}
    r = np.random.default_rng(82)
    t = R.Tree(r.integers(100, 900, 24), r.integers(1, 13, 24), 8, 2, D, 16, pool, seed=83, **fp8)
    o = R.Tree([700, 0, 300, 90], [100, 64, 7, 200], 8, 2, D, 16, "bf16", seed=84)
    d, ws, e = t.device(), t.workspace(), o.device()
    q1 = e["q"][:4].contiguous()
    wsd = torch.empty(max(1, wf.wf_paged_decode_workspace_size(4, 8, o.max_len, wf.pool_desc(e["k"]))), dtype=torch.uint8,
                      device="cuda")
    dec = torch.zeros_like(q1)

    def prefill(stream=None):
        wf.wf_paged_prefill(e["out"], e["q"], e["k"], e["v"], e["table"], e["lens"], e["cu"], o.max_q, o.max_len, o.scale,
                            e["status"], stream=stream)

    def decode(stream=None):
        wf.wf_paged_decode(dec, q1, e["k"], e["v"], e["table"], e["lens"], o.max_len, o.scale, wsd, e["status"],
                           stream=stream)

    prefill()
    decode()
    first = t.run(d, ws).clone(), e["out"].clone(), dec.clone()
    torch.cuda.synchronize()
    a, b, c = (torch.cuda.Stream() for _ in range(3))
    for _ in range(20):
        t.run(d, ws, stream=a)
        prefill(b)
        decode(c)
    torch.cuda.synchronize()
    for x, y in zip(first, (d["out"], e["out"], dec)):
        assert torch.equal(x, y)
    assert wf.wf_device_status_fetch(d["status"]) == wf.wf_device_status_fetch(e["status"]) == 0

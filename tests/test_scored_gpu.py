"""wf_paged_scored_attention against the softmax in 64 bits."""
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
# cached, new, H_q, H_kv, D, P, pool: every instance of the kernels
SHAPES = {
    # bf16, blocks of 16: the tensor cores, up to 128 rows a block and more
    "one token": ([700], [1], 8, 2, 128, 16, "bf16"),
    "first token": ([0], [1], 8, 2, 64, 16, "bf16"),
    "decode": ([1, 130, 127, 5, 260, 0], [1] * 6, 8, 2, 128, 16, "bf16"),
    "decode d64 mha": ([1, 130, 127, 5, 260, 0], [1] * 6, 3, 3, 64, 32, "bf16"),
    "decode group of 8": ([300, 17, 128], [1, 1, 1], 16, 2, 128, 16, "bf16"),
    "few": ([200, 90, 0], [5, 31, 9], 8, 2, 128, 16, "bf16"),
    "few d64": ([30, 0, 20, 7, 0], [0, 0, 4, 16, 6], 10, 2, 64, 48, "bf16"),
    "prompts": ([150, 0, 301], [133, 270, 64], 8, 2, 128, 16, "bf16"),
    "prompts d64": ([0, 40], [400, 90], 4, 4, 64, 16, "bf16"),
    "prompts group of 7": ([33, 0, 5], [90, 1, 41], 7, 1, 128, 64, "bf16"),
    "mixed": ([600, 3, 200, 77], [1, 150, 1, 6], 8, 2, 64, 16, "bf16"),
    # fp8
    "fp8 decode": ([64, 300, 1, 127], [1, 1, 1, 1], 8, 2, 128, 16, "fp8"),
    "fp8 decode d64": ([64, 300, 1, 127], [1, 1, 1, 1], 8, 2, 64, 16, "fp8"),
    "fp8 prompts": ([64, 0], [140, 33], 8, 2, 128, 32, "fp8"),
    "fp8 prompts d64": ([64, 0], [140, 33], 6, 2, 64, 16, "fp8"),
    # the CUDA cores: 1, 2 and 4 rows a warp
    "fp32": ([64, 300, 1], [1, 1, 1], 12, 12, 64, 16, "f32"),
    "fp32 16 rows": ([64, 130, 0], [5, 1, 7], 4, 2, 64, 16, "f32"),
    "fp32 prompts": ([64, 0], [70, 101], 4, 2, 64, 16, "f32"),
    "fp32 d128": ([64, 130], [2, 1], 8, 2, 128, 5, "f32"),
    "fp32 d128 16 rows": ([64, 130], [4, 1], 8, 2, 128, 16, "f32"),
    "fp32 d128 prompts": ([64, 0], [20, 75], 8, 2, 128, 16, "f32"),
    "blocks of 7": ([77, 200], [1, 2], 8, 2, 128, 7, "bf16"),
    "blocks of 7, 16 rows": ([77, 200], [4, 3], 8, 2, 128, 7, "bf16"),
    "blocks of 7, prompts": ([77, 0], [40, 91], 8, 2, 128, 7, "bf16"),
    "blocks of 1 d64": ([20, 3], [1, 2], 4, 2, 64, 1, "bf16"),
    "blocks of 9 d64, 16 rows": ([64, 130], [5, 3], 6, 2, 64, 9, "bf16"),
    "blocks of 24 d64, prompts": ([64, 130], [33, 70], 4, 2, 64, 24, "bf16"),
    "fp8 blocks of 7": ([64, 130], [1, 2], 8, 2, 64, 7, "fp8"),
    "fp8 blocks of 7, 16 rows": ([64, 130], [4, 2], 8, 2, 64, 7, "fp8"),
    "fp8 blocks of 7, prompts": ([64, 30], [7, 60], 8, 2, 64, 7, "fp8"),
    "fp8 blocks of 9 d128": ([64, 130], [1, 2], 8, 2, 128, 9, "fp8"),
    "fp8 blocks of 9 d128, 16 rows": ([64, 130], [4, 2], 8, 2, 128, 9, "fp8"),
    "fp8 blocks of 9 d128, prompts": ([64, 0], [13, 50], 8, 2, 128, 9, "fp8"),
}
RULES = {
    "causal": dict(),
    "window": dict(window=50),
    "window of one": dict(window=1, view="prefix"),
    "documents": dict(view="documents"),
    "any": dict(view="any"),
    "slopes": dict(slopes=True),
    "slopes, prefix": dict(slopes=True, view="prefix"),
    "cap": dict(cap=3.0),
    "cap, any": dict(cap=30.0, view="any", q_size=12.0),
    "all": dict(cap=5.0, slopes=True, window=130, view="documents"),
    "all, ahead": dict(cap=5.0, slopes=True, view="any"),
}


def make(shape, rule, seed=0, **kw):
    pool = SHAPES[shape][-1]
    return Scored(*SHAPES[shape], seed=seed, **{**(FP8 if pool == "fp8" else {}), **RULES[rule], **kw})


def check(t, d, bit=0):
    R.check(t, d["out"])
    assert wf.wf_device_status_fetch(d["status"]) == bit
    assert (d["out"][int(t.cu[-1]):] == 7.0).all()      # rows behind the last request are left as they were


@pytest.mark.parametrize("rule", list(RULES))
@pytest.mark.parametrize("shape", list(SHAPES))
def test_against_the_softmax(shape, rule):
    t = make(shape, rule, seed=len(shape) + 31 * len(rule), extra_rows=3)
    d = t.device()
    t.run(d, t.workspace())
    check(t, d)


@pytest.mark.parametrize("shape", ["decode", "few", "prompts", "fp8 prompts", "fp32 prompts", "blocks of 7"])
def test_rows_that_see_nothing_give_zeros(shape):
    t = make(shape, "causal", view="empty")
    d = t.device()
    t.run(d, t.workspace())
    assert (d["out"] == 0).all() and wf.wf_device_status_fetch(d["status"]) == 0


def test_a_negative_scale_and_a_scale_of_zero():
    for shape in ("decode", "prompts", "fp8 decode", "fp32 prompts"):
        for rule in ("window", "cap", "slopes"):
            for scale in (-0.11, 0.0):
                t = make(shape, rule, seed=4)
                t.scale = scale
                d = t.device()
                t.run(d, t.workspace())
                check(t, d)


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("shape", ["decode", "few", "prompts", "prompts d64", "fp8 prompts", "fp8 prompts d64", "fp32 prompts",
                                   "blocks of 7, prompts"])
def test_what_a_row_does_not_see_does_not_reach_it(shape, value):
    """K and V elements that are no numbers: rows that see them are not finite there, the others as if they were 0."""
    if SHAPES[shape][-1] == "fp8" and not np.isnan(value):
        pytest.skip("e4m3 has no infinities")
    rules = dict(view="any", cap=20.0) if len(SHAPES[shape][0]) % 2 else dict(view="documents", slopes=True)
    t = Scored(*SHAPES[shape], seed=5, **(FP8 if SHAPES[shape][-1] == "fp8" else {}), **rules)
    r = np.random.default_rng(1)
    code = 0x7F if t.pool == "fp8" else float(value)
    wild_v, wild_k = {}, {}
    for b in range(t.B):
        places = np.nonzero(t.seen(b))[0]
        if len(places):
            wild_v[b] = sorted({int(r.choice(places)), int(places[0])})
    clean = t.device()
    ref = t.reference()
    t.run(clean, t.workspace())
    R.check(t, clean["out"], ref)
    for b, where in wild_v.items():
        for p in where:
            t.v[int(t.table[b, p // t.P]), p % t.P, :, 3] = code
    d = t.device()
    t.run(d, t.workspace())
    got, plain = d["out"].double().cpu().numpy(), clean["out"].double().cpu().numpy()
    for b in range(t.B):
        for i in range(int(t.drafted[b])):
            lo, hi = t.range(b, i)
            row = t.cu[b] + i
            hit = any(lo <= p < hi for p in wild_v.get(b, ()))
            assert np.isfinite(np.delete(got[row], 3, -1)).all(), (b, i)
            if not hit:
                assert np.array_equal(got[row], plain[row]), (b, i)
            elif np.isnan(value):
                assert np.isnan(got[row][:, 3]).all(), (b, i)
            else:
                assert (got[row][:, 3] == value).all() or np.isnan(got[row][:, 3]).any(), (b, i)
    # the same of K: rows that see it are NaN, the others finite
    t2 = Scored(*SHAPES[shape], seed=5, **(FP8 if t.pool == "fp8" else {}), **rules)
    for b, where in wild_v.items():
        t2.k[int(t2.table[b, where[0] // t2.P]), where[0] % t2.P] = 0x7F if t2.pool == "fp8" else np.nan
    d = t2.device()
    t2.run(d, t2.workspace())
    got = d["out"].double().cpu().numpy()
    for b in range(t2.B):
        for i in range(int(t2.drafted[b])):
            lo, hi = t2.range(b, i)
            hit = b in wild_v and lo <= wild_v[b][0] < hi
            assert np.isnan(got[t2.cu[b] + i]).all() == hit or not hit, (b, i)
            if not hit:
                assert np.array_equal(got[t2.cu[b] + i], plain[t2.cu[b] + i]), (b, i)


def test_bad_requests_and_blocks():
    for shape in ("decode", "prompts", "fp32 prompts", "fp8 prompts"):
        t = make(shape, "cap", seed=6)
        bad = {(0, 1)} if int(t.lens[0]) > 2 * t.P else {(1, 1)}
        (b, j), = bad
        t.table[b, j] = t.N
        d = t.device()
        t.run(d, t.workspace())
        got, (ref, W, S) = d["out"].double().cpu().numpy(), t.reference(bad_blocks=bad)
        assert (np.abs(got - ref) <= t.bound(ref, W, S)).all()
        assert wf.wf_device_status_fetch(d["status"]) == wf.WF_DEV_BAD_BLOCK
        # a length past the table, or below the request's rows: skipped, its rows left as they were
        for length in (t.max_len + 1, int(t.drafted[-1]) - 1, -4):
            t = make(shape, "window", seed=7)
            d = t.device()
            d["lens"][-1] = length
            t.run(d, t.workspace())
            got = d["out"].double().cpu().numpy()
            ref, W, S = t.reference()
            n = int(t.cu[-2])
            assert (np.abs(got[:n] - ref[:n]) <= t.bound(ref, W, S)[:n]).all() and (got[n:] == 7.0).all()
            assert wf.wf_device_status_fetch(d["status"]) == wf.WF_DEV_BAD_SEQLEN


def test_offsets_out_of_order():
    """Requests whose offsets go backwards or past the rows are skipped; rows named twice are never more than there is room
    for."""
    t = make("prompts", "cap", seed=8)
    d = t.device()
    d["cu"][1] = 2 ** 30
    t.run(d, t.workspace())
    assert wf.wf_device_status_fetch(d["status"]) == wf.WF_DEV_BAD_SEQLEN
    assert (d["out"][:int(t.cu[2])] == 7.0).all() and torch.isfinite(d["out"].float()).all()
    t = Scored([0] * 40, [1] * 40, 8, 2, 128, 16, "bf16", seed=9)
    d = t.device()
    d["cu"].copy_(torch.tensor([0, 40] * 20 + [0], dtype=torch.int32))
    d["lens"].fill_(1)
    t.run(d, t.workspace())
    assert wf.wf_device_status_fetch(d["status"]) & wf.WF_DEV_BAD_SEQLEN


def test_as_decode_and_prefill():
    t = make("decode", "causal", seed=10)
    d = t.device()
    t.run(d, t.workspace())
    out = torch.empty_like(d["q"])
    ws = torch.empty(wf.wf_paged_decode_workspace_size(t.B, t.H_q, t.max_len, t.desc()), dtype=torch.uint8, device="cuda")
    wf.wf_paged_decode(out, d["q"], d["k"], d["v"], d["table"].clamp(0, t.N - 1), d["lens"], t.max_len, t.scale, ws)
    R.check(t, out)
    R.check(t, d["out"])
    t = make("prompts", "causal", seed=11)
    d = t.device()
    t.run(d, t.workspace())
    out = torch.empty_like(d["q"])
    wf.wf_paged_prefill(out, d["q"], d["k"], d["v"], d["table"], d["lens"], d["cu"], t.max_q, t.max_len, t.scale)
    R.check(t, out)
    R.check(t, d["out"])


@pytest.mark.parametrize("shape, rule", [("decode", "cap"), ("prompts", "all"), ("fp8 prompts", "cap"), ("fp32 prompts", "slopes"),
                                         ("mixed", "documents")])
def test_the_largest_limits_and_repeated_calls(shape, rule):
    """The same bytes from the same call; larger limits, a longer table and a larger workspace change nothing but rounding."""
    t = make(shape, rule, seed=12)
    d = t.device()
    ws = t.workspace()
    first = t.run(d, ws).clone()
    d["out"].fill_(7.0)
    assert torch.equal(t.run(d, ws), first)
    t.table = np.concatenate([t.table, np.full((t.B, 9), -1, np.int32)], 1)
    t.max_len = t.table.shape[1] * t.P
    t.max_q = min(t.max_len, 700)
    d = t.device()
    t.run(d, t.workspace())
    check(t, d)


def test_many_requests():
    """More requests than the list keeps in shared memory, some without rows."""
    n = 2500
    t = Scored(np.arange(n) * 7 % 150, (np.arange(n) % 5 != 3).astype(int), 4, 1, 64, 16, "bf16", seed=13, cap=4.0, window=33)
    d = t.device()
    t.run(d, t.workspace())
    check(t, d)
    t = Scored(np.arange(n) * 7 % 40, np.arange(n) % 4, 2, 2, 64, 16, "bf16", seed=14, view="any", slopes=True)
    d = t.device()
    t.run(d, t.workspace())
    check(t, d)


def test_rows_of_many_ranges():
    """Enough rows that a cluster looks at their ranges."""
    for view in ("documents", "prefix", "any"):
        t = Scored([0, 100, 3], [1500, 701, 64], 2, 2, 64, 16, "bf16", seed=15, view=view, window=300)
        d = t.device()
        t.run(d, t.workspace())
        check(t, d)


def test_long_contexts():
    for rule in (dict(slopes=True), dict(cap=9.0), dict(window=777)):
        t = Scored([9000, 2], [3, 1], 4, 1, 128, 16, "bf16", seed=16, **rule)
        d = t.device()
        t.run(d, t.workspace())
        check(t, d)


def test_distances_of_far_rows_stay_exact():
    """Rows that see only positions a long way back: a bias of millions, of which only differences matter."""
    n, far = 40, 1 << 17
    t = Scored([0], [n], 4, 4, 64, 16, "f32", seed=17, slopes=True)
    t.slopes[:] = [0.5, 0.25, 1.0, -0.125]
    table = np.full((1, (far + n) // 16 + 1), -1, np.int32)
    for pool in ("f32", "bf16"):
        t = Scored([0], [n], 4, 4, 64, 16, pool, seed=17, slopes=True)
        t.slopes[:] = [0.5, 0.25, 1.0, -0.125]
        near = t.device()
        near["ranges"] = torch.tensor([[0, n]] * n, dtype=torch.int32, device="cuda")
        table[0, :t.table.shape[1]] = t.table[0]
        d = dict(near, table=torch.from_numpy(table).cuda(), lens=torch.tensor([far + n], dtype=torch.int32, device="cuda"))
        t.max_len = far + n
        t.run(d, t.workspace())
        assert wf.wf_device_status_fetch(d["status"]) == 0
        # the reference: every row at the same distance, which is that of position n - 1 and 1 more for each before it
        q, k, v = (x.double().cpu().numpy() for x in (t.q, t.k, t.v))
        blk, off = t.table[0, np.arange(n) // 16], np.arange(n) % 16
        s = np.einsum("nhd,lhd->hnl", q, k[blk, off]) * t.scale + t.slopes.astype(float)[:, None, None] * (np.arange(n) - n + 1)
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        want = np.einsum("hnl,lhd->nhd", w, v[blk, off])
        err = np.abs(d["out"].double().cpu().numpy() - want).max()
        assert err < (1e-5 if pool == "f32" else 0.03), err


def test_pool_rows_past_32_bits_of_offset():
    for pool in ("bf16", "fp8", "f32"):
        t = Scored([50, 20], [3, 20], 8, 2, 128, 16, pool, seed=18, cap=6.0, **(FP8 if pool == "fp8" else {}))
        N = 2 ** 33 // (16 * 2 * 128) + 50 if pool == "fp8" else 2 ** 32 // (16 * 2 * 128) + 50
        d = t.device()
        kp, vp = (torch.empty((N, 16, 2, 128), dtype=d["k"].dtype, device="cuda") for _ in range(2))
        kp[N - t.N:], vp[N - t.N:] = d["k"], d["v"]
        d.update(k=kp, v=vp, table=d["table"] + (N - t.N))
        t.run(d, t.workspace())
        check(t, d)
        del kp, vp, d


@pytest.mark.parametrize("shape", ["decode", "few", "prompts", "fp8 prompts", "fp32 prompts"])
def test_buffers_aligned_to_16_bytes(shape):
    t = make(shape, "all", seed=22)
    d = t.device()
    for name in ("q", "out"):
        x = torch.empty(d[name].numel() + 16 // d[name].element_size(), dtype=d[name].dtype, device="cuda")
        x = x[16 // x.element_size():].view(d[name].shape)
        d[name] = x.copy_(d[name])
    ws = torch.cat([t.workspace(), torch.zeros(16, dtype=torch.uint8, device="cuda")])[16:]
    assert d["out"].data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
    t.run(d, ws)
    check(t, d)


def test_in_a_graph_beside_other_streams():
    """Two captured calls with workspaces of their own, replayed at once on two streams beside an eager one."""
    a, b, c = make("decode", "cap", seed=19), make("prompts", "all", seed=20), make("fp8 prompts", "window", seed=21)
    da, db, dc = a.device(), b.device(), c.device()
    wa, wb, wc = a.workspace(), b.workspace(), c.workspace()
    graphs = []
    for t, d, ws in ((a, da, wa), (b, db, wb)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            t.run(d, ws)
        graphs.append(g)
    side = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
        c.run(dc, wc, stream=side[2])
    torch.cuda.synchronize()
    for t, d in ((a, da), (b, db), (c, dc)):
        check(t, d)

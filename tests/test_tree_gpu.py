"""wf_paged_tree_decode against the softmax in 64 bits."""
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


def T(*a, **kw):
    return lambda: R.Tree(*a, **kw)


FP8 = dict(k_scale=1 / 64, v_scale=1 / 96)
CASES = {
    # bf16, blocks of 16: the tensor-core shapes
    "one request": T([700], [8], 8, 2, 128, 16, "bf16"),
    "one draft, one position": T([0], [1], 8, 2, 128, 16, "bf16"),
    "no context": T([0, 0], [5, 40], 8, 2, 128, 16, "bf16", seed=1),
    "ragged": T([1, 130, 127, 5, 260], [3, 1, 2, 17, 33], 8, 2, 128, 16, "bf16", seed=2),
    "requests without drafts": T([30, 0, 20, 7, 0], [0, 0, 4, 0, 6], 8, 2, 128, 16, "bf16", seed=3),
    "128 rows": T([200, 90], [32, 31], 8, 2, 128, 16, "bf16", seed=4),
    "more than 128 rows": T([150, 301], [33, 64], 8, 2, 128, 16, "bf16", seed=5),
    "several row blocks": T([150, 20], [130, 70], 8, 2, 64, 16, "bf16", seed=6),
    "drafts over several tiles": T([100], [300], 2, 2, 64, 16, "bf16", seed=7),
    "one query head a kv head": T([77, 200], [40, 9], 3, 3, 128, 16, "bf16", seed=8),
    "group of 3": T([77, 200], [11, 44], 6, 2, 64, 16, "bf16", seed=9),
    "group of 5": T([77, 200], [11, 30], 10, 2, 128, 16, "bf16", seed=10),
    "group of 7": T([77, 40], [11, 20], 7, 1, 64, 16, "bf16", seed=11),
    "group of 8": T([77, 200], [11, 40], 16, 2, 128, 16, "bf16", seed=12),
    "blocks of 32": T([77, 200], [11, 40], 8, 2, 128, 32, "bf16", seed=13),
    "blocks of 64": T([77, 200, 513], [11, 40, 3], 8, 2, 64, 64, "bf16", seed=14),
    "blocks of 48": T([77, 200], [11, 40], 8, 2, 128, 48, "bf16", seed=15),
    "any mask": T([0, 40, 0, 3], [33, 20, 7, 70], 4, 2, 128, 16, "bf16", seed=16, density=0.3),
    "almost empty masks": T([0, 0, 5], [33, 20, 40], 4, 2, 64, 16, "bf16", seed=17, density=0.03),
    "empty masks": T([0, 9], [5, 6], 4, 2, 128, 16, "bf16", seed=18, density=0.0),
    "peaked": T([300, 40], [9, 20], 8, 2, 128, 16, "bf16", seed=19, q_size=40.0),
    "spare rows and mask words": T([30, 20], [4, 9], 8, 2, 128, 16, "bf16", seed=20, extra_rows=7, spare_words=3),
    "many requests": T(np.arange(90) * 7 % 150, np.arange(90) % 12, 8, 2, 64, 16, "bf16", seed=21),
    "long": T([6000], [12], 4, 1, 128, 16, "bf16", seed=22),
    # other block sizes: the CUDA cores
    "blocks of 7": T([77, 200], [11, 40], 8, 2, 128, 7, "bf16", seed=23),
    "blocks of 1": T([20, 3], [11, 4], 4, 2, 64, 1, "bf16", seed=24),
    "any mask, blocks of 7": T([0, 40], [33, 20], 4, 2, 128, 7, "bf16", seed=25, density=0.2),
    # fp32
    "fp32": T([64, 300, 1], [7, 1, 5], 12, 12, 64, 16, "f32", seed=26),
    "fp32 d128": T([64, 300, 0], [9, 20, 30], 8, 2, 128, 16, "f32", seed=27),
    "fp32 any mask": T([0, 3], [40, 35], 6, 2, 64, 16, "f32", seed=28, density=0.1),
    "fp32 group of 8, blocks of 5": T([64, 30], [9, 20], 8, 1, 64, 5, "f32", seed=29),
    "fp32 peaked": T([300, 40], [9, 20], 8, 2, 128, 16, "f32", seed=30, q_size=30.0),
    # rows of a warp of the CUDA-core kernel
    "fp32, 8 rows d128": T([64, 300, 1, 0], [4, 1, 2, 3], 8, 4, 128, 16, "f32", seed=52),
    "fp32, 16 rows": T([64, 300, 1, 0], [16, 1, 9, 11], 3, 3, 64, 16, "f32", seed=53),
    "fp32, 16 rows d128 any mask": T([0, 70], [7, 5], 4, 2, 128, 48, "f32", seed=54, density=0.3),
    "blocks of 7, 8 rows": T([64, 300, 1, 0], [2, 1, 2, 1], 8, 2, 64, 7, "bf16", seed=55),
    "blocks of 7, 16 rows": T([64, 130], [5, 3], 6, 2, 128, 7, "bf16", seed=56),
    "fp8 blocks of 7, 8 rows": T([64, 130], [1, 1], 16, 2, 128, 7, "fp8", seed=57, **FP8),
    "fp8 blocks of 7, 16 rows": T([64, 130, 0], [2, 1, 2], 8, 1, 64, 7, "fp8", seed=58, **FP8),
    "blocks of 24, 16 rows": T([64, 130, 3], [5, 8, 2], 8, 4, 64, 24, "bf16", seed=75),
    "blocks of 1000, 8 rows d128": T([1400, 130], [2, 2], 8, 2, 128, 1000, "bf16", seed=76),
    "fp8 blocks of 9, 8 rows": T([64, 130, 0], [3, 8, 1], 3, 3, 64, 9, "fp8", seed=77, **FP8),
    "fp8 blocks of 9, 16 rows d128": T([64, 130, 0], [3, 2, 1], 10, 2, 128, 9, "fp8", seed=78, **FP8),
    "fp8 blocks of 9, d128": T([64, 130, 0], [13, 20, 1], 14, 2, 128, 9, "fp8", seed=79, **FP8),
    # fp8
    "fp8": T([64, 300, 1], [7, 33, 5], 8, 2, 128, 16, "fp8", seed=31, **FP8),
    "fp8 d64": T([64, 300, 0], [7, 70, 30], 8, 2, 64, 16, "fp8", seed=32, **FP8),
    "fp8 llama-3-8b heads": T([500, 17], [24, 8], 32, 8, 128, 16, "fp8", seed=33, **FP8),
    "fp8 any mask": T([0, 30], [40, 70], 4, 2, 128, 16, "fp8", seed=34, density=0.1, **FP8),
    "fp8 blocks of 7": T([64, 30], [7, 20], 8, 2, 64, 7, "fp8", seed=35, **FP8),
    "fp8 one query head": T([164, 30], [70, 140], 2, 2, 128, 32, "fp8", seed=36, **FP8),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_softmax(name):
    t = CASES[name]()
    d = t.device()
    R.check(t, t.run(d, t.workspace()))
    assert wf.wf_device_status_fetch(d["status"]) == 0
    # rows behind the last request are left as they were
    assert (d["out"][int(t.cu[-1]):] == 7.0).all()


def test_the_largest_limits_change_nothing():
    """max_q_len, max_seq_len above what the batch has, and a longer table."""
    t = CASES["ragged"]()
    d = t.device()
    first = t.run(d, t.workspace()).clone()
    t.table = np.concatenate([t.table, np.full((t.B, 5), -1, np.int32)], 1)
    d = t.device()
    t.max_len = t.table.shape[1] * t.P
    t.max_q = 64
    d["mask"] = torch.cat([d["mask"], torch.full((t.T, 2 - t.words), -1, dtype=torch.int32, device="cuda")], 1) \
        if t.words < 2 else d["mask"]
    t.run(d, t.workspace())
    R.check(t, d["out"])
    assert (first.float() - d["out"].float()).abs().max() < 0.05


def test_a_chain_is_a_prefill():
    """A mask that names every earlier draft is wf_paged_prefill's causal mask."""
    t = R.Tree([100, 0, 300], [30, 64, 7], 8, 2, 128, 16, "bf16", seed=40)
    for b in range(3):
        for i in range(int(t.drafted[b])):
            m = (1 << (i + 1)) - 1
            t.bits[t.cu[b] + i] = [(m >> (32 * w)) & 0xFFFFFFFF for w in range(t.words)]
    d = t.device()
    t.run(d, t.workspace())
    other = torch.empty_like(d["out"])
    wf.wf_paged_prefill(other, d["q"], d["k"], d["v"], d["table"], d["lens"], d["cu"], t.max_q, t.max_len, t.scale,
                        d["status"])
    ref = t.reference()
    R.check(t, d["out"], ref)
    lim = t.bound(*ref) + t.bound(*ref, rounded=True)   # the prefill's weights are rounded to bf16
    off = np.abs(other.double().cpu().numpy() - d["out"].double().cpu().numpy())
    assert (off <= lim).all()


def test_one_draft_is_a_decode():
    t = R.Tree([100, 0, 300, 15], [1, 1, 1, 1], 8, 2, 64, 16, "f32", seed=41)
    d = t.device()
    t.run(d, t.workspace())
    other = torch.empty_like(d["out"])
    n = wf.wf_paged_decode_workspace_size(4, 8, t.max_len, wf.pool_desc(d["k"]))
    wf.wf_paged_decode(other, d["q"], d["k"], d["v"], d["table"], d["lens"], t.max_len, t.scale,
                       torch.empty(n, dtype=torch.uint8, device="cuda"), d["status"])
    ref = t.reference()
    R.check(t, d["out"], ref)
    assert (np.abs((other - d["out"]).double().cpu().numpy()) <= 2 * t.bound(*ref)).all()


def _poisoned(pool, P, value_k, value_v, D=128):
    """A batch whose draft 3 of request 1 has `value` in its rows, seen by itself and its descendants only."""
    t = R.Tree([40, 50, 130], [6, 9, 5], 8, 2, D, P, pool, seed=42, **(FP8 if pool == "fp8" else {}))
    clean = R.Tree([40, 50, 130], [6, 9, 5], 8, 2, D, P, pool, seed=42, **(FP8 if pool == "fp8" else {}))
    pos = 50 + 3
    at = (int(t.table[1, pos // P]), pos % P)
    if pool == "fp8":
        t.k[at][:, 7] = 0x7F
        t.v[at][:, 9] = 0x7F
    else:
        t.k[at][:, 7] = value_k
        t.v[at][:, 9] = value_v
    sees = [int(t.cu[1]) + i for i in range(9) if pos in t.sees(1, i)]
    return t, clean, sees


@pytest.mark.parametrize("pool,P,D", [("bf16", 16, 128), ("bf16", 16, 64), ("bf16", 7, 128), ("f32", 16, 64), ("fp8", 16, 128),
                                      ("fp8", 16, 64), ("fp8", 5, 64)])
@pytest.mark.parametrize("k,v", [(float("nan"), float("nan")), (float("inf"), float("-inf")), (0.0, float("inf")),
                                 (1.0, float("nan"))])
def test_what_a_row_does_not_see_has_no_effect(pool, P, D, k, v):
    t, clean, sees = _poisoned(pool, P, k, v, D)
    rest = [i for i in range(t.T) if i not in sees]
    assert sees and rest
    a, b = clean.device(), t.device()
    ws = t.workspace()
    clean.run(a, ws)
    t.run(b, ws)
    assert torch.equal(a["out"][rest], b["out"][rest]), "rows that do not see the draft changed"
    got = b["out"][sees].float()
    if pool == "fp8" or k != k:
        assert torch.isnan(got).all()                      # the score is NaN
    elif k == 0.0:
        assert torch.equal(got[:, :, 9], torch.full_like(got[:, :, 9], v))
        keep = [c for c in range(D) if c != 9]
        assert torch.isfinite(got[:, :, keep]).all()
    elif k == 1.0:
        assert torch.isnan(got[:, :, 9]).all()
        assert torch.isfinite(got[:, :, :9]).all() and torch.isfinite(got[:, :, 10:]).all()


@pytest.mark.parametrize("pool,P", [("bf16", 16), ("bf16", 7), ("f32", 16), ("fp8", 16)])
def test_bad_lengths_skip_the_request(pool, P):
    kw = FP8 if pool == "fp8" else {}
    for length in (3, -1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        t = R.Tree([40, 50, 130], [6, 9, 5], 8, 2, 128, P, pool, seed=43, **kw)
        ref = t.reference()
        t.lens[1] = length
        d = t.device()
        t.run(d, t.workspace())
        rows = slice(int(t.cu[1]), int(t.cu[2]))
        assert (d["out"][rows] == 7.0).all()
        d["out"][rows] = torch.from_numpy(ref[0][rows]).cuda().to(d["out"].dtype)
        R.check(t, d["out"], ref)
        assert wf.wf_device_status_fetch(d["status"]) == wf.WF_DEV_BAD_SEQLEN


def test_bad_offsets_skip_the_request():
    for cu in ([0, 6, 3, 20], [0, 6, 100, 20], [0, 6, 15, 21]):
        t = R.Tree([40, 50, 130], [6, 9, 5], 8, 2, 128, 16, "bf16", seed=43)
        t.cu = np.array(cu, np.int32)
        d = t.device()
        t.run(d, t.workspace())
        assert torch.isfinite(d["out"].float()).all()
        assert wf.wf_device_status_fetch(d["status"]) & wf.WF_DEV_BAD_SEQLEN


@pytest.mark.parametrize("pool,P", [("bf16", 16), ("bf16", 48), ("bf16", 7), ("f32", 16), ("fp8", 16)])
@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31])
def test_positions_of_bad_blocks_are_left_out(pool, P, bad):
    t = R.Tree([300, 50, 40], [6, 9, 20], 8, 2, 128, P, pool, seed=44, **(FP8 if pool == "fp8" else {}))
    last = (40 + 20 - 1) // P
    ref = t.reference(bad_blocks={(0, 1), (2, last)})
    t.table[0, 1] = bad
    t.table[2, last] = bad
    d = t.device()
    t.run(d, t.workspace())
    R.check(t, d["out"], ref)
    assert wf.wf_device_status_fetch(d["status"]) == wf.WF_DEV_BAD_BLOCK


def test_every_block_bad_gives_zeros():
    for pool, P in (("bf16", 16), ("f32", 16), ("fp8", 16)):
        t = R.Tree([300], [6], 8, 2, 128, P, pool, seed=45, **(FP8 if pool == "fp8" else {}))
        t.table[:] = -1
        d = t.device()
        t.run(d, t.workspace())
        assert (d["out"] == 0).all()


@pytest.mark.parametrize("name", ["ragged", "more than 128 rows", "fp32", "fp8", "blocks of 7", "long"])
def test_the_same_bytes_again_and_from_a_graph(name):
    t = CASES[name]()
    d = t.device()
    ws = t.workspace()
    first = t.run(d, ws).clone()
    for _ in range(3):
        d["out"].fill_(7.0)
        assert torch.equal(t.run(d, ws), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        t.run(d, ws)
    d["out"].fill_(7.0)
    ws.fill_(0xFF)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(d["out"], first)
    # the same graph on other contents of the same buffers
    other = CASES[name]()
    other.q = -other.q
    d["q"].copy_(other.q)
    g.replay()
    torch.cuda.synchronize()
    R.check(other, d["out"])


@pytest.mark.parametrize("pool,D", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64), ("f32", 64)])
@pytest.mark.parametrize("drafts", [5, 40, 64])
def test_pieces_of_every_length_back_to_back(pool, D, drafts):
    """Contexts of 1 to 17 tiles of 128 positions in an order that gives every CTA odd and even pieces, many calls
    without a pause: each has to give the bytes of the first, and no wait may give up."""
    r = np.random.default_rng(50)
    cached = 128 * r.integers(0, 17, 70) + r.integers(0, 128, 70)
    t = R.Tree([1], [1], 8, 2, D, 16, pool, seed=51, **(FP8 if pool == "fp8" else {}))
    # the pools are random and shared: 2300 positions a request out of 300 blocks
    t.cached, t.drafted = cached, np.full(70, drafts)
    t.B, t.lens, t.cu = 70, (cached + drafts).astype(np.int32), (np.arange(71) * drafts).astype(np.int32)
    t.T, t.max_q, t.max_len, t.N = 70 * drafts, drafts, int((cached + drafts).max()), 300
    t.table = r.integers(0, 300, (70, -(-t.max_len // 16))).astype(np.int32)
    t.k, t.v = (R.to_pool((64.0 if pool == "fp8" else 1.0) * r.standard_normal((300, 16, 2, D)), pool) for _ in range(2))
    t.q = torch.from_numpy(r.standard_normal((t.T, 8, D))).float().to(R.act(pool))
    t.words = -(-drafts // 32)
    t.bits = r.integers(0, 2 ** 32, (t.T, t.words), dtype=np.uint32)
    d = t.device()
    ws = t.workspace()
    first = t.run(d, ws).clone()
    few = [0, 1, 2, 33, 69]
    t2 = R.Tree([1], [1], 8, 2, D, 16, pool, seed=51, **(FP8 if pool == "fp8" else {}))
    t2.__dict__.update(t.__dict__)
    t2.cached, t2.drafted, t2.table = t.cached[few], t.drafted[few], t.table[few]
    t2.B, t2.cu = 5, (np.arange(6) * drafts).astype(np.int32)
    rows = np.concatenate([np.arange(drafts) + b * drafts for b in few])
    t2.T, t2.q, t2.bits = len(rows), t.q[rows], t.bits[rows]
    R.check(t2, first[torch.from_numpy(rows).cuda()])
    for _ in range(60):
        t.run(d, ws)
    assert torch.equal(d["out"], first)
    d["out"].fill_(7.0)
    for _ in range(60):
        t.run(d, ws)
    assert torch.equal(d["out"], first)
    assert wf.wf_device_status_fetch(d["status"]) == 0


def test_two_streams_with_their_own_workspaces():
    a, b = CASES["several row blocks"](), CASES["many requests"]()
    da, db = a.device(), b.device()
    wa, wb = a.workspace(), b.workspace()
    ra, rb = a.run(da, wa).clone(), b.run(db, wb).clone()
    torch.cuda.synchronize()
    s, u = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.run(da, wa, stream=s)
        b.run(db, wb, stream=u)
    torch.cuda.synchronize()
    assert torch.equal(da["out"], ra) and torch.equal(db["out"], rb)


def test_negative_and_zero_scale():
    for scale in (0.0, -0.2):
        for pool in ("bf16", "f32"):
            t = R.Tree([40, 50], [6, 9], 8, 2, 128, 16, pool, seed=46)
            t.scale = scale
            d = t.device()
            R.check(t, t.run(d, t.workspace()))


@pytest.mark.parametrize("pool,D,P", [("bf16", 128, 16), ("bf16", 64, 7), ("fp8", 128, 16), ("fp8", 64, 16), ("fp8", 64, 7),
                                      ("f32", 64, 16)])
def test_a_long_tail_of_small_weights(pool, D, P):
    """One position of weight 1 whose values are 0 and 900 of 2^-26: the outputs are the tail's."""
    t = R.Tree([900], [3], 8, 2, D, P, pool, seed=80, **(FP8 if pool == "fp8" else {}))
    r = np.random.default_rng(81)
    own = torch.from_numpy(t.table[0].astype(np.int64))
    spike = R.to_pool(np.array([1.0 / t.ks]), pool)[0]
    t.k[own], t.v[own] = 0, R.to_pool(2.0 / t.vs * r.random((len(own), P, 2, D)), pool)
    t.k[own[0], 0, :, 0], t.v[own[0], 0] = spike, 0
    t.q[:], t.scale = 0, 1.0
    t.q[..., 0] = 18.0            # 18 log2(e) = 25.97
    d = t.device()
    R.check(t, t.run(d, t.workspace()))
    assert float(d["out"].float().abs().min()) > 2.0 ** -18

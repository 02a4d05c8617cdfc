"""wf_qk_norm_rope_and_cache against the formula in 64 bits."""
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


class Step:
    def __init__(self, T, H_q, H_kv, D, P, pool, rot, interleaved=False, norm=(True, True), fused=False, pads=(),
                 seed=0, eps=1e-6, ks=1.0, vs=1.0, rows=500, size=1.0):
        r = np.random.default_rng(seed)
        dt = R.act(pool)
        self.T, self.H_q, self.H_kv, self.D, self.P, self.pool = T, H_q, H_kv, D, P, pool
        self.interleaved, self.eps, self.ks, self.vs = interleaved, eps, ks, vs
        x = torch.from_numpy(size * r.standard_normal((T, H_q + 2 * H_kv, D))).float().to(dt).cuda()
        self.q, self.k, self.v = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
        if not fused:
            self.q, self.k, self.v = self.q.contiguous(), self.k.contiguous(), self.v.contiguous()
        self.qw, self.kw = (torch.from_numpy(1 + 0.3 * r.standard_normal(D)).float().to(dt).cuda() if n else None
                            for n in norm)
        self.table = R.cos_sin_table(rows, rot).cuda() if rot else None
        self.positions = r.integers(0, rows, T).astype(np.int32)
        self.N = -(-T // P) + 1
        self.slots = r.permutation(self.N * P)[:T].astype(np.int64)
        self.slots[list(pads)] = -1
        self.live = np.setdiff1d(np.arange(T), list(pads))
        fill = 0x11 if pool == "fp8" else 3.0
        self.kp = torch.full((self.N, P, H_kv, D), fill, dtype=R.DT[pool], device="cuda")
        self.vp = self.kp.clone()
        self.q_out = torch.full((T, H_q, D), 5.0, dtype=dt, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        kw = dict(k_scale=self.ks, v_scale=self.vs) if self.pool == "fp8" else {}
        wf.wf_qk_norm_rope_and_cache(self.q_out, self.q, self.k, self.v, self.qw, self.kw, self.eps, self.table,
                                     torch.from_numpy(self.positions).cuda(), self.kp, self.vp,
                                     torch.from_numpy(self.slots).cuda(), interleaved=self.interleaved,
                                     dev_status=self.status, stream=stream, **kw)

    def check(self, live=None):
        live = self.live if live is None else np.asarray(live)
        t = R.act(self.pool)
        # The sum of D squares in fp32 is off by at most D roundings, the mean, its reciprocal root (two steps) and
        # the two products by five more; the root halves the sum's part.  A rotation multiplies and adds its pair.
        rel = (self.D / 2 + 9) * 2.0 ** -24
        q, size = R.norm_rope_reference(self.q[live], self.qw, self.eps, self.table, self.positions[live],
                                        self.interleaved)
        got = self.q_out.cpu().to(torch.float64).numpy()
        tol = R.half_step(t) * np.abs(q) + rel * size * (1 + R.half_step(t))
        assert (np.abs(got[live] - q) <= tol).all(), (np.abs(got[live] - q) / tol).max()
        rest = np.setdiff1d(np.arange(self.T), live)
        assert (got[rest] == 5.0).all()
        k, size = R.norm_rope_reference(self.k[live], self.kw, self.eps, self.table, self.positions[live],
                                        self.interleaved)
        v = self.v[live].cpu().to(torch.float64).numpy()
        free = np.setdiff1d(np.arange(self.N * self.P), self.slots[live])
        for x, err, pool, scale in ((k, rel * size, self.kp, self.ks), (v, 0 * v, self.vp, self.vs)):
            got = R.pool_values(pool).reshape(-1, self.H_kv, self.D)
            if self.pool == "fp8":
                inv = np.float32(1) / np.asarray(scale, np.float32)
                inv = np.broadcast_to(inv.astype(np.float64).reshape(-1, 1), (self.H_kv, 1))
                want, err = np.clip(x * inv, -448, 448), err * inv
                # half a step of e4m3: 2^-4 of the value, 2^-10 below its smallest normal number; the product
                # with the reciprocal is one more fp32 rounding
                tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + (err + 2.0 ** -24 * np.abs(want)) * (1 + 2.0 ** -4)
            else:
                want = x
                tol = R.half_step(R.DT[self.pool]) * np.abs(x) * (err > 0) + err * (1 + R.half_step(t))
            off = np.abs(got[self.slots[live]] - want)
            assert (off <= tol).all(), (off - tol).max()
            untouched = pool.view(-1, self.H_kv, self.D)[torch.from_numpy(free).cuda()]
            assert (untouched == (0x11 if self.pool == "fp8" else 3.0)).all()


CASES = {
    "one token, llama-3-8b heads": lambda: Step(1, 32, 8, 128, 16, "bf16", 128),
    "fused projection": lambda: Step(37, 32, 8, 128, 16, "bf16", 128, fused=True),
    "d64": lambda: Step(19, 12, 12, 64, 16, "bf16", 64, fused=True),
    "fp32": lambda: Step(23, 4, 2, 64, 16, "f32", 64, fused=True),
    "fp32 d128": lambda: Step(9, 6, 3, 128, 7, "f32", 128),
    "interleaved": lambda: Step(11, 8, 2, 128, 16, "bf16", 128, interleaved=True),
    "interleaved fp32 half": lambda: Step(11, 8, 2, 64, 16, "f32", 32, interleaved=True),
    "half rotated": lambda: Step(5, 8, 8, 128, 32, "bf16", 64),
    "odd width": lambda: Step(6, 5, 1, 64, 3, "bf16", 20),
    "width of two": lambda: Step(6, 5, 1, 64, 3, "f32", 2),
    "odd width, interleaved": lambda: Step(7, 4, 4, 128, 16, "bf16", 42, interleaved=True),
    "odd width 126": lambda: Step(7, 4, 4, 128, 16, "f32", 126),
    "no rotation": lambda: Step(8, 4, 2, 128, 16, "bf16", 0),
    "neither norm nor rotation": lambda: Step(8, 4, 2, 128, 16, "bf16", 0, norm=(False, False)),
    "only keys normed": lambda: Step(8, 4, 2, 128, 16, "bf16", 128, norm=(False, True)),
    "only queries normed, odd width": lambda: Step(8, 4, 2, 128, 16, "bf16", 24, norm=(True, False)),
    "padding inside and at the end": lambda: Step(40, 8, 2, 64, 16, "bf16", 64, pads=(0, 7, 38, 39)),
    "all padding": lambda: Step(3, 8, 2, 64, 16, "bf16", 64, pads=(0, 1, 2)),
    "many tokens": lambda: Step(1500, 8, 2, 128, 16, "bf16", 128, pads=(1499,)),
    "many tokens fp32": lambda: Step(700, 4, 2, 64, 16, "f32", 64, fused=True),
    "fp8": lambda: Step(33, 32, 8, 128, 16, "fp8", 128, fused=True, ks=1 / 64, vs=1 / 96),
    "fp8 d64 per head": lambda: Step(33, 6, 3, 64, 16, "fp8", 64, ks=[1 / 64, 1 / 32, 1 / 100], vs=[1 / 8, 1 / 77, 2.0]),
    "fp8 many tokens": lambda: Step(900, 8, 4, 128, 16, "fp8", 128, ks=1 / 64, vs=1 / 64, norm=(False, False), pads=(3,)),
    "fp8 saturated": lambda: Step(12, 4, 2, 64, 16, "fp8", 32, ks=1 / 512, vs=1 / 512),
    "large values": lambda: Step(12, 4, 2, 64, 16, "bf16", 64, size=1e4),
    "small values, large eps": lambda: Step(12, 4, 2, 64, 16, "f32", 64, size=1e-3, eps=1e-2),
    "block of one": lambda: Step(12, 4, 2, 64, 1, "bf16", 64),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_formula(name):
    s = CASES[name]()
    s.run()
    s.check()
    assert wf.wf_device_status_fetch(s.status) == 0


def test_v_and_untouched_k_are_byte_copies():
    s = Step(21, 4, 2, 128, 16, "bf16", 0, norm=(False, False), fused=True)
    s.run()
    at = torch.from_numpy(s.slots).cuda()
    assert torch.equal(s.kp.view(-1, 2, 128)[at], s.k)
    assert torch.equal(s.vp.view(-1, 2, 128)[at], s.v)
    assert torch.equal(s.q_out, s.q)


def test_bad_slots_and_positions_are_flagged_and_skipped():
    s = Step(10, 4, 2, 64, 16, "bf16", 64)
    good = s.slots.copy()
    s.slots[4] = s.N * s.P
    s.run()
    s.check(live=[t for t in range(10) if t != 4])
    assert wf.wf_device_status_fetch(s.status) == wf.WF_DEV_BAD_SLOT
    for value in (-1, 500, -2 ** 31, 2 ** 31 - 1):
        s = Step(10, 4, 2, 64, 16, "bf16", 64)
        s.positions[7] = value
        s.run()
        s.check(live=[t for t in range(10) if t != 7])
        assert wf.wf_device_status_fetch(s.status) == wf.WF_DEV_BAD_POSITION
    # a padding token's position is not looked at
    s = Step(10, 4, 2, 64, 16, "bf16", 64, pads=(7,))
    s.positions[7] = -5
    s.run()
    s.check()
    assert wf.wf_device_status_fetch(s.status) == 0
    assert (good >= 0).all()


def test_nan_and_infinity_stay_in_their_row():
    s = Step(6, 4, 2, 64, 16, "fp8", 64, ks=1 / 64, vs=1 / 64)
    s.q[2, 1, 5] = float("nan")
    s.k[3, 1, 5] = float("inf")
    s.v[4, 0, 9] = float("nan")
    s.v[4, 0, 10] = float("-inf")
    s.run()
    q = s.q_out.float()
    assert torch.isnan(q[2, 1]).all() and torch.isfinite(q[2, 0]).all() and torch.isfinite(q[3]).all()
    v = s.vp.view(torch.float8_e4m3fn).float().view(-1, 2, 64)[int(s.slots[4])]
    assert torch.isnan(v[0, 9]) and v[0, 10] == -448 and torch.isfinite(v[1]).all()
    k = s.kp.view(torch.float8_e4m3fn).float().view(-1, 2, 64)[int(s.slots[3])]
    assert torch.isfinite(k[0]).all() and torch.isnan(k[1, 5])


def test_repeated_and_captured_calls_give_the_same_bytes():
    s = Step(300, 8, 2, 128, 16, "bf16", 128, fused=True)
    s.run()
    first = [x.clone() for x in (s.q_out, s.kp, s.vp)]
    pos, slots = torch.from_numpy(s.positions).cuda(), torch.from_numpy(s.slots).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        wf.wf_qk_norm_rope_and_cache(s.q_out, s.q, s.k, s.v, s.qw, s.kw, s.eps, s.table, pos, s.kp, s.vp, slots)
    for x in (s.q_out, s.kp, s.vp):
        x.fill_(3.0)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (s.q_out, s.kp, s.vp)):
        assert torch.equal(a, b)


def test_far_token_strides():
    """Tokens far apart in a larger buffer (a view of more columns than the heads need)."""
    s = Step(17, 4, 2, 64, 16, "bf16", 64)
    wide = torch.full((17, 50, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:7], wide[:, 20:22], wide[:, 48:50] = s.q, s.k, s.v
    s.q, s.k, s.v = wide[:, 3:7], wide[:, 20:22], wide[:, 48:50]
    s.run()
    s.check()

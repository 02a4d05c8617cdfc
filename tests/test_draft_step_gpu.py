"""The verification step of speculative decoding as it is used: drafts normed, rotated and
scattered, their tree attended to over the cache, the accepted path kept, and again."""
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


class Loop:
    """B requests whose buffers stay where they are from step to step.  Request 1 has no drafts; the last
    `PADS` rows belong to nobody and have a slot of -1."""
    PADS = 3
    ROWS = 400     # of the table of cosines and sines

    def __init__(self, cached, drafted, H_q, H_kv, D, P, pool, seed, k_scale=1.0, v_scale=1.0):
        self.rng = np.random.default_rng(seed)
        self.cached, self.drafted = np.asarray(cached), np.asarray(drafted)
        self.B, self.H_q, self.H_kv, self.D, self.P, self.pool = len(cached), H_q, H_kv, D, P, pool
        self.ks, self.vs = k_scale, v_scale
        self.cu = np.concatenate([[0], np.cumsum(drafted)]).astype(np.int32)
        self.T = int(self.cu[-1]) + self.PADS
        self.max_q, self.max_len = int(max(drafted)), 200
        self.M = -(-self.max_len // P)
        self.N = self.B * self.M
        self.table = self.rng.permutation(self.N).reshape(self.B, self.M).astype(np.int32)
        self.words = -(-self.max_q // 32)
        size = 64.0 if pool == "fp8" else 1.0
        self.kp, self.vp = (R.to_pool(size * self.rng.standard_normal((self.N, P, H_kv, D)), pool).cuda()
                            for _ in range(2))
        dt = R.act(pool)
        dev = dict(device="cuda")
        self.qw, self.kw = (torch.from_numpy(1 + 0.3 * self.rng.standard_normal(D)).float().to(dt).cuda()
                            for _ in range(2))
        self.cos_sin = R.cos_sin_table(self.ROWS, D).cuda()
        self.x = torch.zeros((self.T, H_q + 2 * H_kv, D), dtype=dt, **dev)
        self.q = torch.zeros((self.T, H_q, D), dtype=dt, **dev)
        self.out = torch.zeros_like(self.q)
        self.positions = torch.zeros(self.T, dtype=torch.int32, **dev)
        self.slots = torch.zeros(self.T, dtype=torch.int64, **dev)
        self.lens = torch.zeros(self.B, dtype=torch.int32, **dev)
        self.mask = torch.zeros((self.T, self.words), dtype=torch.int32, **dev)
        self.path = torch.zeros((self.B, 6), dtype=torch.int32, **dev)
        self.count = torch.zeros(self.B, dtype=torch.int32, **dev)
        self.new = torch.zeros(self.B, dtype=torch.int32, **dev)
        self.status = torch.zeros(1, dtype=torch.int32, **dev)
        self.d_table, self.d_cu = torch.from_numpy(self.table).cuda(), torch.from_numpy(self.cu).cuda()
        desc = wf.pool_desc(self.kp, **self.scales())
        n = wf.wf_paged_tree_decode_workspace_size(self.B, H_q, self.max_q, self.max_len, desc)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, **dev)
        self.scale = D ** -0.5

    def scales(self):
        return dict(k_scale=self.ks, v_scale=self.vs) if self.pool == "fp8" else {}

    def slot(self, b, pos):
        return int(self.table[b, pos // self.P]) * self.P + pos % self.P

    def feed(self):
        """New drafts: a random tree a request, its values, and a path of it that is accepted."""
        r = self.rng
        bits = np.zeros((self.T, self.words), np.uint32)
        pos = np.zeros(self.T, np.int32)
        slots = np.full(self.T, -1, np.int64)
        path, count = np.full((self.B, 6), -1, np.int32), np.zeros(self.B, np.int32)
        for b in range(self.B):
            n, c, at = int(self.drafted[b]), int(self.cached[b]), int(self.cu[b])
            parent = [int(r.integers(-1, i)) for i in range(n)]
            for i in range(n):
                chain = [i]
                while parent[chain[0]] >= 0:
                    chain.insert(0, parent[chain[0]])
                for j in chain:
                    bits[at + i, j // 32] |= np.uint32(1 << (j % 32))
                pos[at + i] = c + len(chain) - 1
                slots[at + i] = self.slot(b, c + i)
                if i == n - 1:       # the last draft's path, cut short
                    count[b] = r.integers(0, min(len(chain), 6) + 1)
                    path[b, :count[b]] = chain[:count[b]]
        self.bits, self.h_pos, self.h_slots, self.h_path, self.h_count = bits, pos, slots, path, count
        x = r.standard_normal(tuple(self.x.shape))
        if self.PADS:
            x[-self.PADS:] = np.nan
        self.x.copy_(torch.from_numpy(x))
        for to, h in ((self.positions, pos), (self.slots, slots), (self.mask, bits.view(np.int32)), (self.path, path),
                      (self.count, count), (self.lens, (self.cached + self.drafted).astype(np.int32))):
            to.copy_(torch.from_numpy(h))

    def scatter(self, stream=None):
        q, k, v = self.x.split([self.H_q, self.H_kv, self.H_kv], 1)
        wf.wf_qk_norm_rope_and_cache(self.q, q, k, v, self.qw, self.kw, 1e-6, self.cos_sin, self.positions, self.kp,
                                     self.vp, self.slots, dev_status=self.status, stream=stream, **self.scales())

    def attend(self, stream=None):
        wf.wf_paged_tree_decode(self.out, self.q, self.kp, self.vp, self.d_table, self.lens, self.d_cu, self.mask,
                                self.max_q, self.max_len, self.scale, self.ws, dev_status=self.status, stream=stream,
                                **self.scales())

    def keep(self, stream=None):
        wf.wf_keep_accepted(self.kp, self.vp, self.d_table, self.lens, self.d_cu, self.path, self.count,
                            new_seq_lens=self.new, dev_status=self.status, stream=stream)

    def advance(self):
        self.cached = self.cached + self.h_count

    def rows(self, pool):
        return pool.view(torch.uint8).view(self.N * self.P, -1).cpu().numpy()

    def sequence(self, b, length):
        return [self.slot(b, p) for p in range(length)]

    def tree(self):
        """The inputs as the 64-bit reference takes them, from what is on the device now."""
        t = R.Tree.__new__(R.Tree)
        n = int(self.cu[-1])
        t.__dict__.update(cached=self.cached, drafted=self.drafted, H_q=self.H_q, H_kv=self.H_kv, D=self.D, P=self.P,
                          pool=self.pool, B=self.B, ks=self.ks, vs=self.vs, N=self.N, table=self.table, cu=self.cu,
                          T=n, k=self.kp.cpu(), v=self.vp.cpu(), q=self.q[:n].cpu(), bits=self.bits, scale=self.scale)
        return t


def check_scattered(s):
    """The rotated queries and the rows of the pools against the formula; bounds as for the call alone."""
    n, t = int(s.cu[-1]), R.act(s.pool)
    q, k, v = (y[:n] for y in s.x.split([s.H_q, s.H_kv, s.H_kv], 1))
    rel = (s.D / 2 + 9) * 2.0 ** -24
    want, size = R.norm_rope_reference(q, s.qw, 1e-6, s.cos_sin, s.h_pos[:n], False)
    got = s.q[:n].cpu().to(torch.float64).numpy()
    assert (np.abs(got - want) <= R.half_step(t) * np.abs(want) + rel * size * (1 + R.half_step(t))).all()
    want, size = R.norm_rope_reference(k, s.kw, 1e-6, s.cos_sin, s.h_pos[:n], False)
    for x, err, pool, scale in ((want, rel * size, s.kp, s.ks), (v.cpu().to(torch.float64).numpy(), 0, s.vp, s.vs)):
        got = R.pool_values(pool).reshape(-1, s.H_kv, s.D)[s.h_slots[:n]]
        if s.pool == "fp8":
            # half a step of e4m3 (2^-4 of the value, 2^-10 below its smallest normal number), the product with the
            # rounded reciprocal of the scale
            inv = float(np.float32(1) / np.float32(scale))
            x = np.clip(x * inv, -448, 448)
            tol = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10) + (err * inv + 2.0 ** -24 * np.abs(x)) * (1 + 2.0 ** -4)
        else:
            tol = R.half_step(t) * np.abs(x) * (np.asarray(err) > 0) + err * (1 + R.half_step(t))
        assert (np.abs(got - x) <= tol).all()


LOOPS = {
    "bf16": lambda: Loop([40, 9, 0, 130, 17], [12, 0, 5, 33, 1], 8, 2, 128, 16, "bf16", 60),
    "bf16, 64-wide heads": lambda: Loop([40, 9, 0, 130, 17], [12, 0, 5, 40, 1], 6, 2, 64, 32, "bf16", 61),
    "bf16, blocks of 7": lambda: Loop([40, 9, 0, 130, 17], [12, 0, 5, 33, 1], 8, 2, 128, 7, "bf16", 62),
    "f32": lambda: Loop([40, 9, 0, 130, 17], [12, 0, 5, 9, 1], 12, 12, 64, 16, "f32", 63),
    "fp8": lambda: Loop([40, 9, 0, 130, 17], [12, 0, 5, 33, 1], 8, 2, 128, 16, "fp8", 64, 1 / 64, 1 / 64),
}


@pytest.mark.parametrize("name", list(LOOPS))
def test_steps_one_after_the_other(name):
    """Three steps: every call against its reference, and the cache against the rows that were accepted, byte for byte."""
    s = LOOPS[name]()
    kept = [[(s.rows(s.kp)[x].copy(), s.rows(s.vp)[x].copy()) for x in s.sequence(b, int(s.cached[b]))]
            for b in range(s.B)]
    for _ in range(3):
        s.feed()
        s.scatter()
        check_scattered(s)
        s.out.fill_(7.0)
        s.attend()
        t = s.tree()
        R.check(t, s.out[:t.T])
        assert (s.out[t.T:] == 7.0).all()
        k, v = s.rows(s.kp), s.rows(s.vp)
        for b in range(s.B):
            for j in s.h_path[b, :s.h_count[b]]:
                x = s.slot(b, int(s.cached[b]) + int(j))
                kept[b].append((k[x].copy(), v[x].copy()))
        s.keep()
        s.advance()
        assert s.new.cpu().tolist() == s.cached.tolist()
        k, v = s.rows(s.kp), s.rows(s.vp)
        for b in range(s.B):
            at = s.sequence(b, int(s.cached[b]))
            assert len(at) == len(kept[b])
            for x, (kx, vx) in zip(at, kept[b]):
                assert (k[x] == kx).all() and (v[x] == vx).all()
    assert wf.wf_device_status_fetch(s.status) == 0


@pytest.mark.parametrize("name", list(LOOPS))
def test_steps_from_one_graph(name):
    """A step captured once and replayed on the contents of three gives the bytes of three steps of calls."""
    a, b = LOOPS[name](), LOOPS[name]()
    side = torch.cuda.Stream()
    a.feed()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        a.scatter()
        a.attend()
        a.keep()
    b.feed()
    for step in range(3):
        if step:
            a.feed()
            b.feed()
        g.replay()
        b.scatter()
        b.attend()
        b.keep()
        torch.cuda.synchronize()
        n = int(a.cu[-1])
        assert torch.equal(a.out[:n], b.out[:n]) and torch.equal(a.new, b.new)
        assert torch.equal(a.kp.view(torch.uint8), b.kp.view(torch.uint8))
        assert torch.equal(a.vp.view(torch.uint8), b.vp.view(torch.uint8))
        a.advance()
        b.advance()
    assert wf.wf_device_status_fetch(a.status) == wf.wf_device_status_fetch(b.status) == 0


def test_the_next_decode_sees_what_was_kept():
    """After a step, wf_paged_decode of the kept lengths attends to the accepted rows and to no other draft."""
    s = LOOPS["bf16"]()
    s.feed()
    s.scatter()
    s.attend()
    s.keep()
    s.advance()
    q = torch.from_numpy(s.rng.standard_normal((s.B, s.H_q, s.D))).float().to(torch.bfloat16).cuda()
    out = torch.zeros_like(q)
    n = wf.wf_paged_decode_workspace_size(s.B, s.H_q, s.max_len, wf.pool_desc(s.kp))
    ws = torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda")
    wf.wf_paged_decode(out, q, s.kp, s.vp, s.d_table, s.new, s.max_len, s.scale, ws, dev_status=s.status)
    t = s.tree()
    have = s.cached > 0                      # request 2 may have kept nothing
    t.cached, t.drafted = s.cached - have, have.astype(np.int64)
    t.cu, t.T = np.concatenate([[0], np.cumsum(t.drafted)]).astype(np.int32), int(have.sum())
    t.bits = np.ones((t.T, 1), np.uint32)
    t.q = q[torch.from_numpy(have).cuda()].cpu()
    ref = t.reference()
    off = np.abs(out[torch.from_numpy(have).cuda()].cpu().to(torch.float64).numpy() - ref[0])
    # a decode that rounds its weights to bf16 is allowed the same as a tree on the tensor cores
    assert (off <= t.bound(*ref, rounded=True)).all()

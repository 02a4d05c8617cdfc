"""A step of speculative decoding that stays on the GPU: its tables built from lengths, the drafts normed, rotated and
scattered, attended to, verified, the accepted path kept, and the other blocks given back."""
import numpy as np
import pytest
import torch

from paged_kv_cache_wf_gb300 import binding as wf
from tests import _draft as R
from tests import _step as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_wf_gb300 import build
    build.build()


class Serving:
    """B requests; buffers stay where they are from step to step.  The last rows of a step are padding."""
    V, MAX, ROWS = 500, 300, 400

    def __init__(self, cached, nodes, H_q, H_kv, D, P, pool, seed, chain):
        self.r = np.random.default_rng(seed)
        self.B, self.nodes, self.chain = len(cached), max(nodes), chain
        self.H_q, self.H_kv, self.D, self.P, self.pool = H_q, H_kv, D, P, pool
        self.q_ = S.Requests(cached, P, 60, M=-(-self.MAX // P), seed=seed)
        dt, dev = R.act(pool), dict(device="cuda")
        N = self.q_.N
        size = 64.0 if pool == "fp8" else 1.0
        self.kp, self.vp = (R.to_pool(size * self.r.standard_normal((N, P, H_kv, D)), pool).cuda() for _ in range(2))
        self.scale_args = dict(k_scale=1 / 64, v_scale=1 / 96) if pool == "fp8" else {}
        self.table, self.lens = S.i32(self.q_.table), S.i32(self.q_.lens)
        self.free, self.num = S.i32(self.q_.free), S.i32([self.q_.num_free])
        i32 = lambda *n: torch.zeros(n, dtype=torch.int32, **dev)   # noqa: E731
        self.T = self.B * self.nodes + 5
        self.new, self.grown, self.cu, self.depths = i32(self.B), i32(self.B), i32(self.B + 1), i32(self.T)
        self.slots, self.positions = torch.zeros(self.T, dtype=torch.int64, **dev), i32(self.T)
        self.mask, self.parents, self.tokens = i32(self.T, -(-self.nodes // 32)), i32(self.T), i32(self.T)
        self.coins, self.picks = torch.zeros(self.T, **dev), torch.zeros(self.B, **dev)
        self.target, self.draft = (torch.zeros((self.T, self.V), **dev) for _ in range(2))
        self.x = torch.zeros((self.T, H_q + 2 * H_kv, D), dtype=dt, **dev)
        self.q, self.out, self.again = (torch.zeros((self.T, H_q, D), dtype=dt, **dev) for _ in range(3))
        self.cos_sin = R.cos_sin_table(self.ROWS, D).cuda()
        self.path, self.count, self.next, self.kept = i32(self.B, self.nodes), i32(self.B), i32(self.B), i32(self.B)
        self.status = i32(1)
        desc = wf.pool_desc(self.kp, **self.scale_args)
        self.ws = torch.full((wf.wf_paged_tree_decode_workspace_size(self.B, H_q, self.nodes, self.MAX, desc),), 0xFF,
                             dtype=torch.uint8, **dev)
        self.ws2 = torch.full((wf.wf_paged_scored_attention_workspace_size(self.B, H_q, self.T, self.nodes, self.MAX, desc),),
                              0xFF, dtype=torch.uint8, **dev)
        # the host's own account
        self.h_table, self.h_lens, self.h_free, self.h_num = self.q_.table.copy(), self.q_.lens.copy(), self.q_.free.copy(), 60

    def feed(self):
        r = self.r
        self.n = r.integers(0, self.nodes + 1, self.B)
        self.n[0] = self.nodes
        self.h_cu = np.concatenate([[0], np.cumsum(self.n)])
        parents, depths = np.full(self.T, -1, np.int32), np.zeros(self.T, np.int32)
        bits = np.zeros((self.T, self.mask.shape[1]), np.uint32)
        for b in range(self.B):
            at = self.h_cu[b]
            for i in range(self.n[b]):
                up = -1 if i == 0 else i - 1 if self.chain else int(r.integers(max(0, i - 3), i))
                parents[at + i], depths[at + i] = up, 0 if i == 0 else depths[at + up] + 1
                if i:
                    bits[at + i] = bits[at + up]
                bits[at + i, i // 32] |= np.uint32(1 << (i % 32))
        self.h_parents, self.h_depths = parents, depths
        logits = 2 * torch.from_numpy(r.standard_normal((self.T, self.V))).float()
        target = torch.softmax(logits, -1)
        draft = torch.softmax(logits + 0.5 * torch.from_numpy(r.standard_normal((self.T, self.V))).float(), -1)
        tokens = np.zeros(self.T, np.int32)
        for b in range(self.B):
            for i in range(1, self.n[b]):
                p = draft[self.h_cu[b] + parents[self.h_cu[b] + i]].double().numpy()
                tokens[self.h_cu[b] + i] = r.choice(self.V, p=p / p.sum())
        x = r.standard_normal(tuple(self.x.shape))
        x[self.h_cu[-1]:] = np.nan
        self.h_coins, self.h_picks = r.random(self.T).astype(np.float32), r.random(self.B).astype(np.float32)
        for to, h in ((self.new, self.n.astype(np.int32)), (self.depths, depths), (self.parents, parents), (self.tokens, tokens),
                      (self.mask, bits.view(np.int32)), (self.coins, self.h_coins), (self.picks, self.h_picks), (self.x, x),
                      (self.target, target.numpy()), (self.draft, draft.numpy())):
            to.copy_(torch.from_numpy(h))
        self.h_tokens = tokens

    def step(self, upto="trim"):
        split = self.x.split([self.H_q, self.H_kv, self.H_kv], 1)
        wf.wf_build_step(self.table, self.lens, self.new, self.free, self.num, self.grown, self.num, self.cu, self.slots,
                         self.positions, self.P, depths=self.depths, dev_status=self.status)
        wf.wf_qk_norm_rope_and_cache(self.q, *split, None, None, 1e-6, self.cos_sin, self.positions, self.kp, self.vp,
                                     self.slots, dev_status=self.status, **self.scale_args)
        wf.wf_paged_tree_decode(self.out, self.q, self.kp, self.vp, self.table, self.grown, self.cu, self.mask, self.nodes,
                                self.MAX, self.D ** -0.5, self.ws, dev_status=self.status, **self.scale_args)
        if self.chain:
            wf.wf_paged_scored_attention(self.again, self.q, self.kp, self.vp, self.table, self.grown, self.cu, self.nodes,
                                         self.MAX, self.D ** -0.5, self.ws2, dev_status=self.status, **self.scale_args)
        wf.wf_verify_drafts(self.path, self.count, self.next, self.target, self.draft, self.tokens, self.parents, self.cu,
                            self.nodes, self.coins, self.picks, dev_status=self.status)
        wf.wf_keep_accepted(self.kp, self.vp, self.table, self.grown, self.cu, self.path, self.count, new_seq_lens=self.kept,
                            dev_status=self.status, **self.scale_args)
        wf.wf_trim_blocks(self.table, self.grown, self.kept, self.free, self.num, self.num, self.P, dev_status=self.status)
        self.lens.copy_(self.kept)

    def rows(self, slots):
        return [p.view(torch.uint8).view(self.q_.N * self.P, -1).cpu().numpy()[slots] for p in (self.kp, self.vp)]

    def check(self, before):
        table, grown, left, cu, slots, positions = S.build(self.h_table, self.h_lens, self.n, self.h_free, self.h_num, self.T,
                                                           self.P, self.h_depths)
        assert int(self.status.item()) == 0
        for got, want in ((self.table, table), (self.cu, cu), (self.slots, slots), (self.positions, positions)):
            assert np.array_equal(got.cpu().numpy(), want)
        target, draft = self.target.double().cpu().numpy(), self.draft.double().cpu().numpy()
        kept = self.h_lens.copy()
        for b in range(self.B):
            lo, hi = cu[b], cu[b + 1]
            if lo == hi:
                assert int(self.count[b]) == 0 and int(self.next[b]) == -1
                continue
            path, token = S.verify(target[lo:hi], draft[lo:hi], self.h_tokens[lo:hi], self.h_parents[lo:hi],
                                   self.h_coins[lo:hi].astype(float), float(self.h_picks[b]), self.nodes)
            assert self.path[b].tolist() == path + [-1] * (self.nodes - len(path)) and int(self.next[b]) == token
            kept[b] = self.h_lens[b] + len(path)
            # the path's rows lie behind the context, as they were scattered; the context is as it was
            at = [int(table[b, p // self.P]) * self.P + p % self.P for p in range(kept[b])]
            now = self.rows(np.array(at, int))
            for pool, old in zip(now, before):
                assert np.array_equal(pool[:self.h_lens[b]], old[np.array(at[:self.h_lens[b]], int)])
            want = self.scattered(slots[lo + np.array(path)], lo + np.array(path))
            assert np.array_equal(now[1][self.h_lens[b]:], want)
        free, num = S.trim(table, grown, kept, self.h_free, left, self.P)
        assert np.array_equal(self.free.cpu().numpy(), free) and int(self.num.item()) == num
        assert np.array_equal(self.lens.cpu().numpy(), kept)
        n = cu[-1]
        if self.chain:
            # chains are causal: the same to the rounding of two ways to compute it
            off = (self.out[:n].double() - self.again[:n].double()).abs().max()
            assert off <= (1e-4 if self.pool == "f32" else 2e-2), off
        self.h_table, self.h_lens, self.h_free, self.h_num = table, kept, free, num

    def scattered(self, slots, rows):
        """What the scatter wrote of V for these rows, as bytes."""
        v = self.x[torch.from_numpy(rows).cuda(), self.H_q + self.H_kv:]
        if self.pool == "fp8":
            v = (v.float() * (1 / (1 / 96))).clamp(-448, 448).to(torch.float8_e4m3fn)
        return v.contiguous().view(torch.uint8).view(len(rows), -1).cpu().numpy()


@pytest.mark.parametrize("pool, H_q, H_kv, D, P", [("bf16", 8, 2, 128, 16), ("fp8", 8, 2, 64, 16), ("f32", 4, 2, 64, 16),
                                                   ("bf16", 8, 4, 64, 7)])
@pytest.mark.parametrize("chain", [True, False])
def test_steps(pool, H_q, H_kv, D, P, chain):
    s = Serving([100, 37, 0, 5, 16], [9], H_q, H_kv, D, P, pool, seed=3, chain=chain)
    everything = np.arange(s.q_.N * s.P)
    for _ in range(3):
        s.feed()
        before = s.rows(everything)
        s.step()
        s.check(before)
    s.feed()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        s.step()
    for _ in range(4):
        before = s.rows(everything)
        g.replay()
        s.check(before)
        s.feed()


def test_a_step_without_room_moves_nothing():
    """Too few blocks: the whole step has no rows, and the next one, with fewer drafts, goes on from where it was."""
    s = Serving([100, 37, 0, 5, 16], [9], 8, 2, 128, 16, "bf16", seed=4, chain=False)
    s.num.fill_(0)
    s.h_num = 0
    s.feed()
    before = s.rows(np.arange(s.q_.N * s.P))
    s.out.fill_(7.0)
    s.step()
    assert int(s.status.item()) == wf.WF_DEV_NO_BLOCKS
    after = s.rows(np.arange(s.q_.N * s.P))
    assert all(np.array_equal(a, b) for a, b in zip(before, after)) and (s.out == 7.0).all()
    assert np.array_equal(s.lens.cpu().numpy(), s.h_lens) and not s.count.any() and (s.next == -1).all()
    s.status.zero_()
    s.num.fill_(60)
    s.h_num = 60
    s.step()
    s.check(before)

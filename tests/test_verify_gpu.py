"""wf_verify_drafts against the method in float64, request by request."""
import numpy as np
import pytest
import torch

from paged_kv_cache_wf_gb300 import binding as wf
from tests import _step as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_wf_gb300 import build
    build.build()


class Batch:
    """Requests of `nodes` nodes with random trees, probabilities and tokens."""

    def __init__(self, nodes, vocab, drawn=True, probs="f32", seed=0, chain=False, depth=None, pad=0, shift=0, sharp=2.0):
        r = np.random.default_rng(seed)
        self.nodes, self.V, self.B, self.drawn = list(nodes), vocab, len(nodes), drawn
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(int)
        self.T = int(self.cu[-1])
        kind = torch.float32 if probs == "f32" else torch.bfloat16
        gen = torch.Generator().manual_seed(seed)
        x = sharp * torch.randn(max(self.T, 1), vocab, generator=gen)
        y = x + 0.7 * torch.randn(max(self.T, 1), vocab, generator=gen)

        def rows(z):       # rows `pad` elements apart, the first `shift` elements into its memory
            wide = torch.full((max(self.T, 1) * (vocab + pad) + shift,), 0.125, dtype=kind)
            view = wide[shift:].view(max(self.T, 1), vocab + pad)[:, :vocab]
            view.copy_(z)
            on = wide.cuda()
            return on[shift:].view(max(self.T, 1), vocab + pad)[:self.T, :vocab]

        self.target = rows(torch.softmax(x, -1))
        q = torch.softmax(y, -1)
        self.draft = rows(q) if drawn else None
        self.parents, self.tokens = [], []
        for b, n in enumerate(self.nodes):
            for i in range(n):
                up = -1 if i == 0 else i - 1 if chain else int(r.integers(max(0, i - 4), i))
                row = q[self.cu[b] + max(up, 0)].double().numpy()
                self.parents.append(up)
                self.tokens.append(int(r.choice(vocab, p=row / row.sum())) if drawn else int(r.integers(0, min(vocab, 6))))
        self.chain = chain
        self.coins, self.picks = r.random(self.T).astype(np.float32), r.random(self.B).astype(np.float32)
        self.depth = depth or max(1, max(self.nodes))

    def to_device(self):
        self.d = dict(tokens=S.i32(self.tokens), parents=None if self.chain else S.i32(self.parents), cu=S.i32(self.cu),
                      coins=torch.from_numpy(self.coins).cuda(), picks=torch.from_numpy(self.picks).cuda())
        self.accepted = torch.full((self.B, self.depth), -5, dtype=torch.int32, device="cuda")
        self.count, self.next = (torch.full((self.B,), -5, dtype=torch.int32, device="cuda") for _ in range(2))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self

    def call(self, stream=None):
        d = self.d
        wf.wf_verify_drafts(self.accepted, self.count, self.next, self.target, self.draft, d["tokens"], d["parents"], d["cu"],
                            max([1] + self.nodes), d["coins"], d["picks"], dev_status=self.status, stream=stream)
        return self

    def want(self, b):
        lo, hi = self.cu[b], self.cu[b + 1]
        if lo == hi:
            return [], -1
        p = self.target[lo:hi].double().cpu().numpy()
        q = self.draft[lo:hi].double().cpu().numpy() if self.drawn else None
        return S.verify(p, q, self.tokens[lo:hi], self.parents[lo:hi], self.coins[lo:hi].astype(float), float(self.picks[b]),
                        self.depth)

    def check(self, bit=0, skipped=()):
        assert int(self.status.item()) == bit
        accepted, count, following = (x.cpu().numpy() for x in (self.accepted, self.count, self.next))
        lengths = []
        for b in range(self.B):
            if b in skipped:
                assert (accepted[b] == -5).all() and count[b] == -5 and following[b] == -5
                continue
            path, x = self.want(b)
            assert count[b] == len(path) and list(accepted[b]) == path + [-1] * (self.depth - len(path)), b
            assert following[b] == x, b
            lengths.append(len(path))
        return lengths


NODES = [5, 1, 0, 3, 24, 8, 2]


@pytest.mark.parametrize("probs", ["f32", "bf16"])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("vocab", [1, 2, 31, 97, 128, 1000, 4097, 32000, 50257])
def test_paths_and_tokens(vocab, drawn, probs):
    for seed in range(3):
        Batch(NODES, vocab, drawn, probs, seed=seed + vocab).to_device().call().check()


@pytest.mark.parametrize("drawn", [True, False])
def test_long_chains_and_wide_trees(drawn):
    lengths = Batch([60, 200, 4096], 301, drawn, seed=1, chain=True, sharp=0.1).to_device().call().check()
    assert max(lengths) > 1 or not drawn
    Batch([300, 61, 1000], 301, drawn, seed=2).to_device().call().check()


@pytest.mark.parametrize("pad, shift", [(0, 0), (3, 0), (0, 1), (4, 4), (5, 3)])
@pytest.mark.parametrize("probs", ["f32", "bf16"])
def test_rows_apart_and_unaligned(probs, pad, shift):
    Batch(NODES, 1001, True, probs, seed=3, pad=pad, shift=shift).to_device().call().check()
    Batch(NODES, 1000, False, probs, seed=4, pad=pad, shift=shift).to_device().call().check()


def test_a_path_ends_at_the_room_for_it():
    for depth in (1, 2, 3, 40):
        for drawn in (True, False):
            b = Batch([30, 7, 1], 40, drawn, seed=5, chain=True, depth=depth, sharp=0.3)
            b.coins[:] = 0.0 if drawn else b.coins
            lengths = b.to_device().call().check()
            if drawn:
                assert lengths == [min(30, depth), min(7, depth), 1]


def single(target, draft, tokens, parents, coins, pick, depth=None):
    """One request of given rows: (path, next token, status)."""
    n = len(tokens)
    t = torch.tensor(target, dtype=torch.float32, device="cuda")
    q = None if draft is None else torch.tensor(draft, dtype=torch.float32, device="cuda")
    accepted = torch.full((1, depth or n), -5, dtype=torch.int32, device="cuda")
    count, following = S.i32([-5]), S.i32([-5])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    wf.wf_verify_drafts(accepted, count, following, t, q, S.i32(tokens), S.i32(parents), S.i32([0, n]), n,
                        torch.tensor(coins, dtype=torch.float32, device="cuda"),
                        torch.tensor([pick], dtype=torch.float32, device="cuda"), dev_status=st)
    c = int(count.item())
    return accepted[0, :max(c, 0)].tolist(), int(following.item()), int(st.item())


def test_at_the_borders():
    """Dyadic numbers: a coin or a pick that lies exactly on a border is not below it."""
    p, q = [0.25, 0.25, 0.5], [0.5, 0.25, 0.25]
    for coin, path in ((0.5, [0]), (0.5 - 2 ** -25, [0, 1])):
        assert single([p, p], [q, q], [9, 0], [-1, 0], [0, coin], 0.9)[0] == path
    for pick, x in ((0.0, 0), (0.25, 1), (0.25 - 2 ** -26, 0), (0.5, 2), (1 - 2 ** -24, 2)):
        assert single([p], None, [0], [-1], [0], pick) == ([0], x, 0)
    # rejected: what is left is (0, 0, 1/4)
    assert single([p, p], [q, q], [9, 0], [-1, 0], [0, 0.75], 0.0) == ([0], 2, 0)
    # fixed candidates: 0 rejected leaves 3/4, of which 1 takes a third
    assert single([p] * 3, None, [9, 0, 1], [-1, 0, 0], [0, 0.25, 0.34], 0.0) == ([0], 2, 0)
    assert single([p] * 3, None, [9, 0, 1], [-1, 0, 0], [0, 0.25, 0.33], 0.0) == ([0, 2], 0, 0)


def test_one_hot_targets_are_greedy():
    eye = np.eye(7).tolist()
    rows = [eye[3], eye[5], eye[1], eye[2]]
    q = [[1 / 7] * 7] * 4
    for draft in (None, q):
        assert single(rows, draft, [0, 3, 5, 6], [-1, 0, 1, 2], [0, 0.99, 0.99, 0.0], 0.99) == ([0, 1, 2], 1, 0)
        assert single(rows, draft, [0, 4, 3, 6], [-1, 0, 0, 2], [0, 0.0, 0.99, 0.0], 0.0) == ([0, 2], 1, 0)


def test_the_same_token_twice():
    p = [0.5, 0.25, 0.25]
    # the second copy has nothing left, and takes nothing off what is left
    assert single([p] * 4, None, [0, 0, 0, 1], [-1, 0, 0, 0], [0, 0.5, 0.0, 0.49], 0.0) == ([0, 3], 0, 0)
    assert single([p] * 4, None, [0, 0, 0, 1], [-1, 0, 0, 0], [0, 0.5, 0.0, 0.51], 0.0) == ([0], 2, 0)


def test_target_and_draft_alike():
    """Nothing is left of the target where a draft is rejected all the same: its own row is drawn from."""
    p = [0.25, 0.25, 0.5]
    assert single([p, p], [p, p], [0, 2], [-1, 0], [0, 1 - 2 ** -24], 0.0)[0] == [0, 1]
    assert single([p] * 3, [p] * 3, [0, 2, 1], [-1, 0, 0], [0, 1.0, 0.5], 0.3) == ([0], 1, 0)


def test_values_that_are_no_probabilities():
    nan, inf = float("nan"), float("inf")
    bad = wf.WF_DEV_BAD_PROBS
    assert single([[nan, -1.0, 0.5, 0.0]], None, [0], [-1], [0], 0.0) == ([0], 2, 0)
    assert single([[0.5, nan, 0.5]] * 2, [[0.5, 0.5, 0.0]] * 2, [0, 1], [-1, 0], [0, 0.0], 0.0) == ([0], 2, 0)
    assert single([[0.5, 0.0, 0.5]] * 2, [[nan, 1.0, 0.0]] * 2, [0, 1], [-1, 0], [0, 0.0], 0.0) == ([0], 0, 0)
    assert single([[0.25, inf, 0.5]] * 2, [[0.5, 0.25, 0.25]] * 2, [0, 0], [-1, 0], [0, 0.9], 0.5) == ([0], -1, bad)
    for row in ([0.0] * 3, [nan] * 3, [0.5, inf, 0.0], [-1.0, -2.0, 0.0]):
        assert single([row], None, [0], [-1], [0], 0.5) == ([0], -1, bad)
        assert single([row] * 3, [row] * 3, [0, 1, 1], [-1, 0, 0], [0, 1.0, 1.0], 0.5) == ([0], -1, bad)


def test_sums_at_the_end_of_the_range():
    """Sums so small that a threshold rounds up to them, and so large that they only just stay finite."""
    tiny = 2.0 ** -149
    for pick in (0.0, 0.4, 0.6, 1 - 2 ** -24):
        assert single([[0.0, tiny, 0.0]], None, [0], [-1], [0], pick) == ([0], 1, 0)
        assert single([[0.0] * 600 + [tiny] + [0.0] * 5000], None, [0], [-1], [0], pick) == ([0], 600, 0)
    assert single([[0.0, 3e38, 1.0]], None, [0], [-1], [0], 0.9) == ([0], 1, 0)
    assert single([[0.0, 3e38, 3e38]], None, [0], [-1], [0], 0.9) == ([0], -1, wf.WF_DEV_BAD_PROBS)


def test_bad_requests_are_left_out():
    def batch():
        b = Batch([4, 6, 3], 100, True, seed=8)
        return b

    b = batch()
    b.parents[b.cu[1] + 2] = 2
    b.to_device().call().check(wf.WF_DEV_BAD_NODE, skipped=(1,))
    b = batch()
    b.parents[b.cu[1] + 2] = -1
    b.to_device().call().check(wf.WF_DEV_BAD_NODE, skipped=(1,))
    for token in (-1, 100):
        b = batch()
        b.tokens[b.cu[1] + 5] = token
        b.to_device().call().check(wf.WF_DEV_BAD_NODE, skipped=(1,))
        b = batch()
        b.tokens[b.cu[1]] = token                       # the root's is not looked at
        b.to_device().call().check()
    for pick in (1.0, -0.1, float("nan")):
        b = batch()
        b.picks[2] = pick
        b.to_device().call().check(wf.WF_DEV_BAD_PROBS, skipped=(2,))
    b = batch().to_device()
    b.d["cu"][1:3] = torch.tensor([13, 10], dtype=torch.int32)    # past the rows, then backwards
    b.call()
    assert int(b.status.item()) == wf.WF_DEV_BAD_SEQLEN
    assert (b.count[:2].cpu() == -5).all() and (b.accepted[:2].cpu() == -5).all() and int(b.count[2].item()) > 0


def test_tokens_are_distributed_as_the_target():
    """Many requests with one row: the first token after the root follows p, whatever was drafted.  With N draws the
    frequency of a token of probability p lies within 5 sqrt(p (1 - p) / N) of p but for one time in a million."""
    V, N = 6, 1 << 16
    r = np.random.default_rng(0)
    p, q = r.dirichlet(np.ones(V)), r.dirichlet(np.ones(V))
    f32 = lambda x: torch.from_numpy(x.astype(np.float32)).cuda()   # noqa: E731
    for drawn, kids in ((True, 1), (True, 3), (False, 3)):
        n = kids + 1
        T = N * n
        target, draft = f32(p).expand(T, V).contiguous(), f32(q).expand(T, V).contiguous()
        tokens = torch.from_numpy(r.choice(V, T, p=q) if drawn else np.tile([0, 3, 1, 4], N)).int().cuda()
        parents = S.i32(np.tile([-1] + [0] * kids, N))
        accepted = torch.zeros((N, 2), dtype=torch.int32, device="cuda")
        count, following = (torch.zeros(N, dtype=torch.int32, device="cuda") for _ in range(2))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        wf.wf_verify_drafts(accepted, count, following, target, draft if drawn else None, tokens, parents,
                            S.i32(np.arange(N + 1) * n), n, f32(r.random(T)), f32(r.random(N) * (1 - 2 ** -24)), dev_status=st)
        first = torch.where(count > 1, tokens.view(N, n).gather(1, accepted[:, 1:].clamp(min=0).long())[:, 0], following)
        freq = torch.bincount(first.long(), minlength=V).double().cpu().numpy() / N
        assert int(st.item()) == 0
        assert (np.abs(freq - p) < 5 * np.sqrt(p * (1 - p) / N)).all(), (drawn, kids, freq, p)
        assert 0.1 < float((count > 1).double().mean()) < 0.999


def test_rows_past_32_bits_of_offset():
    V, T = 70001, 40000                                # 2.8e9 elements
    target = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    target[T - 2, 69990] = 1.0
    target[T - 1, 70000] = 1.0
    accepted, count, following = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), S.i32([0, 0]), S.i32([0, 0])
    tokens = torch.full((T,), 69990, dtype=torch.int32, device="cuda")
    cu, st = S.i32([T - 2, T, T]), torch.zeros(1, dtype=torch.int32, device="cuda")
    wf.wf_verify_drafts(accepted, count, following, target, None, tokens, None, cu, 2, torch.zeros(T, device="cuda"),
                        torch.zeros(2, device="cuda"), dev_status=st)
    assert accepted.tolist() == [[0, 1], [-1, -1]] and count.tolist() == [2, 0] and following.tolist() == [70000, -1]
    assert int(st.item()) == 0


def test_in_a_graph_and_beside_another_stream():
    a, b = Batch(NODES, 5000, True, seed=10).to_device(), Batch([9] * 40, 3001, False, "bf16", seed=11).to_device()
    a.call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        a.call()
    for x in (a.accepted, a.count, a.next):
        x.fill_(-5)
    g.replay()
    b.call(stream=side)
    torch.cuda.synchronize()
    a.check()
    b.check()

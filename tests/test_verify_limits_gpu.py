"""wf_verify_drafts where numbers lie next to their borders."""
import numpy as np
import pytest
import torch

from paged_kv_cache_wf_gb300 import binding as wf
from tests import _step as S
from tests.test_verify_gpu import single

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_wf_gb300 import build
    build.build()


U = 2.0 ** -48     # a step of the smaller number in a sum's pair (1, 2^-25)


def near(row, pick, x):
    """Whether x has a weight and the threshold lies in its part of the running sum, up to 2^-44 of the whole."""
    up = np.cumsum(np.asarray(row, np.longdouble))
    at = np.longdouble(pick) * up[-1]
    return row[x] > 0 and up[x] - row[x] <= at + up[-1] * 2.0 ** -44 and up[x] >= at - up[-1] * 2.0 ** -44


def sparse(vocab, items):
    row = np.zeros(vocab)
    for x, w in items:
        row[x] = np.float32(w)
    return row


HALF = [(0, 1), (1, 2.0 ** -25)]
ROWS = {
    # Weights of parts of a step, each lost where they are added one by one and not where they are added to one another
    # first, and a tail that makes half of the whole one of the two sums.  Slices of 1024 tokens, four of them a lane:
    # the second lane's sum is the larger one as the lanes add it up.
    f"slices {a}": sparse(16384, HALF + [(4096, a * U), (5120, a * U), (6144, a * U), (8192, 1), (8193, 2.0 ** -25)])
    for a in (0.3, 0.35, 0.4, 0.45)}
# The same of lanes of four tokens with one that has no weight before the one that is looked in.
for i, (parts, tail, more) in enumerate([((0.45, 0.3, 0.6, 0.7, 0.74), 28, 1), ((0.74, 0.4, 0.45, 0.45, 0.7, 0.6), 40, 3),
                                         ((0.45, 0.6, 0.7), 20, 0), ((0.74, 0.4, 0.74, 0.3, 0.6, 0.74), 40, 2),
                                         ((0.4, 0.3, 0.74, 0.4, 0.74), 36, 2)]):
    ROWS[f"lanes {i}"] = sparse(200, HALF + [(4 * k + 4, a * U) for k, a in enumerate(parts)] +
                                [(tail, 1), (tail + 1, 2.0 ** -25), (tail + 2, more * U)])


@pytest.mark.parametrize("name", list(ROWS))
def test_a_threshold_between_two_roundings_of_a_sum(name):
    row = ROWS[name]
    path, x, status = single([row.tolist()], None, [0], [-1], [0], 0.5)
    assert (path, status) == ([0], 0) and 0 <= x < len(row) and near(row, 0.5, x), x


@pytest.mark.parametrize("p0, p2, q0, q2", [
    (0.4157509207725525, 0.8542814254760742, 0.3601817488670349, 0.7555696964263916),
    (0.36879801750183105, 0.8342269659042358, 0.32532966136932373, 0.7440820932388306),
    (0.45207345485687256, 0.8837578296661377, 0.3929266035556793, 0.7923756837844849)])
def test_a_weight_that_is_only_a_rounding_error(p0, p2, q0, q2):
    """Two rejected children leave p - c q, c = 1 + (p0 - q0) + (p2 - q2): above 0 for token 0 alone, by 2^-27 or so, where p0 is
    the rounded product."""
    p, q = [p0, 0.0, p2], [q0, 0.25, q2]
    assert single([p] * 3, [q] * 3, [0, 1, 1], [-1, 0, 0], [0, 0.5, 0.5], 0.3) == ([0], 0, 0)


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("vocab, weight", [((1 << 26) - 5, 0.1), ((1 << 25) + 3, 0.7234567), ((1 << 26) - 64, 1 / 3)])
def test_sums_of_many_equal_tokens(vocab, weight, drawn):
    """One row of a long vocabulary in a batch that leaves it a single CTA: 2^17 and more tokens a thread, whose additions round
    alike.  With equal weights the next token is floor(pick vocab); sums off by 2^-40 move that by 2^-14 of a token."""
    B = 700
    target = torch.full((1, vocab), weight, dtype=torch.float32, device="cuda")
    draft = torch.zeros_like(target) if drawn else None
    accepted, count, following = torch.full((B, 1), -5, dtype=torch.int32, device="cuda"), S.i32([-5] * B), S.i32([-5] * B)
    for pick in (0.3, 0.41, 0.77, 0.93):
        pick = float(np.float32(pick))
        at = np.longdouble(pick) * vocab
        assert 0.01 < at - np.floor(at) < 0.99
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        wf.wf_verify_drafts(accepted, count, following, target, draft, S.i32([0]), None, S.i32([0] * 70 + [1] * (B - 69)), 1,
                            torch.zeros(1, device="cuda"), torch.full((B,), pick, device="cuda"), dev_status=st)
        assert int(st.item()) == 0 and int(following[69].item()) == int(np.floor(at)), (pick, int(following[69].item()) - int(np.floor(at)))
        assert following.sum().item() == int(np.floor(at)) - (B - 1) and count.sum().item() == 1


class Rows:
    """Trees over a long vocabulary, made on the GPU; `some` of the requests are looked at in float64."""

    def __init__(self, B, vocab, drawn, probs, seed, some=10):
        r = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.drawn = B, drawn
        self.nodes = r.integers(0, 4, B)
        self.nodes[:some] = r.integers(3, 8, some)
        self.cu = np.concatenate([[0], np.cumsum(self.nodes)])
        T, kind = int(self.cu[-1]), torch.float32 if probs == "f32" else torch.bfloat16
        self.target, self.draft = (torch.empty((T, vocab), dtype=kind, device="cuda") for _ in range(2))
        for at in range(0, T, 64):
            x = 2.5 * torch.randn((min(64, T - at), vocab), generator=gen, device="cuda")
            self.target[at:at + 64] = torch.softmax(x, -1)
            self.draft[at:at + 64] = torch.softmax(x + 1.2 * torch.randn(x.shape, generator=gen, device="cuda"), -1)
        self.parents = np.array([-1 if i == 0 else r.integers(max(0, i - 3), i) for n in self.nodes for i in range(n)])
        up = torch.from_numpy(np.repeat(self.cu[:-1], self.nodes) + np.maximum(self.parents, 0)).cuda()
        rows = self.draft[up] if drawn else self.target[up]
        self.tokens = torch.multinomial(rows.float(), 1, generator=gen)[:, 0].int()
        self.coins, self.picks = r.random(T).astype(np.float32), r.random(B).astype(np.float32)
        # (a draw that rounds up to 1 is none)
        self.coins, self.picks = (np.minimum(x, np.float32(1 - 2.0 ** -24)) for x in (self.coins, self.picks))
        self.some = np.concatenate([np.arange(some), r.integers(some, B, 4), [B - 1]])

    def check(self):
        depth = 8
        accepted = torch.full((self.B, depth), -5, dtype=torch.int32, device="cuda")
        count, following = S.i32([-5] * self.B), S.i32([-5] * self.B)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        draft = self.draft if self.drawn else None
        wf.wf_verify_drafts(accepted, count, following, self.target, draft, self.tokens, S.i32(self.parents), S.i32(self.cu),
                            int(self.nodes.max()), torch.from_numpy(self.coins).cuda(), torch.from_numpy(self.picks).cuda(),
                            dev_status=st)
        assert int(st.item()) == 0
        path, count, following, tokens = (x.cpu().numpy() for x in (accepted, count, following, self.tokens))
        rejected = 0
        for b in self.some:
            lo, hi = self.cu[b], self.cu[b + 1]
            if lo == hi:
                assert count[b] == 0 and following[b] == -1
                continue
            p, q = (x[lo:hi].double().cpu().numpy() for x in (self.target, self.draft))
            want, x = S.verify(p, q if self.drawn else None, tokens[lo:hi], self.parents[lo:hi], self.coins[lo:hi].astype(float),
                               float(self.picks[b]), depth)
            assert list(path[b][:count[b]]) == want and (path[b][count[b]:] == -1).all() and following[b] == x, b
            rejected += len(want) < hi - lo
        assert rejected > 0
        live = self.nodes > 0
        assert (following[live] >= 0).all() and (following[live] < self.target.shape[1]).all() and (count[~live] == 0).all()


# Clusters of 16, 8, 4, 2 CTAs and single ones, whose slices of a row are 1024 to 16384 tokens.
@pytest.mark.parametrize("probs", ["f32", "bf16"])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("B, vocab", [(19, 128000), (70, 100003), (160, 128000), (231, 100003), (300, 128000), (400, 100003),
                                      (600, 128000), (700, 50257)])
def test_batches_of_every_cluster_size(B, vocab, drawn, probs):
    Rows(B, vocab, drawn, probs, seed=B + vocab).check()

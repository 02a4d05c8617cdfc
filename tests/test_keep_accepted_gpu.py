"""wf_keep_accepted: rows of the accepted path, byte for byte, against numpy."""
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


class Kept:
    def __init__(self, cached, drafted, H_kv, D, P, pool, depth, seed=0, counts=None):
        r = np.random.default_rng(seed)
        self.cached, self.drafted, self.P = np.asarray(cached), np.asarray(drafted), P
        self.B = len(cached)
        self.lens = (self.cached + self.drafted).astype(np.int32)
        need = -(-self.lens // P)
        self.N = int(need.sum()) + 1
        ids = r.permutation(self.N)
        self.table = np.full((self.B, max(1, int(need.max()))), ids[-1], np.int32)
        at = 0
        for b in range(self.B):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
        self.cu = np.concatenate([[0], np.cumsum(self.drafted)]).astype(np.int32)
        top = np.minimum(depth, self.drafted)
        self.count = (r.integers(0, top + 1) if counts is None else np.asarray(counts)).astype(np.int32)
        self.path = np.full((self.B, depth), -7, np.int32)
        for b in range(self.B):
            self.path[b, :self.count[b]] = np.sort(r.permutation(int(self.drafted[b]))[:self.count[b]])
        size = {"f32": 4, "bf16": 2, "fp8": 1}[pool]
        raw = r.integers(0, 256, (2, self.N, P, H_kv, D * size)).astype(np.uint8)   # any bytes, NaN patterns included
        self.raw = raw
        self.kp, self.vp = (torch.from_numpy(x).cuda().view(R.DT[pool]).view(self.N, P, H_kv, D) for x in raw)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.new = torch.full((self.B,), -9, dtype=torch.int32, device="cuda")

    def args(self):
        return [torch.from_numpy(x).cuda() for x in (self.table, self.lens, self.cu, self.path, self.count)]

    def run(self, new=True):
        wf.wf_keep_accepted(self.kp, self.vp, *self.args(), new_seq_lens=self.new if new else None,
                            dev_status=self.status)

    def check(self, skip=(), skip_rows=()):
        want = self.raw.copy()
        for b in range(self.B):
            if b in skip:
                continue
            for j in range(int(self.count[b])):
                if (b, j) in skip_rows:
                    continue
                f, t = int(self.cached[b] + self.path[b, j]), int(self.cached[b] + j)
                want[:, self.table[b, t // self.P], t % self.P] = self.raw[:, self.table[b, f // self.P], f % self.P]
        for i, pool in enumerate((self.kp, self.vp)):
            got = pool.contiguous().view(torch.uint8).cpu().numpy().reshape(want[i].shape)
            assert np.array_equal(got, want[i])
        new = np.where(np.isin(np.arange(self.B), list(skip)), -9, self.cached + self.count)
        return new


CASES = {
    "one request": lambda: Kept([700], [8], 8, 128, 16, "bf16", 4, counts=[4]),
    "ragged": lambda: Kept([0, 5, 100, 33, 16], [1, 9, 64, 0, 31], 8, 128, 16, "bf16", 12, seed=1),
    "everything kept": lambda: Kept([3, 17], [20, 40], 2, 64, 16, "bf16", 40, seed=2, counts=[20, 40]),
    "nothing kept": lambda: Kept([3, 17], [20, 40], 2, 64, 16, "bf16", 40, seed=2, counts=[0, 0]),
    "long paths": lambda: Kept([3, 0], [300, 200], 2, 64, 16, "f32", 260, seed=3, counts=[260, 131]),
    "one kv head of codes": lambda: Kept([13, 2, 0], [24, 24, 3], 1, 64, 16, "fp8", 8, seed=4),
    "wide rows": lambda: Kept([13, 2], [24, 24], 20, 128, 16, "f32", 9, seed=5),
    "odd blocks": lambda: Kept([13, 2, 50], [24, 24, 61], 5, 128, 7, "bf16", 9, seed=6),
    "blocks of one": lambda: Kept([4, 1], [6, 9], 2, 64, 1, "bf16", 5, seed=7),
    "a batch": lambda: Kept(np.arange(231) % 97, 1 + np.arange(231) % 61, 8, 128, 16, "bf16", 9, seed=8),
}


@pytest.mark.parametrize("name", list(CASES))
def test_rows_move_as_if_all_were_read_first(name):
    s = CASES[name]()
    s.run()
    assert np.array_equal(s.new.cpu().numpy(), s.check())
    assert wf.wf_device_status_fetch(s.status) == 0


def test_without_new_lengths():
    s = CASES["ragged"]()
    s.run(new=False)
    s.check()
    assert (s.new == -9).all()


def test_path_of_depth_zero():
    s = Kept([3, 5], [4, 4], 2, 64, 16, "bf16", 1, counts=[0, 0])
    s.path = np.zeros((2, 0), np.int32)
    s.run()
    assert np.array_equal(s.new.cpu().numpy(), s.check())


@pytest.mark.parametrize("path", [[2, 2, 5], [3, 1, 2], [-1, 0, 1], [0, 1, 9], [0, 2 ** 31 - 1, 3], [-2 ** 31, 0, 1]])
def test_bad_paths_skip_the_request(path):
    s = Kept([10, 20, 30], [9, 9, 9], 2, 64, 16, "bf16", 3, seed=9, counts=[3, 3, 3])
    s.path[1] = path
    s.run()
    assert np.array_equal(s.new.cpu().numpy(), s.check(skip=(1,)))
    assert wf.wf_device_status_fetch(s.status) == wf.WF_DEV_BAD_NODE


@pytest.mark.parametrize("count", [-1, 4, 100, 2 ** 31 - 1, -2 ** 31])
def test_bad_counts_skip_the_request(count):
    s = Kept([10, 20, 30], [9, 9, 9], 2, 64, 16, "bf16", 3, seed=9, counts=[3, 3, 3])
    s.count[1] = count
    s.run()
    new = s.check(skip=(1,))
    assert np.array_equal(s.new.cpu().numpy(), new)
    assert wf.wf_device_status_fetch(s.status) == wf.WF_DEV_BAD_NODE


def test_count_above_the_drafts_skips_the_request():
    s = Kept([10, 20], [2, 9], 2, 64, 16, "bf16", 3, seed=9, counts=[2, 3])
    s.count[0], s.path[0] = 3, [0, 1, 2]
    s.run()
    s.check(skip=(0,))
    assert wf.wf_device_status_fetch(s.status) == wf.WF_DEV_BAD_NODE


@pytest.mark.parametrize("length", [8, -1, 1 << 20, 2 ** 31 - 1, -2 ** 31])
def test_bad_lengths_skip_the_request(length):
    s = Kept([10, 20, 30], [9, 9, 9], 2, 64, 16, "bf16", 3, seed=9, counts=[3, 3, 3])
    s.lens[1] = length
    s.run()
    assert np.array_equal(s.new.cpu().numpy(), s.check(skip=(1,)))
    assert wf.wf_device_status_fetch(s.status) == wf.WF_DEV_BAD_SEQLEN


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_bad_blocks_are_not_touched(bad):
    s = Kept([14, 40], [9, 9], 2, 64, 16, "bf16", 3, seed=9, counts=[3, 3])
    s.path[0] = [1, 2, 6]                 # positions 15, 16, 20 -> 14, 15, 16; block 1 holds 16 ..
    s.table[0, 1] = bad
    s.run()
    s.check(skip_rows=((0, 1), (0, 2)))
    assert wf.wf_device_status_fetch(s.status) == wf.WF_DEV_BAD_BLOCK


def test_captured():
    s = CASES["ragged"]()
    args = s.args()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        wf.wf_keep_accepted(s.kp, s.vp, *args, new_seq_lens=s.new, dev_status=s.status)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(s.new.cpu().numpy(), s.check())

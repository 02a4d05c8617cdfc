"""wf_build_step and wf_trim_blocks against a step built token by token on the host."""
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


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Built:
    """A call of wf_build_step over its own buffers, outputs filled with what no step holds."""

    def __init__(self, q, new, rows, depths=None, in_place=False, free=None, num_free=None):
        self.q, self.new, self.rows, self.depths = q, np.asarray(new, np.int64), rows, depths
        self.table, self.lens, self.d_new = S.i32(q.table), S.i32(q.lens), S.i32(new)
        self.free = S.i32(q.free if free is None else free)
        self.num = S.i32([q.num_free if num_free is None else num_free])
        self.out_lens = self.lens if in_place else torch.full_like(self.lens, -5)
        self.out_num = self.num if in_place else torch.full_like(self.num, -5)
        self.cu = torch.full((q.B + 1,), -5, dtype=torch.int32, device="cuda")
        self.slots = torch.full((rows,), -5, dtype=torch.int64, device="cuda")
        self.positions = torch.full((rows,), -5, dtype=torch.int32, device="cuda")
        self.d_depths = None if depths is None else S.i32(depths)
        self.status = status()

    def call(self, stream=None):
        wf.wf_build_step(self.table, self.lens, self.d_new, self.free, self.num, self.out_lens, self.out_num, self.cu,
                         self.slots, self.positions, self.q.block, depths=self.d_depths, dev_status=self.status,
                         stream=stream)
        return self

    def got(self):
        return [x.cpu().numpy() for x in (self.table, self.out_lens, self.out_num, self.cu, self.slots, self.positions)]

    def check(self):
        q = self.q
        want = S.build(q.table, q.lens, self.new, q.free, q.num_free, self.rows, q.block, self.depths)
        for name, a, b in zip(("table", "lens", "left", "offsets", "slots", "positions"), self.got(), want):
            assert np.array_equal(a.reshape(-1), np.asarray(b).reshape(-1)), name
        assert int(self.status.item()) == 0

    def check_refused(self, bit):
        q = self.q
        table, lens, num, cu, slots, positions = self.got()
        assert int(self.status.item()) == bit
        assert np.array_equal(table, q.table) and np.array_equal(lens, self.lens.cpu().numpy())
        assert num[0] == int(self.num.item()) and not cu.any() and (slots == -1).all() and not positions.any()


CASES = {
    "one_token": ([700], [1], 16, 3),
    "none": ([5, 0, 16], [0, 0, 0], 16, 2),
    "first_token": ([0], [1], 16, 1),
    "fills_a_block": ([15, 31, 16], [1, 1, 16], 16, 4),
    "crosses": ([15, 30, 1], [2, 40, 100], 16, 12),
    "blocks_of_one": ([3, 0, 9], [4, 1, 0], 1, 7),
    "odd_blocks": ([3, 0, 9, 700, 13], [4, 1, 0, 33, 8], 7, 20),
    "large_blocks": ([1023, 1024, 5], [1, 2000, 1019], 1024, 9),
    "new_prompts": ([0] * 9, [2048, 1, 0, 17, 16, 15, 300, 1, 2], 16, 200),
    "decode_231": (list(range(1, 232)), [1] * 231, 16, 60),
    "mixed": (list(np.arange(128) * 61 % 8192), [1500 if i % 16 == 0 else i % 9 for i in range(128)], 16, 2000),
    "many_requests": (list(np.arange(5000) % 40), list(np.arange(5000) % 3), 16, 5200),
    "all_requests": ([1] * 16384, [1] * 16384, 2, 5),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_build(name, in_place):
    lens, new, block, spare = CASES[name]
    q = S.Requests(lens, block, spare, M=max(1, max(-(-(a + n) // block) for a, n in zip(lens, new))), seed=len(lens))
    for extra in (0, 5):
        Built(q, new, int(np.sum(new)) + extra, in_place=in_place).call().check()


def test_depths_replace_the_place_in_the_request():
    q = S.Requests([100, 37, 5], 16, 8, M=20, seed=2)
    new = [6, 0, 20]
    depths = np.random.default_rng(0).integers(0, 7, 29)
    Built(q, new, 29, depths=depths).call().check()


def test_no_requests():
    q = S.Requests([], 16, 3, M=4)
    q.table = q.table.reshape(0, 4)
    Built(q, [], 6).call().check()


def test_exactly_the_free_blocks_and_one_too_few():
    q = S.Requests([16, 32, 7], 16, 5, M=9, seed=3)
    Built(q, [16, 33, 9], 60).call().check()                         # 1 + 3 + 0 blocks, and
    Built(q, [17, 33, 9], 60).call().check()                         # all 5
    Built(q, [17, 33, 10], 60).call().check_refused(wf.WF_DEV_NO_BLOCKS)
    Built(q, [17, 33, 10], 60, in_place=True).call().check_refused(wf.WF_DEV_NO_BLOCKS)


def test_a_step_that_cannot_be_built_changes_nothing():
    def requests():
        return S.Requests([16, 33, 7], 16, 6, M=5, seed=4)

    good = [2, 3, 4]
    bad_len = wf.WF_DEV_BAD_SEQLEN
    Built(requests(), good, 9).call().check()
    Built(requests(), good, 8).call().check_refused(bad_len)                       # more rows than there is room for
    Built(requests(), [2, -1, 4], 20).call().check_refused(bad_len)
    Built(requests(), [2, 48, 4], 60).call().check_refused(bad_len)                # 81 tokens of 5 blocks
    Built(requests(), [2, 2 ** 31 - 1, 4], 60).call().check_refused(bad_len)
    Built(requests(), [2 ** 31 - 1] * 3, 60).call().check_refused(bad_len)
    q = requests()
    q.lens = np.array([16, -1, 7])
    Built(q, good, 20).call().check_refused(bad_len)
    q = requests()
    q.table[1, 2] = q.N                                                            # the block that is partly filled
    Built(q, good, 20).call().check_refused(wf.WF_DEV_BAD_BLOCK)
    q = requests()
    q.table[1, 2] = -1
    Built(q, [2, 0, 4], 20).call().check()                                         # is not touched
    q = requests()
    q.free[4] = -1
    Built(q, [2, 40, 4], 60).call().check_refused(wf.WF_DEV_BAD_BLOCK)
    Built(q, [2, 3, 4], 60).call().check()                                         # takes the one above it only
    for num in (-1, q.N + 1):
        Built(requests(), good, 20, num_free=num).call().check_refused(wf.WF_DEV_BAD_BLOCK | (wf.WF_DEV_NO_BLOCKS if num < 0 else 0))


def trimmed(q, kept, num_free=None, in_place=False):
    free, num = S.i32(q.free), S.i32([q.num_free if num_free is None else num_free])
    left, st = num if in_place else torch.full_like(num, -5), status()
    wf.wf_trim_blocks(S.i32(q.table), S.i32(q.lens), S.i32(kept), free, num, left, q.block, dev_status=st)
    return free.cpu().numpy(), int(left.item()), int(st.item())


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens, kept, block", [
    ([700], [690], 16), ([700], [0], 16), ([16, 17, 0, 1], [16, 16, 0, 0], 16), ([5, 9], [4, 9], 1),
    (list(range(231)), [max(0, i - i % 61) for i in range(231)], 16), ([8192, 4096, 3], [1, 0, 3], 7),
    (list(np.arange(4000) % 90), list(np.arange(4000) % 90 // 2), 16), ([2] * 16384, [i % 3 for i in range(16384)], 1)])
def test_trim(lens, kept, block, in_place):
    q = S.Requests(lens, block, 4, seed=1)
    free, left, st = trimmed(q, kept, in_place=in_place)
    want, n = S.trim(q.table, q.lens, kept, q.free, q.num_free, block)
    assert st == 0 and left == n and np.array_equal(free, want)


def test_trims_that_cannot_be_done_change_nothing():
    def refused(q, kept, bit, num_free=None):
        free, left, st = trimmed(q, kept, num_free)
        assert st == bit and left == (q.num_free if num_free is None else num_free) and np.array_equal(free, q.free)

    def requests():
        return S.Requests([40, 33, 7], 16, 6, M=5, seed=4)

    refused(requests(), [40, 34, 7], wf.WF_DEV_BAD_SEQLEN)
    refused(requests(), [40, -1, 7], wf.WF_DEV_BAD_SEQLEN)
    q = requests()
    q.lens = np.array([40, 81, 7])
    refused(q, [40, 0, 7], wf.WF_DEV_BAD_SEQLEN)
    q = requests()
    q.table[0, 1] = q.N
    refused(q, [3, 33, 7], wf.WF_DEV_BAD_BLOCK)
    assert trimmed(q, [17, 33, 7])[2] == 0            # the bad one stays
    q.table[0, 1] = -1
    refused(q, [3, 33, 7], wf.WF_DEV_BAD_BLOCK)
    refused(requests(), [0, 0, 0], wf.WF_DEV_BAD_BLOCK, num_free=8)      # more blocks than there are
    refused(requests(), [0, 0, 0], wf.WF_DEV_BAD_BLOCK, num_free=-1)


def test_a_trim_undoes_a_build():
    q = S.Requests([16, 33, 7, 0, 512], 16, 40, M=60, seed=5)
    x = Built(q, [100, 3, 0, 41, 77], 230).call()
    x.check()
    left = torch.zeros_like(x.num)
    wf.wf_trim_blocks(x.table, x.out_lens, x.lens, x.free, x.out_num, left, 16, dev_status=x.status)
    assert int(left.item()) == q.num_free and np.array_equal(x.free.cpu().numpy(), q.free)
    before = x.got()
    x.call().check()
    assert all(np.array_equal(a, b) for a, b in zip(before, x.got()))


def test_as_the_block_manager_does():
    """The same blocks as the host's manager gives, from the same list."""
    N, P, B = 64, 16, 5
    bm = wf.BlockManager(N, P, shuffle_seed=3)
    probe = wf.BlockManager(N, P, shuffle_seed=3)
    order = [int(probe.append(9, P)[0][0]) // P for _ in range(N)]       # the order its list is handed out in
    q = S.Requests([0] * B, P, 0, M=20)
    q.N, q.free, q.num_free = N, np.array(order[::-1]), N
    table, lens = S.i32(q.table), S.i32([0] * B)
    free, num = S.i32(q.free), S.i32([N])
    cu, st = S.i32([0] * (B + 1)), status()
    r = np.random.default_rng(7)
    for _ in range(6):
        new = r.integers(0, 30, B)
        slots, positions = torch.zeros(200, dtype=torch.int64, device="cuda"), S.i32([0] * 200)
        wf.wf_build_step(table, lens, S.i32(new), free, num, lens, num, cu, slots, positions, P, dev_status=st)
        want = np.concatenate([bm.append(b, int(n))[0] for b, n in enumerate(new)])
        assert np.array_equal(slots.cpu().numpy()[:len(want)], want)
        held, host_lens = bm.tables(range(B), 20, -7)
        assert np.array_equal(lens.cpu().numpy(), host_lens) and int(num.item()) == bm.num_free()
        assert np.array_equal(table.cpu().numpy(), held)
    assert int(st.item()) == 0


def test_steps_from_a_graph_update_their_lengths_in_place():
    q = S.Requests([16, 33, 7, 0], 16, 60, M=30, seed=6)
    x = Built(q, [3, 0, 17, 30], 60, in_place=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        x.call()
    lens, left, table = q.lens.copy(), q.num_free, q.table
    for _ in range(4):
        g.replay()
        table, lens, left, cu, slots, positions = S.build(table, lens, x.new, q.free, left, 60, 16)
        got = x.got()
        for a, b in zip(got, (table, lens, left, cu, slots, positions)):
            assert np.array_equal(a.reshape(-1), np.asarray(b).reshape(-1))
    assert int(x.status.item()) == 0


def test_slots_past_32_bits():
    """Block ids whose slots need 64 bits."""
    N = 2 ** 22 + 3
    free = torch.arange(N, dtype=torch.int32, device="cuda")
    table, lens = S.i32([[-7, -7]]), S.i32([0])
    left, cu, st = S.i32([0]), S.i32([0, 0]), status()
    slots, positions = torch.zeros(1025, dtype=torch.int64, device="cuda"), S.i32([0] * 1025)
    wf.wf_build_step(table, lens, S.i32([1025]), free, S.i32([N]), lens, left, cu, slots, positions, 1024, dev_status=st)
    want = np.concatenate([(N - 1) * 1024 + np.arange(1024), [(N - 2) * 1024]])
    assert np.array_equal(slots.cpu().numpy(), want) and int(st.item()) == 0

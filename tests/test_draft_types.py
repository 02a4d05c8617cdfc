"""CPU checks of the draft calls' binding: tensor types that the kernels would misread are refused before the library
is called, and those of its documentation reach it."""
import pytest
import torch

from paged_kv_cache_wf_gb300 import binding as wf

I32, I64 = torch.int32, torch.int64


class Stub:
    """Takes the library's place: notes which call was reached."""

    def __init__(self):
        self.reached = []

    def __getattr__(self, name):
        def call(*args):
            self.reached.append(name)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    stub = Stub()
    monkeypatch.setattr(wf, "_lib", stub)
    return stub


def tree_args(pool=torch.bfloat16, act=torch.bfloat16):
    k = torch.zeros(4, 16, 2, 64).to(pool)
    q = torch.zeros(3, 4, 64).to(act)
    return dict(out=torch.zeros_like(q), q=q, k_pool=k, v_pool=k.clone(), block_tables=torch.zeros(1, 2, dtype=I32),
                seq_lens=torch.full((1,), 9, dtype=I32), cu_q_lens=torch.tensor([0, 3], dtype=I32),
                tree_mask=torch.zeros(3, 1, dtype=I32), max_q_len=3, max_seq_len=32, scale=0.1,
                workspace=torch.zeros(64, dtype=torch.uint8), stream=0)


def keep_args(pool=torch.bfloat16):
    k = torch.zeros(4, 16, 2, 64).to(pool)
    return dict(k_pool=k, v_pool=k.clone(), block_tables=torch.zeros(1, 2, dtype=I32),
                seq_lens=torch.full((1,), 9, dtype=I32), cu_q_lens=torch.tensor([0, 3], dtype=I32),
                accepted=torch.zeros(1, 2, dtype=I32), num_accepted=torch.ones(1, dtype=I32),
                new_seq_lens=torch.zeros(1, dtype=I32), stream=0)


@pytest.mark.parametrize("pool,act", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                      (torch.uint8, torch.bfloat16)])
def test_tree_takes_the_documented_types(lib, pool, act):
    wf.wf_paged_tree_decode(**tree_args(pool, act))
    a = tree_args(pool, act)
    a["tree_mask"] = torch.zeros(3, 1, dtype=torch.uint32)
    wf.wf_paged_tree_decode(**a)
    assert lib.reached == ["wf_paged_tree_decode"] * 2


@pytest.mark.parametrize("pool,act", [(torch.bfloat16, torch.float16), (torch.uint8, torch.float16),
                                      (torch.bfloat16, torch.int16), (torch.uint8, torch.int16),
                                      (torch.float32, torch.int32), (torch.float32, torch.bfloat16),
                                      (torch.bfloat16, torch.float32)])
def test_tree_refuses_queries_of_another_type(lib, pool, act):
    with pytest.raises(ValueError):
        wf.wf_paged_tree_decode(**tree_args(pool, act))
    assert lib.reached == []


@pytest.mark.parametrize("name", ["block_tables", "seq_lens", "cu_q_lens", "tree_mask"])
@pytest.mark.parametrize("dtype", [I64, torch.int16, torch.float32])
def test_tree_refuses_other_integers(lib, name, dtype):
    a = tree_args()
    a[name] = a[name].to(dtype)
    with pytest.raises(ValueError):
        wf.wf_paged_tree_decode(**a)
    assert lib.reached == []


def test_tree_refuses_pools_of_two_types(lib):
    a = tree_args()
    a["v_pool"] = torch.zeros(4, 16, 2, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        wf.wf_paged_tree_decode(**a)
    assert lib.reached == []


@pytest.mark.parametrize("pool", [torch.bfloat16, torch.float32, torch.uint8])
def test_keep_takes_the_documented_types(lib, pool):
    wf.wf_keep_accepted(**keep_args(pool))
    a = keep_args(pool)
    a["new_seq_lens"] = None
    wf.wf_keep_accepted(**a)
    assert lib.reached == ["wf_keep_accepted"] * 2


@pytest.mark.parametrize("k,v", [(torch.bfloat16, torch.uint8), (torch.float32, torch.bfloat16), (torch.uint8, torch.bfloat16),
                                 (torch.bfloat16, torch.float16), (torch.uint8, torch.int8)])
def test_keep_refuses_pools_of_two_types(lib, k, v):
    a = keep_args(k)
    a["v_pool"] = torch.zeros(4, 16, 2, 64).to(v)
    with pytest.raises(ValueError):
        wf.wf_keep_accepted(**a)
    assert lib.reached == []


@pytest.mark.parametrize("name", ["block_tables", "seq_lens", "cu_q_lens", "accepted", "num_accepted", "new_seq_lens"])
@pytest.mark.parametrize("dtype", [I64, torch.int16, torch.float32])
def test_keep_refuses_other_integers(lib, name, dtype):
    a = keep_args()
    a[name] = a[name].to(dtype)
    with pytest.raises(ValueError):
        wf.wf_keep_accepted(**a)
    assert lib.reached == []

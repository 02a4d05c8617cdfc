"""CPU checks of the step calls: what they refuse before any launch."""
import pytest
import torch

from paged_kv_cache_wf_gb300 import binding as wf
from paged_kv_cache_wf_gb300 import build

FAKE = 0x10000   # never dereferenced by calls that are refused
FAR = 1 << 30


@pytest.fixture(scope="module")
def lib():
    build.build()
    return wf.load()


def test_verify_refusals(lib):
    f = lib.wf_verify_drafts
    ok = dict(acc=FAKE, depth=4, num=FAKE, nxt=FAKE, t=FAKE, ts=100, d=FAKE, ds=100, V=100, dt=wf.WF_DTYPE_F32, tok=FAKE,
              par=FAKE, cu=FAKE, coins=FAKE, picks=FAKE, B=0, T=10, mq=5)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["acc"], a["depth"], a["num"], a["nxt"], a["t"], a["ts"], a["d"], a["ds"], a["V"], a["dt"], a["tok"],
                 a["par"], a["cu"], a["coins"], a["picks"], a["B"], a["T"], a["mq"], None, None)

    assert call() == wf.WF_OK
    assert call(acc=None, t=None, tok=None, cu=None) == wf.WF_OK
    for bad in (dict(B=-1), dict(T=-1), dict(mq=-1), dict(depth=0), dict(V=0), dict(V=-5)):
        assert call(**bad) == wf.WF_ERR_INVALID_ARG, bad
    for bad in (dict(dt=wf.WF_DTYPE_FP8_E4M3), dict(dt=7), dict(mq=4097), dict(V=(1 << 28) + 1), dict(B=(1 << 24) + 1)):
        assert call(**bad) == wf.WF_ERR_UNSUPPORTED, bad
    for bad in (dict(acc=None), dict(num=None), dict(nxt=None), dict(t=None), dict(tok=None), dict(cu=None), dict(coins=None),
                dict(picks=None), dict(ts=99), dict(ds=99), dict(ts=(1 << 40) + 1), dict(t=FAKE + 2), dict(d=FAKE + 1),
                dict(acc=FAKE + 2), dict(num=FAKE + 1), dict(nxt=FAKE + 2), dict(tok=FAKE + 2), dict(par=FAKE + 2),
                dict(cu=FAKE + 3), dict(coins=FAKE + 2), dict(picks=FAKE + 1),
                dict(dt=wf.WF_DTYPE_BF16, t=FAKE + 1)):
        assert call(B=2, **bad) == wf.WF_ERR_INVALID_ARG, bad


def test_verify_refuses_outputs_over_inputs_or_one_another(lib):
    at = lambda i: FAKE + i * FAR   # noqa: E731
    ok = dict(acc=at(0), num=at(1), nxt=at(2), t=at(3), d=at(4), tok=at(5), par=at(6), cu=at(7), coins=at(8), picks=at(9))
    last = (9 * 120 + 100) * 4 - 4                       # the last element of the last row
    for bad in (dict(acc=at(3) + last), dict(acc=at(4)), dict(acc=at(5) + 36), dict(acc=at(6) - 28), dict(num=at(1), nxt=at(1) + 4),
                dict(num=at(7) + 8), dict(nxt=at(8) + 36), dict(nxt=at(9) + 4), dict(num=at(0) + 28), dict(nxt=at(5))):
        a = dict(ok, **bad)
        assert lib.wf_verify_drafts(a["acc"], 4, a["num"], a["nxt"], a["t"], 120, a["d"], 120, 100, wf.WF_DTYPE_F32, a["tok"],
                                    a["par"], a["cu"], a["coins"], a["picks"], 2, 10, 5, None, None) == wf.WF_ERR_INVALID_ARG, bad


def test_build_refusals(lib):
    f = lib.wf_build_step
    at = lambda i: FAKE + i * FAR   # noqa: E731
    ok = dict(bt=at(0), M=4, sl=at(1), nl=at(2), fb=at(3), nf=at(4), dp=at(5), ol=at(6), of=at(7), cu=at(8), sm=at(9),
              pos=at(10), B=3, T=10, N=20, P=16)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["bt"], a["M"], a["sl"], a["nl"], a["fb"], a["nf"], a["dp"], a["ol"], a["of"], a["cu"], a["sm"], a["pos"],
                 a["B"], a["T"], a["N"], a["P"], None, None)

    for bad in (dict(B=-1), dict(T=-1), dict(M=0), dict(N=0), dict(P=0), dict(P=1025), dict(fb=None), dict(nf=None),
                dict(of=None), dict(cu=None), dict(bt=None), dict(sl=None), dict(nl=None), dict(ol=None), dict(sm=None),
                dict(pos=None), dict(sm=at(9) + 4), dict(bt=at(0) + 2), dict(dp=at(5) + 1), dict(cu=at(8) + 2),
                # over one another
                dict(ol=at(1) + 4), dict(ol=at(2)), dict(of=at(1)), dict(cu=at(6) + 8), dict(pos=at(9) + 76),
                dict(pos=at(8)), dict(cu=at(8), pos=at(8)), dict(sm=at(5)), dict(bt=at(3) + 76), dict(nf=at(0) + 44),
                dict(ol=at(4)), dict(of=at(6) + 8)):
        assert call(**bad) == wf.WF_ERR_INVALID_ARG, bad
    assert call(B=16385) == wf.WF_ERR_UNSUPPORTED


def test_trim_refusals(lib):
    f = lib.wf_trim_blocks
    at = lambda i: FAKE + i * FAR   # noqa: E731
    ok = dict(bt=at(0), M=4, sl=at(1), kl=at(2), fb=at(3), nf=at(4), of=at(5), B=3, N=20, P=16)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["bt"], a["M"], a["sl"], a["kl"], a["fb"], a["nf"], a["of"], a["B"], a["N"], a["P"], None, None)

    for bad in (dict(B=-1), dict(M=0), dict(N=0), dict(P=0), dict(P=1025), dict(bt=None), dict(sl=None), dict(kl=None),
                dict(fb=None), dict(nf=None), dict(of=None), dict(bt=at(0) + 2), dict(fb=at(3) + 1), dict(of=at(5) + 2),
                dict(fb=at(0) + 44), dict(fb=at(1) - 76), dict(nf=at(3)), dict(of=at(3) + 4), dict(of=at(2) + 8)):
        assert call(**bad) == wf.WF_ERR_INVALID_ARG, bad
    assert call(B=16385) == wf.WF_ERR_UNSUPPORTED


def test_tensors_of_other_types_or_shapes_are_refused(lib):
    i = lambda *n: torch.zeros(n, dtype=torch.int32)   # noqa: E731
    p = torch.zeros(6, 50)
    ok = dict(accepted=i(2, 3), num_accepted=i(2), next_tokens=i(2), target=p, draft=p, tokens=i(6), parents=i(6),
              cu_q_lens=i(3), max_q_len=3, coins=torch.zeros(6), picks=torch.zeros(2))
    for bad in (dict(target=p.half()), dict(draft=p.bfloat16()), dict(draft=p[:5]), dict(target=torch.zeros(50, 6).t()),
                dict(tokens=i(5)), dict(tokens=torch.zeros(6, dtype=torch.int64)), dict(parents=i(7)), dict(coins=i(6)),
                dict(picks=torch.zeros(3)), dict(picks=torch.zeros(2).double()), dict(cu_q_lens=i(2)), dict(next_tokens=i(3)),
                dict(num_accepted=i(1)), dict(accepted=torch.zeros(2, 3))):
        with pytest.raises(ValueError):
            wf.wf_verify_drafts(**dict(ok, **bad))
    step = dict(block_tables=i(2, 4), seq_lens=i(2), new_lens=i(2), free_blocks=i(9), num_free=i(1), new_seq_lens=i(2),
                new_num_free=i(1), cu_q_lens=i(3), slot_mapping=torch.zeros(7, dtype=torch.int64), positions=i(7),
                block_size=16)
    for bad in (dict(slot_mapping=i(7)), dict(positions=i(6)), dict(depths=i(6)), dict(seq_lens=i(3)), dict(cu_q_lens=i(2)),
                dict(new_lens=i(1)), dict(num_free=i(2)), dict(free_blocks=i(3, 3)), dict(new_seq_lens=torch.zeros(2)),
                dict(block_tables=i(4, 2).t())):
        with pytest.raises(ValueError):
            wf.wf_build_step(**dict(step, **bad))
    trim = dict(block_tables=i(2, 4), seq_lens=i(2), kept_lens=i(2), free_blocks=i(9), num_free=i(1), new_num_free=i(1),
                block_size=16)
    for bad in (dict(seq_lens=i(3)), dict(kept_lens=torch.zeros(2)), dict(num_free=i(2)), dict(free_blocks=i(3, 3))):
        with pytest.raises(ValueError):
            wf.wf_trim_blocks(**dict(trim, **bad))

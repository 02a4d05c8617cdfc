"""CPU checks of the draft-verification entry points: what they refuse before any launch."""
import math

import pytest

from paged_kv_cache_wf_gb300 import binding as wf
from paged_kv_cache_wf_gb300 import build

FAKE = 0x10000   # 16-byte aligned, never dereferenced by calls that are refused


@pytest.fixture(scope="module")
def lib():
    build.build()
    return wf.load()


def _desc(N=10, P=16, H=2, D=64, dt=wf.WF_DTYPE_BF16, ks=0.0, vs=0.0):
    return wf.wf_pool_desc(N, P, H, D, dt, ks, vs)


def test_norm_rope_refusals(lib):
    f = lib.wf_qk_norm_rope_and_cache
    ok = dict(qo=FAKE + (1 << 24), q=FAKE, qs=512, k=FAKE, ks=128, v=FAKE, vs=128, qw=FAKE, kw=FAKE, eps=1e-6, cs=FAKE,
              mp=100, rot=64, il=0, pos=FAKE, kp=FAKE, vp=FAKE, sm=FAKE, T=3, Hq=8, d=_desc())

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["qo"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qw"], a["kw"], a["eps"], a["cs"],
                 a["mp"], a["rot"], a["il"], a["pos"], a["kp"], a["vp"], a["sm"], a["T"], a["Hq"], a["d"], None, None)

    assert call(T=0) == wf.WF_OK
    assert call(T=0, q=None, k=None, v=None) == wf.WF_OK
    for bad in (dict(T=-1), dict(Hq=0), dict(Hq=7), dict(rot=-2), dict(rot=66), dict(rot=63), dict(mp=0),
                dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(q=None), dict(k=None), dict(v=None),
                dict(qo=None), dict(kp=None), dict(vp=None), dict(sm=None), dict(cs=None), dict(pos=None),
                dict(q=FAKE + 2), dict(k=FAKE + 8), dict(v=FAKE + 4), dict(qo=FAKE + (1 << 24) + 8),
                dict(qw=FAKE + 2), dict(kw=FAKE + 8), dict(cs=FAKE + 4), dict(pos=FAKE + 2), dict(sm=FAKE + 4),
                dict(qs=511), dict(qs=504 + 4), dict(ks=120), dict(vs=127), dict(ks=132), dict(qs=1 << 41),
                dict(qo=FAKE), dict(qo=FAKE + 3 * 512 * 2 - 16), dict(qo=FAKE - 16)):
        assert call(**bad) == wf.WF_ERR_INVALID_ARG, bad
    assert call(d=_desc(D=96)) == wf.WF_ERR_UNSUPPORTED
    assert call(d=_desc(dt=5)) == wf.WF_ERR_UNSUPPORTED
    assert call(d=_desc(dt=wf.WF_DTYPE_FP8_E4M3, ks=0.0, vs=1.0)) == wf.WF_ERR_INVALID_ARG


def test_tree_refusals(lib):
    f = lib.wf_paged_tree_decode
    d = _desc(N=10, P=16, H=2, D=64)
    need = wf.wf_paged_tree_decode_workspace_size(2, 8, 7, 64, d)
    ok = dict(out=FAKE, q=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, M=4, sl=FAKE, cu=FAKE, tm=FAKE, W=1, B=2, T=10, mq=7,
              msl=64, Hq=8, scale=0.1, d=d, ws=FAKE, wsb=need)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["out"], a["q"], a["kp"], a["vp"], a["bt"], a["M"], a["sl"], a["cu"], a["tm"], a["W"], a["B"], a["T"],
                 a["mq"], a["msl"], a["Hq"], a["scale"], a["d"], a["ws"], a["wsb"], None, None)

    for none in (dict(B=0), dict(T=0), dict(mq=0)):
        assert call(**none) == wf.WF_OK
    for bad in (dict(B=-1), dict(T=-1), dict(mq=-1), dict(msl=-1), dict(Hq=0), dict(Hq=7), dict(M=0), dict(msl=65),
                dict(mq=65), dict(W=0), dict(mq=33), dict(W=-1), dict(scale=math.inf), dict(scale=math.nan),
                dict(out=None), dict(q=None), dict(kp=None), dict(vp=None), dict(bt=None), dict(sl=None),
                dict(cu=None), dict(tm=None), dict(out=FAKE + 8), dict(q=FAKE + 2), dict(kp=FAKE + 4),
                dict(vp=FAKE + 8), dict(bt=FAKE + 2), dict(sl=FAKE + 1), dict(cu=FAKE + 2), dict(tm=FAKE + 2)):
        assert call(**bad) == wf.WF_ERR_INVALID_ARG, bad
    assert call(Hq=18) == wf.WF_ERR_UNSUPPORTED          # G = 9
    assert call(d=_desc(D=80)) == wf.WF_ERR_UNSUPPORTED
    for bad in (dict(ws=None), dict(ws=FAKE + 8), dict(wsb=need - 1), dict(wsb=0)):
        assert call(**bad) == wf.WF_ERR_WORKSPACE, bad


def test_outputs_over_inputs_and_lengths_that_leave_no_room_are_refused(lib):
    d = _desc(N=10, P=16, H=2, D=64)
    need = wf.wf_paged_tree_decode_workspace_size(2, 8, 7, 64, d)
    rows = 10 * 8 * 64 * 2
    far = FAKE + (1 << 30)

    def tree(out, msl=64, M=4, wsb=need):
        return lib.wf_paged_tree_decode(out, far, FAKE, FAKE, FAKE, M, FAKE, FAKE, FAKE, 1, 2, 10, 7, msl, 8, 0.1, d, FAKE,
                                        wsb, None, None)

    for at in (far, far + rows - 16, far - rows + 16):
        assert tree(at) == wf.WF_ERR_INVALID_ARG
    for msl in (2 ** 31 - 1, 2 ** 31 - 1024):
        assert tree(FAKE, msl=msl, M=1 << 27, wsb=1 << 40) == wf.WF_ERR_INVALID_ARG
    assert tree(FAKE, msl=2 ** 31 - 1025, M=1 << 27, wsb=0) == wf.WF_ERR_WORKSPACE     # the largest that passes

    def rope(qo, T=3):
        return lib.wf_qk_norm_rope_and_cache(qo, FAKE, 768, FAKE + 1024, 768, FAKE + 1280, 768, None, None, 0.0, None, 0, 0,
                                             0, None, far, far, far, T, 8, d, None, None)

    for qo in (FAKE + 1024, FAKE + 1280, FAKE + 1264 + 256):     # the k and v parts of one token, T = 1
        assert rope(qo, 1) == wf.WF_ERR_INVALID_ARG
    assert rope(FAKE + 3 * 768 * 2 - 16) == wf.WF_ERR_INVALID_ARG   # the last token's v


def test_tree_workspace_size(lib):
    d = _desc(N=100, P=16, H=8, D=128)
    size = wf.wf_paged_tree_decode_workspace_size
    one, many = size(1, 32, 8, 64, d), size(231, 32, 8, 8704, d)
    assert 0 < one <= many
    # pieces of two units a CTA: the context's length does not add to it
    assert size(231, 32, 64, 1 << 20, d) == size(231, 32, 64, 1 << 16, d)
    assert size(4, 31, 8, 100, d) == 0 and size(-1, 32, 8, 100, d) == 0
    assert size(1 << 30, 32, 1 << 30, (1 << 31) - 1, d) < 1 << 30
    assert size(0, 32, 8, 100, d) > 0 and size(3, 32, 0, 0, d) > 0


def test_keep_refusals(lib):
    f = lib.wf_keep_accepted
    ok = dict(kp=FAKE, vp=FAKE, bt=FAKE, M=4, sl=FAKE, cu=FAKE, acc=FAKE, A=4, na=FAKE + 64, nl=FAKE + 128, B=2, d=_desc())

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["kp"], a["vp"], a["bt"], a["M"], a["sl"], a["cu"], a["acc"], a["A"], a["na"], a["nl"], a["B"], a["d"],
                 None, None)

    assert call(B=0) == wf.WF_OK
    for bad in (dict(B=-1), dict(A=-1), dict(M=0), dict(kp=None), dict(vp=None), dict(bt=None), dict(sl=None),
                dict(cu=None), dict(acc=None), dict(na=None), dict(kp=FAKE + 8), dict(vp=FAKE + 4), dict(bt=FAKE + 2),
                dict(sl=FAKE + 2), dict(cu=FAKE + 2), dict(acc=FAKE + 2), dict(na=FAKE + 2), dict(nl=FAKE + 130),
                dict(nl=FAKE), dict(nl=FAKE + 64)):
        assert call(**bad) == wf.WF_ERR_INVALID_ARG, bad
    assert call(d=_desc(D=80)) == wf.WF_ERR_UNSUPPORTED


def test_binding_refuses_what_the_abi_cannot_see(lib):
    import torch
    pool = torch.zeros(4, 16, 2, 64)
    x = torch.zeros(3, 4, 64)
    kv = torch.zeros(3, 2, 64)
    table = torch.zeros(8, 64)
    pos, slots = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)

    def rope(**kw):
        a = dict(q_out=torch.zeros_like(x), q=x, k=kv, v=kv, cos_sin=table, positions=pos, slot_mapping=slots, w=None)
        a.update(kw)
        wf.wf_qk_norm_rope_and_cache(a["q_out"], a["q"], a["k"], a["v"], a["w"], None, 1e-6, a["cos_sin"],
                                     a["positions"], pool, pool.clone(), a["slot_mapping"], stream=0)

    for bad in (dict(q=x.transpose(0, 1)), dict(k=torch.zeros(3, 2, 128)[..., ::2]), dict(k=torch.zeros(2, 2, 64)),
                dict(v=torch.zeros(3, 4, 64)), dict(q=x.bfloat16()), dict(q_out=torch.zeros(3, 4, 64).bfloat16()),
                dict(positions=pos.long()), dict(positions=pos[:2]), dict(slot_mapping=slots.int()),
                dict(slot_mapping=slots[:2]), dict(cos_sin=table.double()), dict(w=torch.zeros(32)),
                dict(w=torch.zeros(64).bfloat16()), dict(cos_sin=torch.zeros(8, 128)[:, :64])):
        with pytest.raises(ValueError):
            rope(**bad)
    cu, lens = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    bt, ws = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(16, dtype=torch.uint8)

    def tree(**kw):
        a = dict(out=torch.zeros_like(x), q=x, mask=torch.zeros(3, 1, dtype=torch.int32), lens=lens, cu=cu)
        a.update(kw)
        wf.wf_paged_tree_decode(a["out"], a["q"], pool, pool.clone(), bt, a["lens"], a["cu"], a["mask"], 3, 16, 0.1, ws,
                                stream=0)

    for bad in (dict(out=torch.zeros(2, 4, 64)), dict(q=x.bfloat16()), dict(mask=torch.zeros(2, 1, dtype=torch.int32)),
                dict(mask=torch.zeros(3, 1, dtype=torch.int64)), dict(lens=cu), dict(cu=lens),
                dict(out=torch.zeros(3, 4, 128)[..., ::2])):
        with pytest.raises(ValueError):
            tree(**bad)
    with pytest.raises(ValueError):
        wf.wf_keep_accepted(pool, pool.clone(), bt, lens, cu, torch.zeros(2, 3, dtype=torch.int32), lens, stream=0)
    with pytest.raises(ValueError):
        wf.wf_keep_accepted(pool, pool.clone(), bt, lens, lens, torch.zeros(1, 3, dtype=torch.int32), lens, stream=0)


def test_descriptors_follow_the_values_of_the_scales(lib):
    import numpy as np
    import torch
    pool = torch.zeros(4, 16, 2, 64, dtype=torch.uint8)
    scales = [0.5, 0.25]
    d = wf._desc(pool, scales, 1.0)
    assert wf._desc(pool, [0.5, 0.25], 1.0) is d and wf._desc(pool, (0.5, 0.25), 1.0) is d
    scales[1] = 0.125          # the same list, other values
    e = wf._desc(pool, scales, 1.0)
    assert e is not d and [e.k_head_scales[h] for h in range(2)] == [0.5, 0.125]
    assert [d.k_head_scales[h] for h in range(2)] == [0.5, 0.25]
    assert wf._desc(pool, 1.0, scales) is not e
    for other in (np.array([0.5, 0.25]), torch.tensor([0.5, 0.25]), [torch.tensor(0.5), torch.tensor(0.25)]):
        x = wf._desc(pool, other, 1.0)
        assert x is not d and [x.k_head_scales[h] for h in range(2)] == [0.5, 0.25]
    with pytest.raises(ValueError):
        wf._desc(pool, [0.5, 0.25, 0.5], 1.0)
    assert wf._desc(torch.zeros(5, 16, 2, 64, dtype=torch.uint8), [0.5, 0.25], 1.0).num_blocks == 5

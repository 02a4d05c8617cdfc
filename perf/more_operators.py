"""Cases of the operators that keep a serving step on the GPU and shape what its attention sees:

    build    the step's block tables, slots, positions and offsets from the requests' lengths and the
             list of free blocks (wf_build_step)
    scored   attention of new tokens over the paged cache, one a request or many, whose scores are capped
             by a tanh, biased by distance, and cut to a window or to a range of each row: documents of a
             packed request, a prefix seen in both directions (wf_paged_scored_attention)
    verify   the accepted path of a tree or chain of drafted tokens and the token after it, from the
             target's probabilities and given random numbers (wf_verify_drafts)
    trim     the blocks that a shortened request no longer needs, back to the list (wf_trim_blocks)

`run` computes them with elementary torch operations, or, where `own` is set, by the framework's
calls.  Head counts, head sizes, block sizes and batches are those of the framework's workloads
(Llama-3-8B, Llama-3.2-1B, GPT-2, the mixed step) or generic.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}
K_SCALE, V_SCALE = 1 / 64, 1 / 96      # fp8 pools: what a code's value is multiplied by
ACCEPTED = 0.76                        # how often a draft of these inputs is accepted, for `work`


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def scored(name, batch, heads, kv, dim, block, pool, new, least, shortest, longest, cap=0.0, window=0, slopes=False,
           view="causal", shape=1):
    """Requests of least..new new tokens behind shortest..longest cached ones.  view: what a row may see: `causal`;
    `documents`: back to the start of its own document, a few rows nothing; `prefix`: the request's prefix whole."""
    return {"name": name, "op": "scored", "batch": batch, "heads": heads, "kv": kv, "dim": dim, "block": block,
            "pool": pool, "new": new, "least": least, "shortest": shortest, "longest": longest, "cap": cap,
            "window": window, "slopes": slopes, "view": view, "shape": shape}


def verify(name, batch, vocab, probs, nodes, least, drawn, shape=1):
    """Trees of least..nodes nodes, the root among them; `drawn`: chains with a sibling now and then, and the draft's
    probabilities."""
    return {"name": name, "op": "verify", "batch": batch, "vocab": vocab, "probs": probs, "nodes": nodes, "least": least,
            "drawn": drawn, "shape": shape}


def build(name, batch, block, new, least, shortest, longest, depths=False, shape=1):
    return {"name": name, "op": "build", "batch": batch, "block": block, "new": new, "least": least,
            "shortest": shortest, "longest": longest, "depths": depths, "shape": shape}


def trim(name, batch, block, cut, shortest, longest, shape=1):
    """Requests that lose up to `cut` tokens; every 16th one all of its own."""
    return {"name": name, "op": "trim", "batch": batch, "block": block, "cut": cut, "shortest": shortest,
            "longest": longest, "shape": shape}


def listed():
    return [
        # one user decodes one token, scores biased by distance: latency
        scored("scored one user", 1, 32, 8, 128, 16, "bf16", 1, 1, 700, 700, slopes=True),
        # the decode step of the Llama-3-8B batch with capped scores
        scored("scored decode 231", 231, 32, 8, 128, 16, "bf16", 1, 1, 64, 8192, cap=50.0),
        # a layer with a window over fp8 pools, capped too
        scored("scored window fp8", 64, 32, 8, 128, 16, "fp8", 1, 1, 128, 8192, cap=30.0, window=1024),
        # the prompts of the mixed step behind their cached prefixes, capped: the largest
        scored("scored prompts", 8, 32, 8, 128, 16, "bf16", 2048, 128, 1, 2048, cap=50.0),
        # packed documents of long requests, Llama-3.2-1B heads, biased by distance
        scored("scored documents", 5, 32, 8, 64, 16, "bf16", 4099, 1021, 0, 0, slopes=True, view="documents"),
        # one user's chain of four drafts: latency
        verify("verify one chain", 1, 128000, "f32", 5, 5, True),
        # chains of a full batch
        verify("verify chains 231", 231, 128000, "f32", 5, 2, True),
        # trees of fixed candidates, an odd vocabulary, probabilities in 16 bits
        verify("verify trees bf16", 64, 50257, "bf16", 24, 8, False),
        # the decode step of a full batch: latency
        build("build decode 231", 231, 16, 1, 1, 64, 8192),
        # a mixed step: prompts and drafts beside single tokens
        build("build mixed 128", 128, 16, 2048, 1, 1, 8192, depths=True),
        # what a verified step of wide trees gives back
        trim("trim drafts 231", 231, 16, 61, 64, 8192),
        # one user's drafts
        trim("trim one user", 1, 16, 61, 700, 700),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scored", "scored", "scored", "verify", "verify", "build", "trim"])
    shape = rng.randint(1, 10 ** 6)
    if op == "scored":
        heads, kv, dim = rng.choice([(32, 8, 128), (32, 8, 64), (12, 12, 64), (4, 2, 64), (16, 2, 128), (10, 2, 128), (5, 5, 128)])
        pool = rng.choice(["bf16", "bf16", "bf16", "fp8", "f32"])
        block = rng.choice([16, 16, 16, 32, 64, 7])
        # the CUDA-core shapes (fp32 pools, odd blocks) over shorter contexts and smaller batches
        small = pool == "f32" or block == 7
        cap, window, slopes = rng.choice([0.0, 20.0, 50.0]), rng.choice([0, 0, spread(rng, 1, 2048)]), rng.random() < 0.4
        view = rng.choice(["causal", "causal", "documents", "prefix"])
        if rng.random() < 0.5:
            longest = spread(rng, 16, 2048 if small else 8192)
            return strip(scored("", spread(rng, 1, 8 if small else 96), heads, kv, dim, block, pool, rng.choice([1, 1, 1, 5]), 1,
                                max(1, longest // rng.randint(2, 16)), longest, cap, window, slopes, view, shape))
        new, longest = spread(rng, 16, 300 if small else 2048), spread(rng, 1, 300 if small else 2048)
        return strip(scored("", rng.randint(1, 3 if small else 6), heads, kv, dim, block, pool, new, rng.randint(0, new), 1, longest,
                            cap, window, slopes, view, shape))
    if op == "verify":
        nodes = spread(rng, 1, 32)
        return strip(verify("", spread(rng, 1, 48), spread(rng, 97, 128000), rng.choice(["f32", "f32", "bf16"]), nodes,
                            rng.randint(1, nodes), rng.random() < 0.6, shape))
    longest, block = spread(rng, 16, 8192), rng.choice([16, 16, 32, 64, 7, 1])
    if op == "build":
        new = rng.choice([1, 1, spread(rng, 2, 2048)])
        return strip(build("", spread(rng, 1, 512), block, new, rng.randint(0, new), 1, longest, rng.random() < 0.3, shape))
    return strip(trim("", spread(rng, 1, 512), block, spread(rng, 1, 512), 1, longest, shape))


def strip(case):
    del case["name"]
    return case


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def lengths(case):
    """(cached, new) tokens of each request: they belong to the case, not to the seed."""
    r = np.random.RandomState(case["shape"])
    b = case["batch"]
    cached = np.exp(r.uniform(math.log(max(case["shortest"], 1)), math.log(max(case["longest"], 1)), b)).round().astype(np.int64)
    cached[0] = case["longest"]
    if case["longest"] == 0:
        cached[:] = 0
    if case["op"] == "build" and case["new"] > 64:
        # one request in sixteen is a prompt, the others decode one token or a few drafts
        new = r.randint(min(case["least"], 8), 9, b)
        new[::16] = r.randint(case["least"], case["new"] + 1, len(new[::16]))
    else:
        new = r.randint(case["least"], case["new"] + 1, b)
    new[-1] = case["new"]
    return cached, new


def ranges(case, cached, new):
    """[begin, end) of the positions that each new row may see, before the window; None where it is all up to itself."""
    if case["view"] == "causal":
        return None
    r = np.random.RandomState(case["shape"] + 1)
    out = []
    for c, n in zip(cached, new):
        at, total = c + np.arange(n), c + n
        begin, end = np.zeros(n, np.int64), at + 1
        if case["view"] == "documents":
            starts = np.unique(np.concatenate([[0], r.randint(0, total + 1, 1 + int(total) // 700)]))
            begin = starts[np.searchsorted(starts, at, side="right") - 1]
            begin[50::101] = end[50::101] = 0           # rows that only pad a document
        else:
            end = np.maximum(end, r.randint(0, total + 1))
        out.append(np.stack([begin, end], 1))
    return np.concatenate(out).astype(np.int32).reshape(-1, 2)


def seen(case, cached, new):
    """[begin, end) of each new row with the window in."""
    at = np.concatenate([c + np.arange(n) for c, n in zip(cached, new)])
    view = ranges(case, cached, new)
    begin, end = (np.zeros_like(at), at + 1) if view is None else view.astype(np.int64).T
    if case["window"]:
        begin = np.maximum(begin, at + 1 - case["window"])
    return begin, np.maximum(end, begin)


def values(shape, pool, gen, scale):
    """Pool contents: normal, in the pool's type; fp8 codes stand for the same through their scale."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if pool == "fp8":
        return (x / scale).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(TYPES[pool])


def tables(need, r):
    """Block tables over one shuffled pool; entries past a request's blocks are a spare block's."""
    n = int(need.sum())
    ids, t = r.permutation(n), np.full((len(need), max(1, int(need.max()))), n, np.int32)
    t[np.arange(t.shape[1])[None, :] < need[:, None]] = ids
    return t, n + 1


def offsets(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    return {"scored": prepare_scored, "verify": prepare_verify, "build": prepare_build, "trim": prepare_trim}[case["op"]](
        case, s, gen, r)


def prepare_scored(case, s, gen, r):
    kv, d, p, pool, h = case["kv"], case["dim"], case["block"], case["pool"], case["heads"]
    cached, new = lengths(case)
    table, n = tables(-(-(cached + new) // p), r)
    s["table"] = torch.from_numpy(table).cuda()
    s["lens"] = torch.from_numpy((cached + new).astype(np.int32)).cuda()
    cu = offsets(new)
    s["cu"] = torch.from_numpy(cu).cuda()
    s["k_pool"], s["v_pool"] = (values((n, p, kv, d), pool, gen, c) for c in (K_SCALE, V_SCALE))
    s["longest"], s["new"] = int((cached + new).max()), int(new.max())
    s["q"] = (4 * torch.randn((int(cu[-1]), h, d), generator=gen, device="cuda")).to(
        torch.float32 if pool == "f32" else torch.bfloat16)
    s["out"] = torch.zeros_like(s["q"])
    view = ranges(case, cached, new)
    s["ranges"] = None if view is None else torch.from_numpy(view).cuda()
    s["slopes"] = None
    if case["slopes"]:
        s["slopes"] = torch.pow(2.0, -8 * torch.arange(1, h + 1, dtype=torch.float64) / h).float().cuda()
    s["host_cu"], s["host_lens"] = cu.tolist(), (cached + new).tolist()      # the scheduler's own copy
    return s


def shapes(case):
    """Nodes of each request and the parent of each node: a chain, or a tree (each node's parent lies before it)."""
    r = np.random.RandomState(case["shape"])
    nodes = r.randint(case["least"], case["nodes"] + 1, case["batch"])
    nodes[-1] = case["nodes"]
    parents = []
    for n in nodes:
        parents += [i - 1 if case["drawn"] and i % 4 else r.randint(max(-1, i - 6), i) if i else -1 for i in range(n)]
    return nodes, np.maximum(np.array(parents, np.int32), -1)


def prepare_verify(case, s, gen, r):
    nodes, parents = shapes(case)
    cu, v, t = offsets(nodes), case["vocab"], int(nodes.sum())
    first = np.repeat(cu[:-1], nodes)
    parents[np.arange(t) == first] = -1
    live = parents.copy()
    live[(parents < 0) & (np.arange(t) != first)] = 0           # a second root hangs on the first
    kind = TYPES[case["probs"]]
    target = 2.5 * torch.randn((t, v), generator=gen, device="cuda")
    draft = torch.softmax(target + 0.6 * torch.randn((t, v), generator=gen, device="cuda"), -1)
    s["target"] = torch.softmax(target, -1).to(kind)
    # a node's token: one of its parent's draft probabilities, drawn, or the most likely ones in turn
    up = torch.from_numpy((first + np.maximum(live, 0)).astype(np.int64)).cuda()
    nth = np.zeros(t, np.int64)                                    # which child of its parent
    for i in range(t):
        nth[i] = int(np.sum(live[first[i]:i] == live[i])) if live[i] >= 0 else 0
    most = int(nth.max()) + 1
    if case["drawn"]:
        picks = torch.multinomial(draft, most, replacement=True, generator=gen)
    else:
        picks = torch.topk(draft, min(most, v), -1).indices
    s["tokens"] = picks[up, torch.from_numpy(np.minimum(nth, picks.shape[1] - 1)).cuda()].to(torch.int32)
    s["draft"] = draft.to(kind) if case["drawn"] else None
    s["parents"] = torch.from_numpy(live.astype(np.int32)).cuda()
    s["cu"] = torch.from_numpy(cu).cuda()
    s["nodes"] = int(nodes.max())
    s["coins"] = torch.rand(t, generator=gen, device="cuda")
    s["picks"] = torch.rand(case["batch"], generator=gen, device="cuda")
    s["accepted"] = torch.zeros((case["batch"], s["nodes"]), dtype=torch.int32, device="cuda")
    s["count"], s["next"] = (torch.zeros(case["batch"], dtype=torch.int32, device="cuda") for _ in range(2))
    return s


def prepare_build(case, s, gen, r):
    cached, new = lengths(case)
    p, b = case["block"], case["batch"]
    held, need = -(-cached // p), -(-(cached + new) // p)
    n = int(need.sum()) + 8
    ids = r.permutation(n).astype(np.int32)
    m = max(1, int(need.max()))
    table = np.full((b, m), n - 1, np.int32)
    table[np.arange(m)[None, :] < held[:, None]] = ids[:int(held.sum())]
    free = np.full(n, -1, np.int32)
    free[:n - int(held.sum())] = ids[int(held.sum()):]
    s["table"], s["free"] = torch.from_numpy(table).cuda(), torch.from_numpy(free).cuda()
    s["num_free"] = torch.tensor([n - int(held.sum())], dtype=torch.int32, device="cuda")
    s["lens"], s["new"] = torch.from_numpy(cached.astype(np.int32)).cuda(), torch.from_numpy(new.astype(np.int32)).cuda()
    s["rows"] = int(new.sum()) + 13                                # a padded batch
    s["depths"] = torch.from_numpy(r.randint(0, 8, s["rows"]).astype(np.int32)).cuda() if case["depths"] else None
    zeros = lambda k, t=torch.int32: torch.zeros(k, dtype=t, device="cuda")   # noqa: E731
    s["new_lens"], s["left"], s["cu"] = zeros(b), zeros(1), zeros(b + 1)
    s["slots"], s["positions"] = zeros(s["rows"], torch.int64), zeros(s["rows"])
    return s


def cuts(case):
    r = np.random.RandomState(case["shape"])
    lens = np.exp(r.uniform(math.log(case["shortest"]), math.log(case["longest"]), case["batch"])).round().astype(np.int64)
    lens[0] = case["longest"]
    kept = np.maximum(0, lens - r.randint(0, case["cut"] + 1, case["batch"]))
    kept[15::16] = 0                                               # requests that are done
    return lens, kept


def prepare_trim(case, s, gen, r):
    lens, kept = cuts(case)
    p = case["block"]
    need = -(-lens // p)
    total, spare = int(need.sum()), 24
    ids = r.permutation(total + spare).astype(np.int32)
    m = max(1, int(need.max()))
    table = np.full((case["batch"], m), ids[-1], np.int32)
    table[np.arange(m)[None, :] < need[:, None]] = ids[:total]
    free = np.full(total + spare, -1, np.int32)
    free[:spare] = ids[total:]
    s["table"], s["free"] = torch.from_numpy(table).cuda(), torch.from_numpy(free).cuda()
    s["num_free"] = torch.tensor([spare], dtype=torch.int32, device="cuda")
    s["lens"], s["kept"] = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (lens, kept))
    s["left"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"scored": own_scored, "verify": own_verify, "build": own_build, "trim": own_trim}[op](s)
    return {"scored": plain_scored, "verify": plain_verify, "build": plain_build, "trim": plain_trim}[op](s)


def coded(pool):
    """A pool as the values that its codes stand for (before their scale)."""
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def own_scored(s):
    from paged_kv_cache_wf_gb300 import binding as wf
    c = s["case"]
    if "workspace" not in s:                   # kept between steps, as for wf_paged_decode
        n = wf.wf_paged_scored_attention_workspace_size(c["batch"], c["heads"], s["q"].shape[0], s["new"], s["longest"],
                                                        wf.pool_desc(s["k_pool"], K_SCALE, V_SCALE))
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    scales = {"k_scale": K_SCALE, "v_scale": V_SCALE} if c["pool"] == "fp8" else {}
    wf.wf_paged_scored_attention(s["out"], s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["cu"], s["new"],
                                 s["longest"], 1 / math.sqrt(c["dim"]), s["workspace"], cap=c["cap"], window=c["window"],
                                 slopes=s["slopes"], row_ranges=s["ranges"], dev_status=s["status"], **scales)
    return s["out"]


def own_verify(s):
    from paged_kv_cache_wf_gb300 import binding as wf
    wf.wf_verify_drafts(s["accepted"], s["count"], s["next"], s["target"], s["draft"], s["tokens"], s["parents"], s["cu"],
                        s["nodes"], s["coins"], s["picks"], dev_status=s["status"])
    return {"accepted": s["accepted"], "count": s["count"], "next": s["next"]}


def own_build(s):
    from paged_kv_cache_wf_gb300 import binding as wf
    wf.wf_build_step(s["table"], s["lens"], s["new"], s["free"], s["num_free"], s["new_lens"], s["left"], s["cu"], s["slots"],
                     s["positions"], s["case"]["block"], depths=s["depths"], dev_status=s["status"])
    return {k: s[k] for k in ("table", "new_lens", "left", "cu", "slots", "positions")}


def own_trim(s):
    from paged_kv_cache_wf_gb300 import binding as wf
    wf.wf_trim_blocks(s["table"], s["lens"], s["kept"], s["free"], s["num_free"], s["left"], s["case"]["block"],
                      dev_status=s["status"])
    return {"free": s["free"], "left": s["left"]}


def plain_view(s, lens, cu, first, last):
    """(begin, end, own position) of rows first..last-1, in 64-bit whole numbers."""
    row = torch.arange(first, last, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    at = lens[b] - cu[b + 1] + row
    if s["ranges"] is None:
        begin, end = torch.zeros_like(at), at + 1
    else:
        begin, end = s["ranges"][first:last].long().unbind(1)
    if s["case"]["window"]:
        begin = torch.maximum(begin, at + 1 - s["case"]["window"])
    return begin, end, at


def plain_attend(s, q, k, v, seen_at, at):
    """q [X, kv, rows, g, d], k and v [X, L, kv, d], seen_at [X, rows, L], at [X, rows] -> [X, rows, kv, g, d]."""
    c = s["case"]
    x, kv, n, g, d = q.shape
    ks, vs = (K_SCALE, V_SCALE) if c["pool"] == "fp8" else (1.0, 1.0)
    score = torch.matmul(q.reshape(x, kv, n * g, d), k.permute(0, 2, 3, 1)).mul_(ks / math.sqrt(d))
    if c["cap"]:
        score.div_(c["cap"]).tanh_().mul_(c["cap"])
    score = score.view(x, kv, n, g, -1)
    if s["slopes"] is not None:
        # by the row's own distance to what it sees last: a shift of the whole row changes nothing
        p = torch.arange(k.shape[1], device="cuda")
        far = (p[None, None, :] - at[..., None]).abs()
        far = (far - torch.where(seen_at, far, 1 << 40).amin(-1, keepdim=True)).float()
        score = score - s["slopes"].view(1, kv, 1, g, 1) * far[:, None, :, None, :]
    score = torch.where(seen_at[:, None, :, None, :], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = weight.sum(-1, keepdim=True)
    o = torch.matmul(weight.view(x, kv, n * g, -1), v.permute(0, 2, 1, 3)).view(x, kv, n, g, d)
    return (o * vs / torch.where(total == 0, 1.0, total)).permute(0, 2, 1, 3, 4)


def plain_scored(s):
    c = s["case"]
    kv, d, g, p = c["kv"], c["dim"], c["heads"] // c["kv"], c["block"]
    lens, cu, table = s["lens"].long(), s["cu"].long(), s["table"].long()
    flat = [coded(s[x].view(-1, kv, d)) for x in ("k_pool", "v_pool")]
    if s["new"] == 1 and s["q"].shape[0] == c["batch"]:             # one row a request: all at once
        at = torch.arange(s["longest"], device="cuda")
        slots = table[:, at // p] * p + at % p
        inside = at[None, :] < lens[:, None]
        k, v = (x[slots].float() for x in flat)
        begin, end, own_at = plain_view(s, lens, cu, 0, c["batch"])
        sees = inside & (at >= begin[:, None]) & (at < end[:, None])
        q = s["q"].float().view(-1, 1, kv, g, d).transpose(1, 2)
        s["out"].copy_(plain_attend(s, q, k, v * inside[..., None, None], sees[:, None], own_at[:, None]).reshape(-1, c["heads"], d))
        return s["out"]
    for b, length in enumerate(s["host_lens"]):
        first, last = s["host_cu"][b], s["host_cu"][b + 1]
        at = torch.arange(length, device="cuda")
        slots = table[b, at // p] * p + at % p
        k, v = (x[slots].float()[None] for x in flat)
        for lo in range(first, last, 1024):                          # so many rows' scores at a time
            hi = min(last, lo + 1024)
            begin, end, own_at = plain_view(s, lens, cu, lo, hi)
            sees = (at >= begin[:, None]) & (at < end[:, None])
            q = s["q"][lo:hi].float().view(1, hi - lo, kv, g, d).transpose(1, 2)
            s["out"][lo:hi] = plain_attend(s, q, k, v, sees[None], own_at[None])[0].reshape(hi - lo, c["heads"], d).to(s["out"].dtype)
    return s["out"]


def plain_verify(s):
    # in 64 bits where a number is compared with a border that it may lie next to
    c = s["case"]
    b, n = c["batch"], s["nodes"]
    cu = s["cu"].long()
    count = cu[1:] - cu[:-1]
    node = torch.arange(n, device="cuda")[None, :].expand(b, -1)
    row = (cu[:-1, None] + node).clamp(max=s["tokens"].shape[0] - 1)
    parent = torch.where(node < count[:, None], s["parents"][row].long(), -2)
    token, coin = s["tokens"][row].long(), s["coins"][row].double()
    here = torch.zeros(b, dtype=torch.long, device="cuda")
    one = torch.arange(b, device="cuda")
    accepted, kept = torch.full((b, n), -1, dtype=torch.long, device="cuda"), torch.ones_like(here)
    accepted[:, 0] = 0
    moving = torch.ones(b, dtype=torch.bool, device="cuda")
    taken = torch.zeros_like(here, dtype=torch.double)             # c: how much of the draft is taken off
    rest = torch.ones_like(taken)
    tried = torch.zeros_like(moving)
    node_row = lambda x: row[one, x]                               # noqa: E731
    for i in range(1, n):                                          # nodes in order: a path only goes forward
        mine = moving & (parent[:, i] == here)
        p = s["target"][node_row(here), token[:, i]].double()
        if s["draft"] is not None:
            q = s["draft"][node_row(here), token[:, i]].double()
            yes = mine & (coin[:, i] * q * rest < (p - taken * q).clamp(min=0))
        else:
            again = ((parent[:, :i] == here[:, None]) & (token[:, :i] == token[:, i:i + 1])).any(1)
            yes = mine & ~again & (coin[:, i] * rest < p)
        no = mine & ~yes
        if s["draft"] is not None:
            more = no & ((parent == here[:, None]) & (node > i)).any(1)
            taken = torch.where(no, taken + rest, taken)
            at = torch.nonzero(more)[:, 0]
            if at.numel():                                         # another sibling is tried against what is left
                rows = node_row(here)[at]
                rest[at] = (s["target"][rows].double() - taken[at, None] * s["draft"][rows].double()).clamp_(min=0).sum(-1)
        else:
            rest = torch.where(no & ~again, rest - p, rest)
        tried = (tried | no) & ~yes
        here = torch.where(yes, i, here)
        accepted[one, torch.where(yes, kept, 0)] = torch.where(yes, i, 0)
        kept, taken, rest = kept + yes, torch.where(yes, 0.0, taken), torch.where(yes, 1.0, rest)
    rows = node_row(here)
    weight = s["target"][rows].double()
    left = weight
    if s["draft"] is not None:
        left = (weight - taken[:, None] * s["draft"][rows].double()).clamp_(min=0)
    else:
        left = weight.clone()
        for i in range(1, n):
            gone = parent[:, i] == here
            left[one[gone], token[gone, i]] = 0
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, weight)
    up = left.cumsum(-1)
    past = up > s["picks"].double()[:, None] * up[:, -1:]
    s["next"].copy_(past.to(torch.uint8).argmax(-1))
    s["accepted"].copy_(accepted)
    s["count"].copy_(kept)
    return {"accepted": s["accepted"], "count": s["count"], "next": s["next"]}


def plain_build(s):
    p, rows = s["case"]["block"], s["rows"]
    lens, new = s["lens"].long(), s["new"].long()
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), new.cumsum(0)])
    held, need = (lens + p - 1) // p, (lens + new + p - 1) // p
    taken = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), (need - held).cumsum(0)])
    column = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    fresh = (column >= held[:, None]) & (column < need[:, None])
    at = (s["num_free"].long() - 1 - taken[:-1, None] - (column - held[:, None])).clamp(0, s["free"].shape[0] - 1)
    s["table"].copy_(torch.where(fresh, s["free"][at], s["table"]))
    row = torch.arange(rows, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True).clamp(max=new.shape[0] - 1)
    position = lens[b] + row - cu[b]
    inside = row < cu[-1]
    block = s["table"][b, torch.where(inside, position // p, 0)].long()
    s["slots"].copy_(torch.where(inside, block * p + position % p, -1))
    if s["depths"] is not None:
        position = lens[b] + s["depths"]
    s["positions"].copy_(torch.where(inside, position, 0))
    s["new_lens"].copy_(lens + new)
    s["left"].copy_(s["num_free"] - taken[-1:])
    s["cu"].copy_(cu)
    return {k: s[k] for k in ("table", "new_lens", "left", "cu", "slots", "positions")}


def plain_trim(s):
    p = s["case"]["block"]
    held, keep = (s["lens"].long() + p - 1) // p, (s["kept"].long() + p - 1) // p
    column = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    back = s["table"][(column >= keep[:, None]) & (column < held[:, None])]       # request by request
    at = s["num_free"].long() + torch.arange(back.shape[0], device="cuda")
    s["free"].index_copy_(0, at, back.flip(0))
    s["left"].copy_(s["num_free"] + back.shape[0])
    return {"free": s["free"], "left": s["left"]}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"scored": exact_scored, "verify": exact_verify, "build": exact_build, "trim": exact_trim}[case["op"]](case, s)


def as_double(pool):
    return (pool.view(torch.float8_e4m3fn).float() if pool.dtype == torch.uint8 else pool).double()


def exact_scored(case, s):
    kv, d, block = case["kv"], case["dim"], case["block"]
    ks, vs = (K_SCALE, V_SCALE) if case["pool"] == "fp8" else (1.0, 1.0)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cached, new = lengths(case)
    begin, end = (torch.from_numpy(x).cuda() for x in seen(case, cached, new))
    cu = offsets(new).tolist()
    slopes = None if s["slopes"] is None else s["slopes"].double().view(kv, -1, 1, 1)
    for b in range(case["batch"]):
        length = int(cached[b] + new[b])
        blocks = s["table"][b, :-(-length // block)].long()
        k, v = (as_double(s[x][blocks]).reshape(-1, kv, d)[:length] for x in ("k_pool", "v_pool"))
        p = torch.arange(length, device="cuda")
        for lo in range(cu[b], cu[b + 1], 512):
            hi = min(cu[b + 1], lo + 512)
            q = s["q"][lo:hi].double().view(hi - lo, kv, -1, d)
            x = torch.einsum("nhgd,lhd->hgnl", q, k) * (ks / math.sqrt(d))
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if slopes is not None:
                at = int(cached[b]) - cu[b] + torch.arange(lo, hi, device="cuda")
                x = x - slopes * (p[None, :] - at[:, None]).abs()
            sees = (p >= begin[lo:hi, None]) & (p < end[lo:hi, None])
            x = torch.softmax(x.masked_fill(~sees, -math.inf), -1).nan_to_num(0.0)
            out[lo:hi] = (torch.einsum("hgnl,lhd->nhgd", x, v) * vs).reshape(hi - lo, -1, d)
    return out


def exact_verify(case, s):
    cu, parents, tokens = s["cu"].tolist(), s["parents"].tolist(), s["tokens"].tolist()
    coins, picks = s["coins"].double().tolist(), s["picks"].double().tolist()
    paths, following = [], []
    for b in range(case["batch"]):
        first, n = cu[b], cu[b + 1] - cu[b]
        up, path = parents[first:first + n], [0]
        while True:
            here = path[-1]
            p = s["target"][first + here].double().cpu().numpy()
            q = s["draft"][first + here].double().cpu().numpy() if case["drawn"] else None
            left, whole, chosen = p, 1.0, None
            for i in range(here + 1, n):
                if up[i] != here:
                    continue
                x = tokens[first + i]
                if case["drawn"]:                # left is not divided by its sum: `whole` stands for it
                    if coins[first + i] * q[x] * whole < left[x]:
                        chosen = i
                        break
                    left = np.maximum(left - whole * q, 0.0)
                    whole = left.sum()
                else:
                    if left[x] > 0 and coins[first + i] * whole < left[x]:
                        chosen = i
                        break
                    left = left.copy()
                    whole, left[x] = whole - left[x], 0.0
            if chosen is None:
                break
            path.append(chosen)
        left = left if left.sum() > 0 else p
        up = np.cumsum(left)
        following.append(int(np.argmax(up > picks[b] * up[-1])))
        paths.append(path)
    accepted = np.full((case["batch"], s["nodes"]), -1, np.int32)
    for b, path in enumerate(paths):
        accepted[b, :len(path)] = path
    return {"accepted": accepted, "count": np.array([len(x) for x in paths], np.int32), "next": np.array(following, np.int32)}


def exact_build(case, s):
    free, p = s["free"].cpu().numpy()[:int(s["num_free"])].tolist(), case["block"]
    table, lens, new = s["table"].cpu().numpy().copy(), s["lens"].tolist(), s["new"].tolist()
    slots, positions, cu = [], [], [0]
    for b in range(case["batch"]):
        for i in range(lens[b], lens[b] + new[b]):
            if i % p == 0:
                table[b, i // p] = free.pop()
            slots.append(int(table[b, i // p]) * p + i % p)
            positions.append(i)
        cu.append(len(slots))
    if case["depths"]:
        depths = s["depths"].tolist()
        positions = [lens[b] + depths[t] for b in range(case["batch"]) for t in range(cu[b], cu[b + 1])]
    pad = s["rows"] - len(slots)
    return {"table": table, "new_lens": np.array(lens, np.int32) + np.array(new, np.int32), "left": np.array([len(free)], np.int32),
            "cu": np.array(cu, np.int32), "slots": np.array(slots + [-1] * pad, np.int64),
            "positions": np.array(positions + [0] * pad, np.int32)}


def exact_trim(case, s):
    table, p = s["table"].cpu().numpy(), case["block"]
    free, n = s["free"].cpu().numpy().copy(), int(s["num_free"])
    back = []
    for b, (length, kept) in enumerate(zip(s["lens"].tolist(), s["kept"].tolist())):
        back += table[b, -(-kept // p):-(-length // p)].tolist()
    free[n:n + len(back)] = back[::-1]
    return {"free": free, "left": np.array([n + len(back)], np.int32)}


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "scored":
        size = {"f32": 4, "bf16": 2, "fp8": 1}[case["pool"]]
        act = 4 if case["pool"] == "f32" else 2
        cached, new = lengths(case)
        begin, end = seen(case, cached, new)
        kv, d, cu = case["kv"], case["dim"], offsets(new)
        read = blocks = 0
        for b in range(case["batch"]):                              # positions that some row of the request sees
            lo, hi = begin[cu[b]:cu[b + 1]], end[cu[b]:cu[b + 1]]
            some = np.zeros(int(cached[b] + new[b]) + 2, np.int64)
            np.add.at(some, lo, 1)
            np.add.at(some, hi, -1)
            live = np.nonzero(np.cumsum(some) > 0)[0]
            read += len(live)
            blocks += len(np.unique(live // case["block"]))
        rows, pairs = len(begin), int((end - begin).sum())
        return {"bytes": 2 * read * kv * d * size + 2 * rows * case["heads"] * d * act + 4 * blocks + 8 * case["batch"] +
                (8 * rows if case["view"] != "causal" else 0), "flops": 4 * pairs * case["heads"] * d}
    if case["op"] == "verify":
        nodes, _ = shapes(case)
        size = 4 if case["probs"] == "f32" else 2
        # the last node's row, and the draft's where a draft was rejected
        rows = case["batch"] + (float((1 - ACCEPTED ** np.maximum(nodes - 1, 0)).sum()) if case["drawn"] else 0)
        return {"bytes": int(rows * case["vocab"] * size) + int(nodes.sum()) * (12 + 2 * size) + 16 * case["batch"],
                "flops": int(2 * rows * case["vocab"])}
    if case["op"] == "build":
        cached, new = lengths(case)
        p, rows = case["block"], int(new.sum()) + 13
        fresh = int((-(-(cached + new) // p) - -(-cached // p)).sum())
        return {"bytes": 8 * fresh + 20 * case["batch"] + rows * (16 if case["depths"] else 12), "flops": 0}
    lens, kept = cuts(case)
    back = int((-(-lens // case["block"]) - -(-kept // case["block"])).sum())
    return {"bytes": 8 * back + 8 * case["batch"], "flops": 0}

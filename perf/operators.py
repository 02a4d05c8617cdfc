"""Cases of the speculative-decoding operators: the step that verifies a tree of drafted
tokens against a paged KV cache.

    rope   norms of queries and keys per head, the rotation by position, and the write of the
           new K and V rows into the pool, in one pass (wf_qk_norm_rope_and_cache)
    tree   attention of every drafted token over its request's cached context and its own
           ancestors in the tree (wf_paged_tree_decode)
    keep   the rows of the accepted path moved to the front of the drafted region
           (wf_keep_accepted)

`run` computes them with elementary torch operations in 32 bits, or, where `own` is set, by
the framework's calls.  Head counts, head sizes and block sizes are those of the framework's
workloads (Llama-3-8B, Llama-3.2-1B, GPT-2 and the small fp32 step) or generic.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}
K_SCALE, V_SCALE = 1 / 64, 1 / 96      # fp8 pools: what a code's value is multiplied by
EPS = 1e-6


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def rope(name, tokens, heads, kv, dim, block, pool, norm=True, rotary=0, interleaved=False, fused=False, pad=0):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv": kv, "dim": dim, "block": block,
            "pool": pool, "norm": norm, "rotary": rotary or dim, "interleaved": interleaved, "fused": fused,
            "pad": pad, "positions": 8192}


def tree(name, batch, heads, kv, dim, block, pool, nodes, least, shortest, longest, shape=1):
    return {"name": name, "op": "tree", "batch": batch, "heads": heads, "kv": kv, "dim": dim, "block": block,
            "pool": pool, "nodes": nodes, "least": least, "shortest": shortest, "longest": longest, "shape": shape}


def keep(name, batch, kv, dim, block, pool, nodes, depth, shortest, longest, shape=1):
    return {"name": name, "op": "keep", "batch": batch, "kv": kv, "dim": dim, "block": block, "pool": pool,
            "nodes": nodes, "depth": depth, "shortest": shortest, "longest": longest, "shape": shape}


def listed():
    return [
        # one sequence decodes one token: nothing but latency
        rope("rope 1 token", 1, 32, 8, 128, 16, "bf16", fused=True),
        # the decode step of the Llama-3-8B batch, cut from one fused projection
        rope("rope decode 231", 231, 32, 8, 128, 16, "bf16", fused=True),
        # the prompts of a mixed step written to fp8 pools; a few rows pad the batch; no norms
        rope("rope prompt fp8", 8193, 32, 8, 128, 16, "fp8", norm=False, pad=5),
        # fp32, as many K heads as Q heads, half of each head rotated in adjacent pairs
        rope("rope f32 partial", 1021, 12, 12, 64, 16, "f32", rotary=32, interleaved=True),
        # one user, a small tree: latency
        tree("tree one user", 1, 32, 8, 128, 16, "bf16", 8, 8, 700, 700),
        # the usual served batch: short drafts over ragged contexts
        tree("tree batch 32", 32, 32, 8, 128, 16, "bf16", 16, 1, 64, 4096),
        # the largest: wide trees over long contexts
        tree("tree wide", 118, 32, 8, 128, 16, "bf16", 61, 33, 256, 8192),
        # fp8 pools
        tree("tree fp8", 64, 32, 8, 128, 16, "fp8", 24, 8, 128, 8192),
        # Llama-3.2-1B heads
        tree("tree 64-wide heads", 64, 32, 8, 64, 16, "bf16", 13, 3, 32, 4096),
        # fp32 pools, one query head a KV head, chains and small trees
        tree("tree f32", 8, 12, 12, 64, 16, "f32", 7, 1, 64, 1024),
        # after the verification: one user's accepted path
        keep("keep one user", 1, 8, 128, 16, "bf16", 8, 4, 700, 700),
        # and that of a full batch
        keep("keep batch 231", 231, 8, 128, 16, "bf16", 61, 9, 64, 1024),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "tree", "tree", "tree", "keep"])
    heads, kv, dim = rng.choice([(32, 8, 128), (32, 8, 64), (12, 12, 64), (4, 2, 64), (16, 2, 128), (10, 2, 128), (5, 5, 128)])
    pool = rng.choice(["bf16", "bf16", "fp8", "f32"])
    block = rng.choice([16, 16, 16, 32, 64, 7])
    if op == "rope":
        rotary = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        t = spread(rng, 1, 4096)
        case = rope("", t, heads, kv, dim, block, pool, norm=rng.random() < 0.7, rotary=rotary,
                    interleaved=rng.random() < 0.3, fused=dim == 128 and rng.random() < 0.5, pad=rng.randint(0, min(3, t - 1)))
    elif op == "tree":
        # the CUDA-core shapes (fp32 pools, odd blocks) over shorter contexts and smaller batches
        small = pool == "f32" or block == 7
        longest = spread(rng, 16, 2048 if small else 8192)
        nodes = spread(rng, 1, 24 if small else 64)
        case = tree("", spread(rng, 1, 8 if small else 32), heads, kv, dim, block, pool, nodes, rng.randint(0, nodes),
                    max(1, longest // rng.randint(2, 16)), longest, rng.randint(1, 10 ** 6))
    else:
        longest, nodes = spread(rng, 16, 1024), spread(rng, 1, 64)
        case = keep("", spread(rng, 1, 231), kv, dim, block, pool, nodes, rng.randint(1, min(nodes, 12)),
                    max(1, longest // rng.randint(1, 16)), longest, rng.randint(1, 10 ** 6))
    del case["name"]
    return case


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def lengths(case):
    """(cached, drafted) tokens of each request: they belong to the case, not to the seed."""
    r = np.random.RandomState(case["shape"])
    lo, hi, b = math.log(case["shortest"]), math.log(case["longest"]), case["batch"]
    cached = np.exp(r.uniform(lo, hi, b)).round().astype(np.int64)
    cached[0] = case["longest"]
    drafted = r.randint(case.get("least", 1), case["nodes"] + 1, b)
    drafted[-1] = case["nodes"]
    return cached, drafted


def values(shape, pool, gen, scale):
    """Pool contents: normal, in the pool's type; fp8 codes stand for the same through their scale."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if pool == "fp8":
        return (x / scale).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(TYPES[pool])


def tables(cached, drafted, block, r):
    """Block tables over one shuffled pool with a spare block at its end."""
    need = -(-(cached + drafted) // block)
    n = int(need.sum())
    ids, t = r.permutation(n), np.full((len(need), max(1, int(need.max()))), n, np.int32)
    t[np.arange(t.shape[1])[None, :] < need[:, None]] = ids
    return t, n + 1


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    kv, d, p, pool = case["kv"], case["dim"], case["block"], case["pool"]
    act = torch.float32 if pool == "f32" else torch.bfloat16
    if case["op"] == "rope":
        t, h, rot = case["tokens"], case["heads"], case["rotary"]
        if case["fused"]:
            x = torch.randn((t, h + 2 * kv, d), generator=gen, device="cuda").to(act)
            s["q"], s["k"], s["v"] = x[:, :h], x[:, h:h + kv], x[:, h + kv:]
        else:
            s["q"], s["k"], s["v"] = (torch.randn((t, n, d), generator=gen, device="cuda").to(act) for n in (h, kv, kv))
        for w in ("q_weight", "k_weight"):
            s[w] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(act) if case["norm"] else None
        angle = torch.arange(case["positions"], device="cuda", dtype=torch.float64)[:, None] * \
            torch.pow(torch.tensor(10000.0, device="cuda", dtype=torch.float64),
                      -2 * torch.arange(rot // 2, device="cuda", dtype=torch.float64) / rot)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        s["positions"] = torch.from_numpy(r.randint(0, case["positions"], t).astype(np.int32)).cuda()
        n = -(-t // p) + 1
        slots = r.permutation(n * p)[:t].astype(np.int64)
        if case["pad"]:
            slots[-case["pad"]:] = -1          # rows that only pad the batch
        s["live"] = torch.arange(t - case["pad"], device="cuda")
        s["slots"] = torch.from_numpy(slots).cuda()
        s["k_pool"], s["v_pool"] = (torch.zeros((n, p, kv, d), dtype=TYPES[pool], device="cuda") for _ in range(2))
        s["q_out"] = torch.zeros((t, h, d), dtype=act, device="cuda")
        return s
    cached, drafted = lengths(case)
    table, n = tables(cached, drafted, p, r)
    s["table"] = torch.from_numpy(table).cuda()
    s["lens"] = torch.from_numpy((cached + drafted).astype(np.int32)).cuda()
    cu = np.concatenate([[0], np.cumsum(drafted)])
    s["cu"] = torch.from_numpy(cu.astype(np.int32)).cuda()
    s["k_pool"], s["v_pool"] = (values((n, p, kv, d), pool, gen, c) for c in (K_SCALE, V_SCALE))
    s["longest"], s["nodes"] = int((cached + drafted).max()), int(drafted.max())
    if case["op"] == "keep":
        # a path down the tree: nodes in increasing order; what follows it in the row is not read
        a = np.full((case["batch"], case["depth"]), -1, np.int32)
        count = np.minimum(r.randint(1, case["depth"] + 1, case["batch"]), drafted)
        for b in range(case["batch"]):
            a[b, :count[b]] = np.sort(r.permutation(int(drafted[b]))[:count[b]])
        s["accepted"], s["count"] = torch.from_numpy(a).cuda(), torch.from_numpy(count.astype(np.int32)).cuda()
        s["new_lens"] = torch.zeros(case["batch"], dtype=torch.int32, device="cuda")
        return s
    total, words = int(cu[-1]), -(-s["nodes"] // 32)
    bits = np.zeros((total, words), np.uint32)
    for b in range(case["batch"]):             # each node sees itself and its ancestors
        for i in range(int(drafted[b])):
            parent = r.randint(-1, i)
            if parent >= 0:
                bits[cu[b] + i] = bits[cu[b] + parent]
            bits[cu[b] + i, i // 32] |= np.uint32(1 << (i % 32))
    s["mask"] = torch.from_numpy(bits.view(np.int32)).cuda()
    s["q"] = (2 * torch.randn((total, case["heads"], d), generator=gen, device="cuda")).to(act)
    s["out"] = torch.zeros_like(s["q"])
    # the padded view a program without such kernels works on: row of (request, node), and back
    node = np.arange(s["nodes"])[None, :]
    s["rows"] = torch.from_numpy(np.minimum(cu[:-1, None] + node, max(total - 1, 0))).cuda()
    s["flat"] = torch.from_numpy(np.concatenate([b * s["nodes"] + np.arange(n) for b, n in enumerate(drafted)])).cuda()
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": own_rope, "tree": own_tree, "keep": own_keep}[op](s)
    return {"rope": plain_rope, "tree": plain_tree, "keep": plain_keep}[op](s)


def scales(s):
    return {"k_scale": K_SCALE, "v_scale": V_SCALE} if s["case"]["pool"] == "fp8" else {}


def coded(pool):
    """A pool as the values that its codes stand for (before their scale)."""
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def own_rope(s):
    from paged_kv_cache_wf_gb300 import binding as wf
    c = s["case"]
    wf.wf_qk_norm_rope_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], EPS, s["cos_sin"],
                                 s["positions"], s["k_pool"], s["v_pool"], s["slots"], interleaved=c["interleaved"],
                                 dev_status=s["status"], **scales(s))
    return {"q": s["q_out"], "k_pool": coded(s["k_pool"]), "v_pool": coded(s["v_pool"])}


def own_tree(s):
    from paged_kv_cache_wf_gb300 import binding as wf
    if "workspace" not in s:                   # kept between steps, as for wf_paged_decode
        n = wf.wf_paged_tree_decode_workspace_size(s["case"]["batch"], s["q"].shape[1], s["nodes"], s["longest"],
                                                   wf.pool_desc(s["k_pool"], K_SCALE, V_SCALE))
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    wf.wf_paged_tree_decode(s["out"], s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["cu"], s["mask"],
                            s["nodes"], s["longest"], 1 / math.sqrt(s["case"]["dim"]), s["workspace"],
                            dev_status=s["status"], **scales(s))
    return s["out"]


def own_keep(s):
    from paged_kv_cache_wf_gb300 import binding as wf
    wf.wf_keep_accepted(s["k_pool"], s["v_pool"], s["table"], s["lens"], s["cu"], s["accepted"], s["count"],
                        new_seq_lens=s["new_lens"], dev_status=s["status"])
    return {"k_pool": coded(s["k_pool"]), "v_pool": coded(s["v_pool"]), "lens": s["new_lens"]}


def plain_rope(s):
    c, live = s["case"], s["live"]
    rot, half = c["rotary"], c["rotary"] // 2
    at = s["cos_sin"][s["positions"][live].long()][:, None, :]
    cos, sin = at[..., :half], at[..., half:]

    def turned(x, w):
        x = x[live].float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        head, rest = x[..., :rot], x[..., rot:]
        if c["interleaved"]:
            a, b = head[..., 0::2], head[..., 1::2]
            return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
        a, b = head[..., :half], head[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)

    def stored(x, scale):
        if c["pool"] == "fp8":
            return (x * (1 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return x.to(TYPES[c["pool"]])

    slots = s["slots"][live]
    s["q_out"].index_copy_(0, live, turned(s["q"], s["q_weight"]).to(s["q_out"].dtype))
    s["k_pool"].view(-1, c["kv"], c["dim"]).index_copy_(0, slots, stored(turned(s["k"], s["k_weight"]), K_SCALE))
    s["v_pool"].view(-1, c["kv"], c["dim"]).index_copy_(0, slots, stored(s["v"][live].float(), V_SCALE))
    return {"q": s["q_out"], "k_pool": coded(s["k_pool"]), "v_pool": coded(s["v_pool"])}


def slot_of(s, position):
    """Rows of the flat pool that hold `position` [B, ...] of each request."""
    p = s["case"]["block"]
    blocks = s["table"].long().gather(1, (position // p).clamp(0, s["table"].shape[1] - 1))
    return blocks * p + position % p


def plain_tree(s):
    c = s["case"]
    kv, d, g, n = c["kv"], c["dim"], c["heads"] // c["kv"], s["nodes"]
    position = torch.arange(s["longest"], device="cuda")[None, :].expand(c["batch"], -1)
    slots = slot_of(s, position)
    lens, drafted = s["lens"].long()[:, None], (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    node = position - (lens - drafted)                                    # < 0: cached context
    inside = position < lens
    k = coded(s["k_pool"].view(-1, kv, d)[slots]).float().permute(0, 2, 3, 1)
    v = coded(s["v_pool"].view(-1, kv, d)[slots]).float() * inside[..., None, None]
    q = s["q"][s["rows"]].float().view(c["batch"], n, kv, g, d).permute(0, 2, 1, 3, 4).reshape(c["batch"], kv, n * g, d)
    ks, vs = (K_SCALE, V_SCALE) if c["pool"] == "fp8" else (1.0, 1.0)
    word = (node.clamp(min=0) // 32).clamp(max=s["mask"].shape[1] - 1)[:, None, :].expand(-1, n, -1)
    bit = (s["mask"][s["rows"]].gather(2, word) >> (node.clamp(min=0) % 32)[:, None, :]) & 1
    seen = (inside & (node < 0))[:, None, :] | (inside & (node >= 0))[:, None, :] & (bit != 0)
    seen = seen[:, None, :, None, :].expand(-1, -1, -1, g, -1).reshape(c["batch"], 1, n * g, -1)
    score = torch.where(seen, torch.matmul(q, k) * (ks / math.sqrt(d)), -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = weight.sum(-1, keepdim=True)
    o = torch.matmul(weight, v.permute(0, 2, 1, 3)) * vs / torch.where(total == 0, 1.0, total)
    o = o.view(c["batch"], kv, n, g, d).permute(0, 2, 1, 3, 4).reshape(c["batch"] * n, c["heads"], d)
    s["out"].copy_(o[s["flat"]])
    return s["out"]


def plain_keep(s):
    c = s["case"]
    start = s["lens"].long()[:, None] - (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    step = torch.arange(c["depth"], device="cuda")[None, :]
    kept = step < s["count"][:, None]
    spare = (s["k_pool"].shape[0] - 1) * c["block"]
    source = torch.where(kept, slot_of(s, start + s["accepted"].clamp(min=0).long()), spare).reshape(-1)
    target = torch.where(kept, slot_of(s, start + step), spare).reshape(-1)
    for pool in (s["k_pool"], s["v_pool"]):
        rows = pool.view(-1, c["kv"], c["dim"])
        rows.index_copy_(0, target, rows[source])
    s["new_lens"].copy_(start[:, 0] + s["count"])
    return {"k_pool": coded(s["k_pool"]), "v_pool": coded(s["v_pool"]), "lens": s["new_lens"]}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": exact_rope, "tree": exact_tree, "keep": exact_keep}[case["op"]](case, s)


def as_double(pool):
    return (pool.view(torch.float8_e4m3fn).float() if pool.dtype == torch.uint8 else pool).double()


def exact_rope(case, s):
    t, rot = case["tokens"] - case["pad"], case["rotary"]
    angle = s["cos_sin"].double()[s["positions"].long()[:t]]
    if case["interleaved"]:
        first = torch.arange(0, rot, 2, device="cuda")
        second = first + 1
    else:
        first = torch.arange(rot // 2, device="cuda")
        second = first + rot // 2

    def rotated(x, weight):
        y = x[:t].double()
        if weight is not None:
            y = y / torch.sqrt(torch.sum(y ** 2, 2, keepdim=True) / case["dim"] + EPS) * weight.double()
        turn = torch.complex(angle[:, None, :rot // 2], angle[:, None, rot // 2:])
        z = torch.complex(y[:, :, first], y[:, :, second]) * turn
        y = y.clone()
        y[:, :, first], y[:, :, second] = z.real, z.imag
        return y

    def written(x, pool, scale):
        out = as_double(pool).view(-1, case["kv"], case["dim"]).clone()
        out[s["slots"][:t]] = (x / scale).clamp(-448, 448) if case["pool"] == "fp8" else x
        return out.view(pool.shape)

    q = s["q_out"].double()
    q[:t] = rotated(s["q"], s["q_weight"])
    return {"q": q, "k_pool": written(rotated(s["k"], s["k_weight"]), s["k_pool"], K_SCALE),
            "v_pool": written(s["v"][:t].double(), s["v_pool"], V_SCALE)}


def exact_tree(case, s):
    out = s["out"].double()
    kv, d, block = case["kv"], case["dim"], case["block"]
    ks, vs = (K_SCALE, V_SCALE) if case["pool"] == "fp8" else (1.0, 1.0)
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        blocks = s["table"][b, :-(-length // block)].long()
        k, v = (as_double(s[x][blocks]).reshape(-1, kv, d)[:length] for x in ("k_pool", "v_pool"))
        q = s["q"][cu[b]:cu[b + 1]].double().view(n, kv, -1, d)
        words = s["mask"][cu[b]:cu[b + 1]].long() & 0xFFFFFFFF
        tree_bits = ((words[:, :, None] >> torch.arange(32, device="cuda")) & 1).reshape(n, -1)[:, :n].bool()
        seen = torch.cat([torch.ones(n, length - n, dtype=torch.bool, device="cuda"), tree_bits], 1)
        x = torch.einsum("nhgd,lhd->hgnl", q, k) * (ks / math.sqrt(d))
        x = torch.softmax(x.masked_fill(~seen, -math.inf), -1).nan_to_num(0.0)
        out[cu[b]:cu[b + 1]] = (torch.einsum("hgnl,lhd->nhgd", x, v) * vs).reshape(n, -1, d)
    return out


def exact_keep(case, s):
    table, lens, cu = s["table"].cpu().numpy(), s["lens"].tolist(), s["cu"].tolist()
    accepted, count, p = s["accepted"].tolist(), s["count"].tolist(), case["block"]
    source, target, new = [], [], []
    for b in range(case["batch"]):
        start = lens[b] - (cu[b + 1] - cu[b])
        for j in range(count[b]):
            for to, at in ((source, start + accepted[b][j]), (target, start + j)):
                to.append(int(table[b, at // p]) * p + at % p)
        new.append(start + count[b])
    got = {"lens": np.array(new, np.int32)}
    for x in ("k_pool", "v_pool"):
        old = as_double(s[x])
        rows = old.clone().view(-1, case["kv"], case["dim"])
        rows[torch.tensor(target, device="cuda")] = old.view(rows.shape)[torch.tensor(source, device="cuda")]
        got[x] = rows.view(old.shape)
    return got


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------
def work(case):
    kv, d = case["kv"], case["dim"]
    size = {"f32": 4, "bf16": 2, "fp8": 1}[case["pool"]]
    act = 4 if case["pool"] == "f32" else 2
    if case["op"] == "rope":
        t, h = case["tokens"] - case["pad"], case["heads"]
        moved = t * d * (2 * h * act + 2 * kv * (act + size)) + 12 * case["tokens"] + 4 * t * case["rotary"]
        return {"bytes": moved + (2 * d * act if case["norm"] else 0),
                "flops": t * (h + kv) * ((4 * d if case["norm"] else 0) + 3 * case["rotary"])}
    cached, drafted = lengths(case)
    total = cached + drafted
    if case["op"] == "tree":
        used = total[drafted > 0]
        blocks = int((-(-used // case["block"])).sum())
        rows = int(drafted.sum())
        pairs = int((drafted * cached + drafted * (drafted + 1) // 2).sum())
        return {"bytes": 2 * int(used.sum()) * kv * d * size + 2 * rows * case["heads"] * d * act + 4 * blocks +
                4 * rows * -(-case["nodes"] // 32) + 8 * case["batch"],
                "flops": 4 * pairs * case["heads"] * d}
    rows = int(np.minimum((case["depth"] + 1) / 2, drafted).sum())
    return {"bytes": 2 * 2 * rows * kv * d * size + case["batch"] * (4 * case["depth"] + 16), "flops": 0}

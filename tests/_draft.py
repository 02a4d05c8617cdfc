"""64-bit references and inputs for the draft-verification calls: norm + rotation +
scatter, tree attention, and the move of the accepted rows."""
import math

import numpy as np
import torch

from paged_kv_cache_wf_gb300 import binding as wf

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}


def act(pool):
    """Element type of q, k, v and the outputs for a pool type."""
    return torch.float32 if pool == "f32" else torch.bfloat16


def half_step(t):
    """Largest relative error of one rounding to type t."""
    return torch.finfo(t).eps / 2


def pool_values(pool):
    """What a pool's elements stand for (before an fp8 scale), as float64 numpy."""
    if pool.dtype == torch.uint8:
        pool = pool.view(torch.float8_e4m3fn)
    return pool.detach().cpu().to(torch.float64).numpy()


def to_pool(x, pool):
    """float64 numpy -> CPU tensor of the pool type (fp8: codes of the clamped values)."""
    t = torch.from_numpy(np.ascontiguousarray(x)).float()
    if pool == "fp8":
        nan = torch.isnan(t)
        t = t.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        t[nan] = 0x7F
        return t
    return t.to(DT[pool])


class Tree:
    """A batch of requests with drafts over a shuffled pool; rows no request owns are NaN."""

    def __init__(self, cached, drafted, H_q, H_kv, D, P, pool, seed=0, k_scale=1.0, v_scale=1.0, density=None,
                 extra_rows=0, spare_words=0, q_size=2.0):
        r = np.random.default_rng(seed)
        self.cached, self.drafted = np.asarray(cached), np.asarray(drafted)
        self.H_q, self.H_kv, self.D, self.P, self.pool = H_q, H_kv, D, P, pool
        self.B = len(cached)
        self.ks, self.vs = k_scale, v_scale
        self.lens = (self.cached + self.drafted).astype(np.int32)
        need = -(-self.lens // P)
        n = int(need.sum())
        ids = r.permutation(n + 1)
        self.N = n + 1
        M = max(1, int(need.max()))
        self.table = np.full((self.B, M), ids[-1], np.int32)    # the last block belongs to nobody
        at = 0
        for b in range(self.B):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
        self.cu = np.concatenate([[0], np.cumsum(self.drafted)]).astype(np.int32)
        self.T = int(self.cu[-1]) + extra_rows
        self.max_q = max(1, int(self.drafted.max()))
        self.max_len = max(1, int(self.lens.max()))
        k = np.full((self.N, P, H_kv, D), np.nan)
        v = np.full((self.N, P, H_kv, D), np.nan)
        size = 64.0 if pool == "fp8" else 1.0
        for b in range(self.B):
            for p in range(self.lens[b]):
                blk = self.table[b, p // P]
                k[blk, p % P] = size * r.standard_normal((H_kv, D))
                v[blk, p % P] = size * r.standard_normal((H_kv, D))
        self.k, self.v = to_pool(k, pool), to_pool(v, pool)
        self.q = torch.from_numpy(q_size * r.standard_normal((max(self.T, 1), H_q, D))).float().to(act(pool))[:self.T]
        self.words = -(-self.max_q // 32) + spare_words
        bits = np.zeros((max(self.T, 1), self.words), np.uint32)
        for b in range(self.B):
            for i in range(int(self.drafted[b])):
                row = self.cu[b] + i
                if density is not None:      # any mask, empty rows among them
                    for j in range(int(self.drafted[b])):
                        if r.random() < density:
                            bits[row, j // 32] |= np.uint32(1 << (j % 32))
                    continue
                parent = r.integers(-1, i)
                if parent >= 0:
                    bits[row] = bits[self.cu[b] + parent]
                bits[row, i // 32] |= np.uint32(1 << (i % 32))
        self.bits = bits[:self.T]
        self.scale = 1.0 / math.sqrt(D)

    def sees(self, b, i):
        """Positions that draft i of request b attends to."""
        c, n = int(self.cached[b]), int(self.drafted[b])
        row = self.bits[self.cu[b] + i]
        return list(range(c)) + [c + j for j in range(n) if (int(row[j // 32]) >> (j % 32)) & 1]

    def reference(self, bad_blocks=()):
        """(out, W, S): the softmax in 64 bits, sum p |v| a row and the largest scale * sum |q k| a row."""
        out = np.zeros((self.T, self.H_q, self.D))
        W = np.zeros_like(out)
        S = np.zeros((self.T, self.H_q, 1))
        K, V = pool_values(self.k) * self.ks, pool_values(self.v) * self.vs
        q = self.q.to(torch.float64).numpy()
        G = self.H_q // self.H_kv
        for b in range(self.B):
            for i in range(int(self.drafted[b])):
                pos = [p for p in self.sees(b, i) if (b, p // self.P) not in bad_blocks]
                if not pos:
                    continue
                blk = self.table[b, np.array(pos) // self.P]
                off = np.array(pos) % self.P
                t = self.cu[b] + i
                for g in range(self.H_q):
                    k, v = K[blk, off, g // G], V[blk, off, g // G]
                    s = k @ q[t, g] * self.scale
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[t, g] = w @ v
                    W[t, g] = w @ np.abs(v)
                    S[t, g] = (np.abs(k) @ np.abs(q[t, g])).max() * abs(self.scale)
                    if self.pool == "fp8" and self.kernel() == wf.WF_KERNEL_TENSOR_CORES:
                        # weights go there as fp16, 2^7 of them: below fp16's smallest normal number the half
                        # step is 2^-25, so 2^-32 of a sum that is at least 1; `bound` multiplies W by 2^-8 or more
                        W[t, g] += np.abs(v).sum(0) * 2.0 ** -24
                        # q goes to the tensor cores as two e4m3 parts: off by at most 2^-17 of the row's largest
                        # element in each; `bound` multiplies S by (D + 4) 2^-24
                        S[t, g] += np.abs(k).sum(-1).max() * np.abs(q[t, g]).max() * abs(self.scale) * 2.0 ** 7 / (self.D + 4)
        return out, W, S

    def device(self):
        d = dict(q=self.q.cuda(), k=self.k.cuda(), v=self.v.cuda(), table=torch.from_numpy(self.table).cuda(),
                 lens=torch.from_numpy(self.lens).cuda(), cu=torch.from_numpy(self.cu).cuda(),
                 mask=torch.from_numpy(self.bits.view(np.int32)).cuda(),
                 status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        d["out"] = torch.full_like(d["q"], 7.0)
        return d

    def scales(self):
        if self.pool != "fp8":
            return {}
        # one scale, or an array [H_kv, 1]
        return {n: x if isinstance(x, float) else x.ravel().tolist() for n, x in (("k_scale", self.ks), ("v_scale", self.vs))}

    def workspace(self):
        desc = wf.wf_pool_desc(self.N, self.P, self.H_kv, self.D, {"f32": 0, "bf16": 1, "fp8": 2}[self.pool],
                               float(np.max(self.ks)), float(np.max(self.vs)))
        n = wf.wf_paged_tree_decode_workspace_size(self.B, self.H_q, self.max_q, self.max_len, desc)
        # what it holds before a call must not matter
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def kernel(self):
        desc = wf.wf_pool_desc(self.N, self.P, self.H_kv, self.D, {"f32": 0, "bf16": 1, "fp8": 2}[self.pool],
                               float(np.max(self.ks)), float(np.max(self.vs)))
        return wf.wf_paged_tree_decode_kernel(desc, self.H_q)

    def run(self, d, ws, stream=None):
        wf.wf_paged_tree_decode(d["out"], d["q"], d["k"], d["v"], d["table"], d["lens"], d["cu"], d["mask"],
                                self.max_q, self.max_len, self.scale, ws, dev_status=d["status"], stream=stream,
                                **self.scales())
        return d["out"]

    def bound(self, ref, W, S, rounded=None):
        """How far an output may be off, element by element.

        A score is a sum of D products in fp32 (relative 2^-24 each, against scale * sum |q k| <= S), scaled and
        turned into an exponent in fp32: two more roundings of at most S.  An error ds in the exponent moves a weight
        by a factor of 1 + 2 ds; exp2 and the sums over positions add at most 2^-20.  Weights that go to the tensor
        cores are rounded to bf16 first (numerator only): half a step (`rounded`; by default as the geometry's kernel
        does).  The numerator and the sum both move, hence the 2.  Last, one rounding of the output.
        """
        if rounded is None:
            rounded = self.kernel() == wf.WF_KERNEL_TENSOR_CORES
        ds = (self.D + 4) * 2.0 ** -24 * S
        weight = 2 * (2 * ds + 2.0 ** -20)
        if rounded:
            weight = weight + half_step(torch.bfloat16)
        t = act(self.pool)
        return half_step(t) * np.abs(ref) + weight * W * (1 + half_step(t)) + 1e-30


def check(tree, got, ref=None):
    ref, W, S = tree.reference() if ref is None else ref
    got = got.detach().cpu().to(torch.float64).numpy()
    n = int(tree.cu[-1])
    lim = tree.bound(ref, W, S)
    off = np.abs(got[:n] - ref[:n])
    assert np.isfinite(got[:n]).all(), "non-finite outputs"
    assert (off <= lim[:n]).all(), f"off by {off.max():.3e}, {(off / lim[:n]).max():.2f} of what is allowed"


# ------------------------------------------------------------------------------------------
# norm and rotation
# ------------------------------------------------------------------------------------------
def cos_sin_table(rows, rot, base=10000.0):
    a = np.arange(rows)[:, None] * base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))[None, :]
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float()


def norm_rope_reference(x, w, eps, table, positions, interleaved):
    """(y, size) in 64 bits of [T, H, D]: the result, and |a| + |b| of each element's pair (what its rotation's
    rounding is relative to)."""
    y = x.detach().cpu().to(torch.float64).numpy().copy()
    if w is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * w.detach().cpu().to(torch.float64).numpy()
    size = np.abs(y)
    if table is None:
        return y, size
    t = table.detach().cpu().to(torch.float64).numpy()
    rot = t.shape[1]
    half = rot // 2
    first = np.arange(0, rot, 2) if interleaved else np.arange(half)
    second = first + (1 if interleaved else half)
    row = t[np.asarray(positions)]
    c, s = row[:, None, :half], row[:, None, half:]
    a, b = y[..., first].copy(), y[..., second].copy()
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = np.abs(a) + np.abs(b)
    return y, size

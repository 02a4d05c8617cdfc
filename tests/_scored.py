"""64-bit references and inputs for scored attention."""
import math

import numpy as np
import torch

from paged_kv_cache_wf_gb300 import binding as wf
from tests import _draft as R


class Scored(R.Tree):
    """New tokens behind their cached ones over a shuffled pool; rows that nobody sees are NaN.

    view: None (a row sees what is not behind it), "documents", "prefix", "any" (random ranges, empty ones and ones past
    the request among them) or "empty"."""

    def __init__(self, cached, new, H_q, H_kv, D, P, pool, seed=0, cap=0.0, window=0, slopes=False, view=None, **kw):
        super().__init__(cached, new, H_q, H_kv, D, P, pool, seed=seed, **kw)
        r = np.random.default_rng(seed + 1000)
        self.cap, self.window, self.view = cap, window, view
        self.slopes = None
        if slopes:
            self.slopes = (2.0 ** (-8 * (1 + np.arange(H_q)) / H_q) * np.where(np.arange(H_q) % 5 == 4, -0.05, 1)).astype(
                np.float32)
        self.ranges = None
        if view is not None:
            rows = []
            for c, n in zip(self.cached, self.drafted):
                at, total = c + np.arange(n), int(c + n)
                if view == "documents":
                    starts = np.unique(np.concatenate([[0], r.integers(0, total + 1, 1 + total // 60)]))
                    x = np.stack([starts[np.searchsorted(starts, at, side="right") - 1], at + 1], 1)
                    x[3::11] = 7
                elif view == "prefix":
                    x = np.stack([np.zeros_like(at), np.maximum(at + 1, r.integers(0, total + 1))], 1)
                elif view == "any":
                    x = np.sort(r.integers(-5, total + 9, (int(n), 2)), 1)
                    x[::7] = x[::7, ::-1]
                else:
                    x = np.zeros((int(n), 2), np.int64)
                rows.append(x)
            x = np.concatenate(rows + [np.full((self.T - int(self.cu[-1]), 2), -3)])
            self.ranges = x.astype(np.int32).reshape(-1, 2)
        self.forget()

    def range(self, b, i):
        """[begin, end) of row i of request b."""
        at, total = int(self.cached[b]) + i, int(self.lens[b])
        lo, hi = (0, at + 1) if self.ranges is None else (int(x) for x in self.ranges[self.cu[b] + i])
        if self.window:
            lo = max(lo, at - self.window + 1)
        lo = min(max(lo, 0), total)
        return lo, max(lo, min(hi, total))

    def sees(self, b, i):
        return list(range(*self.range(b, i)))

    def seen(self, b):
        some = np.zeros(int(self.lens[b]), bool)
        for i in range(int(self.drafted[b])):
            some[slice(*self.range(b, i))] = True
        return some

    def forget(self):
        """Pool rows that no row of their request sees become NaN, and blocks before the first and behind the last position
        that one sees lose their place."""
        for b in range(self.B):
            some = self.seen(b)
            for p in np.nonzero(~some)[0]:
                for pool in (self.k, self.v):
                    pool[int(self.table[b, p // self.P]), p % self.P] = 0x7F if self.pool == "fp8" else math.nan
            for j in range(-(-int(self.lens[b]) // self.P)):
                if not some[j * self.P:].any() or not some[:(j + 1) * self.P].any():
                    self.table[b, j] = -1 if j % 2 else self.N + 5

    def reference(self, bad_blocks=()):
        """(out, W, S) as R.Tree's: the error of the rules is in S, in units of its factor in `bound`."""
        out = np.zeros((self.T, self.H_q, self.D))
        W, S = np.zeros_like(out), np.zeros((self.T, self.H_q, 1))
        K, V = R.pool_values(self.k) * self.ks, R.pool_values(self.v) * self.vs
        q = self.q.to(torch.float64).numpy()
        G, tc = self.H_q // self.H_kv, self.kernel() == wf.WF_KERNEL_TENSOR_CORES
        unit = (self.D + 4) * 2.0 ** -24
        for b in range(self.B):
            for i in range(int(self.drafted[b])):
                pos = np.array([p for p in self.sees(b, i) if (b, p // self.P) not in bad_blocks], int)
                if not len(pos):
                    continue
                blk, off, t, at = self.table[b, pos // self.P], pos % self.P, self.cu[b] + i, int(self.cached[b]) + i
                k, v = K[blk, off], V[blk, off]                                  # [L, H_kv, D]
                qg = q[t].reshape(self.H_kv, G, self.D)
                s = np.einsum("hgd,lhd->hgl", qg, k).reshape(self.H_q, -1) * self.scale
                size = np.einsum("hgd,lhd->hgl", np.abs(qg), np.abs(k)).reshape(self.H_q, -1).max(-1) * abs(self.scale)
                if self.pool == "fp8" and tc:      # as R.Tree.reference says
                    part = np.abs(k).sum(-1).max(0)[:, None] * np.abs(qg).max(-1) * abs(self.scale)
                    size = size + part.reshape(-1) * 2.0 ** 7 / (self.D + 4)
                more = np.zeros(self.H_q)
                if self.cap:
                    # tanh does not grow errors.  The tensor cores' 1 - 2 / (1 + 2^z): 2^z is off by 2^-22 and z's own
                    # rounding (0.45 2^-24 of a tanh at most), the sum by 2^-24, the reciprocal by 2^-23, of a number below 1
                    # and times 2 cap, and the result is rounded: below cap 2^-20.  Their polynomial of small arguments:
                    # 2^-20.1 and six roundings of at most 0.4 2^-24, below cap 2^-19.  tanhf: 2^-22, and two roundings.
                    s = self.cap * np.tanh(s / self.cap)
                    more += self.cap * 2.0 ** (-19 if tc else -21)
                if self.slopes is not None:
                    # a slope and its product with a distance round, and so does the sum: 4 half steps of each, from the
                    # position that the kernel measures distances from
                    lo, hi = self.range(b, i)
                    near = min(at, hi - 1)
                    bias = np.abs(self.slopes.astype(float))[:, None] * np.abs(pos - near)[None, :]
                    more += 2.0 ** -22 * (bias.max(-1) + np.abs(s).max(-1))
                    s = s - self.slopes.astype(float)[:, None] * np.abs(pos - at)[None, :]
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                wg = w.reshape(self.H_kv, G, -1)
                out[t] = np.einsum("hgl,lhd->hgd", wg, v).reshape(self.H_q, self.D)
                W[t] = np.einsum("hgl,lhd->hgd", wg, np.abs(v)).reshape(self.H_q, self.D)
                if self.pool == "fp8" and tc:
                    W[t] += np.repeat(np.abs(v).sum(0), G, 0) * 2.0 ** -24
                S[t, :, 0] = size + more / unit
        return out, W, S

    def device(self):
        d = super().device()
        d["ranges"] = None if self.ranges is None else torch.from_numpy(self.ranges).cuda()
        d["slopes"] = None if self.slopes is None else torch.from_numpy(self.slopes).cuda()
        return d

    def desc(self):
        return wf.wf_pool_desc(self.N, self.P, self.H_kv, self.D, {"f32": 0, "bf16": 1, "fp8": 2}[self.pool],
                               float(np.max(self.ks)), float(np.max(self.vs)))

    def workspace(self):
        n = wf.wf_paged_scored_attention_workspace_size(self.B, self.H_q, self.T, self.max_q, self.max_len, self.desc())
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, d, ws, stream=None):
        wf.wf_paged_scored_attention(d["out"], d["q"], d["k"], d["v"], d["table"], d["lens"], d["cu"], self.max_q, self.max_len,
                                     self.scale, ws, cap=self.cap, window=self.window, slopes=d["slopes"],
                                     row_ranges=d["ranges"], dev_status=d["status"], stream=stream, **self.scales())
        return d["out"]

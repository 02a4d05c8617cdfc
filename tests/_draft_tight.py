"""The bound on tree attention over fp8 pools on the tensor cores, with the weights' own rounding: fp16."""
import numpy as np
import torch

from tests import _draft as R

FP8 = dict(k_scale=1 / 64, v_scale=1 / 96)
CASES = {
    # few positions a row: a weight's rounding is not averaged away, and stands out from the output's where values cancel
    "few positions d128": lambda: Tight([0, 1, 2, 3, 5, 1], [1, 4, 3, 2, 4, 5], 32, 8, 128, 16, "fp8", seed=100, **FP8),
    "few positions d64": lambda: Tight([1, 2, 0, 3, 1, 4], [2, 4, 3, 1, 5, 4], 32, 8, 64, 16, "fp8", seed=101, **FP8),
    "one query head": lambda: Tight([1, 2, 3, 0, 4], [4, 3, 2, 5, 1], 12, 12, 64, 32, "fp8", seed=102, **FP8),
    "ragged d128": lambda: Tight([40, 130, 3], [9, 33, 5], 8, 2, 128, 16, "fp8", seed=103, **FP8),
    "ragged d64": lambda: Tight([40, 260, 3], [9, 33, 70], 8, 2, 64, 16, "fp8", seed=104, **FP8),
}


class Tight(R.Tree):
    def tight(self, weights=None):
        """(ref, bound) an output; with `weights`, what a kernel that rounds its weights so (softmax weights relative
        to the row's largest, float64 -> float64) would give in the place of the reference.

        As R.Tree.bound, of which only what belongs to fp8 pools is kept: half a step of fp16 (2^-11) for a weight, and
        2^-25 of 2^7 where it is below fp16's normal numbers, against a sum that is at least 1.  The products of P V are
        added 16 positions at a time in fp32, cut rather than rounded: 2^-23 a step of what is added so far, at most W;
        the join of the streams and the scale add a few.
        """
        ref, _, S = self.reference()
        K, V = R.pool_values(self.k) * self.ks, R.pool_values(self.v) * self.vs
        q = self.q.to(torch.float64).numpy()
        G = self.H_q // self.H_kv
        lim, got = np.zeros_like(ref), np.zeros_like(ref)
        h = R.half_step(torch.bfloat16)
        for b in range(self.B):
            for i in range(int(self.drafted[b])):
                pos = np.array(self.sees(b, i))
                t = self.cu[b] + i
                if not len(pos):
                    continue
                blk, off = self.table[b, pos // self.P], pos % self.P
                for g in range(self.H_q):
                    k, v = K[blk, off, g // G], V[blk, off, g // G]
                    s = k @ q[t, g] * self.scale
                    w = np.exp(s - s.max())
                    if weights is not None:
                        got[t, g] = (weights(w) @ v) / w.sum()
                    W, A = (w / w.sum()) @ np.abs(v), np.abs(v).sum(0)
                    ds = (self.D + 4) * 2.0 ** -24 * S[t, g]
                    share = 2 * (2 * ds + 2.0 ** -20) + R.half_step(torch.float16) + (len(pos) / 16 + 16) * 2.0 ** -23
                    lim[t, g] = h * np.abs(ref[t, g]) + (share * W + 2.0 ** -32 * A) * (1 + h) + 1e-30
        return (ref if weights is None else got), lim

"""64-bit references of the calls that keep a step on the GPU: verification of drafts, a step's tables, trimmed blocks."""
import numpy as np
import torch


def verify(target, draft, tokens, parents, coins, pick, max_accepted):
    """(path, next token) of one request.  target, draft [n, V] float64 (draft None: fixed candidates); what is left of
    the target is divided by its sum at each step, as the method is usually written."""
    n = len(tokens)
    path = [0]
    clean = lambda x: np.where(x > 0, x, 0.0)    # noqa: E731  (NaN and negatives count as 0)
    draft = None if draft is None else clean(draft)
    while True:
        u = path[-1]
        p = clean(target[u])
        left = p.copy()
        if len(path) < max_accepted:
            kept = None
            for i in range(u + 1, n):
                if parents[i] != u:
                    continue
                x = tokens[i]
                if draft is not None:
                    if coins[i] * draft[u][x] < left[x]:
                        kept = i
                        break
                    left = clean(left - draft[u])
                    if left.sum() > 0:
                        left = left / left.sum()
                else:
                    rest = 1.0 - sum(p[y] for y in {tokens[j] for j in range(u + 1, i) if parents[j] == u})
                    if coins[i] * rest < left[x]:
                        kept = i
                        break
                    left[x] = 0.0
            if kept is not None:
                path.append(kept)
                continue
        if not left.sum() > 0:
            left = p
        up = np.cumsum(left)
        if not (up[-1] > 0 and np.isfinite(up[-1])):
            return path, -1
        return path, int(np.argmax(up > pick * up[-1]))


def build(table, lens, new, free, num_free, rows, block, depths=None):
    """(table, new lengths, free left, offsets, slots, positions) of a step, token by token."""
    table, stack = np.array(table), list(free[:num_free])
    slots, positions, cu = [], [], [0]
    for b, (length, n) in enumerate(zip(lens, new)):
        for i in range(length, length + n):
            if i % block == 0:
                table[b, i // block] = stack.pop()
            slots.append(int(table[b, i // block]) * block + i % block)
            positions.append(i if depths is None else length + int(depths[len(positions)]))
        cu.append(len(slots))
    pad = rows - len(slots)
    assert pad >= 0
    return (table, np.asarray(lens) + np.asarray(new), len(stack), np.array(cu), np.array(slots + [-1] * pad),
            np.array(positions + [0] * pad))


def trim(table, lens, kept, free, num_free, block):
    """(free list, its length)."""
    back = [int(table[b][j]) for b in range(len(lens)) for j in range(-(-kept[b] // block), -(-lens[b] // block))]
    free = np.array(free)
    free[num_free:num_free + len(back)] = back[::-1]
    return free, num_free + len(back)


def i32(x):
    return torch.as_tensor(np.array(x), dtype=torch.int32).cuda()


class Requests:
    """Requests over a shuffled pool: `lens` tokens held each, `spare` blocks free."""

    def __init__(self, lens, block, spare, M=None, seed=0):
        r = np.random.default_rng(seed)
        self.lens, self.block = np.asarray(lens, np.int64), block
        self.B = len(lens)
        need = -(-self.lens // block)
        total = int(need.sum())
        self.N = total + spare
        ids = r.permutation(self.N)
        self.M = M or max(1, int(need.max(initial=0)) + spare)
        self.table = np.full((self.B, self.M), -7, np.int64)       # what is not held is nobody's
        self.table[np.arange(self.M)[None, :] < need[:, None]] = ids[:total]
        self.free = np.full(self.N, -9, np.int64)
        self.free[:spare] = ids[total:]
        self.num_free = spare

"""Plain 64-bit references of the drafted-step operators (tree attention, step
plan, commit), and random trees and pools for their tests."""
from __future__ import annotations

import math

import numpy as np

SCALE = 1.0 / math.sqrt(192.0)
PAGE = 64


def random_parents(g, n, roots=1):
    """Parents in topological order; the first `roots` nodes (at least one) have none."""
    return [-1 if i < max(1, roots) else int(g.integers(0, i)) for i in range(n)]


def ancestors(parents):
    """Boolean [n, n]: k is i or an ancestor of i."""
    n = len(parents)
    a = np.zeros((n, n), bool)
    for i, p in enumerate(parents):
        if p >= 0:
            a[i] = a[p]
        a[i, i] = True
    return a


def pack_mask(seen, words):
    """Boolean [rows, n] -> int64 [rows, words] (bit k of word w: column 64 w + k)."""
    out = np.zeros((seen.shape[0], words), np.uint64)
    for k in range(min(seen.shape[1], 64 * words)):
        out[:, k // 64] |= seen[:, k].astype(np.uint64) << np.uint64(k % 64)
    return out.view(np.int64)


def page_table(lens, spare, g, width=None):
    """A permuted pool: block table [B, width] (-1 past each sequence's pages) and the pool size."""
    need = [-(-int(x) // PAGE) for x in lens]
    total = sum(need) + spare
    ids = g.permutation(total).astype(np.int32)
    bt = np.full((len(lens), width or max(1, max(need))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    return bt, total


def attend(q, rows, seen, scale=SCALE):
    """One drafted token: q [H, 576], rows [L, 576], seen [L] (float64 torch) ->
    (o [H, 512], lse [H], a [H, 512] = sum p |c| / sum p, l [H] = sum e^{z - max z})."""
    import torch
    H = q.shape[0]
    if not bool(seen.any()):
        z0 = torch.zeros((H, 512), dtype=torch.float64, device=q.device)
        inf = torch.full((H,), -math.inf, dtype=torch.float64, device=q.device)
        return z0, inf, z0, torch.ones_like(inf)
    x = rows[seen]
    z = scale * (q @ x.T)
    m = z.amax(1, keepdim=True)
    e = (z - m).exp()
    l = e.sum(1, keepdim=True)
    c = x[:, :512]
    return e @ c / l, (m + l.log())[:, 0], e @ c.abs() / l, l[:, 0]


class Plan:
    """mla_step_plan, sequence by sequence, on Python integers."""

    def __init__(self, lens, counts, held, table, free, free_count, num_pages, parents=None, words=0, max_rows=None,
                 chain_mask=False):
        B, width = table.shape
        self.table, self.free = table.copy(), free.copy()
        need = [-(-(l + n) // PAGE) for l, n in zip(lens, counts)]
        stack = [int(x) for x in free[:free_count]]
        for b in range(B):
            for k in range(need[b], held[b]):
                stack.append(int(self.table[b, k]))
                self.table[b, k] = -1
        self.free[free_count:len(stack)] = stack[free_count:]
        for b in range(B):
            for k in range(held[b], need[b]):
                self.table[b, k] = stack.pop()
        self.held, self.free_count = need, len(stack)
        self.row_start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        N = int(self.row_start[-1])
        R = N if max_rows is None else max_rows
        self.kv_lens = [l + n for l, n in zip(lens, counts)]
        self.seq_ids = np.full(R, -1, np.int32)
        self.slots = np.full(R, -1, np.int32)
        self.positions = np.zeros(R, np.int32)
        self.mask = np.zeros((R, words), np.int64)
        for b in range(B):
            s, n = int(self.row_start[b]), counts[b]
            if n == 0:
                continue
            par = list(range(-1, n - 1)) if parents is None else [int(x) for x in parents[s:s + n]]
            a = ancestors(par)
            for i in range(n):
                r = lens[b] + i
                self.seq_ids[s + i] = b
                self.slots[s + i] = self.table[b, r // PAGE] * PAGE + r % PAGE
                self.positions[s + i] = lens[b] + int(a[i].sum()) - 1
            if words:
                self.mask[s:s + n] = pack_mask(a, words)


def commit_rows(rows, table, kv_lens, row_start, counts, nodes):
    """Logical pool rows [num_pages*64, ...] after the commit, and the new lengths."""
    out = rows.copy()
    lens = []
    for b in range(len(counts)):
        n = int(row_start[b + 1] - row_start[b])
        base = int(kv_lens[b]) - n
        slot = lambda r: int(table[b, r // PAGE]) * PAGE + r % PAGE  # noqa: E731
        for j in range(counts[b]):
            out[slot(base + j)] = rows[slot(base + int(nodes[row_start[b] + j]))]
        lens.append(base + counts[b])
    return out, lens

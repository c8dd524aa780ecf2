"""Plain 64-bit and whole-number implementations of the page tables, the rotary
positions of several axes, and the attention over selected blocks, for the tests."""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------------------
# page tables
# ---------------------------------------------------------------------------

class Pages:
    """The page tables of a batch as lists, updated one page at a time."""

    def __init__(self, B, max_blocks, page, num_pages, order):
        self.page, self.max_blocks, self.num_pages = page, max_blocks, num_pages
        self.table = [[-1] * max_blocks for _ in range(B)]
        self.stack = list(order)          # all places; the first self.count are free
        self.count = num_pages
        self.lens = [0] * B

    def need(self, n):
        return -(-n // self.page)

    def update(self, new):
        """(pos, row_offsets, slots, positions, some sequence was refused)"""
        new = [n if 0 <= n <= self.max_blocks * self.page else old for n, old in zip(new, self.lens)]
        gone = []
        for b, n in enumerate(new):
            for j in range(self.need(n), self.need(self.lens[b])):
                gone.append(self.table[b][j])
                self.table[b][j] = -1
        for p in reversed(gone):
            self.stack[self.count] = p
            self.count += 1
        pos, offsets, slots, positions, refused = list(self.lens), [0], [], [], False
        for b, n in enumerate(new):
            old, want = self.lens[b], self.need(n) - self.need(self.lens[b])
            if want > 0 and (refused or want > self.count):
                refused, n = True, old
            for j in range(self.need(old), self.need(n)):
                self.count -= 1
                self.table[b][j] = self.stack[self.count]
            for t in range(old, n):
                slots.append(self.table[b][t // self.page] * self.page + t % self.page)
                positions.append(t)
            offsets.append(len(slots))
            self.lens[b] = n
        return pos, offsets, slots, positions, refused


# ---------------------------------------------------------------------------
# rotary positions of several axes
# ---------------------------------------------------------------------------

def axes_of(sections, dealt):
    if not dealt:
        return np.repeat(np.arange(len(sections)), sections)
    left, out, a = list(sections), [], 0
    while sum(left):
        if left[a]:
            out.append(a)
            left[a] -= 1
        a = (a + 1) % len(left)
    return np.array(out)


def turn_exact(x, positions, turns, axes, factor, interleaved):
    """float64 rows [N, H, D] turned by positions [A, N]: phases in whole 2^-64 turns."""
    half = len(turns)
    p = positions.astype(np.int64)[axes].T  # [N, half]
    with np.errstate(over="ignore"):
        phase = p.astype(np.uint64) * turns[None, :]
    angle = phase.astype(np.float64) / 2.0 ** 64 * 2 * np.pi  # (angles below 2 pi: float64 of the phase is exact to 2^-53)
    turn = factor * np.exp(1j * angle)[:, None, :]
    y = x.copy()
    if interleaved:
        z = (x[..., 0:2 * half:2] + 1j * x[..., 1:2 * half:2]) * turn
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
    else:
        z = (x[..., :half] + 1j * x[..., half:2 * half]) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    return y


# ---------------------------------------------------------------------------
# bounds, selection, attention
# ---------------------------------------------------------------------------

def bounds(rows):
    """(codes int8 [Hkv, 2, D], scales float32 [Hkv]) of a block's keys, float32 [block, Hkv, D]."""
    hi, lo = rows.max(0), rows.min(0)
    with np.errstate(invalid="ignore", divide="ignore"):
        s = np.abs(rows).max((0, 2)).astype(np.float32) / np.float32(127)
        up, down = np.ceil(hi / s[:, None]), np.floor(lo / s[:, None])
    bad = ~np.isfinite(rows).all((0, 2))
    s = np.where(bad, np.float32(np.nan), s).astype(np.float32)
    codes = np.stack([up, down], 1)
    codes = np.where((bad | (s == 0))[:, None, None], 0, codes)
    return np.clip(codes, -127, 127).astype(np.int8), s


def score(q, codes, scales):
    """float32 scores [n] of blocks (codes [n, 2, D], scales [n]) for one group's query rows, float32 [G, D]."""
    best = np.full(len(scales), -np.inf, np.float32)
    with np.errstate(all="ignore"):
        for row in q:
            if not np.isfinite(row).all():
                continue
            s = np.abs(row).max().astype(np.float32) / np.float32(127)
            c = np.clip(np.rint(row / s), -127, 127) if s > 0 else np.zeros_like(row)
            c = c.astype(np.int64)
            whole = codes[:, 0].astype(np.int64) @ np.maximum(c, 0) + codes[:, 1].astype(np.int64) @ np.minimum(c, 0)
            best = np.maximum(best, whole.astype(np.float32) * s)
        best = best * scales
    return np.where(np.isnan(best), np.float32(np.inf), best) + np.float32(0)


def select(scores, keep, first, last, missing=()):
    """The kept blocks, ascending, -1 behind; `missing` blocks rank below all others."""
    n = len(scores)
    if n <= keep:
        return list(range(n)) + [-1] * (keep - n)
    rank = []
    for j in range(n):
        forced = j < first or j >= n - last
        rank.append((0, 0, j) if forced else (2, 0, j) if j in missing else (1, -float(scores[j]), j))
    return sorted(j for _, _, j in sorted(rank)[:keep])


def attend(q, k, v, blocks, seen, block, scale):
    """One KV head of one query token: q [G, D], k, v [S, D] (float64), blocks a list; (out, lse, spread [G, D])."""
    tokens = []
    for j in blocks:
        if j >= 0:
            tokens += range(min(j * block, max(seen, 0)), min((j + 1) * block, max(seen, 0)))
    G, D = q.shape
    if not tokens:
        return np.zeros((G, D)), np.full(G, -np.inf), np.zeros((G, D))
    s = scale * (q @ k[tokens].T)
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    l = w.sum(1, keepdims=True)
    w /= l
    out = w @ v[tokens]
    spread = np.stack([(w[g][:, None] * np.abs(v[tokens] - out[g])).sum(0) for g in range(G)])
    return out, (m + np.log(l))[:, 0], spread

"""Plain CPU oracle of the prompt path: rotary positions, attention of several
new tokens, and the page pool.

TEST INFRASTRUCTURE ONLY, like kvq_oracle.py: fp64 numpy and plain loops,
written from the definitions in include/kvq.h, sharing no code with the CUDA
library.
"""
from __future__ import annotations

import math

import numpy as np


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

def rope_frequencies(rd, base=10000.0, scaling="none", factor=1.0, context=0, low=0.0, high=0.0):
    """Radians per position of each of the rd / 2 pairs, and the amplitude."""
    low = low or 1.0
    high = high or (32.0 if scaling == "yarn" else 4.0)
    amp = 1.0
    if scaling == "ntk":
        base = base * factor ** (rd / (rd - 2))
    ws = []
    if scaling == "yarn":
        def pair(turns):
            return rd * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(pair(high)), 0)
        hi = min(math.ceil(pair(low)), rd - 1)
        if factor > 1:
            amp = 0.1 * math.log(factor) + 1.0
    for i in range(rd // 2):
        w = base ** (-2.0 * i / rd)
        if scaling == "linear":
            w = w / factor
        elif scaling == "bands":
            turns = context * w / (2 * math.pi)
            if turns <= low:
                w = w / factor
            elif turns < high:
                m = (turns - low) / (high - low)
                w = m * w + (1 - m) * w / factor
        elif scaling == "yarn":
            m = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = (1 - m) * w + m * w / factor
        ws.append(w)
    return np.array(ws), amp


def rope_rotate(x16, positions, ws, amp, rd, interleaved):
    """Rotated vectors in fp64, and a bound on this oracle's own error.

    x16 fp16 [..., H, D], positions integer [...]; one position per H rows.
    The angle position * w carries the roundings of w and of the product, up
    to 2^-50 of itself; the library's w is a whole number of 2^-64 turns, so
    its angle may differ by position * pi 2^-64 more, and it works the turn out
    to 2^-42."""
    x = np.asarray(x16, dtype=np.float64)
    pos = np.asarray(positions, dtype=np.float64)[..., None]
    angle = pos * ws
    c, s = (amp * np.cos(angle))[..., None, :], (amp * np.sin(angle))[..., None, :]
    own = (np.abs(angle) * 2.0 ** -50 + np.abs(pos) * math.pi * 2.0 ** -64 + 2.0 ** -42)[..., None, :] * amp
    y, err = x.copy(), np.zeros_like(x)
    if interleaved:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y[..., 0:rd:2], y[..., 1:rd:2] = a * c - b * s, b * c + a * s
        err[..., 0:rd:2] = err[..., 1:rd:2] = own * (np.abs(a) + np.abs(b))
    else:
        h = rd // 2
        a, b = x[..., :h], x[..., h:rd]
        y[..., :h], y[..., h:rd] = a * c - b * s, b * c + a * s
        err[..., :h] = err[..., h:rd] = own * (np.abs(a) + np.abs(b))
    return y, err


# ---------------------------------------------------------------------------
# Attention of several new tokens of one sequence
# ---------------------------------------------------------------------------

def extend_attention(q, k, v, before, scale, mapped=None):
    """q [n][Hq][D], k and v [Hkv][before + n][D] in fp64: out [n][Hq][D], and
    per output the sum of weights times |v| (what the roundings scale with).
    mapped[j] False leaves position j out."""
    n, Hq, D = q.shape
    G = Hq // k.shape[0]
    L = k.shape[1]
    out, mass = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    for t in range(n):
        see = np.arange(L) <= before + t
        if mapped is not None:
            see &= mapped
        if not see.any():
            continue
        for h in range(Hq):
            s = k[h // G][see] @ q[t, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[t, h] = p @ v[h // G][see]
            mass[t, h] = p @ np.abs(v[h // G][see])
    return out, mass


# ---------------------------------------------------------------------------
# Page pool, in plain loops over sequences and blocks
# ---------------------------------------------------------------------------

class Pool:
    def __init__(self, ref, table, page):
        self.ref = [int(r) for r in ref]
        self.table = [[int(e) for e in row] for row in table]
        self.page = page

    def _valid(self, e):
        return 0 <= e < len(self.ref)

    def reorder(self, parent, keep=None):
        old = [list(r) for r in self.table]
        M = len(old[0]) if old else 0
        for b, p in enumerate(parent):
            row = [-1] * M
            if 0 <= p < len(old):
                blocks = M if keep is None else -(-keep[b] // self.page)
                if keep is not None and not 0 <= keep[b] <= M * self.page:
                    blocks = 0
                row = [e if j < blocks and self._valid(e) else -1 for j, e in enumerate(old[p])]
            self.table[b] = row
        for row, step in ((old, -1), (self.table, 1)):
            for r in row:
                for e in r:
                    if self._valid(e):
                        self.ref[e] += step

    def reserve(self, before, new):
        """(src, dst, granted), or None when the free pages do not suffice."""
        B = len(self.table)
        free = [i for i, r in enumerate(self.ref) if r == 0]
        src, dst, granted, takes = [-1] * B, [-1] * B, [0] * B, []
        asked = {}
        for b in range(B):
            if not 0 < new[b] or before[b] < 0 or before[b] + new[b] > len(self.table[b]) * self.page:
                continue
            granted[b] = new[b]
            for j in range(before[b] // self.page, -(-(before[b] + new[b]) // self.page)):
                e = self.table[b][j]
                holds = j * self.page < before[b]
                if not self._valid(e):
                    takes.append((b, j, -1))
                    continue
                refs = self.ref[e]
                if holds:
                    refs -= asked.get(e, 0)
                    asked[e] = asked.get(e, 0) + 1
                if refs > 1:
                    takes.append((b, j, e))
        if len(takes) > len(free):
            return None
        for page, (b, j, e) in zip(free, takes):
            self.table[b][j] = page
            if e >= 0 and j * self.page < before[b]:
                src[b], dst[b] = e, page
        for page, (_, _, e) in zip(free, takes):
            self.ref[page] = 1
            if e >= 0:
                self.ref[e] -= 1
        return src, dst, granted

    def compact(self):
        live = [i for i, r in enumerate(self.ref) if r > 0]
        n = len(live)
        movers = [i for i in live if i >= n]
        holes = [i for i in range(n) if self.ref[i] <= 0]
        to = dict(zip(movers, holes))
        for row in self.table:
            for j, e in enumerate(row):
                if e >= 0:
                    row[j] = to.get(e, e) if self._valid(e) and self.ref[e] > 0 else -1
        for s, d in to.items():
            self.ref[d], self.ref[s] = self.ref[s], 0
        return movers, holes, n

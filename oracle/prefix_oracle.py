"""Plain CPU oracle of rotary positions by axis and of shared prefixes.

TEST INFRASTRUCTURE ONLY, like kvq_oracle.py: fp64 numpy and plain loops,
written from the definitions in include/kvq.h, sharing no code with the CUDA
library.
"""
from __future__ import annotations

import math

import numpy as np

from . import prompt_oracle as P


def axis_table(pairs, cycled):
    """(axis, which of the axis' pairs) of every pair."""
    if not cycled:
        return [(a, j) for a, n in enumerate(pairs) for j in range(n)]
    out, used, a = [], [0] * len(pairs), 0
    while len(out) < sum(pairs):
        if used[a] < pairs[a]:
            out.append((a, used[a]))
            used[a] += 1
        a = (a + 1) % len(pairs)
    return out


def axis_frequencies(pairs, cycled=False, own_ladders=False, base=10000.0, scaling="none", factor=1.0, context=0):
    """Radians a position of every pair, each pair's axis, and the amplitude."""
    table = axis_table(pairs, cycled)
    whole, amp = P.rope_frequencies(2 * sum(pairs), base, scaling, factor, context)
    if own_ladders:
        ladders = [P.rope_frequencies(2 * n, base, scaling, factor, context)[0] for n in pairs]
        whole = np.array([ladders[a][j] for a, j in table])
    return whole, np.array([a for a, _ in table]), amp


def rotate_axes(x16, positions, ws, axis, amp, rd, interleaved):
    """Rotated vectors in fp64 and a bound on this oracle's error: x16 fp16
    [..., H, D], positions integer [..., axes].  As prompt_oracle.rope_rotate,
    pair by pair."""
    x = np.asarray(x16, dtype=np.float64)
    y, err = x.copy(), np.zeros_like(x)
    for i in range(rd // 2):
        pos = np.asarray(positions, dtype=np.float64)[..., axis[i], None]
        angle = pos * ws[i]
        c, s = amp * np.cos(angle), amp * np.sin(angle)
        own = (np.abs(angle) * 2.0 ** -50 + np.abs(pos) * math.pi * 2.0 ** -64 + 2.0 ** -42) * amp
        i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + rd // 2)
        a, b = x[..., i0], x[..., i1]
        y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
        err[..., i0] = err[..., i1] = own * (np.abs(a) + np.abs(b))
    return y, err


def find_prefixes(table, pages, page, lens, min_tokens, most):
    """kvq_prefix_find in plain loops: (prefix_of, prefix_lens, prefix_table,
    tail_table, tail_lens, found)."""
    B, M = len(table), len(table[0]) if len(table) else 0
    k = max(1, -(-min_tokens // page))
    whole = [n // page if 0 <= n <= M * page else 0 for n in lens]

    def valid(e):
        return 0 <= e < pages

    groups = {}
    runs = {}
    for b in range(B):
        if whole[b] < k or not valid(table[b][k - 1]):
            continue
        lead = next(x for x in range(B) if whole[x] >= k and table[x][k - 1] == table[b][k - 1])
        run = 0
        while run < min(whole[b], whole[lead]) and valid(table[b][run]) and table[b][run] == table[lead][run]:
            run += 1
        if run >= k:
            groups.setdefault(lead, []).append(b)
            runs[b] = run
    of, plens = [-1] * B, [0] * most
    ptable = [[-1] * M for _ in range(most)]
    found = 0
    for lead in sorted(groups):
        best = max(((sum(runs[y] >= runs[x] for y in groups[lead]) - 1) * runs[x], runs[x]) for x in groups[lead])
        if best[0] == 0:
            continue
        if found < most:
            plens[found] = best[1] * page
            ptable[found][:best[1]] = list(table[lead][:best[1]])
            for b in groups[lead]:
                if runs[b] >= best[1]:
                    of[b] = found
        found += 1
    tails, tlens = [], []
    for b in range(B):
        n = plens[of[b]] if of[b] >= 0 else 0
        row = list(table[b][n // page:])
        tails.append(row + [-1] * (M - len(row)))
        tlens.append(lens[b] - n)
    return of, plens, ptable, tails, tlens, found


def prefix_attention(q, kp, vp, kt, vt, before, scale, prefix_mapped=None, tail_mapped=None):
    """One sequence: q [n][Hq][D], prefix K and V [Hkv][P][D], tail K and V
    [Hkv][before + n][D], all fp64.  The prefix and the tail as one context."""
    k, v = np.concatenate((kp, kt), 1), np.concatenate((vp, vt), 1)
    mapped = None
    if prefix_mapped is not None or tail_mapped is not None:
        mapped = np.concatenate((np.ones(kp.shape[1], bool) if prefix_mapped is None else prefix_mapped,
                                 np.ones(kt.shape[1], bool) if tail_mapped is None else tail_mapped))
    return P.extend_attention(q, k, v, kp.shape[1] + before, scale, mapped)

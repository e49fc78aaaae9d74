"""Helpers of the shared-prefix GPU tests: a batch of prefixes and tails in
caches of any format, the error bound of kvq_prefix_attn, and its check."""
from __future__ import annotations

import numpy as np

from oracle import prefix_oracle as X
from tests._prompt import FORMATS, expected_rows, extend_bound, new_cache, read_rows


class Shared:
    """N prefixes and B tails with known rows.  lens are per prefix, and per
    tail before the new tokens; every row of the padded batch is appended."""

    def __init__(self, prefix_fmt, tail_fmt, D, Hkv, G, prefix_lens, prefix_of, before, new, T=None, prefix_page=0,
                 tail_page=0, seed=0):
        import torch
        import quantized_kv_decode_gb300 as K
        self.K, self.D, self.Hkv, self.G, self.T = K, D, Hkv, G, T or max(max(new), 1)
        self.fmts = prefix_fmt, tail_fmt
        self.plens, self.of, self.before, self.new = (np.asarray(x, dtype=np.int32) for x in
                                                      (prefix_lens, prefix_of, before, new))
        self.N, self.B = len(prefix_lens), len(prefix_of)
        rng = np.random.default_rng(seed)
        self.P, self.L = int(self.plens.max(initial=0)), int((self.before + self.new).max())
        self.q = rng.standard_normal((self.B, self.T, Hkv * G, D)).astype(np.float16)
        self.prefix, self.pk, self.pv = self._cache(rng, prefix_fmt, self.plens, prefix_page, seed + 1)
        self.tail, self.tk, self.tv = self._cache(rng, tail_fmt, self.before + self.new, tail_page, seed + 2)
        self.dev = {n: torch.from_numpy(getattr(self, n)).cuda() for n in ("plens", "of", "before", "new", "q")}
        self.plan = K.kvq_prefix_plan(self.dev["of"], self.dev["plens"])

    def _cache(self, rng, fmt, lens, page, seed):
        """A cache of len(lens) sequences and its rows in fp64, [rows][most][Hkv][D]."""
        import torch
        rows, most = len(lens), max(int(lens.max(initial=0)), 1)
        if rows == 0:
            return None, None, None
        cache = new_cache(fmt, self.Hkv, self.D, rows, most, page, seed)
        kch = FORMATS[fmt][2].get("k_per_channel", False)
        x = [rng.standard_normal((rows, most, self.Hkv, self.D)).astype(np.float16) for _ in "kv"]
        x[0][..., rng.permutation(self.D)[:2]] *= 4  # keys' persistent large channels
        t = [torch.from_numpy(a).cuda() for a in x]
        if kch:  # an axis-aware sequence's length is what has been appended to it: one call each
            for r, n in enumerate(lens):
                if n:
                    self._append_one(cache, r, [a[r:r + 1, :n].contiguous() for a in t])
            got = read_rows(cache, lens.tolist(), most)
            return cache, *(g.astype(np.float64) for g in got)
        self.K.kvq_append(cache, t[0], t[1], torch.zeros(rows, dtype=torch.int32, device="cuda"))
        return cache, expected_rows(fmt, x[0]), expected_rows(fmt, x[1])

    def _append_one(self, cache, r, kv):
        import torch
        from dataclasses import replace
        kw = {n: getattr(cache, n)[r:r + 1] for n in ("k_window", "v_window")}
        if cache.block_table is not None:
            kw["block_table"] = cache.block_table[r:r + 1].contiguous()
            if kw["block_table"].data_ptr() % 16:
                kw["block_table"] = kw["block_table"].clone()
        else:
            kw.update({n: getattr(cache, n)[r:r + 1] for n in ("k_codes", "v_codes", "k_scale", "k_zero", "v_scale",
                                                               "v_zero")})
        one = replace(cache, batch=1, **kw)
        self.K.kvq_append(one, kv[0], kv[1], torch.zeros(1, dtype=torch.int32, device="cuda"))

    def call(self, **kw):
        args = dict(new_lens=self.dev["new"])
        args.update(kw)
        return self.K.kvq_prefix_attn(self.prefix, self.tail, self.plan, self.dev["q"], self.dev["before"], self.P,
                                      self.L, **args)

    def check(self, got, only=None, prefix_mapped=None, tail_mapped=None, plens=None, of=None):
        """Every live row of got [B][T][Hq][D] (numpy) against the oracle."""
        scale = self.D ** -0.5
        rounded = any(FORMATS[f][2].get("k_per_channel", False) for f in self.fmts)
        plens = self.plens if plens is None else plens
        of = self.of if of is None else of
        for b in range(self.B) if only is None else only:
            n, n0 = int(self.new[b]), int(self.before[b])
            if n == 0:
                continue
            p = int(of[b])
            P = int(plens[p]) if p >= 0 else 0
            kp, vp = ((a[p, :P] if P else np.zeros((0, self.Hkv, self.D))).transpose(1, 0, 2) for a in
                      (self.pk if P else self.tk, self.pv if P else self.tv))
            kt, vt = (a[b, :n0 + n].transpose(1, 0, 2) for a in (self.tk, self.tv))
            q = self.q[b, :n].astype(np.float64)
            want, mass = X.prefix_attention(q, kp, vp, kt, vt, n0, scale,
                                            None if prefix_mapped is None or P == 0 else prefix_mapped[p, :P],
                                            None if tail_mapped is None else tail_mapped[b, :n0 + n])
            k = np.concatenate((kp, kt), 1)
            assert max(np.abs(vp).max(initial=0), np.abs(vt).max(initial=0)) <= 8.0
            bound = extend_bound(q, k, mass, want, scale, rounded)
            if self.T == 1:
                bound = bound + decode_extra(q, kt, mass, scale, FORMATS[self.fmts[1]][0])
            out = got[b, :n].astype(np.float64)
            assert np.isfinite(out).all()
            worst = (np.abs(out - want) / bound).max()
            assert worst <= 1.0, f"sequence {b}: {worst:.2f} times the bound"


def decode_extra(q, k, mass, scale, bits):
    """What a tail of one new token may add to extend_bound: the decode kernels
    take scale and zero-point out of the products.  Scores sum q code and z sum
    q apart: code s and z s reach 3 times the largest |k|, so D roundings of fp32
    at 3 |q| max|k| more.  Weights enter times V's scale, rounded to fp16 once
    more (2^-11 relative, 2^-25 absolute times codes up to 2^bits), and the
    weighted codes and zero-points are summed apart in fp32, at up to 3 max|v| =
    24.  The sum of weights is at least 1."""
    if bits == 16:
        return 0.0
    D, L = q.shape[-1], k.shape[1]
    S = 3.0 * float(np.abs(q).max(axis=(0, 1)).sum()) * float(np.abs(k).max(initial=0))
    rel = 2.0 ** -11 + 2 * 1.5 * scale * (D + 4) * 2.0 ** -24 * S
    return mass * rel + L * 2.0 ** -25 * 2.0 ** bits + 2 * L * 2.0 ** -24 * 24.0

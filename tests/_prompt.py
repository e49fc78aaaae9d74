"""Helpers of the prompt-path GPU tests: caches of every format filled through
kvq_append, their rows read by plain index arithmetic, and the error bound of
kvq_extend_attn."""
from __future__ import annotations

import numpy as np

import oracle as O
from oracle import prompt_oracle as P
from quantized_kv_decode_gb300 import synth

# name -> (bits, group, flags)
FORMATS = {
    "int4": (4, 32, {}),
    "int4_g8": (4, 8, {}),
    "int8": (8, 64, {}),
    "int2": (2, 32, {}),
    "sym4": (4, 32, dict(symmetric=True)),
    "sym8": (8, 16, dict(symmetric=True)),
    "nf4": (4, 32, dict(nf4=True)),
    "fp16": (16, 0, {}),
    "kch4": (4, 32, dict(k_per_channel=True, sink_tokens=3)),
    "kch8": (8, 16, dict(k_per_channel=True, sink_tokens=0)),
}


def new_cache(fmt, Hkv, D, B, cap, page=0, seed=0, spare=3):
    """An empty cache for B sequences of up to `cap` tokens; pages scattered."""
    import torch
    import quantized_kv_decode_gb300 as K
    bits, g, kw = FORMATS[fmt]
    kch = kw.get("k_per_channel", False)
    if page:
        if kch:
            page = -(-page // g) * g
        table, pages = synth.block_table(np.random.default_rng(seed), np.full(B, cap), page, spare_pages=spare)
        desc = K.make_desc(bits, g, Hkv, D, K.KVQ_PAGED, page, pages, table.shape[1], **kw)
        return K.KVCache.allocate(desc, B, "cuda", torch.from_numpy(table))
    if kch:
        cap = -(-(cap + 1) // g) * g
    desc = K.make_desc(bits, g, Hkv, D, K.KVQ_DENSE, cap, **kw)
    return K.KVCache.allocate(desc, B, "cuda")


def expected_rows(fmt, x):
    """What the cache makes of fp16 rows x [..., D] (per-token formats): the
    dequantized values in fp64."""
    bits, g, kw = FORMATS[fmt]
    if bits == 16:
        return x.astype(np.float64)
    if kw.get("nf4"):
        r = O.quantize_groups_nf4(x, g)
        return O.dequantize_nf4(r["codes"], r["scale"], g)
    quantize = O.quantize_groups_symmetric if kw.get("symmetric") else O.quantize_groups
    r = quantize(x, bits, g)
    return O.dequantize(r["codes"], r["scale"], r["zero"], g)


def hold16(x):
    """fp64 -> fp16, held at the largest finite value."""
    return np.clip(x, -65504, 65504).astype(np.float16)


def read_rows(cache, lens, most):
    """K and V [B][most][Hkv][D] of a cache through kvq_cache_read."""
    import torch
    import quantized_kv_decode_gb300 as K
    d = cache.desc
    B = len(lens)
    out = [torch.zeros((B, most, d.num_kv_heads, d.head_dim), dtype=torch.float16, device="cuda") for _ in "kv"]
    K.kvq_cache_read(cache, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                     torch.zeros(B, dtype=torch.int32, device="cuda"), *out)
    return [o.cpu().numpy() for o in out]


def extend_bound(q, k, mass, out, scale, rounded=False):
    """How far an output may be from the formula's on the dequantized K and V.

    Per score: D products accumulated in fp32, error at most D 2^-24 of the
    sum of magnitudes S = sum |q_d k_d| (taken over the largest row of K and
    q); in the exponent that is a relative 1.5 scale D 2^-24 S, plus 2^-20 for
    the exponentials and their reference.  Each probability is rounded to
    fp16: half a step is 2^-11 relative, or 2^-25 absolute below 2^-14.  The
    weighted sum and the sum of probabilities accumulate L terms in fp32, the
    output is rounded to fp16 once more.  K and V enter with 22 bits: 2^-22 of
    S in a score, like four more of the D roundings, and of the mass.

    rounded: k and v are what kvq_cache_read returns, each a rounding to fp16
    (2^-11) from what the call uses: in V directly, in K by 2^-11 S a score,
    felt in a weight and in the sum of weights."""
    D, L = q.shape[-1], k.shape[1]
    S = float((np.abs(q).max(axis=(0, 1)) * np.abs(k).max(axis=(0, 1))).sum())
    rel = 2.0 ** -11 + 2 * 1.5 * scale * (D + 4) * 2.0 ** -24 * S + 2.0 ** -19 + 2 * L * 2.0 ** -24
    if rounded:
        rel += 2.0 ** -11 + 2 * scale * 2.0 ** -11 * S
    return mass * rel + 2.0 ** -11 * np.abs(out) + L * 2.0 ** -25 * 8.0 + 2.0 ** -24


def check_extend(got, q, k16, v16, before, n, scale, mapped=None, rounded=False):
    """One sequence: got [n][Hq][D] against the oracle on K / V [L][Hkv][D]."""
    L = before + n
    k = k16[:L].astype(np.float64).transpose(1, 0, 2)
    v = v16[:L].astype(np.float64).transpose(1, 0, 2)
    q = q[:n].astype(np.float64)
    want, mass = P.extend_attention(q, k, v, before, scale, mapped)
    assert np.abs(v).max(initial=0) <= 8.0  # extend_bound's last term
    bound = extend_bound(q, k, mass, want, scale, rounded)
    off = np.abs(got[:n].astype(np.float64) - want)
    assert np.isfinite(got[:n]).all()
    worst = (off / bound).max()
    assert worst <= 1.0, f"error {off.max():.3e} is {worst:.2f} times the bound"

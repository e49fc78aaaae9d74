"""GPU tests of kvq_prefix_attn over few rows (codes in registers) on values that
fp16 has few bits for, or no room: small V, rows where one key has most of the
weight, q and K far from one."""
import numpy as np
import pytest

import oracle as O
from oracle import prefix_oracle as X

pytestmark = pytest.mark.gpu

# name -> (bits, group, flags): what the kernel for few rows takes
FEW = {
    "int4": (4, 32, {}),
    "int8": (8, 32, {}),
    "int8_g64": (8, 64, {}),
    "sym4": (4, 64, dict(symmetric=True)),
    "sym8": (8, 32, dict(symmetric=True)),
    "nf4": (4, 32, dict(nf4=True)),
}


class Rows:
    """One prefix of P keys that B sequences of T new tokens (G heads) share; tails of
    T keys with all-zero K and V in fp16.  k, v: [P][D] fp16, the same in `heads` KV
    heads."""

    def __init__(self, fmt, k, v, q, heads=1):
        import torch
        import quantized_kv_decode_gb300 as K
        bits, g, kw = FEW[fmt]
        self.K, (self.P, self.D), (self.B, self.T, self.G, _) = K, k.shape, q.shape
        self.kw, self.g, self.bits = kw, g, bits
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.prefix = K.KVCache.allocate(K.make_desc(bits, g, heads, self.D, K.KVQ_DENSE, self.P, **kw), 1, "cuda")
        self.tail = K.KVCache.allocate(K.make_desc(16, 0, heads, self.D, K.KVQ_DENSE, self.T), self.B, "cuda")
        for c in (self.tail.k_codes, self.tail.v_codes):
            c.zero_()
        t = [torch.from_numpy(x[None, :, None]).cuda().expand(1, -1, heads, -1).contiguous() for x in (k, v)]
        K.kvq_append(self.prefix, *t, i32([0]))
        self.k, self.kmag = self._rows(k)
        self.v, self.vmag = self._rows(v)
        self.q, self.before = q, i32([0] * self.B)
        self.plan = K.kvq_prefix_plan(i32([0] * self.B), i32([self.P]))
        self.dev_q = torch.from_numpy(q).cuda().repeat(1, 1, heads, 1)

    def _rows(self, x):
        """The dequantized rows, and what their parts amount to where scale and
        zero-point are taken apart: (code + |zero|) |scale|."""
        x = x[None]
        if self.kw.get("nf4"):
            r = O.quantize_groups_nf4(x, self.g)
            y = O.dequantize_nf4(r["codes"], r["scale"], self.g)
            return y[0], np.abs(y[0])
        r = (O.quantize_groups_symmetric if self.kw.get("symmetric") else O.quantize_groups)(x, self.bits, self.g)
        y = O.dequantize(r["codes"], r["scale"], r["zero"], self.g)
        s, z = (np.repeat(r[n].astype(np.float64), self.g, -1) for n in ("scale", "zero"))
        return y[0], ((r["codes"] + np.abs(z)) * s)[0]

    def worst(self, scale, splits):
        """The largest error over its bound.

        A score: 2 (D + 8) steps of 2^-24 of the sum over the channels of |q| (code +
        |zero|) s (products in fp32, sums that may cut off instead of rounding, and 2^-22
        of the zero-point's term left out); it is felt by its weight and by the sum of
        weights.  2^-18 for the exponentials, their reference and the join.  A weight is
        rounded to fp16 and so is its product with V's scale: 2^-11 of itself each, or
        2^-25 of 2^-7 of the row's largest, and 2^-25 of 2^-11 of the largest times the
        largest scale, which codes up to 2^bits (at most 2 max|v| / scale) multiply.  The
        weighted codes and zero-points are summed apart, (code + |zero|) s at most; a
        block's four warps add sixteen keys at a time, so each sum is rounded P / 64 times
        and a few more in the join, by up to 4 steps of 2^-24 (cut off, sixteen terms at
        once); the weights' sum alike.  The output is rounded to fp16: 2^-11 of itself, or
        half of the smallest step, 2^-25."""
        out = self.K.kvq_prefix_attn(self.prefix, self.tail, self.plan, self.dev_q, self.before, self.P, self.T,
                                     softmax_scale=scale, prefix_splits=splits)
        out = out.unflatten(2, (-1, self.G))
        assert (out == out[:, :, :1]).all()  # every KV head's
        out = out[:, :, 0].cpu().numpy().astype(np.float64)
        worst = 0.0
        zero = np.zeros((1, self.T, self.D))
        for b in range(self.B):
            q = self.q[b].astype(np.float64)
            want, mass = X.prefix_attention(q, self.k[None], self.v[None], zero, zero, 0, scale)
            S = float((np.abs(q).reshape(-1, self.D) @ self.kmag.T).max())
            sums = 4 * (self.P / 64 + 20) * 2.0 ** -24
            rel = 2 * 2.0 ** -11 + 2 * scale * 2 * (self.D + 8) * 2.0 ** -24 * S + 2.0 ** -18 + sums
            low = 2.0 ** -25 + self.P * 2.0 ** -31 * np.abs(self.v).max() + 2 * sums * self.vmag.max()
            bound = mass * rel + 2.0 ** -11 * np.abs(want) + low
            worst = max(worst, float((np.abs(out[b] - want) / bound).max()))
        return worst


def _rows_of(fmt, D, T, size_k, size_v, P=700, seed=3):
    rng = np.random.default_rng(seed)
    q = (rng.standard_normal((3, T, 4, D)) / size_k).astype(np.float16)
    k = (size_k * rng.standard_normal((P, D))).astype(np.float16)
    v = (size_v * (0.5 + rng.standard_normal((P, D)))).astype(np.float16)
    return Rows(fmt, k, v, q)


@pytest.mark.parametrize("size", [1e3, 1e-1, 2e-2, 1e-4])
@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("fmt,D", [(f, D) for f in FEW for D in (64, 128) if (f, D) not in (("int8_g64", 64), ("sym4", 64))])
def test_small_and_large_values(fmt, D, T, size):
    r = _rows_of(fmt, D, T, 1.0, size)
    for splits in (1, 3):
        assert r.worst(2.0 * D ** -0.5, splits) <= 1.0


@pytest.mark.parametrize("heavy", [6.0, 8.0, 10.0])
@pytest.mark.parametrize("size", [1.0, 0.1, 0.02])
@pytest.mark.parametrize("fmt", list(FEW))
def test_one_heavy_key(fmt, size, heavy):
    """One key `heavy` nats above thousands, its V small beside theirs: what the
    others add together must not be lost.  (Enough KV heads that the kernel for few
    rows takes the prefix unsplit.)"""
    rng = np.random.default_rng(int(heavy))
    D, P, G = 128, 6000, 4
    base = rng.standard_normal(D)
    q = (base + 0.05 * rng.standard_normal((2, 1, G, D))).astype(np.float16)
    k = 0.2 * rng.standard_normal((P, D))
    k -= np.outer(k @ base, base) / (base @ base)
    v = size * (0.3 + rng.standard_normal((P, D)))
    k[1234] = base * heavy * D ** 0.5 / (base @ base)
    v[1234] *= 0.05
    r = Rows(fmt, k.astype(np.float16), v.astype(np.float16), q, heads=208)
    assert r.worst(D ** -0.5, 1) <= 1.0
    assert r.worst(D ** -0.5, 0) <= 1.0


@pytest.mark.parametrize("fmt", list(FEW))
def test_scales_that_grow_along_the_prefix(fmt):
    """V grows by 2^-10 .. 2^10 from the first key to the last and back, group by
    group: the sums so far are rescaled many times."""
    rng = np.random.default_rng(8)
    D, P = 128, 900
    e = np.interp(np.arange(P)[:, None] + 40 * (np.arange(D) // 32), [0, P // 2, P + 120], [-10, 10, -10])
    k = rng.standard_normal((P, D)).astype(np.float16)
    v = (2.0 ** e * rng.standard_normal((P, D))).astype(np.float16)
    r = Rows(fmt, k, v, rng.standard_normal((3, 1, 4, D)).astype(np.float16))
    for splits in (1, 2):
        assert r.worst(D ** -0.5, splits) <= 1.0


@pytest.mark.parametrize("size_q,size_k,shift", [(1e4, 1e-4, 0.0), (100.0, 1e-2, 0.0), (3000.0, 1.0, 1.0), (8000.0, 1.0, 0.0),
                                                 (1e-3, 1e3, 0.0), (1e-5, 1e4, 0.0), (60000.0, 1e-5, 0.0)])
@pytest.mark.parametrize("fmt", list(FEW))
def test_scores_of_any_size(fmt, size_q, size_k, shift):
    """q far from one, K as far or not at all: scores of a few units by the softmax
    scale.  shift: channels of one sign, whose sum fp16 does not hold."""
    rng = np.random.default_rng(9)
    D, P = 128, 500
    q = np.clip(size_q * (shift + rng.standard_normal((3, 1, 4, D)) * (0.2 if shift else 1.0)), -65504, 65504).astype(np.float16)
    k = np.clip(size_k * rng.standard_normal((P, D)), -65504, 65504).astype(np.float16)
    r = Rows(fmt, k, (0.5 + rng.standard_normal((P, D))).astype(np.float16), q)
    scale = 2.0 / float(np.std(q.astype(np.float64)[0, 0] @ r.k.T))
    for splits in (1, 2):
        assert r.worst(scale, splits) <= 1.0


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 65504.0, 1e-7])
@pytest.mark.parametrize("fmt", ["int4", "int8"])
def test_a_row_does_not_change_another(fmt, value):
    """Rows of one tile whose q has an infinity, a NaN, fp16's largest or nearly
    nothing: the others are to the bit what they are beside ordinary rows."""
    r = _rows_of(fmt, 128, 1, 1.0, 1.0)
    call = lambda: r.K.kvq_prefix_attn(r.prefix, r.tail, r.plan, r.dev_q, r.before, r.P, r.T, prefix_splits=2)  # noqa: E731
    want = call()
    r.dev_q[1, 0, 2, 5] = value
    if value == 1e-7:
        r.dev_q[1, 0, 2] = value
    got = call()
    same = (want == got).all(-1)
    assert [bool(x) for x in same.flatten()] == [i != 6 for i in range(12)]


@pytest.mark.parametrize("scale", [1e-12, 1e-20, 1e-37])
@pytest.mark.parametrize("size", [1.0, 1e-6])
@pytest.mark.parametrize("fmt", ["int4", "int8", "nf4"])
def test_a_softmax_scale_of_nearly_nothing(fmt, size, scale):
    """All weights alike, and keys that do not count (the last tile is not full)
    count for nothing."""
    rng = np.random.default_rng(4)
    x = [(s * rng.standard_normal(n)).astype(np.float16) for s, n in ((size, (333, 128)), (1.0, (333, 128)), (size, (2, 1, 4, 128)))]
    assert Rows(fmt, *x).worst(scale, 1) <= 1.0

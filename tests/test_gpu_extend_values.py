"""GPU tests of kvq_extend_attn on values that a softmax and its weighted sum
must not lose: an infinity or NaN in V alone, seen by some of a tile's rows
and not by others; K and V so small that fp16 has few bits for them."""
import numpy as np
import pytest

from oracle import prompt_oracle as P
from tests._prompt import FORMATS, check_extend, expected_rows, new_cache, read_rows

pytestmark = pytest.mark.gpu


def _fp16_call(rng, D, Hq, T, before):
    """A filled fp16 cache of one KV head, q, the call's lengths, and K and V."""
    import torch
    import quantized_kv_decode_gb300 as K
    L = before + T
    cache = new_cache("fp16", 1, D, 1, L)
    k, v = (torch.from_numpy(rng.standard_normal((1, L, 1, D)).astype(np.float16)).cuda() for _ in "kv")
    K.kvq_append(cache, k, v, torch.zeros(1, dtype=torch.int32, device="cuda"))
    k16, v16 = read_rows(cache, [L], L)
    q = rng.standard_normal((1, T, Hq, D)).astype(np.float16)
    return cache, q, torch.tensor([before], dtype=torch.int32, device="cuda"), k16, v16


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,before,Hq", [(300, 0, 1), (300, 37, 1), (520, 1, 1), (260, 63, 2), (100, 5, 1), (31, 0, 4)])
def test_every_row_that_sees_a_value_takes_part(T, before, Hq, D, splits, value):
    """V alone holds the infinity or NaN, so that nothing but the weighted sum
    can carry it: the channel is not finite in any row from that token on
    (weights that vanish make a NaN of it too), and the rows before come out
    as without it."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(21)
    cache, q, tb, k16, v16 = _fp16_call(rng, D, Hq, T, before)
    tq = torch.from_numpy(q).cuda()
    v = cache.v_codes.view(torch.float16)[0, 0]
    for at in sorted({0, 10, 64, T // 2, T - 1}):
        if at >= T:
            continue
        held = v[before + at, 3].item()
        v[before + at, 3] = value
        got = K.kvq_extend_attn(cache, tq, tb, before + T, num_splits=splits).cpu().numpy()
        v[before + at, 3] = held
        assert not np.isfinite(got[0, at:, :, 3]).any(), f"a row behind token {at} came out finite"
        if at:
            check_extend(got[0], q[0], k16[0], v16[0], before, at, D ** -0.5)
    if before:  # a cached token: every row sees it
        v[before - 1, 5] = value
        got = K.kvq_extend_attn(cache, tq, tb, before + T, num_splits=splits).cpu().numpy()
        assert not np.isfinite(got[0, :, :, 5]).any()


def _small_bound(q, k, mass, out, scale, v, nf4):
    """How far an output may be from the formula's where K and V enter exactly.

    Per score: D products in fp32, error at most D 2^-24 of S = sum |q_d k_d|
    (over the largest row of K and q), felt by its weight and by the sum of
    weights, 1.5 in the exponent's base; 2^-19 for the exponentials and their
    reference.  A weight is rounded to fp16: 2^-11 of itself, or 2^-25 in units
    of 2^-7 of the row's largest.  The weighted sum and the sum of weights take
    L terms in fp32.  The output is rounded to fp16: 2^-11 of itself, or half of
    the smallest step, 2^-25.  NF4: K and V are each off by up to 2^-25."""
    D, L = q.shape[-1], k.shape[1]
    qs = np.abs(q).max(axis=(0, 1))
    S = float((qs * np.abs(k).max(axis=(0, 1))).sum())
    rel = 2.0 ** -11 + 2 * 1.5 * scale * D * 2.0 ** -24 * S + 2.0 ** -19 + 2 * L * 2.0 ** -24
    low = 2.0 ** -25 + L * 2.0 ** -32 * np.abs(v).max()
    if nf4:
        rel += 2 * scale * 2.0 ** -25 * float(qs.sum())
        low += 2.0 ** -25
    return mass * rel + 2.0 ** -11 * np.abs(out) + low


@pytest.mark.parametrize("size", [1e-2, 1e-4])
@pytest.mark.parametrize("T", [5, 140])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["int4", "int8", "int2", "sym8", "nf4"])
def test_small_values_enter_whole(fmt, D, T, size):
    """K and V of 1e-2 and 1e-4, where a single fp16 number has few bits left
    and the second one's steps are fp16's smallest: scores of several units (q
    as much larger) and outputs against (q - z) s itself."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(17)
    before, Hq, Hkv = 150, 2, 1
    L = before + T
    cache = new_cache(fmt, Hkv, D, 1, L)
    k, v = ((size * rng.standard_normal((1, L, Hkv, D))).astype(np.float16) for _ in "kv")
    K.kvq_append(cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(),
                 torch.zeros(1, dtype=torch.int32, device="cuda"))
    q = (rng.standard_normal((1, T, Hq, D)) / size).astype(np.float16)
    scale = 2.0 * D ** -0.5
    got = K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), torch.tensor([before], dtype=torch.int32, device="cuda"),
                            L, softmax_scale=scale, num_splits=1).cpu().numpy()[0].astype(np.float64)
    kx, vx = (expected_rows(fmt, x[0]).transpose(1, 0, 2) for x in (k, v))
    want, mass = P.extend_attention(q[0].astype(np.float64), kx, vx, before, scale)
    off = np.abs(got - want) / _small_bound(q[0].astype(np.float64), kx, mass, want, scale, vx, fmt == "nf4")
    assert off.max() <= 1.0, off.max()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,before", [(90, 0), (31, 59)])
def test_values_of_an_axis_aware_window(T, before, D, value):
    """The same for the rows that an axis-aware cache keeps in fp16: the sinks
    and the unfinished block, V alone and K and V."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(23)
    bits, g, kw = FORMATS["kch4"]
    S, L, Hq = kw["sink_tokens"], before + T, 2
    cache = new_cache("kch4", 1, D, 1, L)
    k, v = (torch.from_numpy(rng.standard_normal((1, L, 1, D)).astype(np.float16)).cuda() for _ in "kv")
    K.kvq_append(cache, k, v, torch.zeros(1, dtype=torch.int32, device="cuda"))
    k16, v16 = read_rows(cache, [L], L)
    q = rng.standard_normal((1, T, Hq, D)).astype(np.float16)
    tb = torch.tensor([before], dtype=torch.int32, device="cuda")
    r0 = S + (L - S) // g * g
    assert r0 < L - 2
    for pos, slot in ((1, 1), (r0, S), (L - 1, S + (L - 1 - S) % g)):
        for windows in ((cache.v_window,), (cache.k_window, cache.v_window)):
            held = [w[0, 0, slot, 3].item() for w in windows]
            for w in windows:
                w[0, 0, slot, 3] = value
            got = K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), tb, L).cpu().numpy()
            for w, x in zip(windows, held):
                w[0, 0, slot, 3] = x
            at = max(pos - before, 0)       # the first row that sees it
            assert not np.isfinite(got[0, at:, :, 3]).any(), (pos, len(windows))
            if at:
                check_extend(got[0], q[0], k16[0], v16[0], before, at, D ** -0.5, rounded=True)

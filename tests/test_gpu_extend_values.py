"""GPU tests of kvq_extend_attn on values that a softmax and its weighted sum
must not lose: an infinity or NaN in V alone, seen by some of a tile's rows
and not by others."""
import numpy as np
import pytest

from tests._prompt import check_extend, new_cache, read_rows

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

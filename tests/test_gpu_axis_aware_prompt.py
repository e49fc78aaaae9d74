"""GPU tests of the prompt calls on axis-aware caches whose sequences differ:
a padded batch of them, appended as include/kvq.h says, attended in one call;
and the lengths a sequence can be cut back to."""
import numpy as np
import pytest

import oracle as O
from tests._prompt import FORMATS, check_extend, new_cache, read_rows

pytestmark = pytest.mark.gpu


def _one(K, cache, b):
    """Sequence b of a cache as a cache of its own, on the same memory."""
    part = {n: getattr(cache, n) for n in ("k_codes", "v_codes", "k_scale", "k_zero", "v_scale", "v_zero")}
    if cache.block_table is None:
        part = {n: t[b:b + 1] for n, t in part.items()}
        table = None
    else:
        table = cache.block_table[b:b + 1].clone()
    return K.KVCache(cache.desc, 1, block_table=table, k_window=cache.k_window[b:b + 1],
                     v_window=cache.v_window[b:b + 1], **part)


def _append(K, cache, b, k, v, at):
    import torch
    K.kvq_append(_one(K, cache, b), torch.from_numpy(k[None]).cuda(), torch.from_numpy(v[None]).cuda(),
                 torch.tensor([at], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("page", [0, 32])
@pytest.mark.parametrize("fmt,D", [("kch4", 64), ("kch4", 128), ("kch8", 128), ("kch8", 256)])
def test_a_ragged_batch(fmt, D, page, splits):
    """Sequences of different lengths and numbers of new tokens (none, one,
    within the sinks, ends inside and on a block's border)."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(41)
    bits, g, kw = FORMATS[fmt]
    S = kw["sink_tokens"]
    Hq, Hkv, T = 6, 2, 70
    before = [0, 0, 1, 100, S + 3 * g, 40, 200]
    new = [70, 2, 33, 1, 70, 0, S + 2 * g]
    B = len(before)
    lens = [a + n for a, n in zip(before, new)]
    most = max(lens)
    cache = new_cache(fmt, Hkv, D, B, most + 1, page)
    k, v = (rng.standard_normal((B, most, Hkv, D)).astype(np.float16) for _ in "kv")
    for b in range(B):
        if before[b]:
            _append(K, cache, b, k[b, :before[b]], v[b, :before[b]], 0)
        if new[b]:
            _append(K, cache, b, k[b, before[b]:lens[b]], v[b, before[b]:lens[b]], before[b])
    q = rng.standard_normal((B, T, Hq, D)).astype(np.float16)
    tb, tn = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (before, new))
    out = torch.full(q.shape, 9.0, dtype=torch.float16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), tb, most, new_lens=tn, out=out, dev_status=st,
                      num_splits=splits)
    assert int(st.item()) == 0
    got = out.cpu().numpy()
    for b in range(B):
        assert (got[b, new[b]:] == 9).all()
        if new[b]:
            r = O.kivi_quantize(*(x[b, :lens[b]].transpose(1, 0, 2) for x in (k, v)), bits, g, S)
            check_extend(got[b], q[b], r["k_hat"].transpose(1, 0, 2), r["v_hat"].transpose(1, 0, 2), before[b],
                         new[b], D ** -0.5)


@pytest.mark.parametrize("fmt", ["kch4", "kch8"])
def test_lengths_a_sequence_can_be_cut_back_to(fmt):
    """Within the sinks, on a block's border and within the unfinished block a
    shortened sequence reads as if the rest had never been, and goes on so."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(43)
    bits, g, kw = FORMATS[fmt]
    S, D, Hkv = kw["sink_tokens"], 64, 2
    L, more = S + 3 * g + g // 2, g + 3
    k, v = (rng.standard_normal((L + more, Hkv, D)).astype(np.float16) for _ in "kv")
    for cut in sorted({0, S // 2, S, S + g, S + 3 * g, S + 3 * g + 1, L - 1, L}):
        long, fresh = (new_cache(fmt, Hkv, D, 1, L + more) for _ in "ab")
        _append(K, long, 0, k[:L], v[:L], 0)
        if cut:
            _append(K, fresh, 0, k[:cut], v[:cut], 0)
        at = cut
        for n in (0, 1, more - 1):               # as cut, one token on, and past a block's end
            if n:
                for c in (long, fresh):
                    _append(K, c, 0, k[L + at - cut:L + at - cut + n], v[L + at - cut:L + at - cut + n], at)
                at += n
            if at:
                for x, y in zip(read_rows(long, [at], at), read_rows(fresh, [at], at)):
                    assert np.array_equal(x, y), (cut, at)
    torch.cuda.synchronize()

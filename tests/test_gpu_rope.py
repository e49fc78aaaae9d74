"""GPU tests of kvq_rope_apply, kvq_rope_append and kvq_cache_read.

Rotated values are compared with the fp64 oracle after one rounding to fp16:
they have to be equal, except where the oracle's own error bound leaves open
on which side of an fp16 tie the value lies.  Appended rows have to be bit for
bit those of the two separate calls, and the rows read back the exactly
rounded products (q - z) s."""
import numpy as np
import pytest

from oracle import prompt_oracle as P
from tests._cases import Guarded, check_guards
from tests._prompt import FORMATS, expected_rows, hold16, new_cache

pytestmark = pytest.mark.gpu


def _same_rounding(got, y, err):
    low, high = (y - err).astype(np.float16), (y + err).astype(np.float16)
    g = got.astype(np.float16)
    ok = (g == low) | (g == high)
    assert ok.all(), f"{(~ok).sum()} of {ok.size} values are not the nearest fp16"
    # where the oracle is sure (almost everywhere) there is one right answer
    assert (low != high).mean() < 1e-3


def _rope(K, rd, inter, scaling="none", factor=1.0, context=0, base=10000.0, **kw):
    r = K.make_rope(rd, base=base, interleaved=inter, scaling=scaling, factor=factor,
                    original_context=context, **kw)
    return r, P.rope_frequencies(rd, base, scaling, factor, context)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rd", [(64, 64), (128, 128), (256, 256), (128, 32), (64, 16), (64, 20), (128, 6),
                                  (8, 2), (40, 24), (96, 96), (256, 2)])
def test_rope_apply_matches_oracle(D, rd, inter):
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(D * 1000 + rd + inter)
    B, T, Hq, Hk = 3, 5, 7, 2
    q = rng.standard_normal((B, T, Hq, D)).astype(np.float16)
    k = (10 * rng.standard_normal((B, T, Hk, D))).astype(np.float16)
    before = np.array([0, 131071, 517], dtype=np.int32)
    r, (ws, amp) = _rope(K, rd, inter)
    dev = "cuda"
    qo, ko = Guarded(q.shape, torch.float16, dev), Guarded(k.shape, torch.float16, dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    K.kvq_rope_apply(r, torch.from_numpy(q).to(dev), torch.from_numpy(k).to(dev),
                     seq_lens_before=torch.from_numpy(before).to(dev), q_out=qo.tensor, k_out=ko.tensor,
                     dev_status=st)
    assert int(st.item()) == 0
    check_guards({"q": qo, "k": ko}, "rope")
    pos = before[:, None].astype(np.int64) + np.arange(T)
    for x, o in ((q, qo), (k, ko)):
        y, err = P.rope_rotate(x, pos, ws, amp, rd, inter)
        got = o.tensor.cpu().numpy()
        _same_rounding(got, y, err)
        assert np.array_equal(got[..., rd:].view(np.uint16), x[..., rd:].view(np.uint16))


@pytest.mark.parametrize("scaling,factor,context,base", [
    ("linear", 4.0, 0, 1e4), ("ntk", 8.0, 0, 1e4), ("bands", 8.0, 8192, 5e5), ("yarn", 16.0, 4096, 1e4)])
def test_rope_scalings_and_positions(scaling, factor, context, base):
    """Explicit positions, negative and far ones among them, one tensor only,
    in place; T of a few thousand tokens so that CTAs hold several tokens."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(5)
    B, T, H, D = 2, 1300, 3, 64
    x = rng.standard_normal((B, T, H, D)).astype(np.float16)
    pos = rng.integers(-4096, 1 << 20, size=(B, T)).astype(np.int32)
    pos[0, :4] = [0, -1, 1 << 20, 1]
    r, (ws, amp) = _rope(K, D, True, scaling, factor, context, base)
    t = torch.from_numpy(x).cuda()
    _, out = K.kvq_rope_apply(r, k=t, positions=torch.from_numpy(pos).cuda(), k_out=t)
    assert out is t
    y, err = P.rope_rotate(x, pos, ws, amp, D, True)
    _same_rounding(t.cpu().numpy(), y, err)


def test_rope_extreme_positions_are_exact_turns():
    """At positions +-2^31 the angle is turns[] times the position modulo one
    turn, worked out here in whole numbers."""
    import torch
    import quantized_kv_decode_gb300 as K
    D = 8
    r = K.make_rope(D)
    pos = np.array([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -7]], dtype=np.int32)
    x = np.zeros((1, 4, 1, D), dtype=np.float16)
    x[..., :D // 2] = 1.0
    got, _ = K.kvq_rope_apply(r, q=torch.from_numpy(x).cuda(), positions=torch.from_numpy(pos).cuda())
    got = got.cpu().numpy()[0, :, 0].astype(np.float64)
    for t in range(4):
        for i in range(D // 2):
            frac = (int(pos[0, t]) * int(r.turns[i])) % 2 ** 64 / 2.0 ** 64
            want = np.array([np.cos(2 * np.pi * frac), np.sin(2 * np.pi * frac)])
            # 2^-11 relative for the rounding; 2^-50 for frac in fp64
            off = np.abs(got[t, [i, i + D // 2]] - want)
            assert (off <= np.abs(want) * 2.0 ** -11 + 2.0 ** -24).all()


def test_rope_amplitude_nonfinite_and_padding():
    import torch
    import quantized_kv_decode_gb300 as K
    r = K.make_rope(64, amplitude=1.5)
    x = torch.ones((2, 3, 2, 64), dtype=torch.float16, device="cuda")
    x[0, 0, 0, 5] = float("inf")
    x[0, 0, 1, 6] = float("nan")
    before = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 7.0)
    new = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_rope_apply(r, x, seq_lens_before=before, new_lens=new, q_out=out, dev_status=st)
    assert int(st.item()) == 0
    o = out.cpu()
    assert torch.isinf(o[0, 0, 0, 5]) and not torch.isfinite(o[0, 0, 0, 37])
    assert torch.isnan(o[0, 0, 1, 6]) and torch.isnan(o[0, 0, 1, 38])
    assert (o[0, 0, 0, 6:37] == 1.5).all()          # position 0: no turn, the amplitude alone
    assert (o[0, 1:] == 7).all() and (o[1, 2:] == 7).all() and (o[1, :2] != 7).all()
    # lengths that cannot be: flagged, the sequence left out
    for bad_new, bad_before in ((4, 0), (-1, 0), (1, -1)):
        st.zero_()
        out.fill_(7)
        K.kvq_rope_apply(r, x, seq_lens_before=torch.tensor([bad_before, 0], dtype=torch.int32, device="cuda"),
                         new_lens=torch.tensor([bad_new, 1], dtype=torch.int32, device="cuda"), q_out=out,
                         dev_status=st)
        assert int(st.item()) == K._lib.KVQ_FLAG_SEQ_LEN
        assert (out[0] == 7).all() and (out[1, 0] != 7).all()


@pytest.mark.parametrize("fmt", [f for f in FORMATS if not f.startswith("kch")])
@pytest.mark.parametrize("D,rd,inter,page", [(128, 128, False, 0), (64, 32, True, 16), (64, 20, False, 8),
                                             (256, 256, False, 0), (128, 24, True, 16)])
def test_rope_append_is_apply_then_append(fmt, D, rd, inter, page):
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(D + rd)
    B, T, Hkv, Hq = 3, 7, 3, 6
    k = rng.standard_normal((B, T, Hkv, D)).astype(np.float16)
    k[..., :2] *= 10
    v = rng.standard_normal((B, T, Hkv, D)).astype(np.float16)
    q = rng.standard_normal((B, T, Hq, D)).astype(np.float16)
    before = np.array([0, 33, 5], dtype=np.int32)
    dev = "cuda"
    r, _ = _rope(K, rd, inter, "linear", 2.0)
    a, b = (new_cache(fmt, Hkv, D, B, 48, page) for _ in "ab")
    tk, tv, tq, tb = (torch.from_numpy(x).to(dev) for x in (k, v, q, before))
    st = torch.zeros(2, dtype=torch.int32, device=dev)
    qa, ka = K.kvq_rope_apply(r, tq, tk, seq_lens_before=tb)
    K.kvq_append(a, ka, tv, tb, st[:1])
    qb = K.kvq_rope_append(b, r, tk, tv, tb, q=tq, dev_status=st[1:])
    assert st.tolist() == [0, 0]
    assert torch.equal(qa, qb)
    for n in ("k_codes", "v_codes", "k_scale", "k_zero", "v_scale", "v_zero"):
        x, y = getattr(a, n), getattr(b, n)
        assert (x is None) == (y is None)
        if x is not None:
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), n
    # and the rows read back are the exactly rounded products
    lens = torch.from_numpy(before + T).to(dev)
    ko, vo = (Guarded(k.shape, torch.float16, dev) for _ in "kv")
    K.kvq_cache_read(b, lens, tb, ko.tensor, vo.tensor, st[:1])
    check_guards({"k": ko, "v": vo}, "read")
    assert int(st[0].item()) == 0
    for src, o in ((ka.cpu().numpy(), ko), (v, vo)):
        assert np.array_equal(o.tensor.cpu().numpy(), hold16(expected_rows(fmt, src)))


def test_rope_append_padding_limits_and_pages():
    """new_lens cuts sequences short; positions beyond the cache and unmapped
    pages are flagged and skipped; q in place; no q."""
    import torch
    import quantized_kv_decode_gb300 as K
    B, T, Hkv, D = 3, 6, 2, 64
    x = torch.randn((B, T, Hkv, D), device="cuda", dtype=torch.float16)
    r = K.make_rope(64)
    cache = new_cache("int8", Hkv, D, B, 16, 8)
    cache.block_table[2, 0] = -1
    before = torch.tensor([0, 13, 4], dtype=torch.int32, device="cuda")
    new = torch.tensor([2, 6, 6], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = x.clone()
    got = K.kvq_rope_append(cache, r, x, x, before, q=q, q_out=q, new_lens=new, dev_status=st)
    assert got is q and torch.equal(q[0, 2:], x[0, 2:])
    assert int(st.item()) == K._lib.KVQ_FLAG_SEQ_LEN | K._lib.KVQ_FLAG_BLOCK_TABLE
    written = cache.k_scale[:, :, :, 0] != 0
    t = cache.block_table.cpu().numpy()
    w = written.any(1).cpu().numpy()
    assert w[t[0, 0]].tolist() == [True] * 2 + [False] * 6 and not w[t[0, 1]].any()
    assert w[t[1, 1]].tolist() == [False] * 5 + [True] * 3   # positions 13..15; 16.. do not exist
    assert w[t[2, 1]].tolist() == [True] * 2 + [False] * 6   # 4..7 unmapped, 8, 9 written
    assert K.kvq_rope_append(cache, r, x, x, before, new_lens=new) is None


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("page", [0, 16])
def test_cache_read_every_format(fmt, page):
    """Rows of every format from any start, the axis-aware window included;
    rows behind the sequence keep what they held."""
    import torch
    import quantized_kv_decode_gb300 as K
    import oracle as O
    B, L, Hkv, D, T = 3, 75, 2, 64, 40
    rng = np.random.default_rng(3)
    k = rng.standard_normal((B, L, Hkv, D)).astype(np.float16)
    v = rng.standard_normal((B, L, Hkv, D)).astype(np.float16)
    cache = new_cache(fmt, Hkv, D, B, L + 6, page)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    K.kvq_append(cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), zero)
    start = torch.tensor([0, 50, 75], dtype=torch.int32, device="cuda")
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    out = [torch.full((B, T, Hkv, D), 9.0, device="cuda", dtype=torch.float16) for _ in "kv"]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_cache_read(cache, lens, start, *out, dev_status=st)
    assert int(st.item()) == 0
    bits, g, kw = FORMATS[fmt]
    if kw.get("k_per_channel"):
        want = [np.empty(x.shape) for x in (k, v)]
        for b in range(B):
            r = O.kivi_quantize(k[b].transpose(1, 0, 2), v[b].transpose(1, 0, 2), bits, g, kw["sink_tokens"])
            want[0][b], want[1][b] = r["k_hat"].transpose(1, 0, 2), r["v_hat"].transpose(1, 0, 2)
        want = [hold16(x) for x in want]
    else:
        want = [hold16(expected_rows(fmt, x)) for x in (k, v)]
    for i in range(2):
        got = out[i].cpu().numpy()
        for b, s in enumerate((0, 50, 75)):
            n = min(T, L - s)
            assert (got[b, n:] == 9).all()
            assert np.array_equal(got[b, :n], want[i][b, s:s + n])
    one, _ = K.kvq_cache_read(cache, lens, start, k_out=torch.full_like(out[0], 9.0))
    assert torch.equal(one, out[0])
    only_v = K.kvq_cache_read(cache, lens, start, v_out=torch.full_like(out[0], 9.0))[1]
    assert torch.equal(only_v, out[1])


def test_cache_read_flags():
    import torch
    import quantized_kv_decode_gb300 as K
    cache = new_cache("int4", 1, 64, 2, 32, 16)
    out = torch.full((2, 4, 1, 64), 9.0, device="cuda", dtype=torch.float16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for lens, start, want in ((i32(33, 4), i32(0, 0), 1), (i32(4, 4), i32(-1, 0), 1), (i32(-1, 4), i32(0, 0), 1)):
        st.zero_()
        out.fill_(9)
        K.kvq_cache_read(cache, lens, start, k_out=out, dev_status=st)
        assert int(st.item()) == want and (out[0] == 9).all() and (out[1] == 0).all()
    cache.block_table[0, 0] = 10 ** 6
    st.zero_()
    out.fill_(9)
    K.kvq_cache_read(cache, i32(4, 4), i32(0, 0), k_out=out, dev_status=st)
    assert int(st.item()) == K._lib.KVQ_FLAG_BLOCK_TABLE and (out[0] == 9).all() and (out[1] == 0).all()

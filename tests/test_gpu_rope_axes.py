"""GPU tests of kvq_rope_axes_apply and kvq_rope_axes_append.

As for one axis: rotated values equal the fp64 oracle's after one rounding to
fp16, and appended caches are bit for bit those of the two separate calls."""
import numpy as np
import pytest

from oracle import prefix_oracle as X
from tests._cases import Guarded, check_guards
from tests._prompt import new_cache
from tests.test_gpu_rope import _same_rounding

pytestmark = pytest.mark.gpu

AXES = [((16, 24, 24), False, False), ((24, 20, 20), True, False), ((3, 7), True, True), ((1, 1, 1, 1), True, False),
        ((5, 1, 2), False, True), ((64,), False, False), ((40, 8, 8, 8), True, True)]


def _positions(rng, shape, axes):
    pos = rng.integers(-4096, 1 << 20, size=shape + (axes,)).astype(np.int32)
    pos[0, 0] = 0
    return pos


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("pairs,cycled,ladders", AXES)
def test_apply_matches_oracle(pairs, cycled, ladders, inter):
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(sum(pairs) * 10 + len(pairs) + inter)
    rd = 2 * sum(pairs)
    B, T, Hq, Hk, D = 3, 5, 7, 2, -(-rd // 8) * 8 + 8 * inter
    q = rng.standard_normal((B, T, Hq, D)).astype(np.float16)
    k = (10 * rng.standard_normal((B, T, Hk, D))).astype(np.float16)
    pos = _positions(rng, (B, T), len(pairs))
    r = K.make_rope_axes(pairs, cycled=cycled, own_ladders=ladders, base=5e5, interleaved=inter)
    ws, axis, amp = X.axis_frequencies(pairs, cycled, ladders, 5e5)
    new = np.array([T, 0, 3], dtype=np.int32)
    qo, ko = Guarded(q.shape, torch.float16, "cuda"), Guarded(k.shape, torch.float16, "cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_rope_axes_apply(r, torch.from_numpy(pos).cuda(), torch.from_numpy(q).cuda(), torch.from_numpy(k).cuda(),
                          new_lens=torch.from_numpy(new).cuda(), q_out=qo.tensor, k_out=ko.tensor, dev_status=st)
    assert int(st.item()) == 0
    check_guards({"q": qo, "k": ko}, "axes")
    for x, o in ((q, qo), (k, ko)):
        y, err = X.rotate_axes(x, pos, ws, axis, amp, rd, inter)
        got = o.tensor.cpu().numpy()
        live = np.arange(T) < new[:, None]
        _same_rounding(got[live], y[live], err[live])
        assert not got[~live].any()
        assert np.array_equal(got[live][..., rd:].view(np.uint16), x[live][..., rd:].view(np.uint16))


@pytest.mark.parametrize("scaling,factor,context", [("linear", 4.0, 0), ("ntk", 8.0, 0), ("bands", 8.0, 8192),
                                                    ("yarn", 16.0, 4096)])
def test_scalings_in_place_and_long(scaling, factor, context):
    """A few thousand tokens, one tensor only, in place."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(7)
    B, T, H, D, pairs = 2, 1300, 3, 64, (8, 12, 12)
    x = rng.standard_normal((B, T, H, D)).astype(np.float16)
    pos = _positions(rng, (B, T), 3)
    r = K.make_rope_axes(pairs, cycled=True, base=1e4, scaling=scaling, factor=factor, original_context=context)
    ws, axis, amp = X.axis_frequencies(pairs, True, False, 1e4, scaling, factor, context)
    t = torch.from_numpy(x).cuda()
    _, out = K.kvq_rope_axes_apply(r, torch.from_numpy(pos).cuda(), k=t, k_out=t)
    assert out is t
    y, err = X.rotate_axes(x, pos, ws, axis, amp, D, False)
    _same_rounding(t.cpu().numpy(), y, err)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("pairs", [(16, 16, 32), (5, 3)])
def test_agreeing_axes_are_one_position(pairs, inter):
    """Where a token's axes agree the rotation is that of one axis, bit for bit."""
    import torch
    import quantized_kv_decode_gb300 as K
    D, B, T = 128, 4, 9
    x = torch.randn((B, T, 3, D), dtype=torch.float16, device="cuda")
    before = torch.tensor([0, 5, 70000, 3], dtype=torch.int32, device="cuda")
    pos = (before[:, None] + torch.arange(T, device="cuda")).int()
    one, _ = K.kvq_rope_apply(K.make_rope(2 * sum(pairs), interleaved=inter), x, seq_lens_before=before)
    for cycled in (False, True):
        r = K.make_rope_axes(pairs, cycled=cycled, interleaved=inter)
        got, _ = K.kvq_rope_axes_apply(r, pos[..., None].expand(-1, -1, len(pairs)).contiguous(), x)
        assert torch.equal(got.view(torch.int16), one.view(torch.int16))


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("fmt", ["int4", "int4_g8", "int8", "int2", "sym4", "sym8", "nf4", "fp16"])
@pytest.mark.parametrize("D,pairs,inter,T", [(128, (16, 24, 24), False, 5), (64, (16, 16), True, 1), (64, (5, 6), False, 3),
                                             (256, (32, 32), False, 2)])
def test_append_is_apply_then_append(fmt, D, pairs, inter, T, page):
    import torch
    import quantized_kv_decode_gb300 as K
    g = torch.Generator(device="cuda").manual_seed(D + T)
    B, Hq, Hkv, cap = 3, 6, 2, 40
    k, v = (torch.randn((B, T, Hkv, D), generator=g, dtype=torch.float16, device="cuda") for _ in "kv")
    q = torch.randn((B, T, Hq, D), generator=g, dtype=torch.float16, device="cuda")
    pos = torch.randint(-100, 40000, (B, T, len(pairs)), generator=g, device="cuda", dtype=torch.int32)
    before = torch.tensor([0, 33, 7], dtype=torch.int32, device="cuda")
    new = torch.tensor([T, T, max(T - 1, 0)], dtype=torch.int32, device="cuda")
    r = K.make_rope_axes(pairs, interleaved=inter)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    one, two = new_cache(fmt, Hkv, D, B, cap, page), new_cache(fmt, Hkv, D, B, cap, page)
    qo = K.kvq_rope_axes_append(one, r, pos, k, v, before, q=q, new_lens=new, dev_status=st)
    q2, k2 = K.kvq_rope_axes_apply(r, pos, q, k, new_lens=new)
    for b in range(B):  # (kvq_append takes every row of its batch)
        n = int(new[b])
        if n:
            kk, vv = (torch.zeros((B, n, Hkv, D), dtype=torch.float16, device="cuda") for _ in "kv")
            kk[b], vv[b] = k2[b, :n], v[b, :n]
            sink = new_cache(fmt, Hkv, D, B, cap, page)
            K.kvq_append(sink, kk, vv, before)
            for name in ("k_codes", "v_codes", "k_scale", "k_zero", "v_scale", "v_zero"):
                dst, src = getattr(two, name), getattr(sink, name)
                if dst is None:
                    continue
                at = range(int(before[b]), int(before[b]) + n)
                for p in at:
                    if page:
                        pg = int(two.block_table[b, p // two.desc.capacity])
                        dst[pg, :, p % two.desc.capacity] = src[pg, :, p % two.desc.capacity]
                    else:
                        dst[b, :, p] = src[b, :, p]
    assert int(st.item()) == 0
    assert torch.equal(qo.view(torch.int16), q2.view(torch.int16))
    for name in ("k_codes", "v_codes", "k_scale", "k_zero", "v_scale", "v_zero"):
        a, b = getattr(one, name), getattr(two, name)
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


def test_bad_lengths_and_pages_are_flagged():
    import torch
    import quantized_kv_decode_gb300 as K
    D, pairs = 64, (16, 16)
    r = K.make_rope_axes(pairs)
    k = torch.randn((2, 1, 2, D), dtype=torch.float16, device="cuda")
    pos = torch.zeros((2, 1, 2), dtype=torch.int32, device="cuda")
    cache = new_cache("int4", 2, D, 2, 32, 16)
    for before, new, unmap, want in (((32, 0), (1, 1), False, K.KVQ_FLAG_SEQ_LEN), ((0, 0), (2, 1), False, K.KVQ_FLAG_SEQ_LEN),
                                     ((-1, 0), (1, 1), False, K.KVQ_FLAG_SEQ_LEN), ((3, 3), (1, 1), True, K.KVQ_FLAG_BLOCK_TABLE)):
        if unmap:
            cache.block_table[0, 0] = -1
        cache.k_codes.fill_(0x5A)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        K.kvq_rope_axes_append(cache, r, pos, k, k, torch.tensor(before, dtype=torch.int32, device="cuda"),
                               new_lens=torch.tensor(new, dtype=torch.int32, device="cuda"), dev_status=st)
        assert int(st.item()) == want
        page = int(cache.block_table[1, 0])
        mine = cache.k_codes[page, :, int(before[1])]
        assert (mine != 0x5A).any()
        cache.k_codes[page, :, int(before[1])] = 0x5A
        assert (cache.k_codes == 0x5A).all()

"""CPU tests of the prompt and page-pool calls: the rotation's table against
the oracle, refusals before any launch, and argument checks of the binding.
Nothing here launches a kernel."""
import ctypes
import math
from ctypes import byref

import numpy as np
import pytest

from oracle import prompt_oracle as P

SCALINGS = [("none", 1.0, 0), ("linear", 4.0, 0), ("ntk", 8.0, 0), ("bands", 8.0, 8192),
            ("yarn", 16.0, 4096), ("yarn", 1.0, 2048)]


@pytest.fixture(scope="module")
def K():
    from quantized_kv_decode_gb300 import build
    build.build()
    import quantized_kv_decode_gb300 as K
    K.lib()
    return K


@pytest.mark.parametrize("scaling,factor,context", SCALINGS)
@pytest.mark.parametrize("rd,base", [(128, 10000.0), (64, 5e5), (20, 1e6)])
def test_rope_table_matches_the_formulas(K, scaling, factor, context, rd, base):
    r = K.make_rope(rd, base=base, scaling=scaling, factor=factor, original_context=context)
    ws, amp = P.rope_frequencies(rd, base, scaling, factor, context)
    got = np.array([r.turns[i] for i in range(rd // 2)], dtype=np.float64) / 2.0 ** 64 * 2 * math.pi
    # two evaluations in fp64 (a power, a handful of products and a division),
    # and turns[] is a whole number of 2^-64 turns: half a unit is pi 2^-64
    assert np.allclose(got, ws, rtol=2.0 ** -48, atol=math.pi * 2.0 ** -64)
    assert abs(r.amplitude / 2.0 ** 61 - amp) <= amp * 2.0 ** -50
    assert all(r.turns[i] == 0 for i in range(rd // 2, 128))


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=258), dict(rotary_dim=64, base=1.0),
    dict(rotary_dim=64, base=float("nan")), dict(rotary_dim=64, factor=2.0),
    dict(rotary_dim=64, scaling="linear", factor=0.5), dict(rotary_dim=64, scaling="bands", factor=2.0),
    dict(rotary_dim=64, scaling="yarn", factor=2.0, original_context=64, low_turns=4.0, high_turns=4.0),
    dict(rotary_dim=64, amplitude=4.0), dict(rotary_dim=64, amplitude=-1.0),
    dict(rotary_dim=2, scaling="ntk", factor=2.0)])
def test_rope_refusals(K, kw):
    with pytest.raises(K.KVQError) as e:
        K.make_rope(**kw)
    assert e.value.status == K.KVQ_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        K.make_rope(64, scaling="other")


def _ptrs(n):
    """n pointers that pass the null and alignment checks; nothing reads them."""
    return [0x10000 * (i + 1) for i in range(n)]


def _cache(K, **kw):
    p = _ptrs(9)
    return K.kvq_cache(*p)


def test_rope_apply_refusals(K):
    lib, r = K.lib(), K.make_rope(64)
    q, qo, k, ko, pos, lens = _ptrs(6)

    def call(rope=r, D=64, B=1, T=1, Hq=1, q=q, qo=qo, Hk=1, k=k, ko=ko, pos=pos, lens=None):
        return lib.kvq_rope_apply(byref(rope), D, B, T, Hq, q, qo, Hk, k, ko, pos, lens, None, None, None)

    bad = K.KVQ_ERR_INVALID_ARG
    assert call(D=60) == bad and call(D=56) == bad and call(B=-1) == bad and call(T=-1) == bad
    assert call(Hq=-1) == bad and call(q=None) == bad and call(ko=None) == bad
    assert call(pos=None) == bad and call(q=q + 2) == bad and call(pos=pos + 4) == bad
    assert call(qo=q + 16) == bad                     # overlaps without being the same array
    assert call(D=512) == K.KVQ_ERR_UNSUPPORTED
    assert call(B=2 ** 20, T=2 ** 20) == K.KVQ_ERR_UNSUPPORTED
    assert call(B=0) == K.KVQ_OK and call(T=0) == K.KVQ_OK and call(Hq=0, Hk=0) == K.KVQ_OK
    broken = K.make_rope(64)
    broken.rotary_dim = 66
    assert call(rope=broken, D=128) in (bad, K.KVQ_ERR_CUDA)
    broken.rotary_dim = 300
    assert call(rope=broken, D=128) == bad
    broken = K.make_rope(64)
    broken.amplitude = 2 ** 63
    assert call(rope=broken) == bad


def test_rope_append_refusals(K):
    lib, r = K.lib(), K.make_rope(64)
    c = _cache(K)
    k, v, q, qo, lens = [x + 0x1000000 for x in _ptrs(5)]

    def call(d, rope=r, B=1, T=1, k=k, v=v, Hq=1, q=q, qo=qo, lens=lens):
        return lib.kvq_rope_append(byref(d), byref(c), byref(rope), B, T, k, v, Hq, q, qo, lens, None,
                                   None, None)

    d = K.make_desc(4, 32, 2, 64, K.KVQ_DENSE, 64)
    bad = K.KVQ_ERR_INVALID_ARG
    assert call(d, k=None) == bad and call(d, lens=None) == bad and call(d, q=None) == bad
    assert call(d, B=-1) == bad and call(d, rope=K.make_rope(128)) == bad and call(d, v=v + 8) == bad
    assert call(d, qo=q + 32) == bad
    assert call(d, B=0) == K.KVQ_OK
    kch = K.make_desc(4, 32, 2, 64, K.KVQ_DENSE, 64, k_per_channel=True)
    assert call(kch) == K.KVQ_ERR_UNSUPPORTED


def test_read_and_extend_refusals(K):
    lib = K.lib()
    c = _cache(K)
    q, out, lens, start, ws = [x + 0x1000000 for x in _ptrs(5)]
    d = K.make_desc(4, 32, 2, 64, K.KVQ_DENSE, 64)
    bad = K.KVQ_ERR_INVALID_ARG

    def read(B=1, T=1, lens=lens, start=start, k=out, v=None):
        return lib.kvq_cache_read(byref(d), byref(c), B, T, lens, start, k, v, None, None)
    assert read(B=-1) == bad and read(T=-1) == bad and read(lens=None) == bad and read(start=None) == bad
    assert read(k=out + 2) == bad
    assert read(B=0) == K.KVQ_OK and read(k=None) == K.KVQ_OK

    def extend(d=d, B=1, T=1, Hq=4, q=q, lens=lens, new=None, most=64, splits=1, scale=0.0, out=out, ws=None,
               n=0):
        return lib.kvq_extend_attn(byref(d), byref(c), B, T, Hq, q, lens, new, most, splits, scale, out, ws,
                                   n, None, None)
    assert extend(B=-1) == bad and extend(T=-1) == bad and extend(Hq=0) == bad and extend(Hq=3) == bad
    assert extend(most=-1) == bad and extend(splits=-1) == bad and extend(scale=-1.0) == bad
    assert extend(scale=float("nan")) == bad and extend(q=None) == bad and extend(out=None) == bad
    assert extend(out=q) == bad and extend(out=q + 16) == bad and extend(lens=lens + 4) == bad
    assert extend(B=65536) == K.KVQ_ERR_UNSUPPORTED
    assert extend(B=60000, T=60000) == K.KVQ_ERR_UNSUPPORTED
    assert extend(B=0) == K.KVQ_OK and extend(T=0) == K.KVQ_OK
    assert K.kvq_extend_num_splits(d, 1, 1, 3, 64, 1) == 0
    assert K.kvq_extend_workspace_size(d, 1, 1, 3, 64, 1) == 0


def test_pool_refusals(K):
    lib = K.lib()
    ref, table, a, b, c, ws = _ptrs(6)

    def pool(pages=64, page=16, batch=4, blocks=8, ref=ref, table=table):
        return K.kvq_page_pool(pages, page, batch, blocks, ref, table)
    bad, un = K.KVQ_ERR_INVALID_ARG, K.KVQ_ERR_UNSUPPORTED
    size = lib.kvq_pages_workspace_size
    assert size(byref(pool())) >= 64 * 8 and size(byref(pool(pages=0))) == 0
    for broken, want in ((pool(pages=0), bad), (pool(page=0), bad), (pool(batch=-1), bad), (pool(blocks=0), bad),
                         (pool(page=2 ** 20, blocks=2 ** 20), bad), (pool(batch=16385), un),
                         (pool(ref=None), bad), (pool(table=None), bad), (pool(table=table + 4), bad)):
        assert lib.kvq_pages_reorder(byref(broken), a, None, None, None) == want
        assert lib.kvq_pages_reserve(byref(broken), a, None, 1, b, c, None, ws, 1 << 20, None, None) == want
        assert lib.kvq_pages_compact(byref(broken), a, b, c, ws, 1 << 20, None, None) == want
    p = pool()
    assert lib.kvq_pages_reorder(byref(p), None, None, None, None) == bad
    assert lib.kvq_pages_reserve(byref(p), None, None, 1, b, c, None, ws, 1 << 20, None, None) == bad
    assert lib.kvq_pages_reserve(byref(p), a, None, -1, b, c, None, ws, 1 << 20, None, None) == bad
    assert lib.kvq_pages_reserve(byref(p), a, None, 1, b, None, None, ws, 1 << 20, None, None) == bad
    assert lib.kvq_pages_reserve(byref(p), a, None, 1, b, c, None, None, 0, None, None) == K.KVQ_ERR_WORKSPACE
    assert lib.kvq_pages_reserve(byref(p), a, None, 1, b, c, None, ws, 8, None, None) == K.KVQ_ERR_WORKSPACE
    assert lib.kvq_pages_compact(byref(p), a, b, None, ws, 1 << 20, None, None) == bad
    assert lib.kvq_pages_compact(byref(p), a, b, c, ws, 8, None, None) == K.KVQ_ERR_WORKSPACE
    assert lib.kvq_pages_reorder(byref(pool(batch=0, table=None)), None, None, None, None) == K.KVQ_OK


def test_reserve_refuses_more_blocks_than_32_bits_count(K):
    """Pages are counted in 32 bits: a call that could ask for more is refused
    before anything is launched."""
    lib = K.lib()
    ref, table, a, b, c, ws = _ptrs(6)
    for num_new, blocks, want in ((8 * 200000, 200000, K.KVQ_ERR_UNSUPPORTED), (2 ** 31 - 1, 2 ** 17, K.KVQ_ERR_UNSUPPORTED),
                                  (8 * 200000, 131071, K.KVQ_ERR_WORKSPACE), (8 * 100000, 200000, K.KVQ_ERR_WORKSPACE)):
        p = K.kvq_page_pool(64, 8, 16384, blocks, ref, table)
        assert lib.kvq_pages_reserve(byref(p), a, None, num_new, b, c, None, ws, 8, None, None) == want


def test_page_copy_refusals(K):
    lib = K.lib()
    caches = (K.kvq_cache * 2)(_cache(K), _cache(K))
    src, dst = _ptrs(2)
    d = K.make_desc(4, 32, 2, 64, K.KVQ_PAGED, 16, 64, 4)
    bad = K.KVQ_ERR_INVALID_ARG

    def call(d=d, caches=caches, n=2, src=src, dst=dst, pairs=4):
        return lib.kvq_pages_copy(byref(d), caches, n, src, dst, pairs, None, None)
    assert call(d=K.make_desc(4, 32, 2, 64, K.KVQ_DENSE, 16)) == bad
    assert call(n=-1) == bad and call(pairs=-1) == bad and call(src=None) == bad and call(dst=dst + 4) == bad
    assert call(n=0) == K.KVQ_OK and call(pairs=0) == K.KVQ_OK
    empty = (K.kvq_cache * 1)(K.kvq_cache(*([None] * 9)))
    assert call(caches=empty, n=1) == bad


def test_binding_checks(K):
    """Host tensors and wrong types are refused before the library is called."""
    import torch
    x = torch.zeros((1, 1, 2, 64), dtype=torch.float16)
    i = torch.zeros(1, dtype=torch.int32)
    r = K.make_rope(64)
    with pytest.raises(ValueError):
        K.kvq_rope_apply(r)
    with pytest.raises(TypeError):
        K.kvq_rope_apply(r, x, seq_lens_before=i)
    with pytest.raises(TypeError):
        K.PagePool(i, i.view(1, 1), 16)
    d = K.make_desc(16, 0, 2, 64, K.KVQ_DENSE, 8)
    cache = K.KVCache(d, 1, torch.zeros((1, 2, 8, 128), dtype=torch.uint8), None, None, None, None, None)
    for call in (lambda: K.kvq_rope_append(cache, r, x, x, i), lambda: K.kvq_extend_attn(cache, x, i, 8),
                 lambda: K.kvq_cache_read(cache, i, i, x)):
        with pytest.raises(TypeError):
            call()
    assert K.kvq_pages_copy([], i, i) is None


def test_structs_match_the_header(K):
    """Sizes of the structures that cross the boundary by layout."""
    assert ctypes.sizeof(K.kvq_rope) == 16 + 8 * 128
    assert ctypes.sizeof(K.kvq_rope_desc) == 16 + 5 * 8
    assert ctypes.sizeof(K.kvq_page_pool) == 32

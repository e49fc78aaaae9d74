"""CPU tests of rotary positions by axis and the shared-prefix calls: the axes'
table against the oracle, refusals before any launch, argument checks of the
binding.  Nothing here launches a kernel."""
import ctypes
import math
from ctypes import byref

import numpy as np
import pytest

from oracle import prefix_oracle as X
from tests.test_prompt_abi import _cache, _ptrs


@pytest.fixture(scope="module")
def K():
    from quantized_kv_decode_gb300 import build
    build.build()
    import quantized_kv_decode_gb300 as K
    K.lib()
    return K


@pytest.mark.parametrize("scaling,factor,context", [("none", 1.0, 0), ("linear", 4.0, 0), ("yarn", 16.0, 4096)])
@pytest.mark.parametrize("pairs,cycled,ladders", [((16, 24, 24), False, False), ((24, 20, 20), True, False),
                                                  ((3, 7), True, True), ((32, 32), False, True), ((9,), True, True),
                                                  ((1, 2, 3, 4), True, False)])
def test_axes_table_matches_the_formulas(K, pairs, cycled, ladders, scaling, factor, context):
    r = K.make_rope_axes(pairs, cycled=cycled, own_ladders=ladders, base=1e4, scaling=scaling, factor=factor,
                         original_context=context)
    ws, axis, amp = X.axis_frequencies(pairs, cycled, ladders, 1e4, scaling, factor, context)
    half = sum(pairs)
    got = np.array([r.rope.turns[i] for i in range(half)], dtype=np.float64) / 2.0 ** 64 * 2 * math.pi
    assert np.allclose(got, ws, rtol=2.0 ** -48, atol=math.pi * 2.0 ** -64)  # as for one axis
    assert [r.axis[i] for i in range(half)] == axis.tolist()
    assert abs(r.rope.amplitude / 2.0 ** 61 - amp) <= amp * 2.0 ** -50
    assert r.rope.rotary_dim == 2 * half and r.num_axes == len(pairs)


@pytest.mark.parametrize("pairs,kw", [((0, 4), {}), ((-1, 4), {}), ((100, 100), {}), ((4, 4), dict(base=1.0)),
                                      ((4, 1), dict(scaling="ntk", factor=2.0, own_ladders=True)), ((129,), {})])
def test_axes_refusals(K, pairs, kw):
    with pytest.raises(K.KVQError) as e:
        K.make_rope_axes(pairs, **kw)
    assert e.value.status == K.KVQ_ERR_INVALID_ARG
    for bad in ((), (1, 1, 1, 1, 1)):
        with pytest.raises(ValueError):
            K.make_rope_axes(bad)
    lib = K.lib()
    d, out = K.kvq_rope_axes_desc(), K.kvq_rope_axes()
    d.rope = K.kvq_rope_desc(16, 0, 0, 0, 1e4, 1.0)
    d.num_axes = 2
    d.pairs[:2] = [4, 4]
    assert lib.kvq_rope_axes_init(byref(d), byref(out)) == K.KVQ_OK
    assert lib.kvq_rope_axes_init(None, byref(out)) == K.KVQ_ERR_INVALID_ARG
    assert lib.kvq_rope_axes_init(byref(d), None) == K.KVQ_ERR_INVALID_ARG
    for name, value in (("num_axes", 0), ("num_axes", 5), ("cycled", 2), ("own_ladders", -1)):
        keep = getattr(d, name)
        setattr(d, name, value)
        assert lib.kvq_rope_axes_init(byref(d), byref(out)) == K.KVQ_ERR_INVALID_ARG
        setattr(d, name, keep)
    d.rope.rotary_dim = 18
    assert lib.kvq_rope_axes_init(byref(d), byref(out)) == K.KVQ_ERR_INVALID_ARG


def test_axes_call_refusals(K):
    lib = K.lib()
    r = K.make_rope_axes((16, 16))
    q, qo, k, ko, pos, lens = _ptrs(6)
    bad = K.KVQ_ERR_INVALID_ARG

    def call(axes=r, D=64, B=1, T=1, Hq=1, q=q, qo=qo, Hk=1, k=k, ko=ko, pos=pos):
        return lib.kvq_rope_axes_apply(byref(axes), D, B, T, Hq, q, qo, Hk, k, ko, pos, None, None, None)
    assert call(D=60) == bad and call(D=56) == bad and call(B=-1) == bad and call(pos=None) == bad
    assert call(q=None) == bad and call(ko=k + 16) == bad and call(pos=pos + 4) == bad
    assert call(D=512) == K.KVQ_ERR_UNSUPPORTED and call(B=2 ** 20, T=2 ** 20) == K.KVQ_ERR_UNSUPPORTED
    assert call(B=0) == K.KVQ_OK and call(Hq=0, Hk=0) == K.KVQ_OK
    assert lib.kvq_rope_axes_apply(None, 64, 1, 1, 1, q, qo, 1, k, ko, pos, None, None, None) == bad
    broken = K.make_rope_axes((16, 16))
    broken.axis[31] = 2
    assert call(axes=broken) == bad
    broken = K.make_rope_axes((16, 16))
    broken.num_axes = 5
    assert call(axes=broken) == bad

    c = _cache(K)
    k, v, q, qo, lens, pos = [x + 0x1000000 for x in _ptrs(6)]

    def append(d, axes=r, B=1, T=1, k=k, v=v, Hq=1, q=q, qo=qo, pos=pos, lens=lens):
        return lib.kvq_rope_axes_append(byref(d), byref(c), byref(axes), B, T, k, v, Hq, q, qo, pos, lens, None, None,
                                        None)
    d = K.make_desc(4, 32, 2, 64, K.KVQ_DENSE, 64)
    assert append(d, k=None) == bad and append(d, lens=None) == bad and append(d, pos=None) == bad
    assert append(d, pos=pos + 8) == bad and append(d, axes=broken) == bad and append(d, qo=q + 32) == bad
    assert append(d, axes=K.make_rope_axes((32, 32))) == bad
    assert append(d, B=0) == K.KVQ_OK
    assert append(K.make_desc(4, 32, 2, 64, K.KVQ_DENSE, 64, k_per_channel=True)) == K.KVQ_ERR_UNSUPPORTED
    assert lib.kvq_rope_axes_append(byref(d), byref(c), None, 1, 1, k, v, 1, q, qo, pos, lens, None, None, None) == bad


def test_plan_and_find_refusals(K):
    lib = K.lib()
    bad, un, ws_err = K.KVQ_ERR_INVALID_ARG, K.KVQ_ERR_UNSUPPORTED, K.KVQ_ERR_WORKSPACE
    a, b, c, d, e, f, ref, table, ws = _ptrs(9)
    size = lib.kvq_prefix_plan_size
    assert size(5, 2) >= 4 * (5 + 5 + 3 + 2) and size(5, 2) % 16 == 0
    assert size(-1, 1) == 0 and size(1, -1) == 0 and size(65536, 1) == 0 and size(1, 65536) == 0

    def plan(B=5, N=2, of=a, lens=b, to=c, n=1 << 20):
        return lib.kvq_prefix_plan(B, N, of, lens, to, n, None, None)
    assert plan(B=-1) == bad and plan(N=-1) == bad and plan(of=None) == bad and plan(lens=None) == bad
    assert plan(of=a + 4) == bad and plan(lens=b + 8) == bad
    assert plan(B=65536) == un and plan(N=65536) == un
    assert plan(to=a) == bad and plan(to=b) == bad and plan(to=b - 16) == bad
    assert plan(to=None) == ws_err and plan(n=size(5, 2) - 1) == ws_err and plan(to=c + 4) == ws_err

    def pool(pages=64, page=16, batch=4, blocks=8, ref=ref, table=table):
        return K.kvq_page_pool(pages, page, batch, blocks, ref, table)

    def find(p=None, lens=a, min_tokens=0, most=2, of=b, plens=c, ptab=d, ttab=e, tlens=f, num=None, ws=ws, n=1 << 20):
        return lib.kvq_prefix_find(byref(p or pool()), lens, min_tokens, most, of, plens, ptab, ttab, tlens, num, ws, n,
                                   None, None)
    assert find(p=pool(pages=0)) == bad and find(p=pool(page=0)) == bad and find(p=pool(ref=None)) == bad
    assert find(p=pool(table=None)) == bad and find(p=pool(batch=16385)) == un
    assert find(p=pool(blocks=2 ** 30 - 1, page=1, batch=16384)) == un  # savings beyond 64 bits
    assert find(min_tokens=-1) == bad and find(most=0) == bad and find(most=65536) == un
    for name in ("lens", "of", "plens", "ptab", "ttab", "tlens"):
        assert find(**{name: None}) == bad and find(**{name: a + 0x900004}) == bad, name
    assert find(ttab=table) == bad and find(ttab=table + 16) == bad and find(tlens=a) == bad and find(num=a + 4) == bad
    assert find(ptab=table) == bad and find(ptab=table + 64) == bad and find(ptab=e) == bad and find(of=a) == bad
    assert find(plens=a) == bad and find(num=ws) == bad and find(ws=table) == bad and find(of=c) == bad
    need = lib.kvq_prefix_find_workspace_size(byref(pool()))
    assert need > 0 and find(ws=None) == ws_err and find(n=need - 1) == ws_err and find(ws=ws + 8) == ws_err
    assert lib.kvq_prefix_find_workspace_size(byref(pool(page=0))) == 0


def test_prefix_attn_refusals(K):
    lib = K.lib()
    pc, c = _cache(K), _cache(K)
    q, out, lens, plan, ws = [x + 0x1000000 for x in _ptrs(5)]
    pd, d = K.make_desc(4, 32, 2, 64, K.KVQ_DENSE, 64), K.make_desc(8, 32, 2, 64, K.KVQ_DENSE, 64)
    bad, un = K.KVQ_ERR_INVALID_ARG, K.KVQ_ERR_UNSUPPORTED

    def call(pd=pd, pc=pc, N=1, d=d, c=c, B=2, T=1, Hq=4, q=q, lens=lens, new=None, plan=plan, pn=1 << 16, mp=64, ml=64,
             ps=1, ts=1, scale=0.0, out=out, ws=None, n=0):
        return lib.kvq_prefix_attn(None if pd is None else byref(pd), None if pc is None else byref(pc), N, byref(d),
                                   byref(c), B, T, Hq, q, lens, new, plan, pn, mp, ml, ps, ts, scale, out, ws, n, None,
                                   None)
    for kw in (dict(N=-1), dict(B=-1), dict(T=-1), dict(Hq=0), dict(Hq=3), dict(mp=-1), dict(ml=-1), dict(ps=-1),
               dict(ts=-1), dict(pd=None), dict(pd=K.make_desc(4, 32, 1, 64, K.KVQ_DENSE, 64)),
               dict(pd=K.make_desc(4, 32, 2, 128, K.KVQ_DENSE, 64)), dict(d=K.make_desc(8, 3, 2, 64, K.KVQ_DENSE, 64))):
        assert call(**kw) == bad, kw
    assert call(N=65536) == un and call(B=65536) == un and call(B=60000, T=60000) == un
    assert call(d=K.make_desc(8, 32, 2, 512, K.KVQ_DENSE, 64), pd=K.make_desc(8, 32, 2, 512, K.KVQ_DENSE, 64)) == un
    assert call(B=0) == K.KVQ_OK and call(T=0) == K.KVQ_OK
    size = K.kvq_prefix_attn_workspace_size
    assert size(pd, d, 1, 2, 1, 3, 64, 64, 1, 1) == 0


def test_binding_checks(K):
    """Host tensors and wrong sizes are refused before the library is called."""
    import torch
    x = torch.zeros((1, 1, 2, 64), dtype=torch.float16)
    i = torch.zeros(1, dtype=torch.int32)
    r = K.make_rope_axes((16, 16))
    d = K.make_desc(16, 0, 2, 64, K.KVQ_DENSE, 8)
    cache = K.KVCache(d, 1, torch.zeros((1, 2, 8, 128), dtype=torch.uint8), None, None, None, None, None)
    with pytest.raises(ValueError):
        K.kvq_rope_axes_apply(r, i)
    for call in (lambda: K.kvq_rope_axes_apply(r, i.view(1, 1, 1), x),
                 lambda: K.kvq_rope_axes_append(cache, r, i.view(1, 1, 1), x, x, i), lambda: K.kvq_prefix_plan(i, i),
                 lambda: K.kvq_prefix_attn(cache, cache, K.PrefixPlan(i, 1, 1), x, i, 8, 8)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):  # a dense cache has no table
        cache.with_table(i.view(1, 1))


def test_structs_match_the_header(K):
    assert ctypes.sizeof(K.kvq_rope_axes_desc) == ctypes.sizeof(K.kvq_rope_desc) + 4 + 4 * 4 + 8 + 4
    assert ctypes.sizeof(K.kvq_rope_axes) == ctypes.sizeof(K.kvq_rope) + 4 + 128 + 4


def test_prefix_attn_arrays_apart(K):
    """out shares no byte with what the call reads (q, the lengths, the plan); what
    it reads may be one array."""
    lib = K.lib()
    pc, c = _cache(K), _cache(K)
    d = K.make_desc(4, 32, 2, 64, K.KVQ_DENSE, 64)
    base = 0x70000000
    q, lens, new, plan, out = [base + i * 0x10000 for i in range(5)]
    n = 2 * 4 * 64 * 2  # bytes of q and out: 2 sequences, 4 heads of 64
    words = int(lib.kvq_prefix_plan_size(2, 1))

    def call(q=q, lens=lens, new=new, plan=plan, out=out):
        return lib.kvq_prefix_attn(byref(d), byref(pc), 1, byref(d), byref(c), 2, 1, 4, q, lens, new, plan, 1 << 16, 64,
                                   64, 1, 1, 0.0, out, None, 0, None, None)
    for at in (q, q + n - 16, q - n + 16, lens, lens - n + 16, new, new - n + 16, plan, plan + words - 16, plan - n + 16):
        assert call(out=at) == K.KVQ_ERR_INVALID_ARG, hex(at)
    # (without a device, or a workspace, the next step refuses with another status)
    for ok in (call(), call(out=q + n), call(out=plan - n), call(new=None), call(new=lens)):
        assert ok in (K.KVQ_ERR_CUDA, K.KVQ_ERR_WORKSPACE)

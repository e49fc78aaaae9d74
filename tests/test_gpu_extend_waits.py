"""GPU tests of what kvq_extend_attn does when one of its kernel's waits runs
out (debug build: kvq_debug_fail_wait lets a chosen wait count as run out, so
nothing really waits): the call is flagged, returns at once with nothing in
flight, writes nothing outside its arrays, leaves thread blocks that did not
give up right, and the next call is as ever."""
import time

import numpy as np
import pytest

from tests._cases import Guarded, check_guards, guarded_cache
from tests._prompt import FORMATS, new_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def debug_lib():
    from quantized_kv_decode_gb300 import _lib, build
    handle = _lib.load(build.build(debug=True))
    prev = _lib.use(handle)
    try:
        yield handle
    finally:
        handle.kvq_debug_fail_wait(_lib.KVQ_WAIT_NONE, 0)
        _lib.use(prev)


# one tile of rows in two streams (T * Hq / Hkv <= 128), and two tiles of rows
@pytest.mark.parametrize("T", [9, 150])
@pytest.mark.parametrize("fmt,D,page", [("int4", 128, 0), ("int8", 64, 0), ("int2", 128, 16), ("nf4", 64, 64),
                                        ("sym8", 128, 0), ("fp16", 128, 0), ("fp16", 64, 16)])
def test_a_wait_that_runs_out(debug_lib, fmt, D, page, T):
    import torch
    import quantized_kv_decode_gb300 as K
    from quantized_kv_decode_gb300 import _lib as L
    rng = np.random.default_rng(31)
    Hq, Hkv = 16, 8
    before = [700, 0, 1500, 30, 448, 700]      # key tiles of 64: 11 to 26, or 1 to 3
    new = [T, min(T, 60), T, min(T, 30), T, 1]
    B, most = len(before), max(before) + T
    cache = new_cache(fmt, Hkv, D, B, most, page)
    table = cache.block_table
    cache, guards = guarded_cache(cache)
    assert cache.block_table is table
    x = [torch.from_numpy(rng.standard_normal((B, most, Hkv, D)).astype(np.float16)).cuda() for _ in "kv"]
    K.kvq_append(cache, *x, torch.zeros(B, dtype=torch.int32, device="cuda"))
    q = torch.from_numpy(rng.standard_normal((B, T, Hq, D)).astype(np.float16)).cuda()
    tb, tn = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in (before, new))
    guards["out"] = out = Guarded(q.shape, torch.float16, "cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        out.tensor.fill_(9)
        st.zero_()
        torch.cuda.synchronize()
        t0 = time.monotonic()
        K.kvq_extend_attn(cache, q, tb, most, new_lens=tn, out=out.tensor, dev_status=st, num_splits=1)
        torch.cuda.synchronize()
        check_guards(guards, "extend")
        return int(st.item()), time.monotonic() - t0, out.tensor.clone()

    status, _, want = call()
    assert status == 0
    codes = FORMATS[fmt][0] != 16
    for wait, tiles in ((L.KVQ_WAIT_SOFTMAX, (0, 2, 6)), (L.KVQ_WAIT_K, (0, 1, 2, 6)), (L.KVQ_WAIT_V, (0, 1, 3, 6)),
                        (L.KVQ_WAIT_LOAD_K, (0, 1, 5, 8)), (L.KVQ_WAIT_LOAD_V, (0, 1, 5, 8)),
                        (L.KVQ_WAIT_SCORES, (2, 6)), (L.KVQ_WAIT_SUM, (0, 2, 6))):
        for tile in tiles:
            assert debug_lib.kvq_debug_fail_wait(wait, tile) == K.KVQ_OK
            status, took, got = call()
            assert debug_lib.kvq_debug_fail_wait(L.KVQ_WAIT_NONE, 0) == K.KVQ_OK
            if not codes and wait in (L.KVQ_WAIT_V, L.KVQ_WAIT_LOAD_V):
                assert status == 0 and torch.equal(got, want)   # fp16 caches have no such wait
                continue
            assert status == L.KVQ_FLAG_TIMEOUT, (wait, tile)
            # the waits that end a block for good found their copies and
            # products done: each of them has two seconds
            assert took < 1.8, (wait, tile, took)
            if tile >= 3:                       # these sequences have fewer key tiles
                assert torch.equal(got[1], want[1]) and torch.equal(got[3], want[3]), (wait, tile)
            status, _, got = call()
            assert status == 0 and torch.equal(got, want), (wait, tile)
    assert debug_lib.kvq_debug_fail_wait(L.KVQ_WAIT_COUNT, 0) == K.KVQ_ERR_INVALID_ARG
    assert debug_lib.kvq_debug_fail_wait(L.KVQ_WAIT_K, -1) == K.KVQ_ERR_INVALID_ARG

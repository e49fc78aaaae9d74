"""GPU tests of kvq_pages_copy on long lists of pairs: what a compaction of a
large pool hands over, with and without mistakes in it."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _cache(pages):
    """The smallest page there is: 8 rows of 64 two-bit codes."""
    import torch
    import quantized_kv_decode_gb300 as K
    desc = K.make_desc(2, 64, 1, 64, K.KVQ_PAGED, 8, pages, 1)
    c = K.KVCache.allocate(desc, 1, "cuda", torch.zeros((1, 1), dtype=torch.int32))
    c.k_codes.random_(0, 256)
    return c


# short lists (checked pair by pair), long ones, and pools beyond one window
@pytest.mark.parametrize("pages,pairs", [(9000, 2048), (9000, 2049), (100000, 33335), (1 << 20, 70001),
                                         ((1 << 21) + 77, 300003)])
def test_mistakes_in_a_list_are_found(pages, pairs):
    import torch
    import quantized_kv_decode_gb300 as K
    from quantized_kv_decode_gb300 import _lib as L
    rng = np.random.default_rng(pairs)
    c = _cache(pages)
    some = rng.permutation(pages)[:2 * pairs] if 2 * pairs <= pages else rng.permutation(pages)
    n = len(some) // 2
    src0, dst0 = np.full(pairs, -1, dtype=np.int32), np.full(pairs, -1, dtype=np.int32)
    live = np.sort(rng.permutation(pairs)[:n // 2])        # the rest is padding
    src0[live], dst0[live] = some[:len(live)], some[n:n + len(live)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def flags(src, dst):
        st.zero_()
        K.kvq_pages_copy([c], torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda(), st)
        return int(st.item())

    old = c.k_codes.clone()
    assert flags(src0, dst0) == 0
    at, to = (torch.from_numpy(x[live].astype(np.int64)).cuda() for x in (src0, dst0))
    want = old.clone()
    want[to] = old[at]
    assert torch.equal(c.k_codes, want)
    for i, j in ((0, -1), (1, 2), (-2, -1), (len(live) // 2, 3)):
        i, j = live[i], live[j]
        for field, take in (("target twice", lambda s, d: d.__setitem__(i, d[j])),
                            ("source is a target", lambda s, d: s.__setitem__(i, d[j])),
                            ("onto itself", lambda s, d: d.__setitem__(i, s[i]))):
            src, dst = src0.copy(), dst0.copy()
            take(src, dst)
            assert flags(src, dst) == L.KVQ_FLAG_PAGE_LIST, (field, i, j)
        # a pair that is skipped copies nothing, whatever it names
        src, dst = src0.copy(), dst0.copy()
        dst[i], src[i] = dst[j], pages
        assert flags(src, dst) == L.KVQ_FLAG_BLOCK_TABLE
        src[i] = -1
        assert flags(src, dst) == 0
    src, dst = src0.copy(), dst0.copy()
    src[live[0]], src[live[1]] = src[live[2]], src[live[2]]  # one source for several targets
    assert flags(src, dst) == 0


def test_a_large_pools_list_is_checked_in_linear_time():
    """500 000 pairs, 200 000 of them copies of 384 bytes (154 MB read and
    written: 25 us of memory time).  A check of every pair against every other
    took 132 ms."""
    import torch
    import quantized_kv_decode_gb300 as K
    pages, movers = 1_000_000, 200_000
    c = _cache(pages)
    src = torch.full((pages // 2,), -1, dtype=torch.int32, device="cuda")
    dst = src.clone()
    src[:movers] = torch.arange(pages - movers, pages, dtype=torch.int32, device="cuda")
    dst[:movers] = torch.arange(movers, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for status in (st, None):
        K.kvq_pages_copy([c], src, dst, status)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(3):
            K.kvq_pages_copy([c], src, dst, status)
        b.record()
        torch.cuda.synchronize()
        assert a.elapsed_time(b) / 3 < 13.0
    assert int(st.item()) == 0
    assert torch.equal(c.k_codes[:movers], c.k_codes[pages - movers:])

"""GPU tests of which shared pages kvq_pages_reserve replaces, as include/kvq.h
states it, and of large batches of forks."""
import numpy as np
import pytest

from oracle import prompt_oracle as P

pytestmark = pytest.mark.gpu

PAGE = 8


def _i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _reserve(ref, table, before, new):
    """(status, src, dst, granted, counts, table) of one call."""
    import torch
    import quantized_kv_decode_gb300 as K
    pool = K.PagePool(_i32(ref), _i32(table), PAGE)
    src, dst, granted = (_i32([7] * len(table)) for _ in range(3))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_pages_reserve(pool, _i32(before), _i32(new), src, dst, granted, max_new=max(new), dev_status=st)
    return (int(st.item()), src.tolist(), dst.tolist(), granted.tolist(), pool.ref_count.tolist(),
            pool.block_table.tolist())


# three forks of one two-page sequence; positions kept, whether all of them write
@pytest.mark.parametrize("before,new,needs,keeps", [
    ([11, 11, 11], [1, 1, 1], 2, 2),   # tokens kept in the shared page, all write: the last keeps it
    ([11, 11, 11], [1, 0, 1], 2, 1),   # one holder does not write
    ([8, 8, 8], [3, 3, 3], 3, None),   # written from its start: replaced for all three, no copies
    ([11, 8, 11], [1, 1, 1], 3, None),  # one of them from its start
    ([3, 3, 3], [9, 9, 9], 2 + 3, 2),  # both pages: the first kept by the last, the second by none
])
def test_which_shared_pages_are_replaced(before, new, needs, keeps):
    from quantized_kv_decode_gb300 import _lib as L
    table = [[0, 1], [0, 1], [0, 1]]
    for spare in (needs, needs - 1):
        ref = [3, 3] + [0] * spare
        got = _reserve(ref, table, before, new)
        o = P.Pool(ref, table, PAGE)
        want = o.reserve(before, new)
        if spare < needs:
            assert want is None
            assert got == (L.KVQ_FLAG_POOL_EMPTY, [-1] * 3, [-1] * 3, [0] * 3, ref, table)
            continue
        assert got == (0, *want, o.ref, o.table) and sum(r == 0 for r in got[4][2:]) == 0
        first = before[0] // PAGE          # the block that tokens are kept in
        for b in range(3):
            part = new[b] > 0 and before[b] % PAGE != 0
            copies = part and b != keeps
            assert got[1][b] == (first if copies else -1)
            assert (got[5][b][first] == first) == (b == keeps or new[b] == 0)


@pytest.mark.parametrize("B,limit_us", [(300, 1000), (5000, 1000), (16384, 1000)])
@pytest.mark.parametrize("others", [0, 1])
def test_large_batches_of_forks(B, limit_us, others):
    """Every row a fork of one of three sequences and writing into its partly
    filled page; with `others`, somebody who does not write holds each of the
    pages too.  The time is that of a few passes over the rows; a look at all
    rows before each took 2580 us for 16384."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(B)
    who = rng.integers(0, 3, size=B)
    table = np.stack([who, np.full(B, -1)], 1).astype(np.int32)
    ref = np.zeros(B + 40, dtype=np.int32)
    ref[:3] = np.bincount(who, minlength=3) + others
    pool = K.PagePool(_i32(ref), _i32(table), PAGE)
    src, dst, granted = (_i32([7] * B) for _ in range(3))
    before = _i32(np.full(B, 5))
    ws = torch.empty(K.kvq_pages_workspace_size(pool), dtype=torch.uint8, device="cuda")
    times = []
    for _ in range(4):
        pool.ref_count.copy_(torch.from_numpy(ref))
        pool.block_table.copy_(torch.from_numpy(table))
        ws.fill_(0xFF)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        K.kvq_pages_reserve(pool, before, None, src, dst, granted, max_new=1, workspace=ws)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    keep = np.zeros(B, dtype=bool)
    if not others:
        for w in range(3):
            keep[np.flatnonzero(who == w)[-1]] = True
    fresh = 3 + np.cumsum(~keep) - 1
    assert src.tolist() == np.where(keep, -1, who).tolist()
    assert dst.tolist() == np.where(keep, -1, fresh).tolist()
    assert granted.tolist() == [1] * B
    assert pool.block_table[:, 0].tolist() == np.where(keep, who, fresh).tolist()
    left = ref.copy()
    left[3:3 + (~keep).sum()] = 1
    left[:3] = 1
    assert pool.ref_count.tolist() == left.tolist()
    assert min(times) < limit_us, times

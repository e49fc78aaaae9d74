"""GPU tests of kvq_prefix_find and kvq_prefix_plan: whole numbers, equal to
the plain loops of the oracle."""
import numpy as np
import pytest

from oracle import prefix_oracle as X
from tests._cases import Guarded, check_guards

pytestmark = pytest.mark.gpu


def _tree(rng, B, M, depth, pages):
    """A block table of sequences forked from one another: each row copies a
    random earlier row's leading blocks and goes on with pages of its own."""
    table = -np.ones((B, M), dtype=np.int32)
    fresh = iter(rng.permutation(pages).tolist())
    held = np.zeros(B, dtype=np.int64)
    for b in range(B):
        held[b] = rng.integers(0, M + 1)
        keep = 0
        if b and rng.random() < depth:
            par = int(rng.integers(0, b))
            keep = int(rng.integers(0, min(held[par], held[b]) + 1))
            table[b, :keep] = table[par, :keep]
        for j in range(keep, held[b]):
            table[b, j] = next(fresh)
    return table, held


def _find(K, table, pages, page, lens, min_tokens, most, dirty=7):
    import torch
    B, M = table.shape
    t = torch.from_numpy(table).cuda()
    pool = K.PagePool(torch.zeros(pages, dtype=torch.int32, device="cuda"), t, page)
    outs = {n: Guarded(s, torch.int32, "cuda") for n, s in (
        ("of", (B,)), ("plens", (most,)), ("ptable", (most, M)), ("ttable", (B, M)), ("tlens", (B,)), ("num", (1,)))}
    for o in outs.values():
        o.tensor.fill_(dirty)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((K.kvq_prefix_find_workspace_size(pool),), 0xA7, dtype=torch.uint8, device="cuda")
    K.kvq_prefix_find(pool, torch.from_numpy(np.asarray(lens, dtype=np.int32)).cuda(),
                      *(outs[n].tensor for n in ("of", "plens", "ptable", "ttable", "tlens")), min_tokens=min_tokens,
                      num_prefixes=outs["num"].tensor, workspace=ws, dev_status=st)
    check_guards(outs, "find")
    assert torch.equal(t.cpu(), torch.from_numpy(table))
    return [o.tensor.cpu().numpy().tolist() for o in outs.values()], int(st.item())


@pytest.mark.parametrize("B,M,page,depth,min_tokens,most", [
    (1, 1, 16, 0.0, 0, 1), (2, 3, 16, 1.0, 0, 1), (7, 5, 8, 0.9, 1, 3), (33, 9, 16, 0.9, 16, 4),
    (40, 130, 16, 0.95, 33, 16), (70, 300, 1, 0.8, 5, 64), (300, 20, 64, 0.9, 100, 8), (64, 12, 16, 0.9, 193, 5),
    (90, 33, 3, 0.97, 7, 90), (5, 40, 16, 1.0, 10000, 2)])
@pytest.mark.parametrize("seed", [0, 1])
def test_find_matches_oracle(B, M, page, depth, min_tokens, most, seed):
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(seed * 1000 + B)
    pages = B * M + 5
    table, held = _tree(rng, B, M, depth, pages)
    lens = [int(rng.integers(max(h * page - 2 * page, 0), h * page + 1)) for h in held]
    want = X.find_prefixes(table.tolist(), pages, page, lens, min_tokens, most)
    got, st = _find(K, table, pages, page, lens, min_tokens, most)
    assert st == 0
    for name, g, w in zip(("of", "plens", "ptable", "ttable", "tlens"), got, want):
        assert g == [list(r) if isinstance(r, (list, tuple)) else r for r in w], name
    assert got[5] == [want[5]]


def test_find_more_sequences_than_keys_held_at_a_time():
    """Leaders far from their members, and groups of two in a batch of many."""
    import quantized_kv_decode_gb300 as K
    B, M, page = 9001, 3, 16
    table = np.arange(B * M, dtype=np.int32).reshape(B, M)
    table[8999, :2] = table[3, :2]
    table[4097, :1] = table[4096, :1]
    table[9000] = table[8999]
    lens = np.full(B, M * page)
    got, st = _find(K, table, B * M, page, lens, 0, 4)
    assert st == 0 and got[5] == [2]
    want_of = np.full(B, -1)
    want_of[[3, 8999, 9000]] = 0       # all three hold the leader's first two blocks
    want_of[[4096, 4097]] = 1
    assert got[0] == want_of.tolist()
    assert got[1] == [32, 16, 0, 0]
    assert got[4][8999] == 16 and got[4][9000] == 16 and got[4][5] == 48


def test_find_bad_lengths_and_pages():
    import quantized_kv_decode_gb300 as K
    page, M = 16, 4
    table = np.array([[0, 1, 2, -1], [0, 1, 3, -1], [0, 1, 2, 4], [0, 99, 5, -1], [0, 99, 6, -1], [7, 7, 7, 7]],
                     dtype=np.int32)
    lens = [48, 48, -3, 48, 48, 65]
    want = X.find_prefixes(table.tolist(), 8, page, lens, 0, 3)
    got, st = _find(K, table, 8, page, lens, 0, 3)
    assert st == K.KVQ_FLAG_SEQ_LEN
    assert got[:5] == [list(w) if not isinstance(w[0], list) else w for w in want[:5]]
    assert got[0] == [0, 0, -1, 0, 0, -1] and got[1] == [16, 0, 0]  # one block of four saves more than two of two
    assert got[4][2] == -3


@pytest.mark.parametrize("B,N", [(1, 1), (5, 0), (33, 2), (257, 12), (1000, 300), (65535, 7)])
def test_plan_lists_members_in_order(B, N):
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(B)
    of = rng.integers(-1, N, size=B).astype(np.int32) if N else np.full(B, -1, dtype=np.int32)
    lens = rng.integers(0, 1000, size=N).astype(np.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = K.kvq_prefix_plan(torch.from_numpy(of).cuda(), torch.from_numpy(lens).cuda(), dev_status=st)
    w = plan.words.cpu().numpy()
    pad = lambda n: (n + 3) // 4 * 4  # noqa: E731
    first_at = 2 * pad(B)
    order = w[pad(B):pad(B) + B]
    first = w[first_at:first_at + N + 1]
    assert int(st.item()) == 0
    assert np.array_equal(w[:B], of)
    assert np.array_equal(first, [int((of[of >= 0] < n).sum()) for n in range(N + 1)])
    assert np.array_equal(order, np.concatenate([np.flatnonzero(of == n) for n in list(range(N)) + [-1]]))
    assert np.array_equal(w[first_at + pad(N + 1):first_at + pad(N + 1) + N], lens)


def test_plan_flags_and_refills():
    import torch
    import quantized_kv_decode_gb300 as K
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([4, 5], dtype=torch.int32, device="cuda")
    plan = K.kvq_prefix_plan(torch.tensor([0, 2, -2, 1], dtype=torch.int32, device="cuda"), lens, dev_status=st)
    assert int(st.item()) == K.KVQ_FLAG_BLOCK_TABLE
    assert plan.words[:4].tolist() == [0, -1, -1, 1]
    st.zero_()
    again = K.kvq_prefix_plan(torch.tensor([1, 1, 1, 1], dtype=torch.int32, device="cuda"),
                              torch.tensor([-1, 9], dtype=torch.int32, device="cuda"), plan=plan, dev_status=st)
    assert again is plan and int(st.item()) == K.KVQ_FLAG_SEQ_LEN
    assert plan.words[:4].tolist() == [1, 1, 1, 1] and plan.words[12:14].tolist() == [0, 9]
    with pytest.raises(ValueError):
        K.kvq_prefix_plan(torch.zeros(5, dtype=torch.int32, device="cuda"), lens, plan=plan)


def test_find_and_plan_captured_and_replayed():
    """One graph of both calls over tables and lengths that change between replays."""
    import torch
    rng = np.random.default_rng(11)
    B, M, page, N = 70, 12, 16, 9
    tables = [rng.integers(0, 3, size=(B, M)).astype(np.int32) for _ in range(3)]
    lens = [rng.integers(0, page * M + 1, size=B).astype(np.int32) for _ in range(3)]
    table, ln = torch.from_numpy(tables[0]).cuda(), torch.from_numpy(lens[0]).cuda()
    K = __import__("quantized_kv_decode_gb300")
    pool = K.PagePool(torch.ones(64, dtype=torch.int32, device="cuda"), table, page)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")
    of, plens, ptab, ttab, tlens, num = i32(B), i32(N), i32(N, M), i32(B, M), i32(B), i32(1)
    ws = torch.empty(K.kvq_prefix_find_workspace_size(pool), dtype=torch.uint8, device="cuda")
    plan = K.kvq_prefix_plan(of, plens)
    run = lambda: (K.kvq_prefix_find(pool, ln, of, plens, ptab, ttab, tlens, num_prefixes=num, workspace=ws),
                   K.kvq_prefix_plan(of, plens, plan))
    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for t, n in zip(tables, lens):
        table.copy_(torch.from_numpy(t))
        ln.copy_(torch.from_numpy(n))
        g.replay()
        got = [x.clone() for x in (of, plens, ptab, ttab, tlens, num, plan.words)]
        of.fill_(7), plens.fill_(7), plan.words.fill_(7)
        run()
        for a, b in zip(got, (of, plens, ptab, ttab, tlens, num, plan.words)):
            assert torch.equal(a, b)

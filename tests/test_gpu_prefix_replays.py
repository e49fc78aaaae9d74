"""GPU tests of the shared-prefix calls one behind the other: search and plan
replayed against the oracle over arrays full of other values."""
import numpy as np
import pytest

from oracle import prefix_oracle as X
from tests.test_gpu_prefix_find import _tree

pytestmark = pytest.mark.gpu


def test_replays_of_find_and_plan_match_the_oracle():
    """Tables and lengths change between replays, and every array that the calls
    write, the workspace too, is full of something else before each."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(5)
    B, M, page, N, min_tokens = 50, 14, 8, 6, 9
    pages = B * M + 1
    table, ln = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B, M), (B,)))
    pool = K.PagePool(torch.ones(pages, dtype=torch.int32, device="cuda"), table, page)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    of, plens, ptab, ttab, tlens, num, st = i32(B), i32(N), i32(N, M), i32(B, M), i32(B), i32(1), i32(1)
    ws = torch.zeros(K.kvq_prefix_find_workspace_size(pool), dtype=torch.uint8, device="cuda")
    plan = K.kvq_prefix_plan(of, plens)

    def run():
        K.kvq_prefix_find(pool, ln, of, plens, ptab, ttab, tlens, min_tokens=min_tokens, num_prefixes=num, workspace=ws,
                          dev_status=st)
        K.kvq_prefix_plan(of, plens, plan, dev_status=st)

    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    pad = lambda n: (n + 3) // 4 * 4  # noqa: E731
    for turn in range(5):
        t, held = _tree(rng, B, M, 0.9, pages)
        lens = [int(rng.integers(max(h * page - 2 * page, 0), h * page + 1)) for h in held]
        table.copy_(torch.from_numpy(t))
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        for x in (of, plens, ptab, ttab, tlens, num, plan.words):
            x.fill_(-77 - turn if turn % 2 else 1 + turn)
        ws.fill_(0xA7 + turn)
        g.replay()
        want = X.find_prefixes(t.tolist(), pages, page, lens, min_tokens, N)
        for name, got, w in zip(("of", "plens", "ptab", "ttab", "tlens"), (of, plens, ptab, ttab, tlens), want):
            assert got.tolist() == [list(r) if isinstance(r, (list, tuple)) else r for r in w], (name, turn)
        assert num.tolist() == [want[5]] and int(st.item()) == 0
        w = plan.words.tolist()
        first_at = 2 * pad(B)
        on = np.asarray(want[0])
        assert w[:B] == on.tolist()
        assert w[pad(B):pad(B) + B] == np.concatenate([np.flatnonzero(on == n) for n in [*range(N), -1]]).tolist()
        assert w[first_at:first_at + N + 1] == [int((on[on >= 0] < n).sum()) for n in range(N + 1)]
        assert w[first_at + pad(N + 1):first_at + pad(N + 1) + N] == list(want[1])

"""GPU tests of the shared-prefix calls one behind the other: search and plan
replayed against the oracle over arrays full of other values, and steps that append
and attend over the same rows with nothing waited for in between."""
import numpy as np
import pytest

from oracle import prefix_oracle as X
from tests._prefix import Shared
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


STEPS = [("int4", 128, 1, 4), ("int8", 64, 1, 2), ("nf4", 128, 1, 1), ("int2", 128, 1, 2), ("fp16", 128, 1, 2),
         ("int4", 128, 3, 4), ("int8", 128, 2, 2), ("fp16", 64, 4, 2), ("int4", 256, 2, 1), ("int4_g8", 64, 1, 4)]


@pytest.mark.parametrize("fmt,D,T,G", STEPS)
@pytest.mark.parametrize("captured", [False, True])
def test_steps_without_a_wait_between(fmt, D, T, G, captured):
    """Append and attend, step after step over the same rows, with new keys, values and
    queries each time and nothing waited for: tails that start beside the pass over the
    prefixes see the rows that the append just before it wrote.  To the bit what the
    same steps give with the device waited for after each call."""
    import torch
    rng = np.random.default_rng(D + T)
    B, Hkv, steps = 40, 2, 30
    s = Shared(fmt, fmt, D, Hkv, G, [257, 90], rng.integers(0, 2, B), [0] * B, [T] * B, T, seed=D)
    K = s.K
    gen = torch.Generator(device="cuda").manual_seed(T)
    new = [[torch.randn(B, T, h, D, generator=gen, dtype=torch.float16, device="cuda") for h in (Hkv, Hkv, Hkv * G)]
           for _ in range(steps)]
    outs = torch.zeros((2, steps, *s.q.shape), dtype=torch.float16, device="cuda")
    ws = torch.full((K.kvq_prefix_attn_workspace_size(s.prefix.desc, s.tail.desc, s.N, B, T, Hkv * G, s.P, T),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(to, wait):
        for (k, v, q), out in zip(new, to):
            K.kvq_append(s.tail, k, v, s.dev["before"], st)
            wait()
            K.kvq_prefix_attn(s.prefix, s.tail, s.plan, q, s.dev["before"], s.P, T, out=out, workspace=ws, dev_status=st)
            wait()

    run(outs[0], torch.cuda.synchronize)
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(outs[1], lambda: None)
        outs[1].zero_()
        for _ in range(3):
            g.replay()
    else:
        for _ in range(3):
            run(outs[1], lambda: None)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and outs[0].any()
    assert torch.equal(outs[0], outs[1])
    assert not torch.equal(outs[0][0], outs[0][1])


@pytest.mark.parametrize("fmt,T", [("int4", 1), ("int8", 2), ("fp16", 3)])
def test_what_a_workspace_held_does_not_matter(fmt, T):
    """Any bits in it before a call, what an earlier call left in it among them."""
    import torch
    rng = np.random.default_rng(T)
    s = Shared(fmt, fmt, 128, 1, 2, [257, 90], rng.integers(0, 2, 9), [5] * 9, [T] * 9, T, seed=T)
    n = s.K.kvq_prefix_attn_workspace_size(s.prefix.desc, s.tail.desc, s.N, s.B, T, 2, s.P, s.L)
    want = s.call(workspace=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    word = torch.tensor([0x6b76715f70726573], dtype=torch.int64, device="cuda").repeat(n // 8).view(torch.uint8)
    for ws in (torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), word):
        for _ in range(3):
            assert torch.equal(s.call(workspace=ws), want)
    assert int(ws[n - 256:n - 248].view(torch.int64).item()) == 0  # cleared for whoever comes next
    s.check(want.cpu().numpy())

"""GPU tests of the page pool against plain loops (oracle/prompt_oracle.py),
of the page copy byte for byte, and of a run of them as a server uses them:
prompts appended, forked, extended with copy-on-write, decoded, freed and
compacted, every step's attention compared with an unshared cache."""
import numpy as np
import pytest

from oracle import prompt_oracle as P
from tests._cases import Guarded, check_guards
from tests._prompt import FORMATS, check_extend, new_cache, read_rows

pytestmark = pytest.mark.gpu


def _i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _random_pool(rng, pages, page, B, M, fill=0.6, share=0.3):
    """Rows holding random pages, some shared; counts that agree."""
    table = np.full((B, M), -1, dtype=np.int32)
    free = list(rng.permutation(pages))
    used = []
    for b in range(B):
        for j in range(int(rng.integers(0, M + 1))):
            if used and rng.random() < share:
                table[b, j] = used[int(rng.integers(len(used)))]
            elif free and len(used) < fill * pages:
                table[b, j] = free.pop()
                used.append(table[b, j])
    ref = np.bincount(table[table >= 0].ravel(), minlength=pages).astype(np.int32)
    return ref, table


def _device(K, ref, table, page):
    import torch
    r, t = Guarded(ref.shape, torch.int32, "cuda"), Guarded(table.shape, torch.int32, "cuda")
    r.tensor.copy_(torch.from_numpy(ref))
    t.tensor.copy_(torch.from_numpy(table))
    return K.PagePool(r.tensor, t.tensor, page), {"ref": r, "table": t}


def _agree(pool, oracle, guards):
    check_guards(guards, "pool")
    assert pool.ref_count.cpu().tolist() == oracle.ref
    assert pool.block_table.cpu().tolist() == oracle.table


@pytest.mark.parametrize("pages,page,B,M", [(1, 16, 1, 1), (40, 16, 5, 7), (300, 8, 33, 70), (5000, 64, 300, 33),
                                            (70000, 16, 1500, 40)])
def test_reorder(pages, page, B, M):
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(pages)
    ref, table = _random_pool(rng, pages, page, B, M)
    o = P.Pool(ref, table, page)
    pool, guards = _device(K, ref, table, page)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(3):
        parent = rng.integers(-1, B, size=B)
        keep = rng.integers(0, M * page + 1, size=B)
        o.reorder(parent.tolist(), None if step == 1 else keep.tolist())
        K.kvq_pages_reorder(pool, _i32(parent), None if step == 1 else _i32(keep), st)
        assert int(st.item()) == 0
        _agree(pool, o, guards)
    K.kvq_pages_reorder(pool, _i32([-1] * B), dev_status=st)
    assert int(st.item()) == 0 and not pool.ref_count.any() and (pool.block_table == -1).all()


def test_reorder_flags():
    import torch
    import quantized_kv_decode_gb300 as K
    pool = K.PagePool(_i32([1, 1, 1, 0]), _i32([[0, 1], [2, -1], [-1, -1]]), 8)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_pages_reorder(pool, _i32([0, 3, 1]), _i32([17, 8, 8]), st)
    assert int(st.item()) == K._lib.KVQ_FLAG_BLOCK_TABLE | K._lib.KVQ_FLAG_SEQ_LEN
    assert pool.block_table.tolist() == [[-1, -1], [-1, -1], [2, -1]]
    assert pool.ref_count.tolist() == [0, 0, 1, 0]
    bad = K.PagePool(_i32([1, 0]), _i32([[0, 9]]), 8)      # an entry outside the pool is dropped
    st.zero_()
    K.kvq_pages_reorder(bad, _i32([0]), dev_status=st)
    assert int(st.item()) == K._lib.KVQ_FLAG_BLOCK_TABLE and bad.block_table.tolist() == [[0, -1]]


@pytest.mark.parametrize("pages,page,B,M", [(40, 16, 5, 7), (300, 8, 33, 70), (5000, 64, 300, 33),
                                            (70000, 16, 1500, 40), (200000, 16, 64, 600)])
@pytest.mark.parametrize("most", [1, 300])
def test_reserve(pages, page, B, M, most):
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(pages + most)
    ref, table = _random_pool(rng, pages, page, B, M, fill=0.5)
    o = P.Pool(ref, table, page)
    pool, guards = _device(K, ref, table, page)
    held = (table >= 0).sum(1)
    before = np.array([rng.integers(max(h * page - page, 0), h * page + 1) for h in held])
    new = np.minimum(rng.integers(0, most + 1, size=B), M * page - before)
    outs = {n: Guarded((B,), torch.int32, "cuda") for n in ("src", "dst", "granted")}
    ws = Guarded((K.kvq_pages_workspace_size(pool),), torch.uint8, "cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = o.reserve(before.tolist(), new.tolist())
    K.kvq_pages_reserve(pool, _i32(before), _i32(new), outs["src"].tensor, outs["dst"].tensor,
                        outs["granted"].tensor, max_new=most, workspace=ws.tensor, dev_status=st)
    check_guards({**outs, "ws": ws}, "reserve")
    _agree(pool, o, guards)
    if want is None:
        assert int(st.item()) == K._lib.KVQ_FLAG_POOL_EMPTY
        want = ([-1] * B, [-1] * B, [0] * B)
    else:
        assert int(st.item()) == 0
    for n, w in zip(("src", "dst", "granted"), want):
        assert outs[n].tensor.tolist() == w, n


def test_reserve_shared_pages():
    """All holders of a page ask: the last keeps it.  Not all ask: every asker
    is given a copy.  A shared whole block ahead is replaced without a copy."""
    import torch
    import quantized_kv_decode_gb300 as K
    table = [[0, -1, -1], [0, -1, -1], [0, -1, -1], [1, -1, -1], [1, -1, -1], [2, 3, -1], [2, 3, -1]]
    ref = [3, 2, 2, 2, 0, 0, 0, 0, 0, 0]
    before, new = [5, 5, 3, 6, 0, 8, 8], [1, 1, 1, 2, 0, 3, 3]
    o = P.Pool(ref, table, 8)
    pool = K.PagePool(_i32(ref), _i32(table), 8)
    src, dst, granted = (_i32([7] * 7) for _ in range(3))
    K.kvq_pages_reserve(pool, _i32(before), _i32(new), src, dst, granted, max_new=3)
    assert (src.tolist(), dst.tolist(), granted.tolist()) == o.reserve(before, new)
    assert src.tolist() == [0, 0, -1, 1, -1, -1, -1] and dst.tolist() == [4, 5, -1, 6, -1, -1, -1]
    assert pool.block_table.tolist() == o.table and pool.ref_count.tolist() == o.ref
    assert o.table[5][1] == 7 and o.table[6][1] == 8 and o.ref[3] == 0


def test_reserve_exhaustion_and_flags():
    import torch
    import quantized_kv_decode_gb300 as K
    ref, table = [2, 0, 1], [[0, -1], [0, -1], [2, -1]]
    pool = K.PagePool(_i32(ref), _i32(table), 8)
    src, dst, granted = (_i32([7] * 3) for _ in range(3))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    # two fresh blocks and one replaced page, one page free
    K.kvq_pages_reserve(pool, _i32([4, 4, 8]), None, src, dst, granted, max_new=5, dev_status=st)
    assert int(st.item()) == K._lib.KVQ_FLAG_POOL_EMPTY
    assert src.tolist() == dst.tolist() == [-1] * 3 and granted.tolist() == [0] * 3
    assert pool.ref_count.tolist() == ref and pool.block_table.tolist() == table
    # unusable lengths: flagged, the others served
    st.zero_()
    K.kvq_pages_reserve(pool, _i32([14, -1, 8]), _i32([5, 1, 6]), src, dst, granted, max_new=5, dev_status=st)
    assert int(st.item()) == K._lib.KVQ_FLAG_SEQ_LEN and granted.tolist() == [0, 0, 0]
    st.zero_()
    K.kvq_pages_reserve(pool, _i32([14, -1, 8]), _i32([5, 1, 5]), src, dst, None, max_new=5, dev_status=st)
    assert int(st.item()) == K._lib.KVQ_FLAG_SEQ_LEN and pool.block_table.tolist() == [[0, -1], [0, -1], [2, 1]]


@pytest.mark.parametrize("pages,B,M", [(1, 1, 1), (2, 1, 1), (40, 5, 7), (3000, 33, 70), (9001, 200, 38),
                                       (150000, 700, 90)])
@pytest.mark.parametrize("fill", [0.0, 0.5, 1.0])
def test_compact(pages, B, M, fill):
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(pages + int(fill * 10))
    ref, table = _random_pool(rng, pages, 16, B, M, fill=fill)
    o = P.Pool(ref, table, 16)
    pool, guards = _device(K, ref, table, 16)
    half = pages // 2
    src, dst = (Guarded((half,), torch.int32, "cuda") for _ in range(2))
    ws = Guarded((K.kvq_pages_workspace_size(pool),), torch.uint8, "cuda")
    live, st = _i32([7]), torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_pages_compact(pool, src.tensor, dst.tensor, live, workspace=ws.tensor, dev_status=st)
    movers, holes, n = o.compact()
    check_guards({"src": src, "dst": dst, "ws": ws}, "compact")
    _agree(pool, o, guards)
    assert live.tolist() == [n] and int(st.item()) == 0
    pad = [-1] * (half - len(movers))
    assert src.tensor.tolist() == movers + pad and dst.tensor.tolist() == holes + pad


def test_compact_drops_entries_of_free_pages():
    import torch
    import quantized_kv_decode_gb300 as K
    pool = K.PagePool(_i32([0, 0, 1, 0]), _i32([[2, 3], [9, -1]]), 8)
    src, dst, live = _i32([7, 7]), _i32([7, 7]), _i32([0])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_pages_compact(pool, src, dst, live, dev_status=st)
    assert int(st.item()) == K._lib.KVQ_FLAG_BLOCK_TABLE
    assert pool.block_table.tolist() == [[0, -1], [-1, -1]] and pool.ref_count.tolist() == [1, 0, 0, 0]
    assert src.tolist() == [2, -1] and dst.tolist() == [0, -1] and live.tolist() == [1]


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("layers,D", [(1, 64), (3, 128), (67, 64)])
def test_copy(fmt, layers, D):
    import torch
    import quantized_kv_decode_gb300 as K
    if layers == 67 and fmt not in ("int4", "kch4"):
        pytest.skip("many layers: two formats")
    B, names = 2, ("k_codes", "v_codes", "k_scale", "k_zero", "v_scale", "v_zero")
    gen = torch.Generator(device="cuda").manual_seed(1)
    caches, guards, before = [], [], []
    from tests._cases import guarded_cache
    for _ in range(layers):
        c, g = guarded_cache(new_cache(fmt, 3, D, B, 100, 16))
        for n in names:
            t = getattr(c, n)
            if t is not None:
                t.view(torch.uint8).random_(0, 256, generator=gen)
        caches.append(c)
        guards.append(g)
        before.append({n: None if getattr(c, n) is None else getattr(c, n).clone() for n in names})
    pages = caches[0].desc.num_pages
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    src, dst = [0, 3, -1, 0, 2, pages - 1], [1, 4, 5, 6 % pages, -1, 7 % pages]
    if pages < 9:
        src, dst = [0, -1, 2], [1, 5, -1]
    K.kvq_pages_copy(caches, _i32(src), _i32(dst), st)
    assert int(st.item()) == 0
    for c, g, old in zip(caches, guards, before):
        check_guards(g, "copy")
        for n in names:
            if old[n] is None:
                continue
            want = old[n].clone()
            for s, d in zip(src, dst):
                if s >= 0 and d >= 0:
                    want[d] = old[n][s]
            assert torch.equal(getattr(c, n).view(torch.uint8), want.view(torch.uint8)), n


def test_copy_flags():
    import torch
    import quantized_kv_decode_gb300 as K
    c = new_cache("fp16", 1, 64, 1, 100, 16)
    c.k_codes.view(torch.float16).normal_()
    old = c.k_codes.clone()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for src, dst, flag in (([0, 1], [2, 2], K._lib.KVQ_FLAG_PAGE_LIST), ([0, 1], [1, 2], K._lib.KVQ_FLAG_PAGE_LIST),
                           ([3], [3], K._lib.KVQ_FLAG_PAGE_LIST), ([0, 0], [1, 2], 0),
                           ([10 ** 6, 4], [1, 5], K._lib.KVQ_FLAG_BLOCK_TABLE),
                           ([0, 4], [10 ** 6, 5], K._lib.KVQ_FLAG_BLOCK_TABLE)):
        st.zero_()
        K.kvq_pages_copy([c], _i32(src), _i32(dst), st)
        assert int(st.item()) == flag, (src, dst)
    assert torch.equal(c.k_codes[0], old[0]) and torch.equal(c.k_codes[5], old[4])
    other = new_cache("fp16", 2, 64, 1, 100, 16)
    with pytest.raises(ValueError):
        K.kvq_pages_copy([c, other], _i32([0]), _i32([1]))


def test_a_served_run_of_all_calls():
    """Two prompts into a shared pool, four children forked from prefixes of
    them, suffixes appended (rotated keys) and attended, one more token for
    everyone, half of the sequences freed, the pool compacted: after each step
    every sequence's rows and attention equal those of its own history."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(11)
    Hq, Hkv, D, page, B, M, layers = 8, 2, 64, 16, 6, 12, 2
    pool = K.PagePool.allocate(60, page, B, M)
    desc = K.make_desc(4, 32, Hkv, D, K.KVQ_PAGED, page, 60, M)
    caches = []
    for _ in range(layers):
        c = K.KVCache.allocate(desc, B, "cuda", pool.block_table)
        c.block_table = pool.block_table
        caches.append(c)
    rope = K.make_rope(D, base=1e4)
    src, dst, granted = (_i32([-1] * B) for _ in range(3))
    ws = torch.empty(K.kvq_pages_workspace_size(pool), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    hist = [[[] for _ in range(B)] for _ in range(layers)]   # per layer and sequence: dequantized (k, v) rows
    lens = np.zeros(B, dtype=np.int64)

    def step(new, T):
        K.kvq_pages_reserve(pool, _i32(lens), _i32(new), src, dst, granted, max_new=T, workspace=ws, dev_status=st)
        assert granted.tolist() == list(new)
        K.kvq_pages_copy(caches, src, dst, st)
        for layer, c in enumerate(caches):
            x = [torch.from_numpy(rng.standard_normal((B, T, h, D)).astype(np.float16)).cuda()
                 for h in (Hkv, Hkv, Hq)]
            q = K.kvq_rope_append(c, rope, x[0], x[1], _i32(lens), q=x[2], new_lens=granted, dev_status=st)
            out = K.kvq_extend_attn(c, q, _i32(lens), int(max(lens + new)), new_lens=granted, dev_status=st)
            total = lens + new
            k16, v16 = read_rows(c, total, int(total.max()))
            for b in range(B):
                kept = hist[layer][b][:lens[b]]
                for i, (k, v) in enumerate(kept):
                    assert np.array_equal(k, k16[b, i]) and np.array_equal(v, v16[b, i]), (b, i)
                hist[layer][b] = kept + [(k16[b, i], v16[b, i]) for i in range(lens[b], total[b])]
                if new[b]:
                    check_extend(out[b].cpu().numpy(), q[b].cpu().numpy(), k16[b], v16[b], int(lens[b]),
                                 int(new[b]), D ** -0.5, rounded=True)
        assert int(st.item()) == 0
        lens[:] = lens + new

    def reorder(parent, keep):
        K.kvq_pages_reorder(pool, _i32(parent), _i32(keep), st)
        for layer in range(layers):
            hist[layer] = [list(hist[layer][p][:k]) if p >= 0 else [] for p, k in zip(parent, keep)]
        lens[:] = keep

    step(np.array([70, 33, 0, 0, 0, 0]), 70)
    reorder([0, 1, 0, 0, 1, 1], [70, 33, 70, 41, 33, 16])
    used = int((pool.ref_count > 0).sum())
    assert used == 5 + 3                                   # nothing was copied yet
    step(np.array([0, 0, 20, 3, 1, 30]), 30)
    step(np.array([1, 1, 1, 1, 1, 1]), 1)
    reorder([3, -1, 5, 0, -1, 2], [lens[3], 0, lens[5] - 2, lens[0], 0, lens[2]])
    n = 60 // 2
    ms, md, live = _i32([-1] * n), _i32([-1] * n), _i32([0])
    K.kvq_pages_compact(pool, ms, md, live, workspace=ws, dev_status=st)
    K.kvq_pages_copy(caches, ms, md, st)
    k = int(live.item())
    assert (pool.ref_count[:k] > 0).all() and not pool.ref_count[k:].any()
    assert int(pool.block_table.max()) < k
    step(np.array([2, 1, 2, 2, 5, 2]), 5)
    assert int(st.item()) == 0


def test_pool_calls_in_a_graph():
    """Reorder, reserve and copy captured once and replayed with other inputs."""
    import torch
    import quantized_kv_decode_gb300 as K
    page, pages, B, M = 8, 40, 4, 6
    rng = np.random.default_rng(2)
    ref, table = _random_pool(rng, pages, page, B, M, fill=0.4, share=0.0)
    pool, guards = _device(K, ref, table, page)
    c = new_cache("int8", 1, 64, B, 48, page)
    c.desc.num_pages = pages
    c.k_codes, c.v_codes = (torch.zeros((pages, 1, page, 64), dtype=torch.uint8, device="cuda").random_(0, 256) for _ in "kv")
    c.k_scale, c.k_zero, c.v_scale, c.v_zero = (torch.randn((pages, 1, page, 1), device="cuda").half() for _ in range(4))
    parent, keep, src, dst, granted = (_i32([0] * B) for _ in range(5))
    ws = torch.empty(K.kvq_pages_workspace_size(pool), dtype=torch.uint8, device="cuda")

    def calls():
        K.kvq_pages_reorder(pool, parent, keep)
        K.kvq_pages_reserve(pool, keep, None, src, dst, granted, max_new=1, workspace=ws)
        K.kvq_pages_copy([c], src, dst)
    state = [t.clone() for t in (pool.ref_count, pool.block_table)]
    parent.copy_(_i32(range(B)))
    calls()                                   # first call outside the capture
    torch.cuda.synchronize()
    pool.ref_count.copy_(state[0])
    pool.block_table.copy_(state[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    o = P.Pool(ref, table, page)
    for _ in range(4):
        par = rng.integers(0, B, size=B)
        kp = np.array([rng.integers(0, M * page) for _ in range(B)])
        parent.copy_(_i32(par))
        keep.copy_(_i32(kp))
        g.replay()
        o.reorder(par.tolist(), kp.tolist())
        assert o.reserve(kp.tolist(), [1] * B) == (src.tolist(), dst.tolist(), granted.tolist())
        _agree(pool, o, guards)

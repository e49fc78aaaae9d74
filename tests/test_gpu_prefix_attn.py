"""GPU tests of kvq_prefix_attn against the fp64 oracle on the dequantized rows,
and of what a call leaves alone."""
import numpy as np
import pytest

from tests._cases import Guarded, check_guards
from tests._prefix import Shared

pytestmark = pytest.mark.gpu

ALL = ["int4", "int4_g8", "int8", "int2", "sym4", "sym8", "nf4", "fp16"]


def _lens(rng, B, most, T, least=0):
    before = rng.integers(least, most + 1, size=B)
    new = rng.integers(0, T + 1, size=B)
    before[0], new[0] = 0, T
    if B > 1:
        before[1], new[1] = most, min(1, T)
    return before, new


def _batch(prefix_fmt, tail_fmt, D, Hkv, G, T, plens, B, most=70, seed=0, none=True, **kw):
    rng = np.random.default_rng(seed + B * 7 + T)
    N = len(plens)
    of = rng.integers(-1 if none else 0, N, size=B)
    before, new = _lens(rng, B, most, T)
    return Shared(prefix_fmt, tail_fmt, D, Hkv, G, plens, of, before, new, T, seed=seed, **kw)


def _run(s, **kw):
    import torch
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = Guarded(s.q.shape, torch.float16, "cuda")
    out.tensor.fill_(7.0)
    got = s.call(out=out.tensor, dev_status=st, **kw)
    assert got is out.tensor and int(st.item()) == 0
    check_guards({"out": out}, "prefix_attn")
    o = got.cpu().numpy()
    for b in range(s.B):
        assert (o[b, s.new[b]:] == 7).all()
    return o


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("T,G", [(1, 4), (3, 2)])
def test_formats(fmt, D, T, G):
    """Every per-token format, pages and dense in turn; prefixes of nothing, one
    key, whole key tiles and one more or less."""
    s = _batch(fmt, fmt, D, 2, G, T, [0, 1, 63, 64, 65, 200], 11, prefix_page=16 * (D == 64), tail_page=8 * (D == 128))
    s.check(_run(s))


@pytest.mark.parametrize("prefix_fmt,tail_fmt", [("int4", "fp16"), ("fp16", "int8"), ("int2", "nf4"), ("kch4", "fp16"),
                                                 ("kch8", "kch4"), ("int4", "kch8")])
@pytest.mark.parametrize("T", [1, 4])
def test_two_formats(prefix_fmt, tail_fmt, T):
    s = _batch(prefix_fmt, tail_fmt, 128, 2, 4, T, [130, 31], 6, prefix_page=16 if "kch" not in prefix_fmt else 32)
    s.check(_run(s))


@pytest.mark.parametrize("fmt", ["int4", "int8", "fp16", "kch4"])
@pytest.mark.parametrize("T", [1, 5])
def test_wide_heads(fmt, T):
    s = _batch(fmt, fmt, 256, 1, 3, T, [33, 70], 5, most=40)
    s.check(_run(s))


@pytest.mark.parametrize("Hkv,G,T,B,plens", [
    (1, 1, 1, 1, [100]),                  # one sequence, one head
    (3, 5, 1, 40, [257, 64]),             # odd groups, many members
    (1, 16, 1, 9, [90]),                  # more heads than a decode kernel takes
    (2, 7, 1, 3, [40] * 9),               # more prefixes than sequences
    (1, 8, 37, 9, [129, 300]),            # more than 128 rows a prefix: two tiles of rows a block
    (2, 4, 1, 150, [70]),
    (1, 1, 300, 2, [65]),
    (1, 1, 1, 70, [3] * 40),              # prefixes over more than one turn of 32
])
@pytest.mark.parametrize("fmt", ["int4", "fp16"])
def test_shapes(Hkv, G, T, B, plens, fmt):
    s = _batch(fmt, fmt, 64, Hkv, G, T, plens, B, none=B > 1)
    s.check(_run(s), only=range(0, B, max(B // 12, 1)))


@pytest.mark.parametrize("prefix_splits,tail_splits", [(1, 1), (2, 1), (3, 4), (50, 50)])
@pytest.mark.parametrize("fmt,T,G", [("int4", 1, 4), ("fp16", 1, 1), ("int8", 6, 2), ("fp16", 40, 8), ("kch8", 1, 2)])
def test_splits_on_a_used_workspace(fmt, T, G, prefix_splits, tail_splits):
    """As many splits as asked for, ragged prefixes that end in different ones,
    over a workspace of NaNs."""
    import torch
    s = _batch(fmt, fmt, 128 if fmt != "kch8" else 64, 1, G, T, [700, 90, 0], 7, most=300)
    n = s.K.kvq_prefix_attn_workspace_size(s.prefix.desc, s.tail.desc, s.N, s.B, s.T, G, s.P, s.L, prefix_splits,
                                           tail_splits)
    ws = torch.full((n // 4,), float("nan"), device="cuda").view(torch.uint8)
    for _ in range(2):
        s.check(_run(s, prefix_splits=prefix_splits, tail_splits=tail_splits, workspace=ws))
    with pytest.raises(s.K.KVQError):
        s.call(prefix_splits=prefix_splits, tail_splits=tail_splits, workspace=ws[:n - 256])


def test_without_prefixes_it_is_extend_attention():
    import torch
    s = _batch("int8", "int8", 128, 2, 4, 5, [50], 6)
    plan = s.K.kvq_prefix_plan(torch.full((6,), -1, dtype=torch.int32, device="cuda"),
                               torch.zeros(0, dtype=torch.int32, device="cuda"))
    got = s.K.kvq_prefix_attn(None, s.tail, plan, s.dev["q"], s.dev["before"], 0, s.L, new_lens=s.dev["new"])
    s.check(got.cpu().numpy(), of=np.full(6, -1))


def test_softmax_scale():
    s = _batch("int8", "int8", 64, 1, 2, 1, [60], 4)
    one, two = s.call(softmax_scale=0.125), s.call()
    assert (one == two).all()
    assert (s.call(softmax_scale=0.5) != two).any()


def test_values_behind_the_ends_do_not_matter():
    """Rows of the caches behind a prefix's or a tail's length: infinities and
    NaN; a key of fp16's lowest value and weights that vanish."""
    import torch
    s = _batch("fp16", "fp16", 128, 1, 4, 1, [70, 130], 6, prefix_page=0)
    for cache, lens in ((s.prefix, s.plens), (s.tail, s.before + s.new)):
        for arr in (cache.k_codes, cache.v_codes):
            x = arr.view(torch.float16)
            for r, n in enumerate(lens):
                x[r, :, int(n):] = float("nan") if r % 2 else float("inf")
    s.check(_run(s))
    # all weight on the tail's own token: the prefix's scores are far below
    s.prefix.k_codes.view(torch.float16).copy_(
        torch.where(s.dev["q"][0, 0, 0] > 0, -2000.0, 2000.0).half().expand_as(s.prefix.k_codes.view(torch.float16)))
    s.prefix.v_codes.view(torch.float16).fill_(60000.0)
    q = s.dev["q"]
    q[:] = q[0, 0, 0]
    out = s.call().cpu().numpy()
    s.q = q.cpu().numpy()
    s.check(out, of=np.full(s.B, -1))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_prefix_value_that_is_not_finite_reaches_its_members(bad):
    import torch
    s = _batch("fp16", "fp16", 64, 1, 2, 2, [70, 70], 6, none=False)
    s.prefix.v_codes.view(torch.float16)[1, 0, 65] = bad
    out = s.call().cpu().numpy()
    for b in range(s.B):
        live = out[b, :s.new[b]]
        if s.of[b] == 1:
            assert not np.isfinite(live).any()
        else:
            assert np.isfinite(live).all()
    s.check(out, only=[b for b in range(s.B) if s.of[b] == 0])


def test_unmapped_pages_are_left_out():
    import torch
    s = _batch("int4", "int8", 128, 2, 4, 1, [80, 40], 6, none=False, prefix_page=16, tail_page=16)
    pm = np.ones((2, s.P), dtype=bool)
    tm = np.ones((s.B, s.L), dtype=bool)
    s.prefix.block_table[0, 1] = -1
    pm[0, 16:32] = False
    s.tail.block_table[1, 0] = 1 << 20
    tm[1, :16] = False
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.call(dev_status=st).cpu().numpy()
    assert int(st.item()) == s.K.KVQ_FLAG_BLOCK_TABLE
    s.check(out, prefix_mapped=pm, tail_mapped=tm)


@pytest.mark.parametrize("T", [1, 3])
def test_lengths_that_cannot_be(T):
    """A tail that does not fit: a zero row; new_lens outside the batch's: its
    rows are left; a prefix longer than the bound: left out."""
    import torch
    s = _batch("int8", "int8", 64, 1, 2, T, [50, 20], 6, none=False)
    K, st = s.K, torch.zeros(1, dtype=torch.int32, device="cuda")
    before, new = s.dev["before"].clone(), s.dev["new"].clone()
    before[0], before[2], new[3], new[4] = s.L + 1, -1, T + 1, -1
    new[2] = 1
    out = torch.full(s.q.shape, 7.0, dtype=torch.float16, device="cuda")
    K.kvq_prefix_attn(s.prefix, s.tail, s.plan, s.dev["q"], before, s.P, s.L, new_lens=new, out=out, dev_status=st)
    assert int(st.item()) == K.KVQ_FLAG_SEQ_LEN
    o = out.cpu().numpy()
    assert not o[0, :s.new[0]].any() and not o[2, :1].any()
    assert (o[3:5] == 7).all()
    s.check(o, only=[1, 5])
    st.zero_()
    long = int(np.argmax(s.plens))
    out = K.kvq_prefix_attn(s.prefix, s.tail, s.plan, s.dev["q"], s.dev["before"], s.P - 1, s.L,
                            new_lens=s.dev["new"], dev_status=st).cpu().numpy()
    assert int(st.item()) == K.KVQ_FLAG_SEQ_LEN
    s.check(out, of=np.where(s.of == long, -1, s.of))


@pytest.mark.parametrize("T", [1, 6])
def test_captured_and_replayed(T):
    """One graph: new queries, lengths and plan between replays."""
    import torch
    s = _batch("int4", "int4", 128, 2, 4, T, [150, 90], 5)
    ws = torch.empty(s.K.kvq_prefix_attn_workspace_size(s.prefix.desc, s.tail.desc, s.N, s.B, T, 8, s.P, s.L),
                     dtype=torch.uint8, device="cuda")
    out = torch.zeros(s.q.shape, dtype=torch.float16, device="cuda")
    s.call(out=out, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.K.kvq_prefix_plan(s.dev["of"], s.dev["plens"], plan=s.plan)
        s.call(out=out, workspace=ws)
    rng = np.random.default_rng(3)
    for _ in range(3):
        s.of = rng.integers(-1, 2, size=5).astype(np.int32)
        s.q = rng.standard_normal(s.q.shape).astype(np.float16)
        s.dev["of"].copy_(torch.from_numpy(s.of))
        s.dev["q"].copy_(torch.from_numpy(s.q))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        s.check(out.cpu().numpy())


def test_two_streams():
    """Calls with their own workspaces on two streams at once."""
    import torch
    a = _batch("int4", "int4", 128, 2, 4, 1, [900], 20, seed=1)
    b = _batch("fp16", "fp16", 128, 2, 4, 3, [900], 20, seed=2)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        x, y = a.call(stream=one), b.call(stream=two)
    torch.cuda.synchronize()
    a.check(x.cpu().numpy(), only=range(0, 20, 4))
    b.check(y.cpu().numpy(), only=range(0, 20, 4))


def test_the_same_result_each_time():
    s = _batch("int8", "int8", 128, 2, 4, 1, [2000], 30)
    first = s.call()
    assert all((s.call() == first).all() for _ in range(3))

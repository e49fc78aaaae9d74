"""GPU tests of the kernels that kvq_prefix_attn picks from by sizes: few rows
with their codes in registers, one, two and four warps a tail, long tails with
splits, and values at the ends of fp16."""
import numpy as np
import pytest

from tests._prefix import Shared
from tests.test_gpu_prefix_attn import _batch, _run

pytestmark = pytest.mark.gpu

CODES = ["int4", "int8", "sym4", "nf4"]


@pytest.mark.parametrize("members", [1, 4, 5, 8, 9, 17])
@pytest.mark.parametrize("fmt", CODES)
@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_one_prefix(fmt, D, members):
    """4 to 68 rows over one prefix: part of a tile of 16 or 32 rows, whole ones,
    and one row more; a prefix of several key tiles a warp and a ragged end."""
    s = _batch(fmt, fmt, D, 2, 4, 1, [333], members, most=20, none=False, seed=members)
    s.check(_run(s))
    s.check(_run(s, prefix_splits=2))


@pytest.mark.parametrize("fmt", CODES)
@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_many_prefixes(fmt, D):
    """16 prefixes of 16 KV heads, 32 rows each on average: tiles of 32 rows are
    one turn over the device, of 16 two."""
    rng = np.random.default_rng(D)
    s = _batch(fmt, fmt, D, 16, 4, 1, rng.integers(90, 300, size=16).tolist(), 128, most=20, none=False, seed=D)
    s.check(_run(s, prefix_splits=1), only=range(0, 128, 5))


@pytest.mark.parametrize("page", [8, 16, 24, 64])
@pytest.mark.parametrize("fmt", CODES)
def test_rows_over_pages(fmt, page):
    """Pages shorter and longer than a warp's key tile, two of them unmapped."""
    import torch
    s = _batch(fmt, fmt, 128, 2, 4, 1, [150, 90], 7, most=30, none=False, prefix_page=page, tail_page=page)
    s.check(_run(s))
    mapped = np.ones((2, s.P), dtype=bool)
    s.prefix.block_table[0, 0] = -1
    s.prefix.block_table[1, 40 // page] = 1 << 30
    mapped[0, :page] = False
    mapped[1, 40 // page * page:(40 // page + 1) * page] = False
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.call(dev_status=st).cpu().numpy()
    assert int(st.item()) == s.K.KVQ_FLAG_BLOCK_TABLE
    s.check(out, prefix_mapped=mapped)


def test_a_prefix_without_any_mapped_page():
    """Nothing to see there: the tail alone; and a sequence whose tail has none
    either gets a zero row."""
    import torch
    s = _batch("int4", "int4", 128, 1, 4, 1, [64], 3, most=30, none=False, prefix_page=16, tail_page=16)
    s.prefix.block_table.fill_(-1)
    s.tail.block_table[1] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.call(dev_status=st).cpu().numpy()
    assert int(st.item()) == s.K.KVQ_FLAG_BLOCK_TABLE
    s.check(out, only=[b for b in (0, 2) if s.new[b]], of=np.full(3, -1))
    assert not out[1, :s.new[1]].any()


@pytest.mark.parametrize("fmt,D,Hkv,G", [("int4", 128, 2, 4), ("int8", 64, 2, 7), ("int2", 128, 2, 2), ("nf4", 64, 2, 1),
                                         ("sym8", 128, 2, 1), ("sym4", 64, 2, 8)])
@pytest.mark.parametrize("B", [3, 200, 400, 700])
def test_warps_of_a_tail(fmt, D, Hkv, G, B):
    """Four, two and one warp a (sequence, KV head), tails shorter than a key tile
    to several of them; a few sequences have no new token."""
    s = _batch(fmt, fmt, D, Hkv, G, 1, [70, 33], B, most=150, seed=B)
    s.check(_run(s), only=list(range(0, B, max(B // 25, 1))) + [B - 1])


@pytest.mark.parametrize("fmt", ["int4", "fp16", "int8", "kch8"])
def test_long_tails_are_split(fmt):
    """Tails beyond the tail kernel's: a decode kernel with splits, and the join."""
    s = _batch(fmt, fmt, 128, 1, 2, 1, [100], 2, most=2600, none=False)
    s.check(_run(s))


@pytest.mark.parametrize("fmt,D", [("int4", 128), ("fp16", 128), ("int2", 128), ("int8", 256)])
def test_prefixes_far_apart(fmt, D):
    """Few of many prefixes have members: in the first 32, at the edge of the next,
    behind many without any; one of them is empty."""
    plens = np.full(230, 12, dtype=np.int32)
    plens[[0, 64, 229]] = 40, 0, 75
    of = [0, 33, 64, 150, 229, 229, 0, -1, 63]
    s = Shared(fmt, fmt, D, 1, 2, plens, of, [3] * 9, [1] * 9, 1, seed=D)
    s.check(_run(s))
    some = Shared(fmt, fmt, D, 1, 2, plens, [0, 31, 5], [3, 0, 9], [1, 2, 1], 2, seed=D)
    some.check(_run(some))


@pytest.mark.parametrize("fmt,members", [("int4", 3), ("int4", 40), ("nf4", 3), ("fp16", 3)])
def test_pages_beyond_four_gigabytes(fmt, members):
    """Codes more than 2^32 bytes behind the arrays' start: what the first pages
    of the pool hold gives the same result to the bit."""
    import torch
    import quantized_kv_decode_gb300 as K
    from tests._prompt import FORMATS
    bits, g, kw = FORMATS[fmt]
    D, G, page, P, own = 128, 4, 64, 200, 40
    far = 2 ** 32 // (page * D * bits // 8) + 100
    gen = torch.Generator(device="cuda").manual_seed(members)
    rand = lambda *n: torch.randn(*n, generator=gen, dtype=torch.float16, device="cuda")
    pkv, tkv, q = [rand(1, P, 1, D) for _ in "kv"], [rand(members, own, 1, D) for _ in "kv"], rand(members, 1, G, D)
    axes = K.make_rope_axes((32, 32))
    outs = []
    for pages in (100, far):
        desc = K.make_desc(bits, g, 1, D, K.KVQ_PAGED, page, pages, 4, **kw)
        rows = pages - 1 - torch.arange(4 + members, dtype=torch.int32, device="cuda")
        table = torch.full((members, 4), -1, dtype=torch.int32, device="cuda")
        table[:, 0] = rows[4:]
        tail = K.KVCache.allocate(desc, members, "cuda", table)
        prefix = tail.with_table(rows[:4].reshape(1, 4).clone())
        for c, (k, v) in ((prefix, pkv), (tail, tkv)):
            n, t = k.shape[:2]
            pos = torch.arange(2 * t, dtype=torch.int32, device="cuda").reshape(1, t, 2).repeat(n, 1, 1)
            K.kvq_rope_axes_append(c, axes, pos, k, v, torch.zeros(n, dtype=torch.int32, device="cuda"))
        of = torch.zeros(members, dtype=torch.int32, device="cuda")
        plan = K.kvq_prefix_plan(of, torch.tensor([P], dtype=torch.int32, device="cuda"))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        outs.append(K.kvq_prefix_attn(prefix, tail, plan, q, of + own - 1, P, own, dev_status=st).cpu())
        assert int(st.item()) == 0
        del tail, prefix
    assert torch.isfinite(outs[0]).all() and outs[0].any() and torch.equal(*outs)


def test_no_new_lens_and_no_prefix_len():
    """Every row live; empty prefixes and a bound of 0 on their lengths."""
    import torch
    for T in (1, 3):
        s = Shared("int8", "int8", 128, 1, 4, [0, 0], [0, 1, -1], [5, 0, 70], [T, T, T], T, seed=T)
        out = s.call(new_lens=None).cpu().numpy()
        s.check(out)
        got = s.K.kvq_prefix_attn(s.prefix, s.tail, s.plan, s.dev["q"], s.dev["before"], 0, s.L).cpu().numpy()
        assert np.array_equal(got, out)


@pytest.mark.parametrize("fmt", CODES + ["fp16"])
def test_values_at_the_ends_of_fp16(fmt):
    """V at +-60000 and keys far from zero: nothing overflows on the way, and the
    result is the formula's.  (The tail's own kernel is kvq_decode_attn's; its
    values are ordinary here.)"""
    import torch
    from tests._prompt import expected_rows, new_cache
    from oracle import prefix_oracle as X
    K = __import__("quantized_kv_decode_gb300")
    rng = np.random.default_rng(5)
    D, H, G, P, B = 128, 1, 4, 200, 3
    k = (rng.standard_normal((1, P, H, D)) + 40.0).astype(np.float16)
    v = np.where(rng.random((1, P, H, D)) < 0.5, -60000.0, 60000.0).astype(np.float16)
    q = (rng.standard_normal((B, 1, H * G, D)) * 0.05).astype(np.float16)
    prefix = new_cache(fmt, H, D, 1, P)
    tail = new_cache("fp16", H, D, B, 1)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_append(prefix, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), zero)
    tk = np.zeros((B, 1, H, D), dtype=np.float16)
    K.kvq_append(tail, torch.from_numpy(tk).cuda(), torch.from_numpy(tk).cuda(), torch.zeros(B, dtype=torch.int32, device="cuda"))
    plan = K.kvq_prefix_plan(torch.zeros(B, dtype=torch.int32, device="cuda"), torch.tensor([P], dtype=torch.int32, device="cuda"))
    out = K.kvq_prefix_attn(prefix, tail, plan, torch.from_numpy(q).cuda(), torch.zeros(B, dtype=torch.int32, device="cuda"), P, 1)
    out = out.cpu().numpy().astype(np.float64)
    kh, vh = (expected_rows(fmt, x)[0].transpose(1, 0, 2) for x in (k, v))
    t0 = np.zeros((H, 1, D))
    scale = D ** -0.5
    S = float(np.abs(q.astype(np.float64)).max(axis=(0, 1, 2)).sum() * np.abs(kh).max())
    # per score D + 4 roundings of fp32 at up to 3 S (scale and zero-point apart),
    # felt twice (weight and sum); a probability's rounding and its product's
    # (2^-11 each), V's own to 11 bits where it enters as one number, the result's;
    # and P sums in fp32 at up to 65504: 200 * 2^-24 * 65504 < 1
    rel = 3 * 2.0 ** -11 + 2 * 1.5 * scale * (D + 4) * 2.0 ** -24 * 3 * S + 2.0 ** -18
    for b in range(B):
        want, mass = X.prefix_attention(q[b].astype(np.float64), kh, np.clip(vh, -65504, 65504), t0, t0, 0, scale)
        off = np.abs(out[b] - want)
        assert np.isfinite(out[b]).all()
        assert (off <= mass * rel + np.abs(want) * 2.0 ** -11 + 1.0).all(), (off / mass).max()


@pytest.mark.parametrize("bits,kw", [(2, {}), (4, {}), (8, {}), (2, dict(symmetric=True)), (4, dict(symmetric=True)),
                                     (8, dict(symmetric=True)), (4, dict(nf4=True)), (16, {})])
def test_one_new_token_in_every_format(bits, kw):
    """Group sizes, head sizes and heads per KV head of every width: whichever kernel
    the tails come to, one that is built for them takes the call, and without prefixes
    the result is what kvq_decode_attn gives."""
    import torch
    import quantized_kv_decode_gb300 as K
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    B, L = 3, 90
    plan = K.kvq_prefix_plan(i32([-1] * B), i32([]))
    gen = torch.Generator(device="cuda").manual_seed(bits)
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float16, device="cuda")  # noqa: E731
    for D in (64, 128, 256):
        for g in (8, 16, 32, 64, 128) if bits != 16 else (0,):
            if g > D:
                continue
            cache = K.KVCache.allocate(K.make_desc(bits, g, 2, D, K.KVQ_DENSE, 96, **kw), B, "cuda")
            K.kvq_append(cache, rand(B, L, 2, D), rand(B, L, 2, D), i32([0] * B))
            for G in (1, 2, 3, 4, 8, 9):
                q = rand(B, 1, 2 * G, D)
                want = K.kvq_decode_attn(cache, q[:, 0].contiguous(), i32([L, 1, 33]), L).float()
                for splits in (0, 2):
                    got = K.kvq_prefix_attn(None, cache, plan, q, i32([L - 1, 0, 32]), 0, L, tail_splits=splits)
                    # two sums in different orders: each 2^-9 (weights and result to 11 bits) of up to 4
                    assert (got[:, 0].float() - want).abs().max() <= 2 * 2.0 ** -9 * 4, (D, g, G, splits)

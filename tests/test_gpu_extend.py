"""GPU tests of kvq_extend_attn against the fp64 oracle on the rows that the
cache holds, dequantized in fp64 (axis-aware caches: read back through
kvq_cache_read, rounded to fp16), with the error bound of tests/_prompt.py; refusals and flags; splits, streams, graphs; and equality with the decode call for one new token."""
import numpy as np
import pytest

from tests._cases import Guarded, check_guards
from oracle import prompt_oracle as P
from tests._prompt import FORMATS, check_extend, expected_rows, new_cache, read_rows

pytestmark = pytest.mark.gpu


def _fill(K, cache, rng, lens, Hkv, D, most):
    """`most` random rows of every sequence appended (keys with large channels)."""
    import torch
    B = len(lens)
    k = rng.standard_normal((B, most, Hkv, D)).astype(np.float16)
    k[..., 1:3] *= 4
    v = rng.standard_normal((B, most, Hkv, D)).astype(np.float16)
    z = torch.zeros(B, dtype=torch.int32, device="cuda")
    K.kvq_append(cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), z)
    return k, v


def _case(fmt, D, Hq, Hkv, T, before, new=None, page=0, splits=0, seed=0, scale=0.0, extra=2):
    """One call on guarded buffers, every sequence checked."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(seed)
    B = len(before)
    new = [T] * B if new is None else new
    lens = [a + n for a, n in zip(before, new)]
    most = max(max(lens), 1)
    kch = FORMATS[fmt][2].get("k_per_channel", False)
    cache = new_cache(fmt, Hkv, D, B, most + extra, page, seed)
    if kch:  # a sequence's window holds its own newest tokens: append to its length
        k = rng.standard_normal((B, most, Hkv, D)).astype(np.float16)
        v = rng.standard_normal((B, most, Hkv, D)).astype(np.float16)
        at = np.zeros(B, dtype=np.int32)
        assert len(set(lens)) == 1, "axis-aware cases use one length"
        K.kvq_append(cache, torch.from_numpy(k[:, :lens[0]].copy()).cuda(),
                     torch.from_numpy(v[:, :lens[0]].copy()).cuda(), torch.from_numpy(at).cuda())
    else:
        k, v = _fill(K, cache, rng, lens, Hkv, D, most)
    kx, vx = read_rows(cache, lens, most) if kch else (expected_rows(fmt, k), expected_rows(fmt, v))
    q = rng.standard_normal((B, T, Hq, D)).astype(np.float16)
    dev = "cuda"
    tq = torch.from_numpy(q).to(dev)
    tb = torch.tensor(before, dtype=torch.int32, device=dev)
    tn = torch.tensor(new, dtype=torch.int32, device=dev)
    out = Guarded(q.shape, torch.float16, dev)
    out.tensor.fill_(9)
    need = K.kvq_extend_workspace_size(cache.desc, B, T, Hq, most, splits)
    ws = Guarded((need,), torch.uint8, dev) if need else None
    if ws is not None:
        ws.tensor.fill_(0xFF)          # NaN in every float
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    for _ in range(2):                 # twice on one workspace
        K.kvq_extend_attn(cache, tq, tb, most, new_lens=tn, out=out.tensor, workspace=None if ws is None else ws.tensor,
                          dev_status=st, num_splits=splits, softmax_scale=scale)
        assert int(st.item()) == 0
        check_guards({"out": out, **({"ws": ws} if ws else {})}, "extend")
        got = out.tensor.cpu().numpy()
        for b in range(B):
            assert (got[b, new[b]:] == 9).all(), "rows behind the sequence"
            if new[b]:
                check_extend(got[b], q[b], kx[b], vx[b], before[b], new[b], scale or D ** -0.5, rounded=kch)
    return got


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_format(fmt, D):
    _case(fmt, D, 4, 2, 37, [60, 60])


@pytest.mark.parametrize("fmt", ["int4", "int8", "fp16", "kch4", "nf4"])
@pytest.mark.parametrize("page", [8, 16, 64])
def test_paged(fmt, page):
    kch = fmt == "kch4"
    _case(fmt, 128, 4, 2, 21, [100, 100] if kch else [100, 3], page=page)


@pytest.mark.parametrize("T", [1, 2, 5, 16, 17, 64, 129, 300])
@pytest.mark.parametrize("before", [0, 1, 63, 64, 700])
def test_lengths(T, before):
    _case("int4", 128, 8, 2, T, [before])


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (7, 1), (8, 1), (14, 2), (17, 1), (5, 5), (40, 2)])
def test_head_groups(Hq, Hkv):
    _case("int8", 64, Hq, Hkv, 19, [33, 150], new=[19, 6])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["fp16", "int4", "int8", "sym4", "int2"])
def test_long_prompts(fmt, D):
    """Several row tiles and key tiles, lengths that are no multiple of them."""
    _case(fmt, D, 4, 2, 391, [0, 517], new=[391, 200], seed=2)


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 50])
@pytest.mark.parametrize("fmt", ["int4", "fp16"])
def test_splits(splits, fmt):
    """Splits past a sequence's end and past a tile's last visible key."""
    _case(fmt, 64, 4, 1, 40, [0, 300, 10], new=[40, 1, 0], splits=splits)


def test_ragged_batch_and_scale():
    _case("int4", 128, 8, 2, 33, [0, 5, 200, 64, 31], new=[33, 1, 0, 17, 32], page=16, scale=0.3)


def test_split_counts_follow_the_request():
    import quantized_kv_decode_gb300 as K
    d = K.make_desc(4, 32, 2, 64, K.KVQ_DENSE, 4096)
    assert K.kvq_extend_num_splits(d, 1, 4, 8, 4096, 5) == 5
    assert K.kvq_extend_num_splits(d, 1, 4, 8, 64, 5) == 1
    assert K.kvq_extend_workspace_size(d, 1, 4, 8, 64, 5) == 0
    s = K.kvq_extend_num_splits(d, 1, 4, 8, 4096)
    assert s > 1 and K.kvq_extend_workspace_size(d, 1, 4, 8, 4096) >= 4 * 8 * s * (64 + 2) * 4


def test_one_new_token_is_the_decode_call():
    """T = 1 and kvq_decode_attn agree within both calls' tolerances."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(1)
    lens = [700, 64, 1]
    cache = new_cache("int4", 2, 128, 3, 701)
    _fill(K, cache, rng, lens, 2, 128, 700)
    q = torch.from_numpy(rng.standard_normal((3, 8, 128)).astype(np.float16)).cuda()
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = K.kvq_decode_attn(cache, q, t, 700)
    b = K.kvq_extend_attn(cache, q[:, None].contiguous(), t - 1, 700)[:, 0]
    # the decode tolerance, and K, V and p rounded to fp16 (2^-11 each of |v| <= 5)
    assert float((a - b).abs().max()) <= 2e-3 + 3 * 5 * 2.0 ** -11


def test_flags_and_left_out_tokens():
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(9)
    B, T, Hkv, Hq, D, L = 4, 5, 1, 3, 64, 40
    cache = new_cache("int8", Hkv, D, B, L, 8)
    _fill(K, cache, rng, [L] * B, Hkv, D, L)
    k16, v16 = read_rows(cache, [L] * B, L)
    q = rng.standard_normal((B, T, Hq, D)).astype(np.float16)
    before = [20, 39, -1, 10]
    cache.block_table[0, 1] = -1            # positions 8..15 of sequence 0
    cache.block_table[3, :2] = 1 << 20      # everything of sequence 3: 0..14
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for splits in (1, 3):
        st.zero_()
        out = torch.full(q.shape, 9.0, dtype=torch.float16, device="cuda")
        K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), torch.tensor(before, dtype=torch.int32, device="cuda"),
                          L, out=out, dev_status=st, num_splits=splits)
        assert int(st.item()) == K._lib.KVQ_FLAG_SEQ_LEN | K._lib.KVQ_FLAG_BLOCK_TABLE
        got = out.cpu().numpy()
        mapped = np.ones(25, dtype=bool)
        mapped[8:16] = False
        check_extend(got[0], q[0], k16[0], v16[0], 20, T, D ** -0.5, mapped, rounded=True)
        assert (got[1:] == 0).all()         # too long, negative, nothing mapped: zero rows
    # an unusable new_lens: that sequence is skipped
    out.fill_(9)
    st.zero_()
    K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), torch.tensor([0, 0, 0, 0], dtype=torch.int32, device="cuda"),
                      L, new_lens=torch.tensor([T + 1, -1, 1, 0], dtype=torch.int32, device="cuda"), out=out,
                      dev_status=st)
    got = out.cpu().numpy()
    assert int(st.item()) & K._lib.KVQ_FLAG_SEQ_LEN
    assert (got[0] == 9).all() and (got[1] == 9).all() and (got[2, 1:] == 9).all() and (got[3] == 9).all()
    check_extend(got[2], q[2], k16[2], v16[2], 0, 1, D ** -0.5, rounded=True)


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("fmt,value", [("fp16", float("nan")), ("fp16", float("inf")), ("int8", None)])
def test_rows_behind_the_sequence_do_not_count(fmt, value, T):
    """NaN and infinities in cached rows that no token may see: behind the
    sequence, and in the causal mask's reach only later tokens'."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(4)
    Hkv, D, L = 2, 64, 150 + T
    cache = new_cache(fmt, Hkv, D, 1, L + 100)
    _fill(K, cache, rng, [L], Hkv, D, L)
    k16, v16 = read_rows(cache, [L], L)
    if fmt == "fp16":
        for t in (cache.k_codes, cache.v_codes):
            t.view(torch.float16)[:, :, L:] = value
    else:
        for t in (cache.k_scale, cache.v_scale, cache.k_zero, cache.v_zero):
            t[:, :, L:] = float("nan")
    q = rng.standard_normal((1, T, 4, D)).astype(np.float16)
    got = K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), torch.tensor([150], dtype=torch.int32, device="cuda"),
                            L + 100).cpu().numpy()
    check_extend(got[0], q[0], k16[0], v16[0], 150, T, D ** -0.5, rounded=True)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,D", [(5, 64), (200, 128), (150, 256)])
def test_a_later_token_does_not_reach_earlier_ones(T, D, value):
    """An infinity or NaN in K and V of one new token: the tokens before it
    come out as without it, its own and later ones are not finite."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(8)
    before, at = 70, T // 2
    L = before + T
    cache = new_cache("fp16", 1, D, 1, L)
    _fill(K, cache, rng, [L], 1, D, L)
    k16, v16 = read_rows(cache, [L], L)
    for t in (cache.k_codes, cache.v_codes):
        t.view(torch.float16)[:, :, before + at, 3] = value
    q = rng.standard_normal((1, T, 4, D)).astype(np.float16)
    got = K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), torch.tensor([before], dtype=torch.int32, device="cuda"),
                            L).cpu().numpy()
    check_extend(got[0], q[0], k16[0], v16[0], before, at, D ** -0.5, rounded=True)
    assert not np.isfinite(got[0, at:]).all(axis=-1).any()


@pytest.mark.parametrize("fmt", ["int4", "int8", "sym4", "nf4"])
@pytest.mark.parametrize("g_is_D", [False, True])
@pytest.mark.parametrize("extra", [0, 1, 2, 5])
def test_header_arrays_of_any_alignment(fmt, g_is_D, extra):
    """Dense capacities that leave a head's scales and zeros at any two-byte
    boundary, down to one header per row; the last head's end the array."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(12)
    bits, g, kw = FORMATS[fmt]
    D, Hkv, B, T, L = 64, 3, 2, 6, 131 + extra
    desc = K.make_desc(bits, D if g_is_D else g, Hkv, D, K.KVQ_DENSE, L, **kw)
    cache = K.KVCache.allocate(desc, B, "cuda")
    _fill(K, cache, rng, [L] * B, Hkv, D, L)
    k16, v16 = read_rows(cache, [L] * B, L)
    q = rng.standard_normal((B, T, 6, D)).astype(np.float16)
    before = [L - T, 57]
    for splits in (1, 2):
        got = K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), torch.tensor(before, dtype=torch.int32, device="cuda"),
                                L, num_splits=splits).cpu().numpy()
        for b in range(B):
            check_extend(got[b], q[b], k16[b], v16[b], before[b], T, D ** -0.5, rounded=True)


def test_far_zero_points_and_large_scales():
    """Groups whose zero-point lies beyond +-1024 and groups that reach fp16's
    end: products that leave the fast fp16 conversion."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(13)
    D, L, T = 64, 90, 7
    cache = new_cache("int8", 1, D, 1, L)
    k = (rng.standard_normal((1, L, 1, D)) * 0.01).astype(np.float16)
    k[0, ::3] += np.float16(0.5)           # range 0.06 around 0.5: z about -2000
    v = rng.standard_normal((1, L, 1, D)).astype(np.float16)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_append(cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), z)
    assert float(cache.k_zero.float().abs().max()) > 1024
    k16, v16 = read_rows(cache, [L], L)
    q = rng.standard_normal((1, T, 2, D)).astype(np.float16)
    b = torch.tensor([L - T], dtype=torch.int32, device="cuda")
    got = K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), b, L).cpu().numpy()
    check_extend(got[0], q[0], k16[0], v16[0], L - T, T, D ** -0.5, rounded=True)
    # one key at the end of fp16's range, all others small: scores stay finite
    k[0, 5, 0, :] = np.linspace(0, 65504, D).astype(np.float16)  # code 255 decodes to 65535
    K.kvq_append(cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), z)
    q[:] = 0
    q[..., 0] = np.float16(1e-3)
    k16, v16 = read_rows(cache, [L], L)
    assert np.abs(k16[0, 5].astype(np.float64)).max() == 65504
    got = K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), b, L, softmax_scale=0.01).cpu().numpy()
    check_extend(got[0], q[0], k16[0], v16[0], L - T, T, 0.01, rounded=True)


def test_large_scores_keep_the_softmax_exact():
    """Scores of several thousand: one key takes all the weight, whichever
    tile it is in, and earlier tiles' sums vanish without overflow."""
    import torch
    import quantized_kv_decode_gb300 as K
    D, L, T = 64, 600, 130
    cache = new_cache("fp16", 1, D, 1, L)
    k = np.zeros((1, L, 1, D), dtype=np.float16)
    k[0, :, 0, 0] = np.arange(L) % 97 * 8
    v = np.random.default_rng(0).standard_normal((1, L, 1, D)).astype(np.float16)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_append(cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), z)
    q = np.zeros((1, T, 2, D), dtype=np.float16)
    q[0, :, 0, 0] = 64.0
    q[0, :, 1, 0] = -64.0
    got = K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), torch.tensor([L - T], dtype=torch.int32, device="cuda"),
                            L, softmax_scale=1.0).cpu().numpy().astype(np.float64)
    for t in range(T):
        see = np.arange(L - T + t + 1)
        top = see[see % 97 == (see % 97).max()]
        low = see[see % 97 == 0]
        for h, w in ((0, top), (1, low)):
            want = v[0, w, 0].astype(np.float64).mean(0)
            # weights are exactly 1 / len(w): the mean's sum in fp32 and one rounding
            assert np.abs(got[0, t, h] - want).max() <= 2.0 ** -11 * 5 + 2.0 ** -18


def test_streams_and_graph_replay():
    """Two calls on two streams with their own workspaces, and a captured call
    replayed on new inputs, give the eager results bit for bit."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(6)
    B, T, Hq, Hkv, D, L = 2, 9, 8, 2, 128, 900
    cache = new_cache("int4", Hkv, D, B, L)
    _fill(K, cache, rng, [L] * B, Hkv, D, L)
    before = torch.tensor([L - T, 100], dtype=torch.int32, device="cuda")
    qs = [torch.from_numpy(rng.standard_normal((B, T, Hq, D)).astype(np.float16)).cuda() for _ in range(3)]
    need = K.kvq_extend_workspace_size(cache.desc, B, T, Hq, L)
    ws = [torch.empty(max(need, 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
    eager = [K.kvq_extend_attn(cache, q, before, L) for q in qs]
    outs = [torch.empty_like(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, s in enumerate(streams):
        K.kvq_extend_attn(cache, qs[i], before, L, out=outs[i], workspace=ws[i], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], eager[0]) and torch.equal(outs[1], eager[1])
    q, out = qs[0].clone(), torch.empty_like(qs[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kvq_extend_attn(cache, q, before, L, out=out, workspace=ws[0])
    for i in (2, 1):
        q.copy_(qs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i])


@pytest.mark.parametrize("T", [3, 140])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["int4", "int8", "int2", "sym8", "nf4"])
def test_scores_follow_the_dequantized_keys(fmt, D, T):
    """Large scores, against (q - z) s itself: keys rounded to 11 bits would be
    off by up to 2^-11 of a score of 80.

    Bound: a score takes K to 22 bits and its scaling in fp32 (2^-22 and four
    roundings of 2^-24, relative to 80 log2(e)), felt by its own weight and by
    the sum of weights; weights and V are rounded to fp16 (2^-11 each, or
    2^-32 absolute for small weights), the sums take L terms in fp32, the
    output is rounded to fp16."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(11)
    before, Hq, Hkv, scale = 150, 2, 1, 0.1
    L = before + T
    cache = new_cache(fmt, Hkv, D, 1, L)
    k = rng.standard_normal((1, L, Hkv, D)).astype(np.float16)
    k[..., 5] = rng.uniform(-25, 25, (1, L, Hkv))
    v = rng.standard_normal((1, L, Hkv, D)).astype(np.float16)
    K.kvq_append(cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(),
                 torch.zeros(1, dtype=torch.int32, device="cuda"))
    q = np.zeros((1, T, Hq, D), dtype=np.float16)
    q[..., 0, 5], q[..., 1, 5] = 32, -32
    got = K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), torch.tensor([before], dtype=torch.int32, device="cuda"),
                            L, softmax_scale=scale, num_splits=1).cpu().numpy()[0].astype(np.float64)
    kx, vx = (expected_rows(fmt, x[0]).transpose(1, 0, 2) for x in (k, v))
    want, mass = P.extend_attention(q[0].astype(np.float64), kx, vx, before, scale)
    top = 32 * scale * np.abs(kx[..., 5]).max() * 1.4427
    rel = 2 * 2.0 ** -11 + 2 * top * (2.0 ** -22 + 4 * 2.0 ** -24) + L * 2.0 ** -23
    bound = mass * rel + 2.0 ** -11 * np.abs(want) + L * 2.0 ** -32 * np.abs(vx).max() + 2.0 ** -24
    assert (np.abs(got - want) / bound).max() <= 1.0


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("T", [3, 140])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_small_weights(D, T, splits):
    """One key whose value is zero, and thousands 2^-20.4 of its weight that
    make up the output: each weight keeps its 11 bits (fp16's own steps at
    2^-20 are an eighth of that).  Scores are exact up to fp32's roundings."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(12)
    before, scale = 2500, 0.0625
    L = before + T
    cache = new_cache("fp16", 1, D, 1, L)
    k = np.zeros((1, L, 1, D), dtype=np.float16)
    k[:, 1:, :, 3] = -14.140625
    v = rng.uniform(1, 2, (1, L, 1, D)).astype(np.float16)
    v[:, 0] = 0
    K.kvq_append(cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(),
                 torch.zeros(1, dtype=torch.int32, device="cuda"))
    q = np.zeros((1, T, 1, D), dtype=np.float16)
    q[..., 3] = 16
    got = K.kvq_extend_attn(cache, torch.from_numpy(q).cuda(), torch.tensor([before], dtype=torch.int32, device="cuda"),
                            L, softmax_scale=scale, num_splits=splits).cpu().numpy()[0].astype(np.float64)
    kx, vx = (x[0].astype(np.float64).transpose(1, 0, 2) for x in (k, v))
    want, mass = P.extend_attention(q[0].astype(np.float64), kx, vx, before, scale)
    rel = 2.0 ** -11 + 2 * 20.4 * 4 * 2.0 ** -24 + 2 * L * 2.0 ** -24
    bound = mass * rel + 2.0 ** -11 * np.abs(want)
    assert (np.abs(got - want) / bound).max() <= 1.0


def test_outputs_made_on_the_calls_stream():
    """Outputs and workspaces made by a call on another stream than the
    current one are made on that stream: work queued on the current stream
    neither comes in between nor afterwards."""
    import torch
    import quantized_kv_decode_gb300 as K
    rng = np.random.default_rng(13)
    B, T, Hq, Hkv, D, L = 2, 9, 8, 2, 128, 900
    cache = new_cache("int4", Hkv, D, B, L)
    _fill(K, cache, rng, [L] * B, Hkv, D, L)
    before = torch.tensor([L - T, 100], dtype=torch.int32, device="cuda")
    new = torch.tensor([T, 5], dtype=torch.int32, device="cuda")
    q = torch.from_numpy(rng.standard_normal((B, T, Hq, D)).astype(np.float16)).cuda()
    rope = K.make_rope(D)
    want = K.kvq_extend_attn(cache, q, before, L, new_lens=new)
    turned = K.kvq_rope_apply(rope, q, seq_lens_before=before, new_lens=new)[0]
    assert want.abs().max() > 0 and (want[1, 5:] == 0).all() and (turned[1, 5:] == 0).all()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        torch.cuda._sleep(100_000_000)  # the current stream is busy meanwhile
        out = K.kvq_extend_attn(cache, q, before, L, new_lens=new, stream=stream)
        y = K.kvq_rope_apply(rope, q, seq_lens_before=before, new_lens=new, stream=stream)[0]
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(y, turned)


def test_workspace_refusal_and_device_checks():
    import torch
    import quantized_kv_decode_gb300 as K
    cache = new_cache("int4", 2, 64, 2, 512)
    q = torch.zeros((2, 3, 4, 64), dtype=torch.float16, device="cuda")
    b = torch.zeros(2, dtype=torch.int32, device="cuda")
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(K.KVQError) as e:
        K.kvq_extend_attn(cache, q, b, 512, workspace=small, num_splits=4)
    assert e.value.status == K.KVQ_ERR_WORKSPACE
    for bad in (dict(seq_lens_before=b.cpu()), dict(seq_lens_before=b.long()), dict(new_lens=b[:1]),
                dict(out=q.float()), dict(dev_status=torch.zeros(1, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            K.kvq_extend_attn(cache, **{"q": q, "seq_lens_before": b, "max_seq_len": 512, **bad})
    with pytest.raises(ValueError):
        K.kvq_extend_attn(cache, q.transpose(1, 2), b, 512)
    with pytest.raises(ValueError):
        K.kvq_extend_attn(cache, torch.cat([q, q]), torch.cat([b, b]), 512)

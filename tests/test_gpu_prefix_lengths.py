"""GPU tests of kvq_prefix_attn on lengths and counts that cannot be, one new
token a sequence (whichever kernel takes the tails, the call flags them and
leaves or zeroes the rows that kvq.h names), and of what it refuses."""
import numpy as np
import pytest

from tests.test_gpu_prefix_attn import _batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tail_splits", [0, 2])
@pytest.mark.parametrize("fmt,D", [("int4", 64), ("int4", 128), ("int8", 64), ("int8", 128), ("int2", 128), ("sym4", 128),
                                   ("sym8", 128), ("nf4", 64), ("nf4", 128), ("fp16", 128)])
def test_counts_and_lengths_of_one_new_token(fmt, D, tail_splits):
    """A count outside {0, 1}: flagged, the row left.  No new token: the row left,
    a length that cannot be flagged all the same.  One new token behind a length
    that does not fit: flagged, a zero row."""
    import torch
    s = _batch(fmt, fmt, D, 2, 2, 1, [50, 20], 7, none=False)
    K, st = s.K, torch.zeros(1, dtype=torch.int32, device="cuda")
    s.dev["new"].fill_(1)
    s.new[:] = 1
    s.before[:] = np.minimum(s.before, s.L - 1)
    s.dev["before"].copy_(torch.from_numpy(s.before))
    for new, before, flagged, row in ((2, None, True, "left"), (-1, None, True, "left"), (1 << 30, None, True, "left"),
                                      (0, None, False, "left"), (0, -1, True, "left"), (0, s.L + 1, True, "left"),
                                      (1, -1, True, "zero"), (1, s.L, True, "zero"), (1, 0x7fffffff, True, "zero")):
        for b in (0, 6):
            lens, counts = s.dev["before"].clone(), s.dev["new"].clone()
            counts[b] = new
            if before is not None:
                lens[b] = before
            st.zero_()
            out = torch.full(s.q.shape, 7.0, dtype=torch.float16, device="cuda")
            K.kvq_prefix_attn(s.prefix, s.tail, s.plan, s.dev["q"], lens, s.P, s.L, new_lens=counts, out=out,
                              dev_status=st, tail_splits=tail_splits)
            o = out.cpu().numpy()
            what = (new, before, b)
            assert int(st.item()) == (K.KVQ_FLAG_SEQ_LEN if flagged else 0), what
            assert (o[b] == (7.0 if row == "left" else 0.0)).all(), what
            s.check(o, only=[x for x in range(s.B) if x != b])


def test_a_workspace_over_another_array_is_refused():
    """The workspace shares no byte with q, the lengths, the plan or out: refused
    before anything is launched."""
    import torch
    s = _batch("int4", "int4", 64, 1, 2, 1, [50, 20], 6, none=False)
    K = s.K
    n = K.kvq_prefix_attn_workspace_size(s.prefix.desc, s.tail.desc, s.N, s.B, 1, 2, s.P, s.L)
    size = s.q.size * 2
    room = torch.full((n + 4096,), 7, dtype=torch.uint8, device="cuda")
    ws = room[2048:2048 + n]
    for at in (0, 2048 - size + 16, 2048, 2048 + n - 16):
        if at % 16:
            at -= at % 16
        over = room[at:at + size]
        for name in ("q", "out"):
            part = over.view(torch.float16).view(s.q.shape)
            args = dict(q=s.dev["q"], out=None)
            args[name] = part
            clash = at + size > 2048
            try:
                K.kvq_prefix_attn(s.prefix, s.tail, s.plan, args["q"], s.dev["before"], s.P, s.L, out=args["out"], workspace=ws)
                assert not clash
            except K.KVQError as e:
                assert clash and e.status == K.KVQ_ERR_INVALID_ARG
    lens = room[2048 + n - 32:2048 + n - 32 + 4 * s.B].view(torch.int32)
    for kw in (dict(new_lens=lens), dict(before=lens)):
        with pytest.raises(K.KVQError) as e:
            K.kvq_prefix_attn(s.prefix, s.tail, s.plan, s.dev["q"], kw.get("before", s.dev["before"]), s.P, s.L,
                              new_lens=kw.get("new_lens"), workspace=ws)
        assert e.value.status == K.KVQ_ERR_INVALID_ARG


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("fmt,T", [("int4", 1), ("fp16", 1), ("int8", 3), ("kch4", 2)])
def test_bounds_beyond_the_caches(fmt, T, splits):
    """Bounds of any size, for a program that knows none: what the caches hold is bound
    enough."""
    import torch
    s = _batch(fmt, fmt, 128, 1, 2, T, [150, 40], 5)
    for bound in (2 ** 31 - 1, 2 ** 31 - 128, 2 ** 30):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = s.K.kvq_prefix_attn(s.prefix, s.tail, s.plan, s.dev["q"], s.dev["before"], bound, bound,
                                  new_lens=s.dev["new"], prefix_splits=splits, tail_splits=splits, dev_status=st)
        s.check(out.cpu().numpy())
        assert int(st.item()) == 0
    size = s.K.kvq_prefix_attn_workspace_size
    sizes = (s.N, s.B, T, 2)
    most = [int(c.desc.capacity) + int(c.desc.sink_tokens) for c in (s.prefix, s.tail)]
    assert size(s.prefix.desc, s.tail.desc, *sizes, bound, bound, splits, splits) == \
        size(s.prefix.desc, s.tail.desc, *sizes, *most, splits, splits)

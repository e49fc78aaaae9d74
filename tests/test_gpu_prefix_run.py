"""The operators together, as a program uses them: a video's tokens go into a
paged cache by (time, height, width), questions fork it, the pool's table tells
the shared prefix, and decode steps attend over it once for all of them.  Every
step equals attention over each sequence's whole context."""
import numpy as np
import pytest

from oracle import prompt_oracle as P
from tests._prompt import expected_rows, extend_bound
from tests._prefix import decode_extra

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,bits,g", [("int4", 4, 32), ("int8", 8, 64), ("fp16", 16, 0)])
def test_questions_about_one_video(fmt, bits, g):
    import torch
    import quantized_kv_decode_gb300 as K
    Hkv, G, D, page, B, layers = 2, 4, 64, 16, 6, 2
    pages, M = 64, 16
    gen = torch.Generator(device="cuda").manual_seed(bits)
    rand = lambda *s: torch.randn(s, generator=gen, dtype=torch.float16, device="cuda")  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    st = i32([0])
    axes = K.make_rope_axes((8, 12, 12), cycled=True)
    pool = K.PagePool.allocate(pages, page, B, M)
    desc = K.make_desc(bits, g, Hkv, D, K.KVQ_PAGED, page, pages, M)
    caches = [K.KVCache.allocate(desc, B, "cuda", pool.block_table) for _ in range(layers)]
    for c in caches:
        c.block_table = pool.block_table  # one table for all layers
    hist = [[[] for _ in range(B)] for _ in range(layers)]  # rotated k and v of every sequence

    def append(T, new, before, pos, granted):
        qs = []
        for layer, c in enumerate(caches):
            k, v, q = rand(B, T, Hkv, D), rand(B, T, Hkv, D), rand(B, T, Hkv * G, D)
            qr, kr = K.kvq_rope_axes_apply(axes, pos, q, k)
            got = K.kvq_rope_axes_append(c, axes, pos, k, v, before, q=q, new_lens=granted, dev_status=st)
            for b in range(B):
                n = new[b]
                assert torch.equal(got[b, :n], qr[b, :n])
                hist[layer][b].append((kr[b, :n].cpu().numpy(), v[b, :n].cpu().numpy()))
            qs.append(got)
        return qs

    def reserve(before, new, most):
        src, dst, granted = i32([-1] * B), i32([-1] * B), i32([0] * B)
        K.kvq_pages_reserve(pool, before, i32(new), src, dst, granted, max_new=most, dev_status=st)
        K.kvq_pages_copy(caches, src, dst, dev_status=st)
        return granted

    # sequence 0: 5 frames of 4 x 5 patches, then the title's 7 tokens; 5: another text
    T, lens = 107, [107, 0, 0, 0, 0, 9]
    cell = np.arange(T)
    pos = np.where((cell < 100)[:, None], np.stack((cell // 20, cell // 5 % 4, cell % 5), -1), cell[:, None] - 95)
    pos = i32(np.broadcast_to(pos, (B, T, 3)).copy())
    before = i32([0] * B)
    append(T, lens, before, pos, reserve(before, lens, T))
    # four questions on the video
    K.kvq_pages_reorder(pool, i32([0, 0, 0, 0, -1, 5]), i32([107, 107, 107, 107, 0, 9]), dev_status=st)
    for layer in range(layers):
        for b in (1, 2, 3):
            hist[layer][b] = list(hist[layer][0])
    lens = [107, 107, 107, 107, 0, 9]
    new = [3, 1, 5, 2, 4, 1]  # (4: a text of its own from here on)
    N = 2
    of, plens, ptab = i32([0] * B), i32([0] * N), torch.zeros((N, M), dtype=torch.int32, device="cuda")
    ttab, tlens = torch.zeros_like(pool.block_table), i32([0] * B)
    plan = None
    for step in range(4):
        most = max(new)
        before = i32(lens)
        at = (before[:, None] + torch.arange(most, device="cuda")).int()[..., None].expand(-1, -1, 3).contiguous()
        granted = reserve(before, new, most)
        qs = append(most, new, before, at, granted)
        K.kvq_prefix_find(pool, before, of, plens, ptab, ttab, tlens, min_tokens=32, dev_status=st)
        plan = K.kvq_prefix_plan(of, plens, plan=plan, dev_status=st)
        assert of.tolist() == [0, 0, 0, 0, -1, -1] and plens.tolist() == [96, 0]
        assert tlens.tolist() == [n - 96 if b < 4 else n for b, n in enumerate(lens)]
        for layer, c in enumerate(caches):
            out = K.kvq_prefix_attn(c.with_table(ptab), c.with_table(ttab), plan, qs[layer], tlens, 112, 64,
                                    new_lens=granted, dev_status=st).cpu().numpy()
            whole = K.kvq_extend_attn(c, qs[layer], before, 160, new_lens=granted, dev_status=st).cpu().numpy()
            for b in range(B):
                n = new[b]
                k, v = (expected_rows(fmt, np.concatenate([x[i] for x in hist[layer][b]])).transpose(1, 0, 2)
                        for i in (0, 1))
                q = qs[layer][b, :n].cpu().numpy().astype(np.float64)
                want, mass = P.extend_attention(q, k, v, lens[b], D ** -0.5)
                bound = extend_bound(q, k, mass, want, D ** -0.5)
                assert (np.abs(whole[b, :n] - want) <= bound).all()
                if most == 1:
                    bound = bound + decode_extra(q, k, mass, D ** -0.5, bits)
                assert (np.abs(out[b, :n] - want) <= bound).all()
                assert not out[b, n:].any()
        lens = [a + b for a, b in zip(lens, new)]
        new = [1] * B
    assert int(st.item()) == 0

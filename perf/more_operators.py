"""Measured cases of many questions about one long context.

Three groups of operators, as a program that serves images, video and long
documents over a low-bit KV cache uses them: rotary positions with several axes
(time, height, width), applied to q and k and on the way into the cache
(kvq_rope_axes_apply, kvq_rope_axes_append); the prefixes that sequences of a
page pool share, found in its block table (kvq_prefix_find); and attention that
reads a shared prefix once for all sequences on it (kvq_prefix_attn), of one new
token per sequence or of several.

`run` computes each one in plain torch, or through the package where `own` is
true.  Caches are fp16, or asymmetric INT4 / INT8 codes with one fp16 scale and
zero-point per group of channels, dense or paged.
"""
import math
import random

import torch

own = False

F16 = torch.float16


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # positions with three axes: a decode step of a small batch (latency),
        # and prompts of video frames and text, the axes taking turns
        {"name": "axes_step", "op": "axes", "B": 8, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "pairs": "16,24,24",
         "cycled": False, "ladder": False, "inter": False, "base": 1e6, "ragged": 0},
        {"name": "axes_video", "op": "axes", "B": 4, "T": 8191, "Hq": 32, "Hkv": 8, "D": 128, "pairs": "24,20,20",
         "cycled": True, "ladder": False, "inter": False, "base": 5e6, "ragged": 1},
        # the same into the cache and read back: the step of a paged small-model
        # batch over images (two axes, a ladder each), and a chunk of long prompts
        {"name": "axes_append_step", "op": "axes_append", "B": 256, "T": 1, "Hq": 14, "Hkv": 2, "D": 64,
         "pairs": "16,16", "cycled": False, "ladder": True, "inter": True, "base": 1e4, "ragged": 2, "far": 4000,
         "bits": 4, "g": 32, "page": 16},
        {"name": "axes_append_chunk", "op": "axes_append", "B": 2, "T": 4095, "Hq": 32, "Hkv": 8, "D": 128,
         "pairs": "16,24,24", "cycled": False, "ladder": False, "inter": False, "base": 1e6, "ragged": 3, "far": 28000,
         "bits": 8, "g": 64, "page": 0},
        # which sequences share pages: a few samples of one prompt, and a large
        # batch over many documents, some of it on a common system prompt only
        {"name": "find_samples", "op": "find", "B": 8, "page": 16, "len": 1000, "docs": 1, "system": 5, "most": 1,
         "min": 1, "ragged": 4},
        {"name": "find_documents", "op": "find", "B": 2048, "page": 16, "len": 16000, "docs": 60, "system": 12,
         "most": 64, "min": 256, "ragged": 5},
        # decode: a few samples of a short prompt (latency); parallel samples of a
        # 7B-class model (one query head per KV head) on a dense prefix; questions
        # about one long document; a small-model batch on several system prompts,
        # some sequences without one
        {"name": "samples", "op": "shared", "B": 4, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "bits": 8, "g": 32,
         "page": 16, "half": False, "N": 1, "prefix": 1000, "tail": 100, "alone": 0, "ragged": 6},
        {"name": "samples_7b", "op": "shared", "B": 32, "T": 1, "Hq": 32, "Hkv": 32, "D": 128, "bits": 4, "g": 32,
         "page": 0, "half": False, "N": 1, "prefix": 4096, "tail": 512, "alone": 0, "ragged": 7},
        {"name": "questions", "op": "shared", "B": 64, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "bits": 4, "g": 32,
         "page": 64, "half": False, "N": 1, "prefix": 32768, "tail": 500, "alone": 0, "ragged": 8},
        {"name": "system_prompts", "op": "shared", "B": 256, "T": 1, "Hq": 14, "Hkv": 2, "D": 64, "bits": 4, "g": 32,
         "page": 16, "half": False, "N": 12, "prefix": 3000, "tail": 700, "alone": 20, "ragged": 9},
        # drafted tokens checked behind a shared INT8 prefix, the tails in fp16
        {"name": "drafts", "op": "shared", "B": 24, "T": 5, "Hq": 32, "Hkv": 8, "D": 128, "bits": 8, "g": 64,
         "page": 0, "half": True, "N": 2, "prefix": 12001, "tail": 900, "alone": 1, "ragged": 10},
        # whole questions (prompts behind the shared part) at once, fp16 pages
        {"name": "suffixes", "op": "shared", "B": 24, "T": 200, "Hq": 32, "Hkv": 8, "D": 128, "bits": 16, "g": 0,
         "page": 16, "half": False, "N": 3, "prefix": 6000, "tail": 0, "alone": 0, "ragged": 11},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["axes", "axes_append", "find", "shared", "shared", "shared", "shared"])
    c = {"op": op, "ragged": rng.choice([0, rng.randrange(1, 1 << 20)])}
    if op == "find":
        B, length, page = _spread(rng, 1, 2048), _spread(rng, 1, 16000), rng.choice([16, 32, 64])
        docs = _spread(rng, 1, 100)
        c.update(B=B, page=page, len=length, docs=docs, system=rng.randrange(0, 20), most=_spread(rng, 1, 100),
                 min=rng.choice([0, 1, _spread(rng, 1, length)]))
        return c
    D = rng.choice([64, 128])
    Hkv, G = rng.choice([(1, 8), (2, 7), (4, 4), (8, 4), (8, 1), (3, 5), (2, 16)])
    bits = rng.choice([4, 4, 8, 16])
    c.update(Hkv=Hkv, Hq=Hkv * G, D=D)
    fmt = {"bits": bits, "g": 0 if bits == 16 else rng.choice([16, 32, 64]), "page": rng.choice([0, 16, 64])}
    if op in ("axes", "axes_append"):
        tokens = _spread(rng, 1, 16000)
        B = _spread(rng, 1, min(tokens, 256))
        half = rng.choice([D, D, D // 2]) // 2
        axes = rng.choice([2, 3, 3, 4])
        cuts = sorted(rng.sample(range(1, half), axes - 1))
        pairs = [b - a for a, b in zip([0] + cuts, cuts + [half])]
        c.update(B=B, T=max(1, tokens // B), pairs=",".join(map(str, pairs)), cycled=rng.random() < 0.5,
                 ladder=rng.random() < 0.3, inter=rng.random() < 0.5, base=rng.choice([1e4, 5e5, 1e6]))
        if op == "axes_append":
            c.update(fmt)
            c["far"] = max(1, min(_spread(rng, 1, 20000), 2_000_000 // (B * Hkv)))
        return c
    B, T, prefix, tail = _spread(rng, 1, 256), _spread(rng, 1, 200), _spread(rng, 1, 32768), _spread(rng, 1, 2000)
    if rng.random() < 0.5:
        T = 1
    while B * T * Hkv * G * (prefix + tail + T) * D > 4e10 or B * (tail + T) * Hkv * D > 4e8:
        if T > 8:
            T = T * 2 // 3
        elif B > 8:
            B = B * 2 // 3
        else:
            prefix, tail = prefix * 2 // 3, tail * 2 // 3
    N = _spread(rng, 1, min(B, 16))
    if prefix * N * Hkv * D > 2e8:
        N = 1
    c.update(fmt, B=B, T=T, N=N, prefix=max(prefix, 1), tail=rng.choice([tail, tail, 0]),
             alone=rng.choice([0, 0, B // 5]), half=fmt["page"] == 0 and bits != 16 and rng.random() < 0.4)
    return c


def _lengths(case, count, most, salt, least=1):
    """`count` lengths up to `most`: all equal, or spread where the case is ragged."""
    if not case["ragged"]:
        return [most] * count
    r = random.Random(case["ragged"] * 16 + salt)
    return [r.randint(min(least, most), most) for _ in range(count)]


def _row_bytes(D, bits, g):
    """Bytes of one cached K or V vector, its scales and zero-points included."""
    return 2 * D if bits == 16 else D * bits // 8 + 4 * (D // g)


def _formats(case):
    """(bits, group) of the prefixes' cache and of the tails'."""
    own_fmt = (case["bits"], case["g"])
    return own_fmt, (16, 0) if case["half"] else own_fmt


def _members(case):
    """The prefix of every sequence, -1 for those without."""
    r = random.Random(case["ragged"] * 16 + 9)
    of = [-1] * case["alone"] + [b % case["N"] for b in range(case["B"] - case["alone"])]
    r.shuffle(of)
    return of


def _shared_lens(case):
    """Tokens of each prefix (whole pages where paged), and of each tail, before and new."""
    prefix = _lengths(case, case["N"], case["prefix"], 3, least=max(case["prefix"] // 2, 1))
    if case["page"]:
        prefix = [max(p // case["page"], 1) * case["page"] for p in prefix]
    return prefix, _lengths(case, case["B"], case["tail"], 2, least=0), _lengths(case, case["B"], case["T"], 1)


def _axes_of(case):
    return [int(p) for p in case["pairs"].split(",")]


def _blocks(case):
    return -(-case["len"] // case["page"]) + case["system"]


def work(case):
    op = case["op"]
    if op == "find":
        table = 4 * case["B"] * _blocks(case)
        return {"bytes": 2 * table + 4 * case["most"] * _blocks(case) + 16 * case["B"], "flops": 0}
    D, Hkv, Hq = case["D"], case["Hkv"], case["Hq"]
    if op in ("axes", "axes_append"):
        tokens, rd = sum(_lengths(case, case["B"], case["T"], 1)), 2 * sum(_axes_of(case))
        at = 4 * tokens * len(_axes_of(case))
        q = tokens * Hq * D * 2 * 2
        if op == "axes":
            return {"bytes": at + q + tokens * Hkv * D * 2 * 2, "flops": 3 * tokens * (Hq + Hkv) * rd}
        # in, cache written and read, rows out
        kv = tokens * Hkv * 2 * (2 * D + 2 * _row_bytes(D, case["bits"], case["g"]) + 2 * D)
        return {"bytes": at + q + kv, "flops": tokens * (3 * (Hq + Hkv) * rd + 2 * Hkv * D * 6)}
    prefix, before, new = _shared_lens(case)
    (pb, pg), (tb, tg) = _formats(case)
    of = _members(case)
    pairs = sum(n * ((prefix[p] if p >= 0 else 0) + b) + n * (n + 1) // 2 for p, b, n in zip(of, before, new))
    cached = 2 * Hkv * (sum(prefix[p] for p in set(of) if p >= 0) * _row_bytes(D, pb, pg)
                        + sum(b + n for b, n in zip(before, new)) * _row_bytes(D, tb, tg))
    return {"bytes": cached + 4 * sum(new) * Hq * D, "flops": 4 * Hq * D * pairs}


# -------------------------------------------------- rotary positions, by axis

def _axis_of_pairs(case):
    """(axis, pair within the axis) of every channel pair."""
    pairs = _axes_of(case)
    if not case["cycled"]:
        return [(a, j) for a, n in enumerate(pairs) for j in range(n)]
    left, out = list(pairs), []
    while any(left):  # the axes take turns while they have pairs left
        for a in range(len(pairs)):
            if left[a]:
                out.append((a, pairs[a] - left[a]))
                left[a] -= 1
    return out


def _turn_rates(case, device):
    """Radians a position of every pair, in 64 bits."""
    half = sum(_axes_of(case))
    i = torch.arange(half, dtype=torch.float64, device=device)
    if not case["ladder"]:
        return case["base"] ** (-i / half)
    at = _axis_of_pairs(case)
    j = torch.tensor([p for _, p in at], dtype=torch.float64, device=device)
    n = torch.tensor([_axes_of(case)[a] for a, _ in at], dtype=torch.float64, device=device)
    return case["base"] ** (-j / n)


def _grid_positions(case, gen, device):
    """[B][T][axes]: frames of patches (time, then rows and columns), then text, on which the axes agree."""
    B, T, A = case["B"], case["T"], len(_axes_of(case))
    side = max(1, min(32, int(math.sqrt(T))))
    t = torch.arange(T, device=device)
    first = torch.randint(0, 20000, (B, 1), generator=gen, device=device)
    media = (t < T - T // 5)[None, :]
    text = first + t
    cell = (torch.div(t, side * side, rounding_mode="floor"), torch.div(t, side, rounding_mode="floor") % side, t % side,
            t % 7)
    cols = [torch.where(media, first + cell[(a if A > 2 else a + 1)], text) for a in range(A)]
    return torch.stack(cols, -1).int().contiguous()


def _rotate(x, angle, case):
    """x [B][T][H][D] turned by angle [B][T][pairs]; computed in x's type."""
    half = angle.shape[-1]
    c, s = torch.cos(angle).to(x.dtype).unsqueeze(2), torch.sin(angle).to(x.dtype).unsqueeze(2)
    if case["inter"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((r, x[..., 2 * half:]), -1)


def _angles(st):
    axis = torch.tensor([a for a, _ in _axis_of_pairs(st["case"])], device=st["at"].device)
    return st["at"].double()[..., axis] * _turn_rates(st["case"], st["at"].device)


def _live(st):
    """Which of the padded rows [B][T] a sequence has."""
    return torch.arange(st["case"]["T"], device=st["new"].device) < st["new"][:, None]


# ------------------------------------------------------------- the cache

def _quantize(x, bits, g):
    """x [..., D] fp16 -> codes, scale, zero, as the cache defines them."""
    v = x.float().unflatten(-1, (-1, g))
    mn, mx = v.amin(-1), v.amax(-1)
    top = 2 ** bits - 1
    span = mx.double() - mn.double()
    s = (span / top).to(F16)
    up = (s.view(torch.int16) + 1).view(F16)
    s = torch.where(s.double() * top < span, up, s)          # the smallest fp16 that is not below
    s = torch.where(span == 0, torch.where(mn == 0, torch.ones_like(mn), mn.abs()).to(F16), s)
    sf = s.float()
    z = torch.round(-mn / sf).clamp(-2048, 2048)
    q = (torch.round(v / sf[..., None]) + z[..., None]).clamp(0, top)
    return q.flatten(-2).to(torch.uint8), s, (z + 0.0).to(F16)


def _pack(q, bits):
    return q if bits == 8 else (q[..., 0::2] | (q[..., 1::2] << 4))


def _dequantize(codes, scale, zero, bits, g, dtype=torch.float32):
    if bits == 16:
        return codes.view(F16).to(dtype)
    q = codes if bits == 8 else torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    q = q.to(dtype).unflatten(-1, (-1, g))
    return ((q - zero.to(dtype)[..., None]) * scale.to(dtype)[..., None]).flatten(-2)


def _empty_cache(D, bits, g, lead, device):
    cache = {"k_codes": torch.zeros(lead + (D * bits // 8,), dtype=torch.uint8, device=device)}
    cache["v_codes"] = torch.zeros_like(cache["k_codes"])
    for n in ("k_scale", "k_zero", "v_scale", "v_zero"):
        cache[n] = None if bits == 16 else torch.zeros(lead + (D // g,), dtype=F16, device=device)
    return cache


def _filled_cache(D, bits, g, lead, gen, device):
    """Random K and V, with the persistent large channels of keys."""
    cache = _empty_cache(D, bits, g, lead, device)
    for which in "kv":
        x = torch.randn(lead + (D,), generator=gen, device=device, dtype=F16)
        if which == "k":
            x[..., torch.randperm(D, generator=gen, device=device)[:4]] *= 10
        if bits == 16:
            cache[which + "_codes"] = x.view(torch.uint8)
            continue
        q, s, z = _quantize(x, bits, g)
        cache[which + "_codes"] = _pack(q, bits).contiguous()
        cache[which + "_scale"], cache[which + "_zero"] = s, z
    return cache


def _tables(blocks, M, pool, gen, device):
    """Rows of `blocks` pages each, scattered over the pool; -1 behind."""
    perm = torch.randperm(pool, generator=gen, device=device).int()
    need = torch.tensor(blocks, device=device)
    at = torch.cumsum(need, 0) - need
    j = torch.arange(M, device=device)
    return torch.where(j < need[:, None], perm[(at[:, None] + j).clamp(max=pool - 1)], -1).int().contiguous()


def _gather(cache, name, table, page, L):
    """[rows][Hkv][L][...] of one cache array."""
    t = cache[name]
    if t is None:
        return None
    if table is None:
        return t[:, :, :L]
    pos = torch.arange(L, device=table.device)
    return t[table[:, pos // page].long().clamp(min=0), :, pos % page].permute(0, 2, 1, 3)


def _kv(st, side, L, dtype):
    """K and V of the prefixes or the tails, [rows][Hkv][L][D]."""
    bits, g = _formats(st["case"])[side == "tail"]
    return (_dequantize(*(_gather(st[side], n + a, st[side + "_table"], st["case"]["page"], L)
                          for a in ("_codes", "_scale", "_zero")), bits, g, dtype) for n in "kv")


def _handle(case, fmt, cache, table, batch):
    """The package's cache over these arrays."""
    import quantized_kv_decode_gb300 as K
    lead = cache["k_codes"].shape
    if table is not None:
        desc = K.make_desc(fmt[0], fmt[1], case["Hkv"], case["D"], K.KVQ_PAGED, case["page"], lead[0], table.shape[1])
    else:
        desc = K.make_desc(fmt[0], fmt[1], case["Hkv"], case["D"], K.KVQ_DENSE, lead[2])
    return K.KVCache(desc, batch, block_table=table, **cache)


# ----------------------------------------------------------------- prepare

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": case}
    if case["op"] in ("axes", "axes_append"):
        _prepare_axes(st, gen, dev)
    elif case["op"] == "find":
        _prepare_find(st, seed, gen, dev)
    else:
        _prepare_shared(st, gen, dev)
    if own:
        _prepare_own(st)
    return st


def _prepare_axes(st, gen, dev):
    case = st["case"]
    B, T, Hkv, D = case["B"], case["T"], case["Hkv"], case["D"]
    st["at"] = _grid_positions(case, gen, dev)
    st["new"] = torch.tensor(_lengths(case, B, T, 1), dtype=torch.int32, device=dev)
    st["q"] = torch.randn((B, T, case["Hq"], D), generator=gen, device=dev, dtype=F16)
    st["k"] = torch.randn((B, T, Hkv, D), generator=gen, device=dev, dtype=F16)
    st["q_out"], st["k_out"] = torch.zeros_like(st["q"]), torch.zeros_like(st["k"])
    if case["op"] == "axes_append":
        st["before"] = torch.randint(0, case["far"], (B,), generator=gen, device=dev, dtype=torch.int32)
        st["v"] = torch.randn((B, T, Hkv, D), generator=gen, device=dev, dtype=F16)
        st["v_out"] = torch.zeros_like(st["v"])
        cap = case["far"] + T
        if case["page"]:
            M = -(-cap // case["page"])
            st["table"] = _tables([M] * B, M, B * M + 5, gen, dev)
            lead = (B * M + 5, Hkv, case["page"])
        else:
            st["table"], lead = None, (B, Hkv, cap)
        st["cache"] = _empty_cache(D, case["bits"], case["g"], lead, dev)


def _prepare_find(st, seed, gen, dev):
    """The table of a pool whose sequences continue documents: a common system
    prompt's pages first, then a part of the document's, then their own."""
    case = st["case"]
    r = random.Random(seed * 1000 + 1)
    B, S, M, sys_blocks = case["B"], case["page"], _blocks(case), case["system"]
    body = M - sys_blocks
    lens, doc, cut = [], [], []
    for _ in range(B):
        lens.append(r.randint(1, case["len"]) + sys_blocks * S if case["ragged"] else M * S)
        doc.append(r.randrange(case["docs"] + 1))  # the last: only the system prompt
        cut.append(r.choice([0, body // 2, body, r.randint(0, body)]))
    docs = torch.arange(case["docs"] + 1, device=dev)[:, None] * body + torch.arange(body, device=dev) + sys_blocks
    pages = sys_blocks + (case["docs"] + 1) * body
    st["pages"] = pages + B * body
    j = torch.arange(body, device=dev)
    doc_t, cut_t = torch.tensor(doc, device=dev), torch.tensor(cut, device=dev)
    cut_t = torch.where(doc_t == case["docs"], 0, cut_t)
    mine = pages + torch.arange(B, device=dev)[:, None] * body + j
    rows = torch.where(j < cut_t[:, None], docs[doc_t], mine)
    rows = torch.cat((torch.arange(sys_blocks, device=dev).expand(B, -1), rows), 1)
    held = -(-torch.tensor(lens, device=dev) // S)
    names = torch.randperm(st["pages"], generator=gen, device=dev)  # pages lie scattered over the pool
    st["table"] = torch.where(torch.arange(M, device=dev) < held[:, None], names[rows], -1).int().contiguous()
    st["ref"] = torch.bincount(st["table"].flatten().long() + 1, minlength=st["pages"] + 1)[1:].int()
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["of"] = torch.empty(B, dtype=torch.int32, device=dev)
    st["prefix_lens"] = torch.empty(case["most"], dtype=torch.int32, device=dev)
    st["prefix_table"] = torch.empty((case["most"], M), dtype=torch.int32, device=dev)
    st["tail_table"], st["tail_lens"] = torch.empty_like(st["table"]), torch.empty_like(st["of"])


def _prepare_shared(st, gen, dev):
    case = st["case"]
    B, T, N, Hkv, D, S = case["B"], case["T"], case["N"], case["Hkv"], case["D"], case["page"]
    prefix, before, new = _shared_lens(case)
    st["of_list"] = _members(case)
    st["prefix_list"] = prefix
    st["of"] = torch.tensor(st["of_list"], dtype=torch.int32, device=dev)
    st["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device=dev)
    st["before"] = torch.tensor(before, dtype=torch.int32, device=dev)
    st["new"] = torch.tensor(new, dtype=torch.int32, device=dev)
    st["P"], st["L"] = max(prefix), max(b + n for b, n in zip(before, new))
    fmt = _formats(case)
    if S:  # one pool: the prefixes' pages and the tails'
        blocks = [-(-n // S) for n in prefix] + [-(-(b + n) // S) for b, n in zip(before, new)]
        table = _tables(blocks, max(blocks), sum(blocks) + 3, gen, dev)
        st["prefix_table"], st["tail_table"] = table[:N].clone(), table[N:].clone()  # (each on a 16-byte boundary)
        st["prefix"] = st["tail"] = _filled_cache(D, *fmt[0], (sum(blocks) + 3, Hkv, S), gen, dev)
    else:
        st["prefix_table"] = st["tail_table"] = None
        st["prefix"] = _filled_cache(D, *fmt[0], (N, Hkv, st["P"]), gen, dev)
        st["tail"] = _filled_cache(D, *fmt[1], (B, Hkv, st["L"]), gen, dev)
    st["q"] = torch.randn((B, T, case["Hq"], D), generator=gen, device=dev, dtype=F16)
    st["out"] = torch.zeros_like(st["q"])


def _prepare_own(st):
    """The handles, plans and workspaces that a program keeps."""
    import quantized_kv_decode_gb300 as K
    case = st["case"]
    if case["op"] in ("axes", "axes_append"):
        st["rope"] = K.make_rope_axes(_axes_of(case), cycled=case["cycled"], own_ladders=case["ladder"],
                                      base=case["base"], interleaved=case["inter"])
    if case["op"] == "axes_append":
        st["kv"] = _handle(case, (case["bits"], case["g"]), st["cache"], st["table"], case["B"])
        st["total"] = st["before"] + st["new"]
    if case["op"] == "find":
        st["pool"] = K.PagePool(st["ref"], st["table"], case["page"])
        st["ws"] = torch.empty(K.kvq_prefix_find_workspace_size(st["pool"]), dtype=torch.uint8, device="cuda")
    if case["op"] == "shared":
        fmt = _formats(case)
        st["prefix_kv"] = _handle(case, fmt[0], st["prefix"], st["prefix_table"], case["N"])
        st["tail_kv"] = _handle(case, fmt[1], st["tail"], st["tail_table"], case["B"])
        # which sequences are on which prefix: the same for every layer of a step
        st["plan"] = K.kvq_prefix_plan(st["of"], st["prefix_lens"])
        n = K.kvq_prefix_attn_workspace_size(st["prefix_kv"].desc, st["tail_kv"].desc, case["N"], case["B"], case["T"],
                                             case["Hq"], st["P"], st["L"])
        st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------------- run

def run(st):
    op = st["case"]["op"]
    if own:
        return {"axes": _own_axes, "axes_append": _own_append, "find": _own_find, "shared": _own_shared}[op](st)
    return {"axes": _plain_axes, "axes_append": _plain_append, "find": _plain_find, "shared": _plain_shared}[op](st)


def _own_axes(st):
    import quantized_kv_decode_gb300 as K
    K.kvq_rope_axes_apply(st["rope"], st["at"], st["q"], st["k"], new_lens=st["new"], q_out=st["q_out"],
                          k_out=st["k_out"])
    return st["q_out"], st["k_out"]


def _own_append(st):
    import quantized_kv_decode_gb300 as K
    K.kvq_rope_axes_append(st["kv"], st["rope"], st["at"], st["k"], st["v"], st["before"], q=st["q"],
                           q_out=st["q_out"], new_lens=st["new"])
    K.kvq_cache_read(st["kv"], st["total"], st["before"], st["k_out"], st["v_out"])
    return st["q_out"], st["k_out"], st["v_out"]


def _own_find(st):
    import quantized_kv_decode_gb300 as K
    K.kvq_prefix_find(st["pool"], st["lens"], st["of"], st["prefix_lens"], st["prefix_table"], st["tail_table"],
                      st["tail_lens"], min_tokens=st["case"]["min"], workspace=st["ws"])
    return st["of"], st["prefix_lens"], st["prefix_table"], st["tail_table"], st["tail_lens"]


def _own_shared(st):
    import quantized_kv_decode_gb300 as K
    K.kvq_prefix_attn(st["prefix_kv"], st["tail_kv"], st["plan"], st["q"], st["before"], st["P"], st["L"],
                      new_lens=st["new"], out=st["out"], workspace=st["ws"])
    return st["out"]


def _plain_axes(st):
    live, angle = _live(st)[..., None, None], _angles(st)
    return tuple(torch.where(live, _rotate(st[n].float(), angle, st["case"]).to(F16), st[n + "_out"]) for n in "qk")


def _plain_append(st):
    case, live = st["case"], _live(st)
    angle = _angles(st)
    q = torch.where(live[..., None, None], _rotate(st["q"].float(), angle, case).to(F16), st["q_out"])
    # keys in 64 bits: their codes change where a value lies next to a border
    rows = {"k": _rotate(st["k"].double(), angle, case).to(F16), "v": st["v"]}
    pos = st["before"].long()[:, None] + torch.arange(case["T"], device=live.device)
    b = torch.arange(case["B"], device=live.device)[:, None].expand_as(pos)
    if case["page"]:
        first, off = st["table"].gather(1, (pos // case["page"])).long(), pos % case["page"]
    else:
        first, off = b, pos
    first, off = torch.where(live, first, first[:, :1]), torch.where(live, off, off[:, :1])
    outs = []
    for n in "kv":
        x = torch.where(live[..., None, None], rows[n], rows[n][:, :1])  # padding rewrites a row's own value
        if case["bits"] == 16:
            st["cache"][n + "_codes"][first, :, off] = x.contiguous().view(torch.uint8)
        else:
            c, s, z = _quantize(x, case["bits"], case["g"])
            st["cache"][n + "_codes"][first, :, off] = _pack(c, case["bits"])
            st["cache"][n + "_scale"][first, :, off] = s
            st["cache"][n + "_zero"][first, :, off] = z
        got = [None if st["cache"][n + a] is None else st["cache"][n + a][first, :, off].contiguous()
               for a in ("_codes", "_scale", "_zero")]
        hat = _dequantize(*got, case["bits"], case["g"]).to(F16)
        outs.append(torch.where(live[..., None, None], hat, st[n + "_out"]))
    return q, outs[0], outs[1]


def _plain_find(st):
    case, table, lens = st["case"], st["table"], st["lens"]
    B, M = table.shape
    S, most = case["page"], case["most"]
    whole = (lens // S).clamp(max=M)
    k = max(1, -(-case["min"] // S))
    idx = torch.arange(B, device=table.device)
    none = torch.full_like(idx, -1)
    if k > M:
        of, value, leader, run = none, torch.zeros_like(idx), idx, torch.zeros_like(idx)
    else:
        key = torch.where(whole >= k, table[:, k - 1].long(), -1)
        same = (key[:, None] == key[None, :]) & (key >= 0)[:, None]
        leader = torch.where(same, idx[None, :], B).amin(1)
        lead = leader.clamp(max=B - 1)
        j = torch.arange(M, device=table.device)
        equal = (table == table[lead]) & (table >= 0) & (j < torch.minimum(whole, whole[lead])[:, None])
        run = equal.int().cumprod(1).sum(1)
        member = (key >= 0) & (run >= k)
        # what a prefix of this run saves: (members with at least it, but one) blocks of it
        pair = member[:, None] & member[None, :] & (leader[:, None] == leader[None, :]) & (run[None, :] >= run[:, None])
        saved = torch.where(member, (pair.sum(1) - 1) * run, 0)
        value = torch.zeros(B, dtype=torch.int64, device=table.device).scatter_reduce(
            0, lead, torch.where(saved > 0, saved * (M + 1) + run, 0), "amax")
        best = value % (M + 1)
        rank = torch.cumsum((value > 0).long(), 0) - 1
        kept = (value > 0) & (rank < most)
        of = torch.where(member & kept[lead] & (run >= best[lead]), rank[lead], -1)
    lens_n = torch.zeros(most, dtype=torch.int64, device=table.device)
    rows = torch.full((most, M), -1, dtype=torch.int32, device=table.device)
    shift = torch.zeros_like(idx)
    if k <= M:
        at = torch.nonzero(kept).flatten()
        lens_n[:len(at)] = best[at] * S
        rows[:len(at)] = torch.where(j < best[at][:, None], table[at], -1)
        shift = torch.where(of >= 0, best[lead], 0)
    j = torch.arange(M, device=table.device)
    src = j + shift[:, None]
    tail = torch.where(src < M, table.gather(1, src.clamp(max=M - 1)), -1)
    return of.int(), lens_n.int(), rows, tail, (lens - shift * S).int()


def _plain_shared(st):
    case = st["case"]
    B, T, Hq, D = st["q"].shape
    Hkv, L = case["Hkv"], st["L"]
    G = Hq // Hkv
    kp, vp = _kv(st, "prefix", st["P"], torch.float32)
    kt, vt = _kv(st, "tail", L, torch.float32)
    # tail position j is seen by new token t when j <= before + t
    seen = torch.arange(L, device=kt.device) <= (st["before"][:, None] + torch.arange(T, device=kt.device))[..., None]
    held = torch.arange(L, device=kt.device) < (st["before"] + st["new"])[:, None]
    vt = torch.where(held[:, None, :, None], vt, 0)
    q = st["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    s = torch.matmul(q, kt.transpose(-1, -2)).mul_(D ** -0.5).view(B, Hkv, G, T, L)
    s.masked_fill_(~(seen & held[:, None, :])[:, None, None], -math.inf)
    s = s.view(B, Hkv, G * T, L)
    out = torch.empty_like(q)
    for n in range(-1, case["N"]):
        who = [b for b in range(B) if st["of_list"][b] == n]
        if not who:
            continue
        who = torch.tensor(who, device=q.device)
        tail, top = s[who], s[who].amax(-1, keepdim=True)
        if n >= 0:
            P = st["prefix_list"][n]
            rows = q[who].transpose(0, 1).reshape(Hkv, -1, D)
            sp = torch.matmul(rows, kp[n, :, :P].transpose(-1, -2)).mul_(D ** -0.5)
            sp = sp.view(Hkv, len(who), G * T, P).transpose(0, 1)
            top = torch.maximum(top, sp.amax(-1, keepdim=True))
            sp = (sp - top).exp_()
        top = torch.where(top == -math.inf, 0, top)
        tail = (tail - top).exp_()
        o, total = torch.matmul(tail, vt[who]), tail.sum(-1, keepdim=True)
        if n >= 0:
            o += torch.matmul(sp.transpose(0, 1).reshape(Hkv, -1, P), vp[n, :, :P]).view(Hkv, -1, G * T, D).transpose(0, 1)
            total = total + sp.sum(-1, keepdim=True)
        out[who] = o / total
    out = out.view(B, Hkv, G, T, D).permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(F16)
    return torch.where(_live(st)[..., None, None], out, st["out"])


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """What run returns, from the definitions in 64 bits; None for whole numbers."""
    global own
    if case["op"] == "find":
        return None
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return _exact_shared(st) if case["op"] == "shared" else _exact_rows(st)


def _exact_turns(st):
    """exp(i position w) of every token and pair, pair by pair."""
    case = st["case"]
    pairs, half, turns = _axes_of(case), sum(_axes_of(case)), []
    used = [0] * len(pairs)
    axis = 0
    for i in range(half):
        if case["cycled"]:
            while used[axis] == pairs[axis]:
                axis = (axis + 1) % len(pairs)
        else:
            axis = next(a for a in range(len(pairs)) if i < sum(pairs[:a + 1]))
        power = used[axis] / pairs[axis] if case["ladder"] else i / half
        used[axis] += 1
        w = math.exp(-power * math.log(case["base"]))
        angle = st["at"][..., axis].double() * w
        turns.append(torch.polar(torch.ones_like(angle), angle))
        if case["cycled"]:
            axis = (axis + 1) % len(pairs)
    return torch.stack(turns, -1)[:, :, None]


def _exact_rows(st):
    """Each pair as a complex number times its turn; then the cache's grid."""
    case = st["case"]
    turn = _exact_turns(st)
    half = turn.shape[-1]
    padding = torch.arange(case["T"], device="cuda").expand(case["B"], -1) >= st["new"][:, None]

    def turned(x):
        y = x.double()
        even = slice(0, 2 * half, 2) if case["inter"] else slice(0, half)
        odd = slice(1, 2 * half, 2) if case["inter"] else slice(half, 2 * half)
        w = torch.complex(y[..., even].contiguous(), y[..., odd].contiguous()) * turn
        y[..., even], y[..., odd] = w.real, w.imag
        return y

    def placed(y):
        y[padding] = 0.0
        return y

    q = placed(turned(st["q"]))
    if case["op"] == "axes":
        return q, placed(turned(st["k"]))
    outs = []
    for x in (turned(st["k"]).to(F16), st["v"]):
        if case["bits"] == 16:
            outs.append(placed(x.double()))
            continue
        y = x.double().view(*x.shape[:-1], -1, case["g"])
        low, high = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        n = float(2 ** case["bits"] - 1)
        step = ((high - low) / n).to(F16).double()
        ulp = 2.0 ** (torch.floor(torch.log2(step.clamp(min=2.0 ** -14))) - 10)
        step = torch.where(step * n < high - low, step + ulp, step)  # the scale is rounded up
        step = torch.where(high == low, torch.where(low == 0, 1.0, low.abs()), step)
        zero = torch.round((-low).float() / step.float()).double().clamp(-2048, 2048)
        code = (torch.round(y.float() / step.float()).double() + zero).clamp(0, n)
        outs.append(placed(((code - zero) * step).view(x.shape)))
    return q, outs[0], outs[1]


def _exact_cached(st, side, n, row, length):
    """[Hkv][length][D] of K or V of one prefix or tail, in 64 bits."""
    case, D = st["case"], st["case"]["D"]
    bits, g = _formats(case)[1 if side == "tail" else 0]
    rows = []
    for a in ("_codes", "_scale", "_zero"):
        t = st[side][n + a]
        if t is None:
            rows.append(None)
        elif case["page"]:
            pages = st[side + "_table"][row, : -(-length // case["page"])].long()
            rows.append(t[pages].transpose(0, 1).flatten(1, 2)[:, :length])
        else:
            rows.append(t[row, :, :length])
    if bits == 16:
        return rows[0].contiguous().view(F16).double()
    c = rows[0].int()
    per = 8 // bits
    q = torch.empty((*c.shape[:2], D), dtype=torch.float64, device=c.device)
    for e in range(per):
        q[..., e::per] = ((c >> (e * bits)) % 2 ** bits).double()
    s, z = (r.double().repeat_interleave(g, -1) for r in rows[1:])
    return (q - z) * s


def _exact_shared(st):
    """Sequence by sequence: its prefix and its tail as one context."""
    case = st["case"]
    B, T, Hq, D = st["q"].shape
    G = Hq // case["Hkv"]
    if B * T * (st["P"] + st["L"]) * Hq * D > 2e12:  # over about 20 seconds in 64 bits
        return None
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    shared = {}
    for b in range(B):
        n, n0, new = int(st["of"][b]), int(st["before"][b]), int(st["new"][b])
        k, v = (_exact_cached(st, "tail", a, b, n0 + new) for a in "kv")
        P = 0
        if n >= 0:
            P = int(st["prefix_lens"][n])
            if n not in shared:
                shared[n] = [_exact_cached(st, "prefix", a, n, P) for a in "kv"]
            k, v = torch.cat((shared[n][0], k), 1), torch.cat((shared[n][1], v), 1)
        later = torch.arange(P + n0 + new, device="cuda") > torch.arange(P + n0, P + n0 + new, device="cuda")[:, None]
        q = st["q"][b, :new].double().view(new, case["Hkv"], G, D).permute(1, 2, 0, 3)
        s = torch.matmul(q, k[:, None].transpose(-1, -2)) / math.sqrt(D)
        s = torch.softmax(s.masked_fill(later, -math.inf), -1)
        out[b, :new] = torch.matmul(s, v[:, None]).permute(2, 0, 1, 3).reshape(new, Hq, D)
    return out

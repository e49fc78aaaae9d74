"""Measured cases of the prompt path over a low-bit KV cache.

Three groups of operators, as a serving program uses them around the decode
step: rotary positions applied to q and k and quantized into the cache
(kvq_rope_apply, kvq_rope_append, read back by kvq_cache_read); the page pool
that forks, extends, frees and compacts paged sequences (kvq_pages_reorder,
kvq_pages_reserve, kvq_pages_compact, kvq_pages_copy); and attention of several
new tokens per sequence over the quantized cache (kvq_extend_attn).

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
        # rotary positions: one decode step of a small batch (latency), and a
        # batch of long prompts past the trained context
        {"name": "rope_step", "op": "rope", "B": 8, "T": 1, "Hq": 32, "Hkv": 32, "D": 128, "rd": 128,
         "inter": False, "scaling": "none", "base": 1e4, "factor": 1.0, "far": 4096, "ragged": 0},
        {"name": "rope_prompts", "op": "rope", "B": 4, "T": 8191, "Hq": 32, "Hkv": 8, "D": 128, "rd": 128,
         "inter": False, "scaling": "bands", "base": 5e5, "factor": 8.0, "far": 120000, "ragged": 1},
        # rotary positions on the way into the cache, and the rows read back:
        # a paged small-model batch's step, and a chunk of long prompts
        {"name": "append_step", "op": "append", "B": 256, "T": 1, "Hq": 14, "Hkv": 2, "D": 64, "rd": 32,
         "inter": True, "scaling": "none", "base": 1e4, "factor": 1.0, "far": 4000, "ragged": 2,
         "bits": 4, "g": 32, "page": 16},
        {"name": "append_chunk", "op": "append", "B": 2, "T": 4095, "Hq": 32, "Hkv": 8, "D": 128, "rd": 128,
         "inter": False, "scaling": "yarn", "base": 1e4, "factor": 16.0, "far": 28000, "ragged": 3,
         "bits": 8, "g": 64, "page": 0},
        # sequences forked from cached prompts and extended by a token: the
        # partly filled page of each child is copied in every layer
        {"name": "fork_small", "op": "fork", "prompts": 1, "kids": 4, "len": 999, "layers": 24, "Hkv": 2, "D": 64,
         "bits": 4, "g": 32, "page": 16, "pool": 128, "new": 1, "ragged": 4},
        {"name": "fork_large", "op": "fork", "prompts": 16, "kids": 240, "len": 3000, "layers": 32, "Hkv": 8,
         "D": 128, "bits": 4, "g": 64, "page": 16, "pool": 6000, "new": 33, "ragged": 5},
        # a pool left half empty by finished sequences, moved to its low end
        {"name": "compact", "op": "compact", "B": 200, "len": 600, "layers": 16, "Hkv": 8, "D": 128, "bits": 16,
         "g": 0, "page": 16, "pool": 9000, "ragged": 6},
        # a few drafted tokens per sequence checked over a ragged long cache
        {"name": "verify", "op": "extend", "B": 16, "T": 5, "Hq": 32, "Hkv": 8, "D": 128, "bits": 4, "g": 64,
         "page": 0, "before": 8000, "ragged": 7},
        # one short continuation of a single long conversation
        {"name": "short_turn", "op": "extend", "B": 1, "T": 17, "Hq": 32, "Hkv": 8, "D": 128, "bits": 8, "g": 32,
         "page": 0, "before": 32768, "ragged": 0},
        # the suffixes of requests that share cached pages, small model
        {"name": "suffixes", "op": "extend", "B": 24, "T": 200, "Hq": 14, "Hkv": 2, "D": 64, "bits": 4, "g": 32,
         "page": 16, "before": 2000, "ragged": 8},
        # whole prompts over an fp16 cache, and a late chunk of a long one
        {"name": "prompts", "op": "extend", "B": 4, "T": 2048, "Hq": 32, "Hkv": 32, "D": 128, "bits": 16, "g": 0,
         "page": 0, "before": 0, "ragged": 0},
        {"name": "late_chunk", "op": "extend", "B": 1, "T": 4096, "Hq": 32, "Hkv": 8, "D": 128, "bits": 4, "g": 32,
         "page": 0, "before": 12288, "ragged": 0},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "append", "fork", "compact", "extend", "extend", "extend"])
    D = rng.choice([64, 128])
    Hkv, G = rng.choice([(1, 8), (2, 7), (4, 4), (8, 4), (8, 1), (3, 5)])
    c = {"op": op, "Hkv": Hkv, "D": D, "ragged": rng.choice([0, rng.randrange(1, 1 << 20)])}
    bits = rng.choice([4, 4, 8, 16])
    fmt = {"bits": bits, "g": 0 if bits == 16 else rng.choice([16, 32, 64]), "page": rng.choice([0, 16, 64])}
    if op in ("rope", "append"):
        tokens = _spread(rng, 1, 16000)
        B = _spread(rng, 1, min(tokens, 256))
        scaling = rng.choice(["none", "linear", "ntk", "bands", "yarn"])
        c.update(B=B, T=max(1, tokens // B), Hq=Hkv * G, rd=rng.choice([D, D, D // 2, D // 4]),
                 inter=rng.random() < 0.5, scaling=scaling, base=rng.choice([1e4, 5e5, 1e6]),
                 factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]), far=_spread(rng, 1, 20000))
        if op == "append":
            c.update(fmt)
            c["far"] = max(1, min(c["far"], 2_000_000 // (B * Hkv)))
    elif op == "fork":
        prompts = _spread(rng, 1, 16)
        length, page, kids, new = _spread(rng, 1, 3000), rng.choice([16, 64]), _spread(rng, 1, 200), _spread(rng, 1, 40)
        need = prompts * -(-length // page) + kids * (2 + new // page)
        c.update(fmt, prompts=prompts, kids=kids, len=length, layers=rng.choice([1, 4, 24]), page=page,
                 pool=need + rng.randrange(1, 300), new=new)
    elif op == "compact":
        B, length, page = _spread(rng, 1, 200), _spread(rng, 1, 600), rng.choice([16, 64])
        c.update(fmt, B=B, len=length, layers=rng.choice([1, 4, 16]), page=page,
                 pool=B * -(-length // page) + rng.randrange(1, 900))
    else:
        B, T, before = _spread(rng, 1, 32), _spread(rng, 1, 4096), _spread(rng, 1, 32768)
        while B * T * (before + T) > 24_000_000:  # at most the largest listed work, and its scores in memory
            if B > 1:
                B //= 2
            elif T > 64:
                T = T * 2 // 3
            else:
                before //= 2
        c.update(fmt, B=B, T=T, Hq=Hkv * G, before=rng.choice([before, before, before, 0]))
    return c


def _lengths(case, count, most, salt, least=1):
    """`count` lengths up to `most`: all equal, or spread where the case is ragged."""
    if not case["ragged"]:
        return [most] * count
    r = random.Random(case["ragged"] * 16 + salt)
    return [r.randint(min(least, most), most) for _ in range(count)]


def _row_bytes(case):
    """Bytes of one cached K or V vector, its scales and zero-points included."""
    if case["bits"] == 16:
        return 2 * case["D"]
    return case["D"] * case["bits"] // 8 + 4 * (case["D"] // case["g"])


def work(case):
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    if op in ("rope", "append"):
        tokens = sum(_lengths(case, case["B"], case["T"], 1))
        q = tokens * case["Hq"] * D * 2 * 2
        if op == "rope":
            return {"bytes": q + tokens * Hkv * D * 2 * 2, "flops": 3 * tokens * (case["Hq"] + Hkv) * case["rd"]}
        kv = tokens * Hkv * 2 * (2 * D + 2 * _row_bytes(case) + 2 * D)  # in, cache written and read, rows out
        return {"bytes": q + kv, "flops": tokens * (3 * (case["Hq"] + Hkv) * case["rd"] + 2 * Hkv * D * 6)}
    if op == "fork":
        lens, parent = _fork_rows(case)
        rows, M = case["prompts"] + case["kids"], _fork_blocks(case)
        copied = sum(1 for p in parent[case["prompts"]:] if lens[p] % case["page"])
        page = 2 * Hkv * case["page"] * _row_bytes(case)
        return {"bytes": 2 * copied * case["layers"] * page + 8 * rows * M + 8 * case["pool"], "flops": 0}
    if op == "compact":
        live = _compact_live(case)
        moved = sum(1 for p in live if p >= len(live))
        page = 2 * Hkv * case["page"] * _row_bytes(case)
        return {"bytes": 2 * moved * case["layers"] * page + 8 * len(live) + 8 * case["pool"], "flops": 0}
    before, new = _extend_lens(case)
    pairs = sum(n * b + n * (n + 1) // 2 for b, n in zip(before, new))
    cached = sum(b + n for b, n in zip(before, new)) * Hkv * 2 * _row_bytes(case)
    return {"bytes": cached + 2 * sum(new) * case["Hq"] * D * 2, "flops": 4 * case["Hq"] * D * pairs}


def _extend_lens(case):
    before = _lengths(case, case["B"], case["before"], 2, least=max(case["before"] // 8, 0))
    return before, _lengths(case, case["B"], case["T"], 1)


def _fork_rows(case):
    """Cached tokens of each prompt, and each row's parent (a prompt is its own)."""
    r = random.Random(case["ragged"] * 16 + 5)
    P = case["prompts"]
    return _lengths(case, P, case["len"], 3), list(range(P)) + [r.randrange(P) for _ in range(case["kids"])]


def _fork_blocks(case):
    return -(-(case["len"] + case["new"]) // case["page"])


def _compact_live(case):
    """The live pages of a pool that random sequences still hold."""
    r = random.Random(case["ragged"] * 16 + 7)
    need = sum(-(-n // case["page"]) for n in _lengths(case, case["B"], case["len"], 4))
    return r.sample(range(case["pool"]), need)


# -------------------------------------------------------- rotary positions

def _inv_freq(case, device):
    """Rotation per position of each channel pair, in radians (64 bits)."""
    rd, base, f = case["rd"], case["base"], case["factor"]
    i = torch.arange(rd // 2, dtype=torch.float64, device=device)
    if case["scaling"] == "ntk":  # the base grown so that the slowest pair turns `factor` times slower
        base = base * f ** (rd / (rd - 2))
    w = base ** (-2.0 * i / rd)
    if case["scaling"] == "linear":
        return w / f
    if case["scaling"] == "bands":  # by wavelength: fast pairs kept, slow ones slowed, a ramp between
        turns = 8192 * w / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return w * (keep + (1 - keep) / f)
    if case["scaling"] == "yarn":  # by pair index, between the pairs that turn 32 times and once in the context
        at = lambda turns: rd * math.log(8192 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rd - 1)
        ramp = ((i - lo) / (max(hi - lo, 0.001))).clamp(0, 1)
        return w * (1 - ramp) + w / f * ramp
    return w


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" and case["factor"] > 1 else 1.0


def _rotate(x, angle, amp, case):
    """x [B][T][H][D] turned by angle [B][T][rd/2]; computed in x's type."""
    rd = case["rd"]
    c = (torch.cos(angle) * amp).to(x.dtype).unsqueeze(2)
    s = (torch.sin(angle) * amp).to(x.dtype).unsqueeze(2)
    if case["inter"]:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., : rd // 2], x[..., rd // 2: rd]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((r, x[..., rd:]), -1)


def _angles(st):
    case = st["case"]
    pos = st["before"].double()[:, None] + torch.arange(case["T"], device=st["before"].device)
    return pos[..., None] * _inv_freq(case, pos.device)


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


def _empty_cache(case, lead, device):
    D, bits, Hkv = case["D"], case["bits"], case["Hkv"]
    cache = {"k_codes": torch.zeros(lead + (D * bits // 8,), dtype=torch.uint8, device=device)}
    cache["v_codes"] = torch.zeros_like(cache["k_codes"])
    for n in ("k_scale", "k_zero", "v_scale", "v_zero"):
        cache[n] = None if bits == 16 else torch.zeros(lead + (D // case["g"],), dtype=F16, device=device)
    return cache


def _random_rows(case, lead, gen, device, keys):
    """Random K or V vectors [*lead][D] with the persistent large channels of keys."""
    x = torch.randn(lead + (case["D"],), generator=gen, device=device, dtype=F16)
    if keys:
        x[..., torch.randperm(case["D"], generator=gen, device=device)[:4]] *= 10
    return x


def _filled_cache(case, lead, gen, device):
    cache = _empty_cache(case, lead, device)
    for which in "kv":
        x = _random_rows(case, lead, gen, device, which == "k")
        if case["bits"] == 16:
            cache[which + "_codes"] = x.view(torch.uint8)
            continue
        q, s, z = _quantize(x, case["bits"], case["g"])
        cache[which + "_codes"] = _pack(q, case["bits"]).contiguous()
        cache[which + "_scale"], cache[which + "_zero"] = s, z
    return cache


def _table(blocks, M, pool, gen, device):
    """A block table [B][M] whose pages are scattered over the pool; -1 behind."""
    perm = torch.randperm(pool, generator=gen, device=device).int()
    need = torch.tensor(blocks, device=device)
    at = torch.cumsum(need, 0) - need
    j = torch.arange(M, device=device)
    return torch.where(j < need[:, None], perm[(at[:, None] + j).clamp(max=pool - 1)], -1).int().contiguous()


def _rows_of(st, L):
    """(index of each cached position's row) for L positions of every sequence."""
    pos = torch.arange(L, device=st["before"].device)
    if not st["case"]["page"]:
        return None
    page = st["table"][:, pos // st["case"]["page"]].long().clamp(min=0)
    return page, pos % st["case"]["page"]


def _gather(st, name, L):
    """[B][Hkv][L][...] of one cache array."""
    t = st["cache"][name]
    if t is None:
        return None
    if not st["case"]["page"]:
        return t[:, :, :L]
    page, off = _rows_of(st, L)
    return t[page, :, off].permute(0, 2, 1, 3)


def _handle(case, cache, table, batch):
    """The package's cache over these arrays."""
    import quantized_kv_decode_gb300 as K
    lead = cache["k_codes"].shape
    if case["page"]:
        desc = K.make_desc(case["bits"], case["g"], case["Hkv"], case["D"], K.KVQ_PAGED, case["page"], lead[0],
                           table.shape[1])
    else:
        desc = K.make_desc(case["bits"], case["g"], case["Hkv"], case["D"], K.KVQ_DENSE, lead[2])
    return K.KVCache(desc, batch, block_table=table, **cache)


# ----------------------------------------------------------------- prepare

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": case}
    if case["op"] in ("rope", "append"):
        B, T, Hkv, D = case["B"], case["T"], case["Hkv"], case["D"]
        st["before"] = torch.randint(0, case["far"], (B,), generator=gen, device=dev, dtype=torch.int32)
        st["new"] = torch.tensor(_lengths(case, B, T, 1), dtype=torch.int32, device=dev)
        st["q"] = torch.randn((B, T, case["Hq"], D), generator=gen, device=dev, dtype=F16)
        st["k"] = torch.randn((B, T, Hkv, D), generator=gen, device=dev, dtype=F16)
        st["q_out"] = torch.zeros_like(st["q"])
        st["k_out"] = torch.zeros_like(st["k"])
        if case["op"] == "append":
            st["v"] = torch.randn((B, T, Hkv, D), generator=gen, device=dev, dtype=F16)
            st["v_out"] = torch.zeros_like(st["v"])
            cap = case["far"] + T
            if case["page"]:
                M = -(-cap // case["page"])
                st["table"] = _table([M] * B, M, B * M + 5, gen, dev)
                lead = (B * M + 5, Hkv, case["page"])
            else:
                st["table"], lead = None, (B, Hkv, cap)
            st["cache"] = _empty_cache(case, lead, dev)
    elif case["op"] == "fork":
        lens, parent = _fork_rows(case)
        P, M, rows = case["prompts"], _fork_blocks(case), case["prompts"] + case["kids"]
        held = [-(-n // case["page"]) for n in lens] + [0] * case["kids"]
        st["table"] = _table(held, M, case["pool"], gen, dev)
        st["ref"] = (torch.bincount(st["table"].flatten().long() + 1, minlength=case["pool"] + 1)[1:]).int()
        st["parent"] = torch.tensor(parent, dtype=torch.int32, device=dev)
        st["keep"] = torch.tensor([lens[p] for p in parent], dtype=torch.int32, device=dev)
        st["new"] = torch.tensor([0] * P + [case["new"]] * case["kids"], dtype=torch.int32, device=dev)
        lead = (case["layers"], case["pool"], case["Hkv"], case["page"])
        st["cache"] = _page_bytes(case, lead, gen, dev)
        st["src"] = torch.full((rows,), -1, dtype=torch.int32, device=dev)
        st["dst"], st["granted"] = st["src"].clone(), st["src"].clone()
    elif case["op"] == "compact":
        live = torch.tensor(_compact_live(case), dtype=torch.int32, device=dev)
        blocks = [-(-n // case["page"]) for n in _lengths(case, case["B"], case["len"], 4)]
        need = torch.tensor(blocks, device=dev)
        j = torch.arange(max(blocks), device=dev)
        at = (torch.cumsum(need, 0) - need)[:, None] + j
        st["table0"] = torch.where(j < need[:, None], live[at.clamp(max=len(live) - 1)], -1).int().contiguous()
        st["ref0"] = torch.zeros(case["pool"], dtype=torch.int32, device=dev)
        st["ref0"][live.long()] = 1
        st["table"], st["ref"] = st["table0"].clone(), st["ref0"].clone()
        st["src"] = torch.full((case["pool"] // 2,), -1, dtype=torch.int32, device=dev)
        st["dst"], st["live"] = st["src"].clone(), torch.zeros(1, dtype=torch.int32, device=dev)
        st["cache"] = _page_bytes(case, (case["layers"], case["pool"], case["Hkv"], case["page"]), gen, dev)
    else:
        B, T, Hkv, D = case["B"], case["T"], case["Hkv"], case["D"]
        before, new = _extend_lens(case)
        st["before"] = torch.tensor(before, dtype=torch.int32, device=dev)
        st["new"] = torch.tensor(new, dtype=torch.int32, device=dev)
        st["L"] = max(b + n for b, n in zip(before, new))
        if case["page"]:
            M = -(-st["L"] // case["page"])
            blocks = [-(-(b + n) // case["page"]) for b, n in zip(before, new)]
            st["table"] = _table(blocks, M, sum(blocks) + 3, gen, dev)
            lead = (sum(blocks) + 3, Hkv, case["page"])
        else:
            st["table"], lead = None, (B, Hkv, st["L"])
        st["cache"] = _filled_cache(case, lead, gen, dev)
        st["q"] = torch.randn((B, T, case["Hq"], D), generator=gen, device=dev, dtype=F16)
        st["out"] = torch.zeros_like(st["q"])
    if own:
        _prepare_own(st)
    return st


def _page_bytes(case, lead, gen, dev):
    """Page contents of every layer: random bytes and small fp16 numbers."""
    cache = _empty_cache(case, lead, dev)
    for t in cache.values():
        if t is not None and t.dtype == torch.uint8:
            t.random_(0, 256, generator=gen) if case["bits"] != 16 else t.view(F16).normal_(generator=gen)
        elif t is not None:
            t.normal_(generator=gen)
    return cache


def _prepare_own(st):
    """The handles and workspaces that a program keeps."""
    import quantized_kv_decode_gb300 as K
    case = st["case"]
    if case["op"] in ("rope", "append"):
        st["rope"] = K.make_rope(case["rd"], base=case["base"], interleaved=case["inter"], scaling=case["scaling"],
                                 factor=case["factor"], original_context=8192)
    if case["op"] in ("append", "extend"):
        st["kv"] = _handle(case, st["cache"], st["table"], case["B"])
    if case["op"] == "append":
        st["total"] = st["before"] + st["new"]
    if case["op"] == "extend":
        n = K.kvq_extend_workspace_size(st["kv"].desc, case["B"], case["T"], case["Hq"], st["L"])
        st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    if case["op"] in ("fork", "compact"):
        st["pool"] = K.PagePool(st["ref"], st["table"], case["page"])
        st["ws"] = torch.empty(K.kvq_pages_workspace_size(st["pool"]), dtype=torch.uint8, device="cuda")
        st["kvs"] = [_handle(case, {n: None if t is None else t[i] for n, t in st["cache"].items()}, st["table"],
                             st["table"].shape[0]) for i in range(case["layers"])]


# --------------------------------------------------------------------- run

def run(st):
    op = st["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "fork": _own_fork, "compact": _own_compact,
                "extend": _own_extend}[op](st)
    return {"rope": _plain_rope, "append": _plain_append, "fork": _plain_fork, "compact": _plain_compact,
            "extend": _plain_extend}[op](st)


def _own_rope(st):
    import quantized_kv_decode_gb300 as K
    K.kvq_rope_apply(st["rope"], st["q"], st["k"], seq_lens_before=st["before"], new_lens=st["new"],
                     q_out=st["q_out"], k_out=st["k_out"])
    return st["q_out"], st["k_out"]


def _own_append(st):
    import quantized_kv_decode_gb300 as K
    K.kvq_rope_append(st["kv"], st["rope"], st["k"], st["v"], st["before"], q=st["q"], q_out=st["q_out"],
                      new_lens=st["new"])
    K.kvq_cache_read(st["kv"], st["total"], st["before"], st["k_out"], st["v_out"])
    return st["q_out"], st["k_out"], st["v_out"]


def _own_fork(st):
    import quantized_kv_decode_gb300 as K
    K.kvq_pages_reorder(st["pool"], st["parent"], st["keep"])
    K.kvq_pages_reserve(st["pool"], st["keep"], st["new"], st["src"], st["dst"], st["granted"],
                        max_new=st["case"]["new"], workspace=st["ws"])
    K.kvq_pages_copy(st["kvs"], st["src"], st["dst"])
    return st["ref"], st["table"], st["src"], st["dst"], st["granted"], _page_state(st)


def _own_compact(st):
    import quantized_kv_decode_gb300 as K
    st["table"].copy_(st["table0"])
    st["ref"].copy_(st["ref0"])
    K.kvq_pages_compact(st["pool"], st["src"], st["dst"], st["live"], workspace=st["ws"])
    K.kvq_pages_copy(st["kvs"], st["src"], st["dst"])
    return st["ref"], st["table"], st["src"], st["dst"], st["live"], _page_state(st)


def _own_extend(st):
    import quantized_kv_decode_gb300 as K
    K.kvq_extend_attn(st["kv"], st["q"], st["before"], st["L"], new_lens=st["new"], out=st["out"],
                      workspace=st["ws"])
    return st["out"]


def _page_state(st):
    """The pages' bytes, fp16 caches as the numbers they hold."""
    c = st["cache"]
    if st["case"]["bits"] == 16:
        return c["k_codes"].view(F16), c["v_codes"].view(F16)
    return tuple(c.values())


def _plain_rope(st):
    live, amp = _live(st)[..., None, None], _amplitude(st["case"])
    angle = _angles(st)
    return tuple(torch.where(live, _rotate(st[n].float(), angle, amp, st["case"]).to(F16), st[n + "_out"])
                 for n in "qk")


def _plain_append(st):
    case, live = st["case"], _live(st)
    amp, angle = _amplitude(case), _angles(st)
    q = torch.where(live[..., None, None], _rotate(st["q"].float(), angle, amp, case).to(F16), st["q_out"])
    # keys in 64 bits: their codes change where a value lies next to a border
    rows = {"k": _rotate(st["k"].double(), angle, amp, case).to(F16), "v": st["v"]}
    pos = st["before"].long()[:, None] + torch.arange(case["T"], device=live.device)
    b = torch.arange(case["B"], device=live.device)[:, None].expand_as(pos)
    if case["page"]:
        first = st["table"].gather(1, (pos // case["page"])).long()
        off = pos % case["page"]
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


def _copy_pages(st, src, dst):
    """pages[dst] = pages[src] in every array and layer; pairs of -1 copy nothing."""
    some = src >= 0
    src, dst = src[some].long(), dst[some].long()
    for t in st["cache"].values():
        if t is not None:
            t[:, dst] = t[:, src]


def _plain_fork(st):
    case, table, ref = st["case"], st["table"], st["ref"]
    page, pool, (B, M) = case["page"], case["pool"], table.shape
    j = torch.arange(M, device=table.device)
    count = lambda t: torch.bincount(t.flatten().long() + 1, minlength=pool + 1)[1:].int()  # noqa: E731
    # every row takes its parent's first blocks
    blocks = (st["keep"] + page - 1) // page
    moved = torch.where(j < blocks[:, None], table[st["parent"].long()], -1)
    ref += count(moved) - count(table)
    # the blocks that [keep, keep + new) touches; a shared one is replaced,
    # but for the last row to touch it when all its owners do
    at, new = st["keep"][:, None], st["new"][:, None]
    touched = (new > 0) & (j >= at // page) & (j * page < at + new)
    partial = touched & (j * page < at) & (moved >= 0)
    mine = torch.where(partial, moved, -1).amax(1)
    below = ((mine[:, None] == mine[None, :]) & (mine[:, None] >= 0)).tril(-1).sum(1)
    refs = ref[moved.clamp(min=0).long()]
    shared = touched & (moved >= 0) & (refs - torch.where(partial, below[:, None], 0) > 1)
    fresh = touched & ((moved < 0) | shared)
    free = torch.argsort((ref != 0).int(), stable=True).int()
    rank = (torch.cumsum(fresh.flatten().long(), 0) - 1).clamp(0, pool - 1).view(B, M)
    taken = torch.where(fresh, free[rank], moved)
    src = torch.where(shared & partial, moved, -1).amax(1)
    dst = torch.where(shared & partial, taken, -1).amax(1)
    ref += count(taken) - count(moved)
    table.copy_(taken)
    _copy_pages(st, src, dst)
    return ref, table, src, dst, st["new"].clone(), _page_state(st)


def _plain_compact(st):
    case, table, ref = st["case"], st["table"], st["ref"]
    table.copy_(st["table0"])
    ref.copy_(st["ref0"])
    idx = torch.arange(case["pool"], device=ref.device)
    n = (ref > 0).sum()
    half = case["pool"] // 2
    # the k-th live page behind the border goes to the k-th hole before it
    mover, hole = (ref > 0) & (idx >= n), (ref == 0) & (idx < n)
    src = torch.argsort((~mover).int(), stable=True)[:half]
    dst = torch.argsort((~hole).int(), stable=True)[:half]
    valid = torch.arange(half, device=ref.device) < mover.sum()
    src, dst = torch.where(valid, src, -1).int(), torch.where(valid, dst, -1).int()
    into = torch.arange(case["pool"] + 1, device=ref.device)
    into[torch.where(valid, src, case["pool"]).long()] = dst.long()
    into[case["pool"]] = -1
    table.copy_(into[torch.where(table >= 0, table, case["pool"]).long()].int())
    ref.copy_(torch.bincount(table.flatten().long() + 1, minlength=case["pool"] + 1)[1:].int())
    _copy_pages(st, src, dst)
    return ref, table, src, dst, n.int().view(1), _page_state(st)


def _plain_extend(st):
    case = st["case"]
    B, T, Hq, D = st["q"].shape
    Hkv, L = case["Hkv"], st["L"]
    k, v = (_dequantize(*(_gather(st, n + a, L) for a in ("_codes", "_scale", "_zero")), case["bits"], case["g"])
            for n in "kv")
    live = _live(st)
    # position j is seen by new token t when j <= before + t
    seen = torch.arange(L, device=k.device) <= (st["before"][:, None] + torch.arange(T, device=k.device))[..., None]
    held = torch.arange(L, device=k.device) < (st["before"] + st["new"])[:, None]
    v = torch.where(held[:, None, :, None], v, 0)
    q = st["q"].float().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(D ** -0.5).view(B, Hkv, Hq // Hkv, T, L)
    s.masked_fill_(~(seen & held[:, None, :])[:, None, None], -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, Hkv, -1, L), v).view(B, Hkv, Hq // Hkv, T, D).div_(total)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(F16)
    return torch.where(live[..., None, None], o, st["out"])


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """What run returns, from the definitions in 64 bits; None for whole numbers."""
    global own
    if case["op"] in ("fork", "compact"):
        return None
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return _exact_extend(st) if case["op"] == "extend" else _exact_rows(st)


def _exact_turns(st):
    """amplitude * exp(i position w) of every token and pair, w pair by pair."""
    case = st["case"]
    rd, f, kind = case["rd"], case["factor"], case["scaling"]
    ws = []
    for i in range(rd // 2):
        base = case["base"] * (f ** (rd / (rd - 2)) if kind == "ntk" else 1.0)
        w = math.exp(-2 * i / rd * math.log(base))
        if kind == "linear":
            w /= f
        elif kind == "bands":
            wave = 2 * math.pi / w
            if wave > 8192 / 1.0:
                w /= f
            elif wave >= 8192 / 4.0:
                m = (8192 / wave - 1.0) / 3.0
                w = (1 - m) * w / f + m * w
        elif kind == "yarn":
            bound = [rd * math.log(8192 / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32.0, 1.0)]
            lo, hi = max(math.floor(bound[0]), 0), min(math.ceil(bound[1]), rd - 1)
            m = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = m * (w / f) + (1 - m) * w
        ws.append(w)
    amp = 1.0 + 0.1 * math.log(f) if kind == "yarn" and f > 1 else 1.0
    pos = torch.stack([st["before"].double() + t for t in range(case["T"])], 1)
    angle = pos[:, :, None, None] * torch.tensor(ws, dtype=torch.float64, device=pos.device)
    return torch.polar(torch.full_like(angle, amp), angle)


def _exact_rows(st):
    """Each pair as a complex number times its turn; then the cache's grid."""
    case = st["case"]
    half = case["rd"] // 2
    turn = _exact_turns(st)
    padding = torch.arange(case["T"], device="cuda").expand(case["B"], -1) >= st["new"][:, None]

    def turned(x):
        y = x.double()
        even = slice(0, case["rd"], 2) if case["inter"] else slice(0, half)
        odd = slice(1, case["rd"], 2) if case["inter"] else slice(half, case["rd"])
        w = torch.complex(y[..., even].contiguous(), y[..., odd].contiguous()) * turn
        y[..., even], y[..., odd] = w.real, w.imag
        return y

    def placed(y):
        y[padding] = 0.0
        return y

    q = placed(turned(st["q"]))
    if case["op"] == "rope":
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


def _exact_cached(st, n, b, length):
    """[Hkv][length][D] of K or V of one sequence, in 64 bits."""
    case, D = st["case"], st["case"]["D"]
    rows = []
    for a in ("_codes", "_scale", "_zero"):
        t = st["cache"][n + a]
        if t is None:
            rows.append(None)
        elif case["page"]:
            pages = st["table"][b, : -(-length // case["page"])].long()
            rows.append(t[pages].transpose(0, 1).flatten(1, 2)[:, :length])
        else:
            rows.append(t[b, :, :length])
    if case["bits"] == 16:
        return rows[0].contiguous().view(F16).double()
    c = rows[0].int()
    per = 8 // case["bits"]
    q = torch.empty((*c.shape[:2], D), dtype=torch.float64, device=c.device)
    for e in range(per):
        q[..., e::per] = ((c >> (e * case["bits"])) % 2 ** case["bits"]).double()
    s, z = (r.double().repeat_interleave(case["g"], -1) for r in rows[1:])
    return (q - z) * s


def _exact_extend(st):
    case = st["case"]
    if case["B"] * case["T"] * st["L"] * case["Hq"] * case["D"] > 5e11:  # over about 20 seconds in 64 bits
        return None
    B, T, Hq, D = st["q"].shape
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        n0, n = int(st["before"][b]), int(st["new"][b])
        k, v = (_exact_cached(st, a, b, n0 + n) for a in "kv")
        later = torch.arange(n0 + n, device="cuda") > torch.arange(n0, n0 + n, device="cuda")[:, None]
        for h in range(Hq):
            s = st["q"][b, :n, h].double() @ k[h // (Hq // case["Hkv"])].T / math.sqrt(D)
            out[b, :n, h] = torch.softmax(s.masked_fill(later, -math.inf), -1) @ v[h // (Hq // case["Hkv"])]
    return out

"""Python entry points of the prompt and page-pool calls (include/kvq.h).

As in api.py, PyTorch provides device memory and streams only: each function
checks dtypes, shapes and devices, passes raw pointers to libkvq.so and
returns.  The tensors of a call live on one device; the call runs on that
device, on its current stream unless `stream` is given.  Outputs and
workspaces made here are made on the call's stream too: what fills them runs
before the kernels, and their memory is not handed to other streams' work
while the kernels may still run.
"""
from __future__ import annotations

from array import array
from ctypes import byref
from dataclasses import dataclass
from operator import attrgetter

import torch

from . import _lib
from ._lib import ROPE_SCALING, kvq_page_pool, kvq_rope, kvq_rope_desc
from .api import KVCache, _ptr


def _check(t, dtype, name, shape, device):
    """A contiguous CUDA tensor of this dtype and shape (None in it: any size),
    on `device` (an index; None: any)."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor of dtype {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    got = t.shape
    if got != shape and (len(got) != len(shape)
                         or any(w is not None and w != n for w, n in zip(shape, got))):
        raise ValueError(f"{name} must have shape {tuple('*' if w is None else w for w in shape)}, "
                         f"not {tuple(got)}")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")


def _optional(t, dtype, name, shape, device):
    if t is not None:
        _check(t, dtype, name, shape, device)


def _status(t, device):
    if t is not None and (not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != device
                          or t.dtype not in (torch.int32, torch.uint32) or t.numel() < 1):
        raise TypeError(f"dev_status must be an int32 tensor on cuda:{device}")


def _bytes(t, device, need, name):
    """(tensor, its bytes) of a workspace; allocated when missing or too small."""
    if t is not None and (not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != device
                          or not t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous tensor on cuda:{device}")
    size = 0 if t is None else t.numel() * t.element_size()
    if need > size:
        t, size = torch.empty(need, dtype=torch.uint8, device=f"cuda:{device}"), need
    return t, size


def _made_like(t, new_lens):
    """An output of a call: rows behind new_lens[b], which no kernel writes, are zeros."""
    return torch.empty_like(t) if new_lens is None else torch.zeros_like(t)


class _on:
    """Makes a call's device and stream current, where they are not already."""
    __slots__ = ("guard",)

    def __init__(self, device, stream):
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                handle = getattr(stream, "cuda_stream", stream)
                stream = (torch.cuda.ExternalStream(handle, device) if handle
                          else torch.cuda.default_stream(device))
            if stream.device.index != device:
                raise ValueError(f"the stream is of {stream.device}, the tensors are on cuda:{device}")
            self.guard = torch.cuda.stream(stream)
        else:
            self.guard = None if device == torch.cuda.current_device() else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _handle(device):
    return torch.cuda.current_stream(device).cuda_stream


def _same_cache_device(cache: KVCache, device):
    if not cache.k_codes.is_cuda or cache.k_codes.get_device() != device:
        raise ValueError(f"the cache is on {cache.k_codes.device}, not on cuda:{device}")


def _batch(cache: KVCache, B):
    """A call's batch fits the cache's arrays."""
    if B > cache.batch:
        raise ValueError(f"a batch of {B} on a cache of {cache.batch} sequences")


def make_rope(rotary_dim: int, base: float = 10000.0, interleaved: bool = False,
              scaling: str = "none", factor: float = 1.0, original_context: int = 0,
              low_turns: float = 0.0, high_turns: float = 0.0,
              amplitude: float = 0.0) -> kvq_rope:
    """A rotation for kvq_rope_apply / kvq_rope_append.  scaling: "none",
    "linear", "ntk", "bands" or "yarn" (see kvq_rope_scaling in kvq.h); a 0
    for low_turns, high_turns or amplitude takes the scaling's default."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {', '.join(ROPE_SCALING)}")
    desc = kvq_rope_desc(int(rotary_dim), int(bool(interleaved)), ROPE_SCALING[scaling],
                         int(original_context), float(base), float(factor), float(low_turns),
                         float(high_turns), float(amplitude))
    rope = kvq_rope()
    _lib.check(_lib.lib().kvq_rope_init(byref(desc), byref(rope)), "kvq_rope_init")
    return rope


def kvq_rope_apply(rope: kvq_rope, q: torch.Tensor | None = None, k: torch.Tensor | None = None,
                   positions: torch.Tensor | None = None,
                   seq_lens_before: torch.Tensor | None = None,
                   new_lens: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                   k_out: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
                   stream=None):
    """Rotate q [B][T][Hq][D] and / or k [B][T][Hk][D] fp16 by positions
    [B][T] or seq_lens_before [B] + t; returns (q_out, k_out).  An output may
    be its input (in place).  Rows behind new_lens[b] keep what they held
    (an output made here starts as zeros)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k must be given")
    _check(x, torch.float16, "q" if q is not None else "k", (None,) * 4, None)
    B, T, _, D = x.shape
    dev = x.get_device()
    if positions is None and seq_lens_before is None:
        raise ValueError("positions or seq_lens_before must be given")
    _optional(positions, torch.int32, "positions", (B, T), dev)
    _optional(seq_lens_before, torch.int32, "seq_lens_before", (B,), dev)
    _optional(new_lens, torch.int32, "new_lens", (B,), dev)
    _status(dev_status, dev)
    for t, o, name in ((q, q_out, "q"), (k, k_out, "k")):
        if t is not None:
            _check(t, torch.float16, name, (B, T, None, D), dev)
            if o is not None:
                _check(o, torch.float16, name + "_out", t.shape, dev)
        elif o is not None:
            raise ValueError(f"{name}_out without {name}")
    with _on(dev, stream):
        outs = [o if t is None or o is not None else _made_like(t, new_lens)
                for t, o in ((q, q_out), (k, k_out))]
        st = _lib.lib().kvq_rope_apply(
            byref(rope), D, B, T, 0 if q is None else q.shape[2], _ptr(q), _ptr(outs[0]),
            0 if k is None else k.shape[2], _ptr(k), _ptr(outs[1]), _ptr(positions),
            _ptr(seq_lens_before), _ptr(new_lens), _ptr(dev_status), _handle(dev))
    _lib.check(st, "kvq_rope_apply")
    return outs[0], outs[1]


def kvq_rope_append(cache: KVCache, rope: kvq_rope, k_new: torch.Tensor, v_new: torch.Tensor,
                    seq_lens_before: torch.Tensor, q: torch.Tensor | None = None,
                    q_out: torch.Tensor | None = None, new_lens: torch.Tensor | None = None,
                    dev_status: torch.Tensor | None = None, stream=None):
    """Rotate k_new [B][T][Hkv][D] fp16 and quantize it and v_new into the
    cache at positions seq_lens_before[b] + t; rotate q [B][T][Hq][D] into
    q_out (which may be q).  Returns q_out (None without q)."""
    d = cache.desc
    _check(k_new, torch.float16, "k_new", (None, None, d.num_kv_heads, d.head_dim), None)
    B, T, _, D = k_new.shape
    dev = k_new.get_device()
    _check(v_new, torch.float16, "v_new", k_new.shape, dev)
    _check(seq_lens_before, torch.int32, "seq_lens_before", (B,), dev)
    _optional(new_lens, torch.int32, "new_lens", (B,), dev)
    _same_cache_device(cache, dev)
    _batch(cache, B)
    _status(dev_status, dev)
    if q is not None:
        _check(q, torch.float16, "q", (B, T, None, D), dev)
        if q_out is not None:
            _check(q_out, torch.float16, "q_out", q.shape, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    with _on(dev, stream):
        if q is not None and q_out is None:
            q_out = _made_like(q, new_lens)
        st = _lib.lib().kvq_rope_append(
            byref(d), byref(cache.ptrs), byref(rope), B, T, _ptr(k_new), _ptr(v_new),
            0 if q is None else q.shape[2], _ptr(q), _ptr(q_out), _ptr(seq_lens_before),
            _ptr(new_lens), _ptr(dev_status), _handle(dev))
    _lib.check(st, "kvq_rope_append")
    return q_out


def kvq_cache_read(cache: KVCache, seq_lens: torch.Tensor, start: torch.Tensor,
                   k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
                   dev_status: torch.Tensor | None = None, stream=None):
    """Rows [start[b], seq_lens[b]) of every sequence as fp16 into k_out and /
    or v_out [B][T][Hkv][D], at most T of them; rows behind keep what they
    held.  Returns (k_out, v_out)."""
    d = cache.desc
    x = k_out if k_out is not None else v_out
    if x is None:
        raise ValueError("k_out or v_out must be given")
    _check(x, torch.float16, "k_out" if k_out is not None else "v_out",
           (None, None, d.num_kv_heads, d.head_dim), None)
    B, T, dev = x.shape[0], x.shape[1], x.get_device()
    _optional(k_out, torch.float16, "k_out", x.shape, dev)
    _optional(v_out, torch.float16, "v_out", x.shape, dev)
    _check(seq_lens, torch.int32, "seq_lens", (B,), dev)
    _check(start, torch.int32, "start", (B,), dev)
    _same_cache_device(cache, dev)
    _batch(cache, B)
    _status(dev_status, dev)
    with _on(dev, stream):
        st = _lib.lib().kvq_cache_read(byref(d), byref(cache.ptrs), B, T, _ptr(seq_lens),
                                       _ptr(start), _ptr(k_out), _ptr(v_out), _ptr(dev_status),
                                       _handle(dev))
    _lib.check(st, "kvq_cache_read")
    return k_out, v_out


def kvq_extend_num_splits(desc, batch, num_new, num_q_heads, max_seq_len, num_splits=0) -> int:
    return int(_lib.lib().kvq_extend_num_splits(byref(desc), batch, num_new, num_q_heads,
                                                max_seq_len, num_splits))


def kvq_extend_workspace_size(desc, batch, num_new, num_q_heads, max_seq_len, num_splits=0) -> int:
    return int(_lib.lib().kvq_extend_workspace_size(byref(desc), batch, num_new, num_q_heads,
                                                    max_seq_len, num_splits))


def kvq_extend_attn(cache: KVCache, q: torch.Tensor, seq_lens_before: torch.Tensor,
                    max_seq_len: int, new_lens: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    dev_status: torch.Tensor | None = None, num_splits: int = 0,
                    softmax_scale: float = 0.0, stream=None) -> torch.Tensor:
    """Causal attention of the new tokens q [B][T][Hq][D] fp16, whose K and V
    rows are already cached at seq_lens_before[b] + t, over positions
    [0, seq_lens_before[b] + t]; returns out.  Rows behind new_lens[b] keep
    what they held (an `out` made here starts as zeros)."""
    d = cache.desc
    _check(q, torch.float16, "q", (None, None, None, d.head_dim), None)
    B, T, Hq, _ = q.shape
    dev = q.get_device()
    _check(seq_lens_before, torch.int32, "seq_lens_before", (B,), dev)
    _optional(new_lens, torch.int32, "new_lens", (B,), dev)
    _same_cache_device(cache, dev)
    _batch(cache, B)
    _status(dev_status, dev)
    if out is not None:
        _check(out, torch.float16, "out", q.shape, dev)
    with _on(dev, stream):
        if out is None:
            out = _made_like(q, new_lens)
        need = 0 if workspace is not None else \
            kvq_extend_workspace_size(d, B, T, Hq, max_seq_len, num_splits)
        workspace, ws_bytes = _bytes(workspace, dev, need, "workspace")
        st = _lib.lib().kvq_extend_attn(
            byref(d), byref(cache.ptrs), B, T, Hq, _ptr(q), _ptr(seq_lens_before), _ptr(new_lens),
            int(max_seq_len), int(num_splits), float(softmax_scale), _ptr(out), _ptr(workspace),
            ws_bytes, _ptr(dev_status), _handle(dev))
    _lib.check(st, "kvq_extend_attn")
    return out


@dataclass
class PagePool:
    """The pages the sequences of paged caches hold: one reference count per
    page (0: free) and the block table that the layers' caches share."""
    ref_count: torch.Tensor    # int32 [num_pages]
    block_table: torch.Tensor  # int32 [batch][max_blocks_per_seq], -1: no page
    page_size: int

    def __post_init__(self):
        _check(self.ref_count, torch.int32, "ref_count", (None,), None)
        _check(self.block_table, torch.int32, "block_table", (None, None), self.ref_count.get_device())

    @classmethod
    def allocate(cls, num_pages: int, page_size: int, batch: int, max_blocks_per_seq: int,
                 device="cuda") -> "PagePool":
        """An empty pool: every page free, every block without a page."""
        return cls(torch.zeros(num_pages, dtype=torch.int32, device=device),
                   torch.full((batch, max_blocks_per_seq), -1, dtype=torch.int32, device=device),
                   page_size)

    @property
    def struct(self) -> kvq_page_pool:
        return kvq_page_pool(self.ref_count.numel(), self.page_size, self.block_table.shape[0],
                             self.block_table.shape[1], _ptr(self.ref_count),
                             _ptr(self.block_table))


def kvq_pages_workspace_size(pool: PagePool) -> int:
    return int(_lib.lib().kvq_pages_workspace_size(byref(pool.struct)))


def kvq_pages_reorder(pool: PagePool, parent: torch.Tensor, keep_lens: torch.Tensor | None = None,
                      dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Row b of the block table becomes the first ceil(keep_lens[b] /
    page_size) entries of row parent[b] (-1: freed); reference counts follow."""
    B, dev = pool.block_table.shape[0], pool.ref_count.get_device()
    _check(parent, torch.int32, "parent", (B,), dev)
    _optional(keep_lens, torch.int32, "keep_lens", (B,), dev)
    _status(dev_status, dev)
    with _on(dev, stream):
        st = _lib.lib().kvq_pages_reorder(byref(pool.struct), _ptr(parent), _ptr(keep_lens),
                                          _ptr(dev_status), _handle(dev))
    _lib.check(st, "kvq_pages_reorder")


def kvq_pages_reserve(pool: PagePool, seq_lens_before: torch.Tensor,
                      new_lens: torch.Tensor | None, copy_src: torch.Tensor,
                      copy_dst: torch.Tensor, granted: torch.Tensor | None = None,
                      max_new: int = 1, workspace: torch.Tensor | None = None,
                      dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Make positions [seq_lens_before[b], seq_lens_before[b] + new_lens[b])
    writable (new_lens None: max_new each); the pages to copy first are left
    in copy_src / copy_dst [B], the tokens granted in granted [B]."""
    B, dev = pool.block_table.shape[0], pool.ref_count.get_device()
    _check(seq_lens_before, torch.int32, "seq_lens_before", (B,), dev)
    _optional(new_lens, torch.int32, "new_lens", (B,), dev)
    _check(copy_src, torch.int32, "copy_src", (B,), dev)
    _check(copy_dst, torch.int32, "copy_dst", (B,), dev)
    _optional(granted, torch.int32, "granted", (B,), dev)
    _status(dev_status, dev)
    pl = pool.struct
    with _on(dev, stream):
        need = int(_lib.lib().kvq_pages_workspace_size(byref(pl)))
        workspace, ws_bytes = _bytes(workspace, dev, need, "workspace")
        st = _lib.lib().kvq_pages_reserve(
            byref(pl), _ptr(seq_lens_before), _ptr(new_lens), int(max_new), _ptr(copy_src),
            _ptr(copy_dst), _ptr(granted), _ptr(workspace), ws_bytes, _ptr(dev_status),
            _handle(dev))
    _lib.check(st, "kvq_pages_reserve")


def kvq_pages_compact(pool: PagePool, move_src: torch.Tensor, move_dst: torch.Tensor,
                      num_live: torch.Tensor, workspace: torch.Tensor | None = None,
                      dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Move the pages in use to the low end of the pool: table and counts
    change here, the moves [num_pages // 2] go to kvq_pages_copy."""
    n, dev = pool.ref_count.numel(), pool.ref_count.get_device()
    _check(move_src, torch.int32, "move_src", (n // 2,), dev)
    _check(move_dst, torch.int32, "move_dst", (n // 2,), dev)
    _check(num_live, torch.int32, "num_live", (1,), dev)
    _status(dev_status, dev)
    pl = pool.struct
    with _on(dev, stream):
        need = int(_lib.lib().kvq_pages_workspace_size(byref(pl)))
        workspace, ws_bytes = _bytes(workspace, dev, need, "workspace")
        st = _lib.lib().kvq_pages_compact(byref(pl), _ptr(move_src), _ptr(move_dst),
                                          _ptr(num_live), _ptr(workspace), ws_bytes,
                                          _ptr(dev_status), _handle(dev))
    _lib.check(st, "kvq_pages_compact")


_PAGED_ARRAYS = attrgetter("k_codes", "v_codes", "k_scale", "k_zero", "v_scale", "v_zero")


def kvq_pages_copy(caches, copy_src: torch.Tensor, copy_dst: torch.Tensor,
                   dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Page copy_dst[i] takes the bytes of page copy_src[i] in every cache of
    `caches` (the layers: one descriptor); pairs with a -1 are skipped."""
    caches = list(caches)
    if not caches:
        return
    dev = caches[0].k_codes.get_device()
    _check(copy_src, torch.int32, "copy_src", (None,), dev)
    _check(copy_dst, torch.int32, "copy_dst", copy_src.shape, dev)
    _status(dev_status, dev)
    desc = caches[0].desc
    first = bytes(desc)
    tail = [0 if t is None else t.data_ptr() for t in
            (caches[0].block_table, caches[0].k_window, caches[0].v_window)]
    flat = []
    for c in caches:
        kc, vc, ks, kz, vs, vz = _PAGED_ARRAYS(c)
        if kc.get_device() != dev:
            _same_cache_device(c, dev)
        if c.desc is not desc and bytes(c.desc) != first:
            raise ValueError("the caches must have one descriptor")
        flat += (kc.data_ptr(), vc.data_ptr(), 0 if ks is None else ks.data_ptr(),
                 0 if kz is None else kz.data_ptr(), 0 if vs is None else vs.data_ptr(),
                 0 if vz is None else vz.data_ptr())
        flat += tail  # (not touched by the copy)
    # the kvq_cache structures: their pointers one after the other
    structs = array("Q", flat)
    arrays = structs.buffer_info()[0]
    with _on(dev, stream):
        st = _lib.lib().kvq_pages_copy(byref(caches[0].desc), arrays, len(caches), _ptr(copy_src),
                                       _ptr(copy_dst), copy_src.numel(), _ptr(dev_status),
                                       _handle(dev))
    _lib.check(st, "kvq_pages_copy")


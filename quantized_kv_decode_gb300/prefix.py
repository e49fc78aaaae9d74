"""Python entry points of the shared-prefix calls (include/kvq.h).

Checks, devices, streams and workspaces as in prompt.py.
"""
from __future__ import annotations

from ctypes import byref
from dataclasses import dataclass

import torch

from . import _lib
from .api import KVCache, _ptr
from .prompt import PagePool, _batch, _bytes, _check, _handle, _made_like, _on, _optional, _same_cache_device, _status


@dataclass
class PrefixPlan:
    """Which sequence of a batch is on which prefix, as kvq_prefix_plan left it."""
    words: torch.Tensor  # int32, opaque
    batch: int
    num_prefixes: int


def kvq_prefix_plan(prefix_of: torch.Tensor, prefix_lens: torch.Tensor, plan: PrefixPlan | None = None,
                    dev_status: torch.Tensor | None = None, stream=None) -> PrefixPlan:
    """The plan of a batch: prefix_of [B] names each sequence's prefix (-1:
    none), prefix_lens [N] their tokens.  `plan`: one of the same sizes, filled
    again in place."""
    _check(prefix_of, torch.int32, "prefix_of", (None,), None)
    dev = prefix_of.get_device()
    _check(prefix_lens, torch.int32, "prefix_lens", (None,), dev)
    _status(dev_status, dev)
    B, N = prefix_of.numel(), prefix_lens.numel()
    need = int(_lib.lib().kvq_prefix_plan_size(B, N))
    if plan is not None:
        if (plan.batch, plan.num_prefixes) != (B, N):
            raise ValueError(f"the plan is for {plan.batch} sequences and {plan.num_prefixes} prefixes, not {B} and {N}")
        _check(plan.words, torch.int32, "plan.words", (max(need // 4, 1),), dev)
    with _on(dev, stream):
        if plan is None:
            plan = PrefixPlan(torch.empty(max(need // 4, 1), dtype=torch.int32, device=f"cuda:{dev}"), B, N)
        st = _lib.lib().kvq_prefix_plan(B, N, _ptr(prefix_of), _ptr(prefix_lens), _ptr(plan.words),
                                        plan.words.numel() * 4, _ptr(dev_status), _handle(dev))
    _lib.check(st, "kvq_prefix_plan")
    return plan


def kvq_prefix_find_workspace_size(pool: PagePool) -> int:
    return int(_lib.lib().kvq_prefix_find_workspace_size(byref(pool.struct)))


def kvq_prefix_find(pool: PagePool, seq_lens_before: torch.Tensor, prefix_of: torch.Tensor,
                    prefix_lens: torch.Tensor, prefix_table: torch.Tensor, tail_table: torch.Tensor,
                    tail_lens: torch.Tensor, min_tokens: int = 0, num_prefixes: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
                    stream=None) -> None:
    """The prefixes of at least min_tokens tokens that the pool's sequences
    share, at most N of them: prefix_of [B], prefix_lens [N], prefix_table
    [N][M], tail_table [B][M], tail_lens [B] (see kvq.h).  Then
    kvq_prefix_plan(prefix_of, prefix_lens), and kvq_prefix_attn with
    cache.with_table(prefix_table) and cache.with_table(tail_table)."""
    B, M = pool.block_table.shape
    dev = pool.ref_count.get_device()
    _check(seq_lens_before, torch.int32, "seq_lens_before", (B,), dev)
    _check(prefix_of, torch.int32, "prefix_of", (B,), dev)
    _check(prefix_lens, torch.int32, "prefix_lens", (None,), dev)
    N = prefix_lens.numel()
    _check(prefix_table, torch.int32, "prefix_table", (N, M), dev)
    _check(tail_table, torch.int32, "tail_table", (B, M), dev)
    _check(tail_lens, torch.int32, "tail_lens", (B,), dev)
    _optional(num_prefixes, torch.int32, "num_prefixes", (1,), dev)
    _status(dev_status, dev)
    pl = pool.struct
    with _on(dev, stream):
        need = int(_lib.lib().kvq_prefix_find_workspace_size(byref(pl)))
        workspace, ws_bytes = _bytes(workspace, dev, need, "workspace")
        st = _lib.lib().kvq_prefix_find(
            byref(pl), _ptr(seq_lens_before), int(min_tokens), N, _ptr(prefix_of), _ptr(prefix_lens),
            _ptr(prefix_table), _ptr(tail_table), _ptr(tail_lens), _ptr(num_prefixes), _ptr(workspace), ws_bytes,
            _ptr(dev_status), _handle(dev))
    _lib.check(st, "kvq_prefix_find")


def kvq_prefix_attn_workspace_size(prefix_desc, desc, num_prefixes, batch, num_new, num_q_heads, max_prefix_len,
                                   max_seq_len, prefix_splits=0, tail_splits=0) -> int:
    return int(_lib.lib().kvq_prefix_attn_workspace_size(
        None if prefix_desc is None else byref(prefix_desc), byref(desc), num_prefixes, batch, num_new, num_q_heads,
        int(max_prefix_len), int(max_seq_len), int(prefix_splits), int(tail_splits)))


def kvq_prefix_attn(prefix: KVCache | None, cache: KVCache, plan: PrefixPlan, q: torch.Tensor,
                    seq_lens_before: torch.Tensor, max_prefix_len: int, max_seq_len: int,
                    new_lens: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
                    prefix_splits: int = 0, tail_splits: int = 0, softmax_scale: float = 0.0,
                    stream=None) -> torch.Tensor:
    """Attention of the new tokens q [B][T][Hq][D] fp16 over each sequence's
    prefix (a sequence of `prefix`, by the plan) and its own tail in `cache`,
    positions [0, seq_lens_before[b] + t]; returns out.  Rows behind new_lens[b]
    keep what they held (an `out` made here starts as zeros)."""
    d = cache.desc
    _check(q, torch.float16, "q", (None, None, None, d.head_dim), None)
    B, T, Hq, _ = q.shape
    dev = q.get_device()
    _check(seq_lens_before, torch.int32, "seq_lens_before", (B,), dev)
    _optional(new_lens, torch.int32, "new_lens", (B,), dev)
    _same_cache_device(cache, dev)
    _batch(cache, B)
    N = plan.num_prefixes
    if plan.batch != B:
        raise ValueError(f"the plan is for {plan.batch} sequences, not {B}")
    _check(plan.words, torch.int32, "plan.words", (None,), dev)
    if N:
        if prefix is None:
            raise ValueError("the plan has prefixes, but there is no cache of them")
        _same_cache_device(prefix, dev)
        _batch(prefix, N)
    _status(dev_status, dev)
    if out is not None:
        _check(out, torch.float16, "out", q.shape, dev)
    pd = None if prefix is None else prefix.desc
    with _on(dev, stream):
        if out is None:
            out = _made_like(q, new_lens)
        need = 0 if workspace is not None else \
            kvq_prefix_attn_workspace_size(pd, d, N, B, T, Hq, max_prefix_len, max_seq_len, prefix_splits, tail_splits)
        workspace, ws_bytes = _bytes(workspace, dev, need, "workspace")
        words = plan.words
        st = _lib.lib().kvq_prefix_attn(
            None if pd is None else byref(pd), None if prefix is None else byref(prefix.ptrs), N, byref(d),
            byref(cache.ptrs), B, T, Hq, q.data_ptr(), seq_lens_before.data_ptr(), _ptr(new_lens), words.data_ptr(),
            words.numel() * 4, int(max_prefix_len), int(max_seq_len), int(prefix_splits), int(tail_splits),
            float(softmax_scale), out.data_ptr(), _ptr(workspace), ws_bytes, _ptr(dev_status), _handle(dev))
    if st:
        _lib.check(st, "kvq_prefix_attn")
    return out

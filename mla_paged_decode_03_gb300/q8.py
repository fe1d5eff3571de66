"""The 8-bit paged cache: a step's tables from request lengths, the quantising store and the
decode over it (C ABI: cp_step_tables, cp_store_q8, mla_decode_q8, mla_decode_shards_q8).

A step of a serving loop, on one rank of ``cp`` (each rank has its own pool and scales, all
share the block table):

    t = cp_step_tables(prev, ctx, new, block_table, free_pages, free_state, bs, N, cp, rank)
    cp_store_q8(kv_new, ctx, t.total_lens, block_table, cache, scales, cp, rank)
    out, lse = mla_decode_q8(q, cache, scales, block_table, t.seq_lens[0], t.total_lens,
                             N, cp, rank, scale)
    # next step: prev = t.total_lens, free_state = t.free_state

Marshalling and checks of arguments only, as in the package's other wrappers.  All tensors
must live on the current CUDA device.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import D_QK, D_V, _lib, _need

__all__ = ["Q8_GROUP", "StepTables", "cp_step_tables", "cp_store_q8", "mla_decode_q8",
           "mla_decode_shards_q8", "workspace_size_q8", "alloc_workspace_q8"]

Q8_GROUP = 16      # consecutive slots of a page that share a scale


class StepTables(NamedTuple):
    """What ``cp_step_tables`` gives besides the updated block table and ring."""
    total_lens: torch.Tensor               # int32 [B], global lengths after the step
    seq_lens: torch.Tensor                 # int32 [n_ranks, B], shard-local lengths
    positions: torch.Tensor                # int64 [B, N], -1 where there is no new token
    slots: torch.Tensor                    # int64 [n_ranks, B, N], PAD_SLOT_ID elsewhere
    free_state: torch.Tensor               # int32 [2], the ring's new {head, count}


# The checks below cost a call's latency (a small step's kernel takes a few microseconds), so
# each argument is tested by one expression; only a failing one is looked at again for its error.

def _here(t: torch.Tensor, name: str) -> None:
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device "
                         f"cuda:{torch.cuda.current_device()}")


def _refuse(t, name: str, dtype, shape) -> None:
    """The error of an argument that is not a contiguous ``dtype`` tensor of ``shape`` on the
    current device."""
    _need(t, name, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    _here(t, name)
    raise ValueError(f"{name} is not usable")


def _check(t, name: str, dtype, shape: tuple, dev: int) -> int:
    """Checks a tensor argument; returns its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        _refuse(t, name, dtype, shape)
    return t.data_ptr()


def _table(t, rows: int, dev: int) -> int:
    """Checks a block table; returns its row stride (a single row's is its width at least)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.dim() == 2 and t.is_cuda):
        raise TypeError("block_table must be a 2-D int32 CUDA tensor")
    n, width = t.shape
    if n != rows or (width > 1 and t.stride(1) != 1):
        raise ValueError(f"block_table must be [{rows}, max_blocks] with contiguous rows, got "
                         f"{list(t.shape)} with strides {list(t.stride())}")
    if t.get_device() != dev:
        _here(t, "block_table")
    return max(t.stride(0), width) if rows <= 1 else t.stride(0)


def _cache(kv_cache, kv_scales, dev: int) -> Tuple[int, int]:
    """Checks the cache and its scales; returns (num_blocks, block_size)."""
    _need(kv_cache, "kv_cache", torch.float8_e4m3fn, 3)
    nb, bs, d = kv_cache.shape
    if d != D_QK or bs % Q8_GROUP:
        raise ValueError(f"kv_cache must be [num_blocks, block_size, {D_QK}] with block_size a "
                         f"multiple of {Q8_GROUP}, got {list(kv_cache.shape)}")
    if kv_cache.get_device() != dev:
        _here(kv_cache, "kv_cache")
    _check(kv_scales, "kv_scales", torch.float32, (nb, bs // Q8_GROUP), dev)
    return nb, bs


def _on(stream, call, *args):
    """``call`` with ``stream`` as the current stream, so that what it allocates (outputs, a
    workspace) belongs to that stream and is not handed out again while its kernels run."""
    dev = torch.cuda.current_device()
    if stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, not on the current device cuda:{dev}")
    with torch.cuda.stream(stream):
        return call(*args)


def _stream(dev: int) -> int:
    """The current stream's handle."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _device() -> int:
    return torch.cuda.current_device()


def cp_step_tables(prev_lens: torch.Tensor, ctx_lens: torch.Tensor, new_lens: torch.Tensor,
                   block_table: torch.Tensor, free_pages: torch.Tensor, free_state: torch.Tensor,
                   block_size: int, N: int, cp_size: int = 1, cp_rank: int = 0, n_ranks: int = 1,
                   interleave: int = 1, total_lens: Optional[torch.Tensor] = None,
                   seq_lens: Optional[torch.Tensor] = None,
                   positions: Optional[torch.Tensor] = None,
                   slots: Optional[torch.Tensor] = None,
                   free_state_out: Optional[torch.Tensor] = None, stream=None) -> StepTables:
    """A step's tables from request lengths, for ranks cp_rank .. cp_rank + n_ranks - 1.

    prev_lens [B] int32: lengths the pages in ``block_table`` were taken for (the last step's
    total_lens, 0 for a new request); ctx_lens [B]: tokens in the cache now (0 when a request
    has finished); new_lens [B]: new tokens, at most N.  Pages that prev_lens held and the
    new lengths do not need go to the end of ``free_pages`` (a ring, free_state = {head,
    count}); missing ones come from its head, in the order of the requests.  A request whose
    pages do not fit the table or the ring's supply gets none of its new tokens (total_lens
    stays at its cached length, its positions are -1) and device_status() reports it.
    ``block_table`` and ``free_pages`` are updated in place; the outputs must not share memory
    with the inputs."""
    if stream is not None:
        return _on(stream, cp_step_tables, prev_lens, ctx_lens, new_lens, block_table, free_pages, free_state,
                   block_size, N, cp_size, cp_rank, n_ranks, interleave, total_lens, seq_lens, positions,
                   slots, free_state_out)
    if not isinstance(prev_lens, torch.Tensor) or prev_lens.dim() != 1:
        raise TypeError("prev_lens must be a 1-D int32 CUDA tensor")
    if not prev_lens.is_cuda:
        raise ValueError("prev_lens must be a CUDA tensor")
    dev = _device()
    B = prev_lens.shape[0]
    i32, i64 = torch.int32, torch.int64
    lens = (_check(prev_lens, "prev_lens", i32, (B,), dev), _check(ctx_lens, "ctx_lens", i32, (B,), dev),
            _check(new_lens, "new_lens", i32, (B,), dev))
    stride = _table(block_table, B, dev)
    _need(free_pages, "free_pages", i32, 1)
    if free_pages.get_device() != dev:
        _here(free_pages, "free_pages")
    state = _check(free_state, "free_state", i32, (2,), dev)
    if n_ranks < 1 or N < 0:
        raise ValueError(f"need n_ranks >= 1 and N >= 0, got {n_ranks} and {N}")
    device = prev_lens.device
    # (outputs made here need no check; a user who cares for the last microseconds passes them)
    if total_lens is None:
        total_lens = torch.empty_like(prev_lens)
        total = total_lens.data_ptr()
    else:
        total = _check(total_lens, "total_lens", i32, (B,), dev)
    if seq_lens is None:
        seq_lens = torch.empty((n_ranks, B), dtype=i32, device=device)
        seq = seq_lens.data_ptr()
    else:
        seq = _check(seq_lens, "seq_lens", i32, (n_ranks, B), dev)
    if free_state_out is None:
        free_state_out = torch.empty_like(free_state)
        state_out = free_state_out.data_ptr()
    else:
        state_out = _check(free_state_out, "free_state_out", i32, (2,), dev)
    if positions is None:
        positions = torch.empty((B, N), dtype=i64, device=device)
        pos = positions.data_ptr()
    else:
        pos = _check(positions, "positions", i64, (B, N), dev)
    if slots is None:
        slots = torch.empty((n_ranks, B, N), dtype=i64, device=device)
        slot = slots.data_ptr()
    else:
        slot = _check(slots, "slots", i64, (n_ranks, B, N), dev)
    rc = _lib.load().cp_step_tables(
        *lens, B, N, block_table.data_ptr(), stride, block_table.shape[1], free_pages.data_ptr(),
        free_pages.shape[0], state, state_out, block_size, cp_size, cp_rank, n_ranks, interleave,
        total, seq, pos, slot, _stream(dev))
    if rc:
        _lib.check(rc)
    return StepTables(total_lens, seq_lens, positions, slots, free_state_out)


def cp_store_q8(kv_new: torch.Tensor, ctx_lens: torch.Tensor, total_lens: torch.Tensor,
                block_table: torch.Tensor, kv_cache: torch.Tensor, kv_scales: torch.Tensor,
                cp_size: int = 1, cp_rank: int = 0, interleave: int = 1,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Quantises the new rows kv_new [B, N, 576] bf16 of positions ctx_lens[b] ..
    total_lens[b] - 1 that rank ``cp_rank`` owns into kv_cache [num_blocks, block_size, 576]
    float8_e4m3fn and kv_scales [num_blocks, block_size / 16] float32 (a power of two for
    each 16 slots; a partly filled group's scale only grows).  Returns (kv_cache, kv_scales)."""
    if stream is not None:
        return _on(stream, cp_store_q8, kv_new, ctx_lens, total_lens, block_table, kv_cache, kv_scales, cp_size,
                   cp_rank, interleave)
    _need(kv_new, "kv_new", torch.bfloat16, 3)
    dev = _device()
    B, N, d = kv_new.shape
    if d != D_QK:
        raise ValueError(f"kv_new must be [B, N, {D_QK}], got {list(kv_new.shape)}")
    if kv_new.get_device() != dev:
        _here(kv_new, "kv_new")
    stride = _table(block_table, B, dev)
    nb, bs = _cache(kv_cache, kv_scales, dev)
    rc = _lib.load().cp_store_q8(
        kv_new.data_ptr(), _check(ctx_lens, "ctx_lens", torch.int32, (B,), dev),
        _check(total_lens, "total_lens", torch.int32, (B,), dev), block_table.data_ptr(), stride,
        block_table.shape[1], B, N, bs, cp_size, cp_rank, interleave, kv_cache.data_ptr(),
        kv_scales.data_ptr(), nb, _stream(dev))
    if rc:
        _lib.check(rc)
    return kv_cache, kv_scales


def workspace_size_q8(B: int, H: int, q_len: int, device=None) -> int:
    """Workspace bytes the decode over the 8-bit cache can use for split-KV on ``device`` (for
    the shards call: with B = n_shards * B)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    return int(_lib.load().mla_decode_q8_workspace_size(B, H, q_len, sms))


def alloc_workspace_q8(B: int, H: int, q_len: int, device=None) -> torch.Tensor:
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return torch.empty(max(workspace_size_q8(B, H, q_len, dev), 256), dtype=torch.uint8, device=dev)


def _decode(shards, q, kv_cache, kv_scales, block_table, seq_lens, gseq, q_len, cp, rank, scale, out,
            lse, lse_base_e, workspace, return_lse, stream, causal, interleave):
    if stream is not None:
        return _on(stream, _decode, shards, q, kv_cache, kv_scales, block_table, seq_lens, gseq, q_len, cp, rank,
                   scale, out, lse, lse_base_e, workspace, return_lse, None, causal, interleave)
    if isinstance(q, torch.Tensor) and q.dim() == 3 and q_len >= 1 and q.shape[0] % q_len == 0:
        q = q.view(-1, q_len, q.shape[1], q.shape[2])
    _need(q, "q", torch.bfloat16, 4)
    dev = _device()
    B, ql, H, d = q.shape
    if ql != q_len or d != D_QK:
        raise ValueError(f"q must be [B, q_len={q_len}, H, {D_QK}], got {list(q.shape)}")
    if q.get_device() != dev:
        _here(q, "q")
    nb, bs = _cache(kv_cache, kv_scales, dev)
    n = shards if shards is not None else 1
    if n < 1:
        raise ValueError(f"need n_shards >= 1, got {n}")
    stride = _table(block_table, n * B, dev)
    seq = _check(seq_lens, "seq_lens", torch.int32, (n * B,), dev)
    g = None if gseq is None else _check(gseq, "causal_seqlens_global", torch.int32, (B,), dev)
    rows = (B * q_len, H) if shards is None else (n, B * q_len, H)
    if out is None:
        out = torch.empty((*rows, D_V), dtype=torch.bfloat16, device=q.device)
        o = out.data_ptr()
    else:
        o = _check(out, "out", torch.bfloat16, (*rows, D_V), dev)
    if lse is not None:
        l = _check(lse, "lse", torch.float32, rows, dev)
    elif return_lse:
        lse = torch.empty(rows, dtype=torch.float32, device=q.device)
        l = lse.data_ptr()
    else:
        l = None
    if workspace is None:
        workspace = alloc_workspace_q8(n * B, H, q_len, q.device)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _need(workspace, "workspace", workspace.dtype)
        _here(workspace, "workspace")
    lib = _lib.load()
    head = (q.data_ptr(), kv_cache.data_ptr(), kv_scales.data_ptr(), block_table.data_ptr(), stride, seq, g,
            B, H, q_len, 1 if causal else 0, bs, nb, block_table.shape[1])
    tail = (int(interleave), float(scale), o, l, 1 if lse_base_e else 0, workspace.data_ptr(), workspace.nbytes,
            _stream(dev))
    if shards is not None:
        rc = lib.mla_decode_shards_q8(*head, n, *tail)
    else:
        rc = lib.mla_decode_q8(*head, cp, rank, *tail)
    if rc:
        _lib.check(rc)
    return out, lse


def mla_decode_q8(q: torch.Tensor, kv_cache: torch.Tensor, kv_scales: torch.Tensor,
                  block_table: torch.Tensor, seq_lens: torch.Tensor,
                  causal_seqlens_global: Optional[torch.Tensor], q_len: int, cp_world: int,
                  cp_rank: int, scale: float, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, lse_base_e: bool = True,
                  workspace: Optional[torch.Tensor] = None, return_lse: bool = True, stream=None,
                  causal: bool = True,
                  interleave: int = 1) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``mla_decode`` over the 8-bit cache: kv_cache [num_blocks, block_size, 576]
    float8_e4m3fn times kv_scales [num_blocks, block_size / 16] float32; the other arguments
    and the results (out [B*q_len, H, 512] bf16, lse [B*q_len, H] float32) as there."""
    return _decode(None, q, kv_cache, kv_scales, block_table, seq_lens, causal_seqlens_global, q_len,
                   cp_world, cp_rank, scale, out, lse, lse_base_e, workspace, return_lse, stream, causal,
                   interleave)


def mla_decode_shards_q8(q: torch.Tensor, kv_cache: torch.Tensor, kv_scales: torch.Tensor,
                         block_table: torch.Tensor, seq_lens: torch.Tensor,
                         causal_seqlens_global: Optional[torch.Tensor], q_len: int, n_shards: int,
                         scale: float, out: Optional[torch.Tensor] = None,
                         lse: Optional[torch.Tensor] = None, lse_base_e: bool = True,
                         workspace: Optional[torch.Tensor] = None, stream=None,
                         causal: bool = True,
                         interleave: int = 1) -> Tuple[torch.Tensor, torch.Tensor]:
    """``mla_decode_shards`` over the 8-bit cache (all shards' pages in one kv_cache and
    kv_scales; shard-major block_table [n_shards*B, max_blocks] and seq_lens [n_shards*B])."""
    return _decode(n_shards, q, kv_cache, kv_scales, block_table, seq_lens, causal_seqlens_global, q_len,
                   None, None, scale, out, lse, lse_base_e, workspace, True, stream, causal, interleave)

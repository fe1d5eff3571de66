"""The 8-bit paged cache: a step's tables from request lengths, the quantising store and the
decode over it (C ABI: cp_step_tables, cp_store_q8, mla_decode_q8, mla_decode_shards_q8).

A step of a serving loop, on one rank of ``cp`` (each rank has its own pool and scales, all
share the block table):

    t = cp_step_tables(prev, ctx, new, block_table, free_pages, free_state, bs, N, cp, rank)
    cp_store_q8(kv_new, ctx, t.total_lens, block_table, cache, scales, cp, rank)
    out, lse = mla_decode_q8(q, cache, scales, block_table, t.seq_lens[0], t.total_lens,
                             N, cp, rank, scale)
    # next step: prev = t.total_lens, free_state = t.free_state

Marshalling and checks of arguments only, as in the package's other wrappers, but in a native
binding (csrc/q8_binding.cpp): these calls' smallest kernels take 3 to 12 us.  All tensors must
live on the current CUDA device.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib

__all__ = ["Q8_GROUP", "StepTables", "cp_step_tables", "cp_store_q8", "mla_decode_q8",
           "mla_decode_shards_q8", "workspace_size_q8", "alloc_workspace_q8"]

Q8_GROUP = 16      # consecutive slots of a page that share a scale


class StepTables(NamedTuple):
    """What ``cp_step_tables`` gives besides the updated block table and ring (new outputs of one
    type share an allocation)."""
    total_lens: torch.Tensor               # int32 [B], global lengths after the step
    seq_lens: torch.Tensor                 # int32 [n_ranks, B], shard-local lengths
    positions: torch.Tensor                # int64 [B, N], -1 where there is no new token
    slots: torch.Tensor                    # int64 [n_ranks, B, N], PAD_SLOT_ID elsewhere
    free_state: torch.Tensor               # int32 [2], the ring's new {head, count}


def _on(stream, call, *args):
    """``call`` with ``stream`` as the current stream, so that what it allocates (outputs, a
    workspace) belongs to that stream and is not handed out again while its kernels run."""
    dev = torch.cuda.current_device()
    if stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, not on the current device cuda:{dev}")
    with torch.cuda.stream(stream):
        return call(*args)


def _native():
    """The binding (checks of arguments, outputs, the current stream)."""
    return _lib.load_q8(StepTables)


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
    return _native().step_tables(prev_lens, ctx_lens, new_lens, block_table, free_pages, free_state, block_size, N,
                                 cp_size, cp_rank, n_ranks, interleave, total_lens, seq_lens, positions, slots,
                                 free_state_out)


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
    return _native().store(kv_new, ctx_lens, total_lens, block_table, kv_cache, kv_scales, cp_size, cp_rank,
                           interleave)


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
    return _native().decode(shards, q, kv_cache, kv_scales, block_table, seq_lens, gseq, q_len, cp, rank, scale, out,
                            lse, lse_base_e, workspace, return_lse, causal, interleave)


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

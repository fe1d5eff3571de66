"""Prompt processing over the paged latent cache: rotary positions, the append of new tokens, the
heads' keys and values, and the attention of chunks of new tokens (C ABI: mla_rope, cp_rope_store,
mla_expand, mla_prefill).

One layer of a step whose requests bring chunks of any and different lengths (cp_step_tables gives
positions and lengths).  The append takes the new tokens as [B, N, ...], padded to the longest
chunk, its padding at position -1 as the step's positions have it; the queries, and what belongs to
them, hold the requests' new tokens one after another without padding:

    freqs = rope_freqs(theta, "yarn", factor=40.0, original_max_position=4096)   # once
    t = cp_step_tables(prev, ctx, new, block_table, free_pages, free_state, bs, N, cp, rank)
    cp_rope_store(latent, k_rope, t.positions, freqs, block_table, kv_cache, cp, rank)
    positions = t.positions[t.positions >= 0]       # (the host waits; with its own lengths it need not)
    mla_rope(q[..., 128:], positions, freqs, out=q[..., 128:])
    seq_lens = t.seq_lens[0]                        # kv_starts = cumsum(seq_lens) - seq_lens
    k, v, kr = mla_expand(kv_cache, block_table, seq_lens, kv_starts, w_kv, S)
    out, lse = mla_prefill(q, k, kr, v, cu_q_lens, kv_starts, seq_lens, t.total_lens, scale, cp, rank)

Tokens without padding are appended as T requests of one token each, latent [T, 1, 512] and positions
[T, 1], with the table's row of each token's request: block_table[request_of_token].

Single tokens beside the chunks may go this way too; where all requests bring one (or a few), the
absorbed form (mla_rope into the absorbed queries, cp_rope_store, mla_decode) reads far less.
Shards' results are joined by lse_merge.  Marshalling and checks of arguments only, in the native
binding (csrc/q8_binding.cpp).  All tensors must live on the current CUDA device.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from . import _lib
from .q8 import _native, _on

__all__ = ["rope_freqs", "mla_rope", "cp_rope_store", "mla_expand", "mla_prefill",
           "workspace_size_prefill", "alloc_workspace_prefill", "D_ROPE", "D_NOPE", "D_HEAD_V"]

D_ROPE, D_NOPE, D_HEAD_V = 64, 128, 128      # a head's rope dims, other key dims, value dims


def rope_freqs(theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_max_position: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
               device=None) -> torch.Tensor:
    """The rotation's 32 frequencies, as mla_rope and cp_rope_store take them: int64 [32], turns a
    position in units of 2^-64.  Pair i turns by theta^(-i/32) radians a position, and

      "none"    as it is;
      "linear"  divided by ``factor`` (positions interpolated);
      "ntk"     with theta grown so that the slowest pair is stretched by ``factor``;
      "yarn"    pairs that turn more than ``beta_fast`` times over ``original_max_position``
                positions as they are, those that turn less than ``beta_slow`` times divided by
                ``factor``, a linear ramp over the pairs between (the values' factor that goes with
                it, 0.1 ln(factor) + 1 by itself, is the calls' ``mscale``)."""
    if not (math.isfinite(theta) and theta > 1.0) or not (math.isfinite(factor) and factor > 0.0):
        raise ValueError(f"need theta > 1 and factor > 0, got {theta} and {factor}")
    half = D_ROPE // 2
    i = torch.arange(half, dtype=torch.float64)
    if scaling == "ntk":
        theta = theta * factor ** (half / (half - 1.0))
        if theta <= 1.0:
            raise ValueError(f"factor {factor} makes theta {theta}")
    f = float(theta) ** (-i / half)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if original_max_position < 1 or not beta_fast > beta_slow > 0.0:
            raise ValueError("yarn needs original_max_position >= 1 and beta_fast > beta_slow > 0")
        lo, hi = (half * math.log(original_max_position / (turns * 2.0 * math.pi)) / math.log(theta)
                  for turns in (beta_fast, beta_slow))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), D_ROPE - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        f = f / factor * ramp + f * (1.0 - ramp)
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    turns = [int(round(x / (2.0 * math.pi) * 2.0 ** 64)) % (1 << 64) for x in f.tolist()]
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=dev)


def mla_rope(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor,
             out: Optional[torch.Tensor] = None, half: bool = False, mscale: float = 1.0,
             stream=None) -> torch.Tensor:
    """Turns x [T, H, 64] (or [B, N, H, 64]) bf16, the rope part of queries (a view of their last
    dims, say: 64 contiguous dims, other strides multiples of 8), by positions [T] ([B, N]) int64.
    ``freqs``: see rope_freqs.  ``half``: pairs are (i, i+32), else (2i, 2i+1).  The result, times
    ``mscale``, goes to ``out`` (of x's shape, strides of its own; x itself for in place), or to a
    new tensor; tokens at negative positions are left as they were there.  Returns out."""
    if stream is not None:
        return _on(stream, mla_rope, x, positions, freqs, out, half, mscale)
    return _native().rope(x, positions, freqs, out, half, mscale)


def cp_rope_store(latent: torch.Tensor, k_rope: torch.Tensor, positions: torch.Tensor,
                  freqs: torch.Tensor, block_table: torch.Tensor, kv_cache: torch.Tensor,
                  cp_size: int = 1, cp_rank: int = 0, interleave: int = 1, half: bool = False,
                  mscale: float = 1.0, slots: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Writes new tokens, latent [B, N, 512] and k_rope [B, N, 64] bf16 (parts of one tensor, or
    two), into kv_cache [num_blocks, block_size, 576] bf16 at the slots that ``cp_local_slot`` gives
    positions [B, N] int64 on rank ``cp_rank``, k_rope turned by its position as mla_rope does it.
    Positions the rank does not own, and negative ones, write nothing.  ``slots`` (int64 [B, N], may
    be None) receives the slots.  Returns kv_cache."""
    if stream is not None:
        return _on(stream, cp_rope_store, latent, k_rope, positions, freqs, block_table, kv_cache, cp_size,
                   cp_rank, interleave, half, mscale, slots)
    return _native().rope_store(latent, k_rope, positions, freqs, block_table, kv_cache, cp_size, cp_rank,
                                interleave, half, mscale, slots)


def mla_expand(kv_cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
               kv_starts: torch.Tensor, w_kv: torch.Tensor, S: int,
               kv_scales: Optional[torch.Tensor] = None, kv: Optional[torch.Tensor] = None,
               k_rope: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Keys and values of all heads from the cache: local key l of request b (block_table [B,
    max_blocks], seq_lens [B] int32) becomes row kv_starts[b] + l of

      k_nope [S, H, 128], v [S, H, 128]   w_kv[h, 0:128] and w_kv[h, 128:256] times the latent part,
      k_rope [S, 64]                      the rope part.

    kv_cache [num_blocks, block_size, 576] bf16, or float8_e4m3fn with kv_scales [num_blocks,
    block_size / 16]; w_kv [H, 256, 512] bf16; kv_starts [B] int32 in order and apart.  ``kv`` bf16
    [H, S, 256] and ``k_rope`` receive the results, else new tensors do; k_nope and v are views of
    kv.  Rows of no request are left as they were."""
    if stream is not None:
        return _on(stream, mla_expand, kv_cache, block_table, seq_lens, kv_starts, w_kv, S, kv_scales, kv, k_rope)
    return _native().expand(kv_cache, kv_scales, block_table, seq_lens, kv_starts, w_kv, S, kv, k_rope)


def workspace_size_prefill(T: int, B: int, H: int, S: int, device=None) -> int:
    """Workspace bytes mla_prefill can use on ``device`` to split the keys of few query rows."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    return int(_lib.load().mla_prefill_workspace_size(T, B, H, S, sms))


def alloc_workspace_prefill(T: int, B: int, H: int, S: int, device=None) -> torch.Tensor:
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return torch.empty(max(workspace_size_prefill(T, B, H, S, dev), 256), dtype=torch.uint8, device=dev)


def mla_prefill(q: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor,
                cu_q_lens: torch.Tensor, kv_starts: torch.Tensor, seq_lens: torch.Tensor,
                causal_seqlens_global: Optional[torch.Tensor], scale: float, cp_world: int = 1,
                cp_rank: int = 0, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, lse_base_e: bool = True,
                workspace: Optional[torch.Tensor] = None, return_lse: bool = True, stream=None,
                causal: bool = True,
                interleave: int = 1) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of chunks of new tokens over expanded keys and values (those of mla_expand).

    q [T, H, 192] bf16 (128 dims, then 64 rotated ones): request b's rows are cu_q_lens[b] ..
    cu_q_lens[b+1] - 1 (int32 [B+1]); k_nope [S, H, 128], k_rope [S, 64], v [S, H, 128] bf16: its
    seq_lens[b] local keys are the rows from kv_starts[b] on (int32 [B]).  Their last dims are
    contiguous, other strides multiples of 8.  causal_seqlens_global [B] int32: global lengths with
    the new tokens (None when cp_world == 1, then seq_lens, or when the block is not causal);
    ``causal``, ``cp_world``, ``cp_rank``, ``interleave``, ``lse_base_e`` as mla_decode.  Returns out
    [T, H, 128] bf16 and lse [T, H] float32 (None with return_lse False and no lse); rows of no
    request are left as they were."""
    if stream is not None:
        return _on(stream, mla_prefill, q, k_nope, k_rope, v, cu_q_lens, kv_starts, seq_lens,
                   causal_seqlens_global, scale, cp_world, cp_rank, out, lse, lse_base_e, workspace, return_lse,
                   None, causal, interleave)
    return _native().prefill(q, k_nope, k_rope, v, cu_q_lens, kv_starts, seq_lens, causal_seqlens_global, scale,
                             cp_world, cp_rank, out, lse, lse_base_e, workspace, return_lse, causal, interleave)

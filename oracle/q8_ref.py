"""CPU oracle for the 8-bit paged cache: a step's tables from request lengths, the quantising
store, and the float64 keys that the stored values stand for.

TEST INFRASTRUCTURE, like ``oracle.mla_ref``: plain definitions, page by page and row by row,
sharing no code with the CUDA library.  The decode over the 8-bit cache is
``mla_ref.ref_mla_decode`` over ``ref_dequantised``.
"""
from __future__ import annotations

import math

import numpy as np

from .mla_ref import PAD_SLOT_ID, ref_cp_local_slot, ref_owned_positions

GROUP = 16
E4M3_MAX = 448.0
SCALE_MIN, SCALE_MAX = 2.0 ** -32, 2.0 ** 64


def ref_e4m3(x) -> np.ndarray:
    """Values rounded to e4m3 (4 significant bits, exponents from -6, subnormals in steps of
    2^-9), to nearest even, beyond +-448 saturated; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(a > 0, np.floor(np.log2(np.where(a > 0, a, 1.0))), -6)
    step = 2.0 ** (np.maximum(np.nan_to_num(e, nan=0.0, posinf=8.0), -6) - 3)
    y = np.rint(x / step) * step
    return np.where(np.isnan(x), np.nan, np.clip(y, -E4M3_MAX, E4M3_MAX))


def ref_scale(amax: float) -> float:
    """Smallest power of two s with amax <= 448 s, inside the scales' range."""
    if amax == 0:
        return SCALE_MIN
    s = 2.0 ** math.floor(math.log2(amax / E4M3_MAX))
    while amax > E4M3_MAX * s:
        s *= 2
    return min(max(s, SCALE_MIN), SCALE_MAX)


def ref_step_tables(prev, ctx, new, table, ring, state, block_size, N, cp, ranks, interleave=1):
    """cp_step_tables, request after request.  Returns (total, seq [R, B], positions, slots
    [R, B, N], table, ring, state) without changing the arguments."""
    table = np.array(table, dtype=np.int64)
    ring = [int(x) for x in ring]
    B, width = table.shape
    vbs, cap = block_size * cp, len(ring)
    head, count = (int(x) for x in state)
    need = lambda x: -(-int(x) // vbs)                                   # noqa: E731
    queue = [ring[(head + k) % cap] for k in range(count)]               # free pages in order
    total = np.zeros(B, np.int64)
    granted = np.zeros(B, bool)
    asked = 0
    back = []
    for b in range(B):
        held, want = need(prev[b]), need(int(ctx[b]) + int(new[b]))
        fits = want <= width
        take = max(0, want - held) if fits else 0
        asked += take
        granted[b] = fits and (take == 0 or asked <= count)
        total[b] = int(ctx[b]) + int(new[b]) if granted[b] else min(int(ctx[b]), int(prev[b]))
        back += [int(x) for x in table[b, need(total[b]):held]]
        if granted[b]:
            for j in range(held, held + take):
                table[b, j] = queue.pop(0)
    taken = count - len(queue)
    for k, page in enumerate(back):
        ring[(head + count + k) % cap] = page
    new_state = ((head + taken) % cap, count - taken + len(back))
    pos = np.full((B, N), -1, np.int64)
    for b in range(B):
        n = int(new[b]) if granted[b] else 0
        pos[b, :n] = int(ctx[b]) + np.arange(n)
    seq = np.array([[len(ref_owned_positions(int(t), cp, r, interleave)) for t in total]
                    for r in ranks], dtype=np.int64).reshape(len(ranks), B)
    slots = (np.stack([ref_cp_local_slot(pos, table, block_size, cp, r, interleave) for r in ranks])
             if B else np.zeros((len(ranks), 0, N), np.int64))
    return total, seq, pos, slots, table, np.array(ring), np.array(new_state)


def ref_store_q8(rows, ctx, total, table, cache, scales, cp, rank, interleave=1):
    """cp_store_q8 on float64 copies of the cache's e4m3 values [num_blocks, bs, 576] and its
    scales [num_blocks, bs / 16]; returns both."""
    cache = np.array(cache, dtype=np.float64)
    scales = np.array(scales, dtype=np.float64)
    bs, d = cache.shape[1:]
    flat, fs = cache.reshape(-1, d), scales.reshape(-1)
    rows = np.asarray(rows, dtype=np.float64)
    for b in range(rows.shape[0]):
        pos = np.arange(int(ctx[b]), int(total[b]), dtype=np.int64)
        slots = ref_cp_local_slot(pos.reshape(1, -1), np.asarray(table)[b:b + 1], bs, cp, rank,
                                  interleave)[0]
        mine = np.nonzero(slots != PAD_SLOT_ID)[0]
        for g in sorted(set(int(s) // GROUP for s in slots[mine])):
            at = [n for n in mine if int(slots[n]) // GROUP == g]
            x = rows[b, at]
            fin = np.abs(x[np.isfinite(x)])
            s = ref_scale(float(fin.max()) if fin.size else 0.0)
            first = int(min(slots[at])) - g * GROUP
            if first > 0:
                old = float(fs[g])
                s = max(s, old)
                if s != old:
                    flat[g * GROUP:g * GROUP + first] = ref_e4m3(flat[g * GROUP:g * GROUP + first] * (old / s))
            flat[slots[at]] = ref_e4m3(np.where(np.isfinite(x), x, np.nan) / s)
            fs[g] = s
    return cache, scales


def ref_dequantised(cache, scales) -> np.ndarray:
    """The rows that an e4m3 cache and its scales stand for, in float64."""
    c = np.asarray(cache, dtype=np.float64)
    return c * np.repeat(np.asarray(scales, dtype=np.float64), GROUP, axis=1)[..., None]

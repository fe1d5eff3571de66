"""Float64 oracle of prompt processing: rotary positions, the append, the expanded keys and values,
and the attention of chunks of new tokens.  Plain NumPy, one row at a time where that is plainest."""
from __future__ import annotations

import math

import numpy as np

import oracle.mla_ref as R


def ref_angles(pos: int, freqs) -> np.ndarray:
    """Angles [32] in radians: the exact product of the position and the 64-bit fraction of a turn."""
    return np.array([2.0 * math.pi * ((int(pos) * (int(f) % (1 << 64))) % (1 << 64)) / 2.0 ** 64
                     for f in freqs])


def ref_rope_row(x, pos: int, freqs, half: bool, mscale: float) -> np.ndarray:
    """x [..., 64] turned by one position."""
    x = np.asarray(x, dtype=np.float64)
    a = ref_angles(pos, freqs)
    y = np.empty_like(x)
    for i in range(32):
        e, o = (i, i + 32) if half else (2 * i, 2 * i + 1)
        y[..., e] = mscale * (x[..., e] * math.cos(a[i]) - x[..., o] * math.sin(a[i]))
        y[..., o] = mscale * (x[..., e] * math.sin(a[i]) + x[..., o] * math.cos(a[i]))
    return y


def ref_rope(x, positions, freqs, half, mscale, out) -> np.ndarray:
    """x [T, H, 64]; tokens at negative positions keep what `out` holds."""
    y = np.array(out, dtype=np.float64)
    for t, p in enumerate(np.asarray(positions)):
        if p >= 0:
            y[t] = ref_rope_row(x[t], int(p), freqs, half, mscale)
    return y


def ref_rope_store(latent, k_rope, positions, freqs, table, cache, cp, rank, il, half, mscale):
    """The updated cache [num_blocks, bs, 576], the rows that were written (flat slots) and the slots."""
    cache = np.array(cache, dtype=np.float64)
    nb, bs, d = cache.shape
    positions = np.asarray(positions)
    slots = np.asarray(R.ref_cp_local_slot(positions, table, bs, cp, rank, il))
    written = []
    flat = cache.reshape(-1, d)
    for b, n in np.argwhere(slots >= 0):
        s = int(slots[b, n])
        if s >= nb * bs:
            continue
        flat[s, :512] = latent[b, n]
        flat[s, 512:] = ref_rope_row(k_rope[b, n], int(positions[b, n]), freqs, half, mscale)
        written.append(s)
    return cache, written, slots


def ref_expand(rows_of, seq_lens, starts, w, S):
    """rows_of(b) -> [seq_lens[b], 576]: kv [H, S, 256], k_rope [S, 64], their sums of magnitudes, and
    which rows are some request's."""
    w = np.asarray(w, dtype=np.float64)
    kv, mag = np.zeros((w.shape[0], S, 256)), np.zeros((w.shape[0], S, 256))
    kr, mine = np.zeros((S, 64)), np.zeros(S, dtype=bool)
    for b, n in enumerate(seq_lens):
        if n == 0:
            continue
        c = np.asarray(rows_of(b), dtype=np.float64)[:n]
        at = slice(starts[b], starts[b] + n)
        kv[:, at] = np.einsum("sc,hdc->hsd", c[:, :512], w)
        mag[:, at] = np.einsum("sc,hdc->hsd", np.abs(c[:, :512]), np.abs(w))
        kr[at] = c[:, 512:]
        mine[at] = True
    return kv, kr, mag, mine


def ref_seen(G, n, have, cp, rank, il, causal):
    """Keys that each of a chunk's n rows sees."""
    if not causal:
        return [have] * n
    return [min(have, int(R.ref_local_len(max(0, G - (n - 1 - i)), cp, rank, il))) for i in range(n)]


def ref_prefill(q, k, kr, v, cu, starts, seq_lens, G, scale, cp, rank, il, causal):
    """out [T, H, 128], lse [T, H] (natural), A = sum_l w_l |v_l| and D = max_l scale sum_d |q_d k_d|
    over a row's keys, and which rows are some request's."""
    q, k, kr, v = (np.asarray(x, dtype=np.float64) for x in (q, k, kr, v))
    T, H, _ = q.shape
    out, A = np.zeros((T, H, 128)), np.zeros((T, H, 128))
    lse, D = np.full((T, H), -np.inf), np.zeros((T, H))
    mine = np.zeros(T, dtype=bool)
    for b in range(len(seq_lens)):
        n, have = cu[b + 1] - cu[b], seq_lens[b]
        mine[cu[b]:cu[b + 1]] = True
        at = slice(starts[b], starts[b] + have)
        for i, L in enumerate(ref_seen(G[b], n, have, cp, rank, il, causal)):
            if L == 0:
                continue
            t = cu[b] + i
            for h in range(H):
                key = np.concatenate([k[at][:L, h], kr[at][:L]], 1)
                s = scale * (key @ q[t, h])
                D[t, h] = scale * (np.abs(key) @ np.abs(q[t, h])).max()
                m = s.max()
                w = np.exp(s - m)
                lse[t, h] = m + math.log(w.sum())
                w /= w.sum()
                out[t, h] = w @ v[at][:L, h]
                A[t, h] = w @ np.abs(v[at][:L, h])
    return out, lse, A, D, mine

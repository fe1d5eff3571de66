"""Prompt processing at the edges that test_gpu_prompt.py leaves out; the tolerances are those of its head."""
import math

import numpy as np
import pytest
import torch

import mla_paged_decode_03_gb300 as M
import oracle.mla_ref as R
import oracle.prompt_ref as P
from test_gpu_prompt import (BAD_STEP, BF, DEV, FREQS, SCALE, U, call, check, gen, i32, i64, n64, paged, pair_sum,
                             prefill_case, randn, starts_of, within)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    M.device_status()
    yield


# =============================================================================================
# attention of chunks
# =============================================================================================
def alone(d, b, rows):
    """The call of request b by itself, with the rows that it has in another one's cu_q_lens."""
    return dict(d, q=d["q"][rows], cu=[0, rows.stop - rows.start], starts=[d["starts"][b]], lens=[d["lens"][b]], G=[d["G"][b]],
                T=rows.stop - rows.start)


# cu_q_lens and which requests are in order: {request: its rows}
BAD_ROWS = [
    ([0, 30, 20, 90], {0: (0, 30)}), ([0, 30, 60, 900], {0: (0, 30), 1: (30, 60)}),
    ([-5, 30, 60, 90], {1: (30, 60), 2: (60, 90)}), ([0, 60, 30, 30], {0: (0, 60)}), ([0, 60, 30, 90], {0: (0, 60)}),
    ([0, 200, 60, 90], {}), ([0, 90, 90, 30], {0: (0, 90)}), ([10, 40, 40, 90], {0: (10, 40), 2: (40, 90)}),
]


@pytest.mark.parametrize("cu,fine", BAD_ROWS)
@pytest.mark.parametrize("split", [True, False])
def test_prefill_leaves_rows_of_skipped_requests(cu, fine, split):
    """Requests whose rows are out of order or beyond T are skipped, their rows left as they were, the others
    complete: also where the keys are split and the parts joined, whatever the workspace holds."""
    d = prefill_case([30, 30, 30], [1500, 10, 1200], 2)
    ws = torch.full((M.workspace_size_prefill(90, 3, 2, d["S"]) if split else 0,), 255, dtype=torch.uint8, device=DEV)
    assert (ws.numel() > 0) == split
    out = torch.full((90, 2, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((90, 2), 9.0, device=DEV)
    call(dict(d, cu=cu), out=out, lse=lse, workspace=ws)
    assert M.device_status() == (0 if cu[0] == 10 else BAD_STEP)
    left = torch.ones(90, dtype=torch.bool)
    for b, (lo, hi) in fine.items():
        left[lo:hi] = False
        check(alone(d, b, slice(lo, hi)), out[lo:hi], lse[lo:hi], split=True)
    left = left.to(DEV)
    assert (out[left] == 9).all() and (lse[left] == 9).all()


def test_prefill_split_skips_among_many_requests():
    """The same behind the first 32 requests, with requests of no rows among them."""
    new = [0 if b % 5 == 3 else 2 for b in range(64)]
    ctx = [(37 * b) % 60 for b in range(64)]
    d = prefill_case(new, ctx, 1)
    T, cu = d["T"], list(d["cu"])
    fine = {b: (cu[b], cu[b + 1]) for b in range(64) if new[b]}
    cu[40] = cu[35] - 1                            # rows of 39 end before those of 35 begin
    for b in (39, 40):
        fine.pop(b, None)
    ws = torch.full((M.workspace_size_prefill(T, 64, 1, d["S"]),), 255, dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0
    out = torch.full((T, 1, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, 1), 9.0, device=DEV)
    call(dict(d, cu=cu), out=out, lse=lse, workspace=ws)
    assert M.device_status() == BAD_STEP
    left = torch.ones(T, dtype=torch.bool)
    for b, (lo, hi) in fine.items():
        left[lo:hi] = False
        check(alone(d, b, slice(lo, hi)), out[lo:hi], lse[lo:hi], split=True)
    left = left.to(DEV)
    assert left.any() and (out[left] == 9).all() and (lse[left] == 9).all()


@pytest.mark.parametrize("what", ["rows", "rows before", "keys", "start"])
@pytest.mark.parametrize("B", [33, 65, 100])
@pytest.mark.parametrize("split", [True, False])
def test_prefill_reports_requests_behind_the_last_rows(what, B, split):
    """A request out of order or range is reported wherever it stands: here behind all rows, in a round of 32
    requests of which no other one has any."""
    new = [1, 1] + [0] * (B - 2)
    d = prefill_case(new, [900, 3] + [1] * (B - 2), 1)
    good, good_lse = call(d)
    assert M.device_status() == 0
    cu, lens, starts = list(d["cu"]), list(d["lens"]), list(d["starts"])
    if what == "rows":
        cu[B] = 3                                  # beyond T
    elif what == "rows before":
        cu[B] = 1
    elif what == "keys":
        lens[B - 1] = -1
    else:
        starts[B - 1] = d["S"] + 1
    n = M.workspace_size_prefill(2, B, 1, d["S"])
    assert n > 0
    ws = torch.empty(n if split else 0, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        out, lse = call(dict(d, cu=cu, lens=lens, starts=starts), workspace=ws)
        assert M.device_status() == BAD_STEP
        check(dict(d, cu=d["cu"][:3], lens=lens[:2], starts=starts[:2], G=d["G"][:2]), out, lse, split=True)


def test_prefill_rows_computed_again_do_not_run_out_of_time():
    """Rows that a NaN in a value they do not see has them computed again take longer than the wait limit, here
    some 3 ms against 0.5; the block's other warps wait that long, and its next unit is complete as well."""
    n, ctx, H = 256, 768, 304                      # two units a block
    d = prefill_case([n], [ctx], H)
    few = [0, 150, 151, 152, H - 1]
    sub = dict(d, q=d["q"][:, few], k=d["k"][:, few], v=d["v"][:, few], H=len(few))
    o, l, A, D, _ = P.ref_prefill(n64(sub["q"]), n64(sub["k"]), n64(sub["kr"]), n64(sub["v"]), d["cu"], d["starts"], d["lens"],
                                  d["G"], SCALE, 1, 0, 1, True)
    d["v"][n + ctx - 1] = math.nan                 # seen by the last row alone
    call(d)
    torch.cuda.synchronize()
    prev = M.set_wait_limit_ns(500_000)
    try:
        out, lse = call(d)
        torch.cuda.synchronize()
        bits = M.device_status()
    finally:
        M.set_wait_limit_ns(prev)
    assert bits == 0
    assert torch.isnan(out[-1]).all() and torch.isfinite(out[:-1]).all() and torch.isfinite(lse).all()
    delta = 60 * U * D + 2.0 ** -20
    tol = BF * np.abs(o) + (BF + 2 * (np.exp(2 * delta) - 1) + (n + ctx + 64) * U)[..., None] * A
    within(n64(out[:-1, few]), o[:-1], tol[:-1], "out")


def test_prefill_many_requests_and_head_groups():
    """More than 32 requests and several groups of heads, the last one smaller: a block that goes on from one
    group to the next finds its request again from the first.  (152 SMs: 111 row tiles, so 6 heads' units
    are four an SM; 33 heads are 5 groups of 7, the last one of 5.)"""
    new = [(11 * b) % 59 for b in range(100)]
    ctx = [(29 * b) % 331 for b in range(100)]
    H = 33
    d = prefill_case(new, ctx, H)
    out, lse = call(d)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    for b in range(100):
        if new[b] == 0:
            continue
        rows = slice(d["cu"][b], d["cu"][b + 1])
        o1, l1 = call(alone(d, b, rows), workspace=none)
        assert torch.equal(o1, out[rows]) and torch.equal(l1, lse[rows]), b
    few = [0, 6, 7, 27, 28, 32]
    check(dict(d, q=d["q"][:, few], k=d["k"][:, few], v=d["v"][:, few], H=len(few)), out[:, few], lse[:, few])
    assert M.device_status() == 0


# =============================================================================================
# expanded keys and values
# =============================================================================================
def expand_case(seed, lens, H, bs, gap, form):
    g = gen(seed)
    table, nb = paged(g, lens, bs)
    starts, S = starts_of(lens, gap)
    w = randn(g, H, 256, 512, scale=512 ** -0.5)
    x = torch.randn(nb, bs, 576, generator=g)
    scales = None
    if form == "bf16":
        cache = x.to(torch.bfloat16).to(DEV)
    else:
        cache = (x * 8).to(torch.float8_e4m3fn).to(DEV)
        s = torch.exp2(torch.randint(-12, 5, (nb, bs // 16), generator=g).float())
        if form == "q8 odd scales":
            s = s * (1 + torch.rand(nb, bs // 16, generator=g))
        scales = s.to(DEV)
    return cache, scales, table, starts, S, w


def source_rows(cache, scales, table, lens, starts, at):
    """The cache rows (float64) behind output rows `at`; None where there is no request."""
    bs = cache.shape[1]
    slot = np.full(len(at), -1)
    for b, n in enumerate(lens):
        l = at - starts[b]
        ok = (l >= 0) & (l < n)
        slot[ok] = table[b].numpy()[l[ok] // bs] * bs + l[ok] % bs
    t = torch.from_numpy(np.maximum(slot, 0)).to(DEV)
    rows = n64(cache.reshape(-1, 576).view(torch.uint8 if scales is not None else torch.bfloat16)[t].view(cache.dtype).float())
    if scales is not None:
        rows = rows * n64(scales.reshape(-1)[t // 16])[:, None]
    return rows, slot >= 0


@pytest.mark.parametrize("form", ["q8 odd scales"])
@pytest.mark.parametrize("lens,H", [([5, 0, 130], 2), ([700], 5)])
def test_expand_8bit_scales_are_exact(lens, H, form):
    """The 8-bit rows' scales multiply the sums in fp32, whatever they are: one rounding to bf16, no other.
    (The sum of exact products: 92 u of the magnitudes, the product with the scale: u |y|.)"""
    cache, scales, table, starts, S, w = expand_case(31 + H, lens, H, 32, 3, form)
    k, v, r = M.mla_expand(cache, table.to(DEV), i32(lens), i32(starts), w, S, kv_scales=scales)
    at = np.arange(S)
    rows, mine = source_rows(cache, scales, table, lens, starts, at)
    want = np.einsum("sc,hdc->shd", rows[mine, :512], n64(w))
    mag = np.einsum("sc,hdc->shd", np.abs(rows[mine, :512]), np.abs(n64(w)))
    got = np.concatenate([n64(k), n64(v)], -1)[mine]
    within(got, want, (BF + U) * np.abs(want) + 92 * U * mag, "kv")
    within(n64(r)[mine], rows[mine, 512:], BF * np.abs(rows[mine, 512:]), "rope key")
    assert M.device_status() == 0


@pytest.mark.parametrize("lens,H,bs,gap", [
    ([9000, 0, 700, 31000, 17], 1, 64, 37),           # more row pairs than clusters of two SMs: several a cluster
    ([21000, 133], 2, 192, 0),
    ([1500, 3, 0, 2000, 600], 128, 64, 5),            # fewer, but too uneven for clusters of their own: cut evenly
])
@pytest.mark.parametrize("form", ["bf16", "q8"])
def test_expand_clusters_go_from_pair_to_pair(lens, H, bs, gap, form):
    """Tiles of all row pairs cut evenly over the clusters: a cluster ends one pair's columns, gathers the
    next pair's rows while products of the last are under way, and begins or ends inside a pair."""
    cache, scales, table, starts, S, w = expand_case(sum(lens) + H, lens, H, bs, gap, form)
    kv = torch.full((H, S, 256), 9.0, dtype=torch.bfloat16, device=DEV)
    kr = torch.full((S, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    M.mla_expand(cache, table.to(DEV), i32(lens), i32(starts), w, S, kv_scales=scales, kv=kv, k_rope=kr)
    rng = np.random.default_rng(S)
    edges = np.concatenate([np.arange(0, S, 128) + x for x in (-1, 0)] + [np.array(starts) + x for x in (-1, 0, 1)] +
                           [np.array(starts) + np.array(lens) + x for x in (-1, 0)])
    at = np.unique(np.concatenate([edges[(edges >= 0) & (edges < S)], rng.integers(0, S, 700)]))
    rows, mine = source_rows(cache, scales, table, lens, starts, at)
    heads = sorted({0, H // 2, H - 1, int(rng.integers(0, H))})
    t = torch.from_numpy(at).to(DEV)
    got, wn = n64(kv[heads][:, t]), n64(w[heads])
    for i in range(len(heads)):
        want, mag = rows[:, :512] @ wn[i].T, np.abs(rows[:, :512]) @ np.abs(wn[i]).T
        within(got[i, mine], want[mine], (BF * np.abs(want) + 92 * U * mag)[mine], f"head {heads[i]}")
    assert np.array_equal(n64(kr[t])[mine], rows[mine, 512:])
    # every row of every head: written where it is somebody's, and there alone
    somebody = torch.zeros(S, dtype=torch.bool)
    for s, n in zip(starts, lens):
        somebody[s:s + n] = True
    somebody = somebody.to(DEV)
    assert (kv[:, ~somebody] == 9).all() and (kr[~somebody] == 9).all()
    assert ((kv == 9).all(-1) == ~somebody).all() and ((kr == 9).all(-1) == ~somebody).all()
    # and equal to a call that has a request alone
    for b in (0, len(lens) - 1):
        k1, v1, r1 = M.mla_expand(cache, table[b:b + 1].to(DEV), i32(lens[b:b + 1]), i32([0]), w, lens[b], kv_scales=scales)
        at = slice(starts[b], starts[b] + lens[b])
        assert torch.equal(kv[:, at, :128].transpose(0, 1), k1) and torch.equal(kv[:, at, 128:].transpose(0, 1), v1)
        assert torch.equal(kr[at], r1)
    assert M.device_status() == 0


# =============================================================================================
# rotation and append
# =============================================================================================
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("T,H,width,into", [(5000, 128, 192, 0), (5000, 128, 192, 576), (4999, 37, 192, 0), (5003, 37, 64, 576),
                                            (70001, 1, 576, 64), (70001, 1, 576, 0), (30000, 4, 64, 0)])
def test_rope_of_many_tokens(T, H, width, into, half):
    """Enough tokens for a warp to take all of a token's heads, several in flight and in several rounds:
    in place, and into rows of another width."""
    g = gen(T + H + into)
    freqs = M.rope_freqs(**FREQS["yarn"])
    q = torch.randn(T, H, width, generator=g, dtype=torch.float32).to(torch.bfloat16).to(DEV)
    x = q[..., width - 64:]
    pos = torch.randint(0, 1 << 20, (T,), generator=g)
    pos[::97] = -1
    whole = torch.full((T, H, into), 9.0, dtype=torch.bfloat16, device=DEV) if into else q.clone()
    start = whole.clone()
    out = whole[..., whole.shape[-1] - 64:]
    y = M.mla_rope(x if into else out, i64(pos), freqs, out=out, half=half, mscale=1.25)
    assert y is out
    at = np.unique(np.concatenate([np.arange(0, T, 97)[:40], np.arange(0, T, 97)[:40] + 1, [T - 1],
                                   np.random.default_rng(T).integers(0, T, 200)]))
    t = torch.from_numpy(at).to(DEV)
    xs = n64(x[t])
    want = P.ref_rope(xs, pos.numpy()[at], freqs.tolist(), half, 1.25, n64(start[t])[..., -64:])
    within(n64(out[t]), want, BF * np.abs(want) + 2.0 ** -20 * 1.25 * pair_sum(xs, half), "rope")
    assert torch.equal(whole[..., :-64], start[..., :-64])
    stay = (pos < 0).to(DEV)
    assert torch.equal(whole[stay], start[stay])
    # every token as in a call of few tokens at a time
    pieces = torch.cat([M.mla_rope(x[a:a + 300], i64(pos[a:a + 300]), freqs, half=half, mscale=1.25)
                        for a in range(0, min(T, 6000), 300)])
    assert torch.equal(out[:len(pieces)][~stay[:len(pieces)]], pieces[~stay[:len(pieces)]])


@pytest.mark.parametrize("B,N", [(1, 4864), (1, 4865), (64, 76), (5, 973), (3, 2731), (1, 16384)])
@pytest.mark.parametrize("cp,rank,il", [(1, 0, 1), (2, 1, 1), (3, 0, 4)])
def test_rope_store_of_thousands(B, N, cp, rank, il):
    """Around the number of positions from which a warp takes 32 of them (32 an SM: 4,864 with 152)."""
    g = gen(B + N + cp)
    freqs, bs = M.rope_freqs(**FREQS["ntk"]), 32
    ctx = torch.randint(0, 2000, (B, 1), generator=g)
    pos = ctx + torch.arange(N)[None]
    pos[:, N - N // 9:] = -1
    width = (2000 + N) // (bs * cp) + 1
    nb = B * width + 1
    table = torch.randperm(nb, generator=g)[:B * width].view(B, width).to(torch.int32).to(DEV)
    kv = torch.randn(B, N, 576, generator=g).to(torch.bfloat16).to(DEV)
    cache = torch.full((nb, bs, 576), 9.0, dtype=torch.bfloat16, device=DEV)
    slots = torch.empty(B, N, dtype=torch.int64, device=DEV)
    M.cp_rope_store(kv[..., :512], kv[..., 512:], i64(pos), freqs, table, cache, cp, rank, il, slots=slots)
    want_slots = R.ref_cp_local_slot(pos.numpy(), table.cpu().numpy(), bs, cp, rank, il)
    assert np.array_equal(n64(slots), want_slots)
    own = torch.from_numpy(want_slots >= 0).to(DEV)
    flat, at = cache.view(-1, 576), slots[own]
    assert torch.equal(flat[at, :512], kv[own][:, :512])
    left = torch.ones(nb * bs, dtype=torch.bool, device=DEV)
    left[at] = False
    assert (flat[left] == 9).all()
    p, x, got = n64(i64(pos)[own]), n64(kv[own][:, 512:]), n64(flat[at, 512:])
    some = np.unique(np.concatenate([np.arange(min(64, len(p))), [len(p) - 1], np.random.default_rng(N).integers(0, len(p), 150)]))
    want = np.stack([P.ref_rope_row(x[i], int(p[i]), freqs.tolist(), False, 1.0) for i in some])
    within(got[some], want, BF * np.abs(want) + 2.0 ** -20 * pair_sum(x[some], False), "rope key")
    turned = M.mla_rope(kv[own][:, None, 512:], i64(pos)[own], freqs)
    assert torch.equal(flat[at, 512:], turned[:, 0])
    assert M.device_status() == 0


# =============================================================================================
# together
# =============================================================================================
@pytest.mark.parametrize("cp,rank", [(1, 0), (2, 1)])
def test_layer_of_uneven_chunks(cp, rank):
    """A step's layer as the module's example has it, for requests of different lengths; the append of
    tokens without padding, as requests of one token each, writes the same rows."""
    g = gen(77 + cp)
    new, ctx, H, bs, N = [37, 130, 0, 1], [20, 0, 5, 300], 2, 16, 130
    B, width = 4, 40
    nb = B * width
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    ring = torch.randperm(nb, generator=g).to(torch.int32).to(DEV)
    w, freqs = randn(g, H, 256, 512, scale=512 ** -0.5), M.rope_freqs(**FREQS["yarn"])
    t0 = M.cp_step_tables(i32([0] * B), i32([0] * B), i32(ctx), table, ring, i32([0, nb]), bs, 300, cp, rank)
    cache = randn(g, nb, bs, 576)                   # what the tokens before left
    t = M.cp_step_tables(t0.total_lens, i32(ctx), i32(new), table, ring, t0.free_state, bs, N, cp, rank)
    again = cache.clone()
    kv = randn(g, B, N, 576)
    M.cp_rope_store(kv[..., :512], kv[..., 512:], t.positions, freqs, table, cache, cp, rank)
    real = t.positions >= 0
    positions = t.positions[real]
    assert positions.tolist() == [c + j for n, c in zip(new, ctx) for j in range(n)]
    flat = kv[real]
    owner = i64([b for b in range(B) for _ in range(new[b])])
    M.cp_rope_store(flat[:, None, :512], flat[:, None, 512:], positions[:, None], freqs, table[owner], again, cp, rank)
    assert torch.equal(cache, again)
    q = randn(g, sum(new), H, 192)
    before = n64(q)
    M.mla_rope(q[..., 128:], positions, freqs, out=q[..., 128:])
    turned = P.ref_rope(before[..., 128:], positions.tolist(), freqs.tolist(), False, 1.0, before[..., 128:])
    within(n64(q)[..., 128:], turned, BF * np.abs(turned) + 2.0 ** -20 * pair_sum(before[..., 128:], False), "rope")
    seq = t.seq_lens[0]
    G = [a + b for a, b in zip(new, ctx)]
    lens = [int(R.ref_local_len(x, cp, rank, 1)) for x in G]
    assert seq.tolist() == lens and t.total_lens.tolist() == G
    starts, S = starts_of(lens)
    kv_starts = torch.cumsum(seq, 0, dtype=torch.int32) - seq
    assert kv_starts.tolist() == starts
    cu = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
    k, v, kr = M.mla_expand(cache, table, seq, kv_starts, w, S)
    want, wr, mag, mine = P.ref_expand(lambda b: R.ref_gather_pages(n64(cache), table[b].cpu().numpy(), lens[b]), lens, starts,
                                       n64(w), S)
    got = np.concatenate([n64(k), n64(v)], -1).transpose(1, 0, 2)
    assert mine.all() and np.array_equal(n64(kr), wr)
    within(got, want, BF * np.abs(want) + 92 * U * mag, "kv")
    out, lse = M.mla_prefill(q, k, kr, v, i32(cu), kv_starts, seq, t.total_lens, SCALE, cp, rank)
    check(dict(q=q, k=k, kr=kr, v=v, cu=cu, starts=starts, lens=lens, G=G, cp=cp, rank=rank, il=1), out, lse, split=True)
    assert M.device_status() == 0


# =============================================================================================
# merge
# =============================================================================================
@pytest.mark.parametrize("n,T,H", [(3, 5, 2), (16, 3, 2), (3, 4000, 2), (40, 300, 4)])
@pytest.mark.parametrize("D", [512, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_merge_nan_lse(n, T, H, D, dtype):
    """A NaN among a row's LSEs, or nothing but NaN and empty shards, gives NaN in both widths; rows of empty
    shards alone give 0 and -inf, and all others are as they would be without such rows."""
    g = gen(n + T + D)
    parts = torch.randn(n, T, H, D, generator=g).to(dtype).to(DEV)
    lses = torch.randn(n, T, H, generator=g).to(DEV)
    clean, clean_lse = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, H, device=DEV)
    M.lse_merge(parts, lses, out=clean, out_lse=clean_lse)
    lses[:, 0, 0] = math.nan
    lses[1, 1, 1] = math.nan
    lses[0, 2, 0], lses[1:, 2, 0] = math.nan, -math.inf
    lses[:, 2, 1] = -math.inf
    out_lse = torch.empty(T, H, device=DEV)
    out, _ = M.lse_merge(parts, lses, out_lse=out_lse)
    bad, empty = torch.isnan(lses).any(0), (lses == -math.inf).all(0)
    assert bad.sum() == 3 and torch.isnan(out[bad]).all() and torch.isnan(out_lse[bad]).all()
    assert (out[empty] == 0).all() and (out_lse[empty] == -math.inf).all()
    rest = ~bad & ~empty
    assert torch.equal(out[rest], clean[rest]) and torch.equal(out_lse[rest], clean_lse[rest])

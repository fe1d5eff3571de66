"""The 8-bit paged cache on the GPU against its float64 oracle: step tables (exact), the
quantising store (exact) and the decode, and a serving run of them together.

Tolerance of the decode, per row, head and dim, with w_l = softmax weights, S_l the key's
scale, v_l the stored e4m3 values, A = sum_l w_l S_l |v_l|, M = max_l w_l S_l:
  * out is rounded to bf16 once: 2^-8 |out|; the warp-level kernel's partials are fp32;
  * a weight that meets v_l is rounded to bf16 (warp-level kernel: 2^-8 of itself), or, in
    [2^e, 2^(e+1)), to an e5m2 value, whose residue is at most 2^(e-3), plus that residue in
    e4m3, whose half step up to there is 2^(e-8): 2^-8 of itself; to half precision before
    (2^-11); and the tcgen05 kernel's partials are in half precision (2^-11 of a mean of at
    most A): 2^-8 + 2^-10 < 2^-7 in all; where the remainder is subnormal, half a step, 2^-10,
    where the row's largest weight times scale is at least 2^5 when the reference is set:
    2^-15 M, doubled to 2^-14 M (half precision's own subnormals, 2^-25, are far below):
    (2^-7) A + 2^-14 M sum_l |v_l|;
  * scores: q times its row's power of two is the sum of two e4m3 values to within 2^-10 of a
    row maximum of at least 2^7 (exact above 2^-9 of the maximum): 2^-17 max|q| sum_d |k_d|;
    the products are exact in fp32 and summed in 36 steps of 32: (31 + 35) u, doubled for
    truncation: 132 u sum_d |q_d k_d|; base-2 exponent arguments are rounded to fp32 three
    times (times scale, plus log2 S, minus the reference): 4 u max|s| log2 e and the like,
    covered by 8 u (|s| + |log2 S| + 64); 2^x by 2^-22.  With delta their sum, weights move by e^{+-delta} against each
    other, the output by 2 (e^{2 delta} - 1) A, the LSE by delta (+ 1e-6 (1 + |lse|) for its own
    rounding and log).
Besides, the norm of the output's error is at most 2^-7 of the output's (roundings are
independent; each is at most that)."""
import ctypes
import math
import re

import numpy as np
import pytest
import torch

import mla_paged_decode_03_gb300 as M
import oracle.mla_ref as R
import oracle.q8_ref as Q
from mla_paged_decode_03_gb300 import _lib

pytestmark = pytest.mark.gpu

DEV = "cuda"
SCALE = 1.0 / math.sqrt(192.0)
BAD_PAGE, TOO_LONG, BAD_VBLOCK, BAD_SCALE, NO_PAGES, BAD_STEP = 1, 2, 4, 16, 32, 64


@pytest.fixture(autouse=True)
def _clean():
    M.device_status()
    prev = M.set_decode_kernel(M.KERNEL_AUTO)
    yield
    M.set_decode_kernel(prev)


_extra_columns = 0


@pytest.fixture(params=["mma", "units32", "units64"])
def kernel(request):
    """The warp-level kernel, and the tcgen05 kernel with units of 32 and (requests of more than
    32 rows only) of 64 rows."""
    global _extra_columns
    prev = M.set_decode_kernel(M.KERNEL_MMA if request.param == "mma" else M.KERNEL_AUTO)
    _extra_columns = 8 * torch.cuda.get_device_properties(DEV).multi_processor_count * 8 \
        if request.param == "units64" else 0
    yield request.param
    _extra_columns = 0
    M.set_decode_kernel(prev)


@pytest.fixture(params=[32, 64])
def units(request):
    """As `kernel`, for tests of the tcgen05 kernel alone."""
    global _extra_columns
    _extra_columns = 8 * torch.cuda.get_device_properties(DEV).multi_processor_count * 8 \
        if request.param == 64 else 0
    yield request.param
    _extra_columns = 0


def bt32(table):
    """A block table on the GPU.  The decode takes units of 64 rows when full tables would give
    every SM some tiles of 128 keys; columns for eight (of 16 slots or more) make it do so at any
    length."""
    return torch.nn.functional.pad(i32(table), (0, _extra_columns), value=-1)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def n64(t):
    return t.detach().cpu().to(torch.float64).numpy() if t.is_floating_point() else t.cpu().numpy()


# =============================================================================================
# step tables
# =============================================================================================
def check_step(prev, ctx, new, table, ring, state, bs, N, cp, rank, ranks, il, bits=0):
    d = dict(table=i32(table), ring=i32(ring), state=i32(state))
    t = M.cp_step_tables(i32(prev), i32(ctx), i32(new), d["table"], d["ring"], d["state"], bs, N,
                         cp, rank, ranks, il)
    want = Q.ref_step_tables(prev, ctx, new, table, ring, state, bs, N, cp,
                             range(rank, rank + ranks), il)
    got = (t.total_lens, t.seq_lens, t.positions, t.slots, d["table"], d["ring"], t.free_state)
    for name, g, w in zip(("total", "seq", "positions", "slots", "table", "ring", "state"), got, want):
        assert np.array_equal(n64(g), w), name
    assert M.device_status() == bits
    # a call does not change what it reads: repeated, it gives the same
    t2 = M.cp_step_tables(i32(prev), i32(ctx), i32(new), d["table"], d["ring"], d["state"], bs, N,
                          cp, rank, ranks, il, seq_lens=torch.empty_like(t.seq_lens))
    for a, b in zip(t, t2):
        assert torch.equal(a, b)
    assert np.array_equal(n64(d["table"]), want[4]) and np.array_equal(n64(d["ring"]), want[5])
    assert M.device_status() == bits
    return want


@pytest.mark.parametrize("B,N,bs,cp,il,ranks,supply", [
    (1, 1, 16, 1, 1, 1, 1.0),
    (8, 1, 64, 1, 1, 1, 1.0),
    (5, 4, 16, 2, 2, 2, 0.5),
    (37, 3, 7, 3, 7, 2, 1.0),          # odd sizes (pages of any size here)
    (256, 4, 64, 8, 1, 8, 1.0),
    (300, 1, 16, 4, 16, 1, 0.3),       # more requests than a block scans at once
    (3, 2500, 16, 2, 1, 2, 1.0),       # more positions than a tile
    (2, 4096, 64, 1, 64, 1, 0.6),
    (70, 33, 16, 16, 4, 16, 0.8),
    (1025, 2, 32, 1, 1, 1, 0.9),
    (4, 0, 16, 2, 1, 2, 1.0),          # lengths only
])
def test_step_tables_over_several_steps(B, N, bs, cp, il, ranks, supply):
    """A simulated loop: requests grow by up to N, have drafts rejected, finish and start over,
    with a pool of `supply` of what they need at most."""
    rng = np.random.default_rng(B * 1000 + N)
    vbs = bs * cp
    longest = 3 * N + 5 * vbs
    width = -(-longest // vbs) + 1
    cap = max(2, int(B * width * supply)) + 3
    table = np.full((B, width), -1)
    ring = rng.permutation(cap)
    state = (int(rng.integers(cap)), cap)
    ring = np.roll(ring, state[0])
    prev = np.zeros(B, np.int64)
    for step in range(4):
        ctx = np.maximum(prev - rng.integers(0, 4, B), 0)
        if step == 0:
            new = rng.integers(0, N + 1, B)
        else:
            new = rng.integers(0, N + 1, B)
            new[ctx + new > longest] = 0
        done = rng.random(B) < 0.2
        ctx[done], new[done] = 0, 0
        asked = np.cumsum([max(0, -(-int(c + n) // vbs) - -(-int(p) // vbs)) for c, n, p in zip(ctx, new, prev)])
        short = bool(np.any((asked > state[1]) & (np.diff(asked, prepend=0) > 0)))
        total, _, _, _, table, ring, state = check_step(
            prev, ctx, new, table, ring, state, bs, N, cp, cp - ranks if cp > ranks else 0, ranks, il,
            NO_PAGES if short else 0)
        held = [int(x) for b in range(B) for x in table[b, :-(-int(total[b]) // vbs)]]
        free = [int(ring[(int(state[0]) + k) % cap]) for k in range(int(state[1]))]
        assert sorted(held + free) == list(range(cap))            # no page lost or used twice
        prev = total


def test_step_tables_refuse_a_request_beyond_its_table():
    table = np.array([[0, 1], [2, -1], [3, -1]])
    check_step([30, 16, 10], [30, 16, 10], [3, 1, 1], table, [4, 5, 6, 7], (1, 3), 16, 4, 1, 0, 1, 1,
               TOO_LONG)
    # the request beyond its table takes no page from those behind it
    check_step([0, 0], [0, 0], [40, 16], np.full((2, 2), -1), [4, 5], (0, 1), 16, 40, 1, 0, 1, 1, TOO_LONG)


def test_step_tables_bad_data_is_flagged_and_bounded():
    def call(prev, ctx, new, state, ring=(4, 5, 6, 7), N=4, width=2):
        tab = torch.full((len(prev), width), -1, dtype=torch.int32, device=DEV)
        r = i32(ring)
        t = M.cp_step_tables(i32(prev), i32(ctx), i32(new), tab, r, i32(state), 16, N)
        return t, tab, r
    # a ring state outside the ring: an empty ring
    for state in ((-1, 2), (4, 1), (0, 5), (0, -1)):
        t, tab, r = call([0], [0], [1], state)
        assert M.device_status() == BAD_STEP | NO_PAGES
        assert t.total_lens.tolist() == [0] and tab.tolist() == [[-1, -1]] and t.free_state.tolist() == [0, 0]
    # negative lengths are 0, more than N new tokens N, prev beyond the table the whole table
    t, tab, _ = call([0, -5], [-3, 0], [2, -1], (0, 4))
    assert M.device_status() == BAD_STEP and t.total_lens.tolist() == [2, 0]
    assert tab.tolist() == [[4, -1], [-1, -1]] and t.positions.tolist() == [[0, 1, -1, -1], [-1] * 4]
    t, _, _ = call([0], [0], [9], (0, 4))
    assert M.device_status() == BAD_STEP and t.total_lens.tolist() == [4]
    t, _, r = call([1000], [0], [0], (0, 1))
    assert M.device_status() == BAD_STEP and t.free_state.tolist() == [0, 3] and r.tolist() == [4, -1, -1, 7]
    # pages given back to a full ring are dropped
    t, _, r = call([20], [0], [0], (1, 4))
    assert M.device_status() == BAD_STEP and t.free_state.tolist() == [1, 4] and r.tolist() == [4, 5, 6, 7]
    # lengths whose sum passes 31 bits
    t, _, _ = call([5], [2 ** 31 - 2], [4], (0, 4))
    assert M.device_status() == TOO_LONG and t.total_lens.tolist() == [5]


def test_step_tables_large_lengths():
    # positions near 2^31 with a virtual block of 2^20: 64-bit slots
    pages = [2 ** 31 - 1, 2 ** 30]
    bs, N = 1 << 20, 3
    table = np.full((1, 2048), -1)
    table[0, 2046] = pages[0]
    ctx = 2047 * bs - 2
    check_step([2047 * bs - 1], [ctx], [3], table, [pages[1], 9], (0, 2), bs, N, 1, 0, 1, 1)


def test_step_tables_empty_batch_copies_the_ring_state():
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    t = M.cp_step_tables(e, e, e, torch.empty(0, 3, dtype=torch.int32, device=DEV), i32([1, 2, 3]), i32([2, 1]),
                         16, 4)
    assert t.free_state.tolist() == [2, 1] and M.device_status() == 0


def test_step_tables_strided_table_and_other_stream():
    wide = torch.full((3, 9), -7, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ring, state = i32([3, 4, 5, 6]), i32([0, 4])
    prev, ctx, new = i32([0, 0, 0]), i32([0, 0, 0]), i32([5, 0, 17])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        t = M.cp_step_tables(prev, ctx, new, wide[:, 2:5], ring, state, 16, 17)
    s.synchronize()
    assert wide[:, 2:5].tolist() == [[3, -7, -7], [-7, -7, -7], [4, 5, -7]]
    assert (wide[:, :2] == -7).all() and (wide[:, 5:] == -7).all() and t.free_state.tolist() == [3, 1]


def test_tables_and_store_on_a_given_stream():
    """Everything on a stream passed to the calls, which allocate their outputs there."""
    s = torch.cuda.Stream()
    rows = torch.randn(3, 17, 576, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).to(DEV)
    table = torch.full((3, 3), -1, dtype=torch.int32, device=DEV)
    ring, state, zero, new = i32([3, 4, 5, 6, 7]), i32([0, 5]), i32([0, 0, 0]), i32([5, 0, 17])
    cache, scales = new_pool(8, 16, poison=False)
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        t = M.cp_step_tables(zero, zero, new, table, ring, state, 16, 17, stream=s)
        M.cp_store_q8(rows, zero, t.total_lens, table, cache, scales, stream=s)
        got.append(t)
        torch.full((1 << 16,), -7, dtype=torch.int32, device=DEV)
    s.synchronize()
    for t in got:
        assert t.total_lens.tolist() == [5, 0, 17] and t.free_state.tolist() == [3, 2]
        assert t.positions[2].tolist() == list(range(17)) and t.slots[0, 0, :5].tolist() == list(range(48, 53))
    want, ws = Q.ref_store_q8(n64(rows), [0, 0, 0], [5, 0, 17], np.maximum(n64(table), 0), np.zeros((8, 16, 576)),
                              np.ones((8, 1)), 1, 0)
    assert np.array_equal(n64(cache.float()), want) and np.array_equal(n64(scales), ws)
    assert M.device_status() == 0


def test_step_tables_refuses_outputs_over_inputs():
    a, tab, ring, st = i32([0, 0]), torch.zeros(2, 2, dtype=torch.int32, device=DEV), i32([1, 2]), i32([0, 2])
    with pytest.raises(M.MlaError):
        M.cp_step_tables(a, i32([0, 0]), i32([1, 1]), tab, ring, st, 16, 1, total_lens=a)
    with pytest.raises(M.MlaError):
        M.cp_step_tables(a, i32([0, 0]), i32([1, 1]), tab, ring, st, 16, 1, free_state_out=st)


# =============================================================================================
# store
# =============================================================================================
def f8(x):
    return torch.tensor(np.asarray(x), dtype=torch.float32, device=DEV).to(torch.float8_e4m3fn)


def new_pool(nb, bs, poison=True):
    """A pool nobody wrote: NaN bytes and NaN scales (or zeros and ones)."""
    c = torch.full((nb, bs, 576), 0x7f if poison else 0, dtype=torch.uint8, device=DEV)
    return c.view(torch.float8_e4m3fn), torch.full((nb, bs // 16), float("nan") if poison else 1.0, device=DEV)


def random_table(rng, B, pages, num_blocks):
    return rng.permutation(num_blocks)[:B * pages].reshape(B, pages)


def check_store(rows, ctx, total, table, cache, scales, cp, rank, il, bits=0):
    want_c, want_s = Q.ref_store_q8(n64(rows), ctx, total, table, n64(cache.float()), n64(scales), cp, rank, il)
    M.cp_store_q8(rows, i32(ctx), i32(total), i32(table), cache, scales, cp, rank, il)
    assert M.device_status() == bits
    assert np.array_equal(n64(cache.float()), want_c, equal_nan=True)
    assert np.array_equal(n64(scales), want_s, equal_nan=True)


@pytest.mark.parametrize("B,N,bs,cp,il,top", [
    (1, 1, 16, 1, 1, 40), (7, 1, 64, 1, 1, 100), (5, 4, 16, 2, 2, 70), (3, 5, 48, 3, 4, 200),
    (4, 37, 64, 4, 16, 90), (2, 333, 16, 1, 1, 50), (2, 700, 128, 8, 1, 3000), (64, 3, 32, 2, 1, 64),
    (3, 17, 16, 16, 16, 700),
])
def test_store_matches_oracle(B, N, bs, cp, il, top):
    """Every rank's pool, two stores in a row (the second begins inside blocks the first left
    partly filled, with rows of very different size)."""
    rng = np.random.default_rng(N * 100 + bs)
    g = torch.Generator().manual_seed(B + N)
    pages = -(-(top + 2 * N) // (bs * cp)) + 1
    nb = B * pages + 2
    table = random_table(rng, B, pages, nb)
    ctx = rng.integers(0, top + 1, B)
    for rank in range(cp):
        cache, scales = new_pool(nb, bs, poison=False)
        cache.view(torch.uint8).copy_(torch.randint(0, 127, (nb, bs, 576), generator=g).to(torch.uint8))
        at = ctx
        for _ in range(2):
            total = at + rng.integers(max(0, N - 3), N + 1, B)
            rows = torch.randn(B, N, 576, generator=g)
            rows *= 10.0 ** torch.randint(-3, 3, (B, N, 1), generator=g)
            check_store(rows.to(torch.bfloat16).to(DEV), at, total, table, cache, scales, cp, rank, il)
            at = total


def test_store_token_by_token_equals_scales_of_the_whole():
    # rows of falling size: the first sets the scale, so one by one gives what one call gives
    rows = (torch.randn(1, 40, 576, generator=torch.Generator().manual_seed(3)).clamp(-2, 2)
            * torch.linspace(8, 1, 40)[None, :, None])
    rows[0, 0, 0] = rows[0, 16, 0] = rows[0, 32, 0] = 32.0
    rows = rows.to(torch.bfloat16).to(DEV)
    table = [[2, 0, 1]]
    a, sa = new_pool(3, 16)
    b, sb = new_pool(3, 16)
    M.cp_store_q8(rows, i32([0]), i32([40]), i32(table), a, sa)
    for n in range(40):
        M.cp_store_q8(rows[:, n:n + 1].contiguous(), i32([n]), i32([n + 1]), i32(table), b, sb)
    assert M.device_status() == 0
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(sa, sb)


@pytest.mark.parametrize("values", [
    [0.0], [float("nan"), 1.0], [float("inf"), -float("inf"), 3.0], [float("nan")], [3.0e38, 1.0],
    [1e-30, -1e-38], [448.0, 449.0], [1.75, 1.7578125], [2.0 ** -40],
])
def test_store_special_values(values):
    rows = torch.zeros(1, 3, 576, dtype=torch.bfloat16, device=DEV)
    rows[0, 1, :len(values)] = torch.tensor(values).to(torch.bfloat16).to(DEV)
    cache, scales = new_pool(2, 16, poison=False)
    check_store(rows, [0], [3], [[1]], cache, scales, 1, 0, 1)
    # behind earlier rows
    rows[0, 0, 3] = 5.0
    check_store(rows, [3], [6], [[1]], cache, scales, 1, 0, 1)


def test_store_keeps_or_grows_any_earlier_scale():
    rows = torch.full((1, 1, 576), 3.0, dtype=torch.bfloat16, device=DEV)
    for old in (0.3, 1.0, 1e-4, 7.7e-3, 2.0 ** -32, 2.0 ** 64):
        cache, scales = new_pool(1, 16, poison=False)
        cache[0, :5] = f8(np.linspace(-448, 448, 5 * 576).reshape(5, 576))
        scales.fill_(old)
        old32 = float(scales[0, 0])
        new = max(old32, 2.0 ** -7)
        M.cp_store_q8(rows, i32([5]), i32([6]), i32([[0]]), cache, scales)
        assert M.device_status() == 0 and float(scales[0, 0]) == new
        stands = n64(cache[0, :5].float()) * new
        was = n64(f8(np.linspace(-448, 448, 5 * 576).reshape(5, 576)).float()) * old32
        # one more rounding: half a step, or half a subnormal step
        assert np.all(np.abs(stands - was) <= np.maximum(2.0 ** -4 * np.abs(was), 2.0 ** -10 * new) * 1.001)
        got = n64(cache[0, 5].float()) * new
        assert np.all(np.abs(got - 3.0) <= max(2.0 ** -4 * 3, 2.0 ** -10 * new) * 1.001)
    # an earlier scale outside the range is taken as 1
    for old in (0.0, -1.0, float("nan"), float("inf"), 1e-12):
        cache, scales = new_pool(1, 16, poison=False)
        scales.fill_(old)
        M.cp_store_q8(rows, i32([5]), i32([6]), i32([[0]]), cache, scales)
        assert M.device_status() == BAD_SCALE and float(scales[0, 0]) == 1.0 and (cache[0, 5].float() == 3).all()


def test_store_bad_data_writes_nothing():
    rows = torch.ones(3, 20, 576, dtype=torch.bfloat16, device=DEV)

    def call(ctx, total, table, bits, N=20):
        cache, scales = new_pool(4, 16)
        before = cache.view(torch.uint8).clone()
        M.cp_store_q8(rows[:len(ctx), :N].contiguous(), i32(ctx), i32(total), i32(table), cache, scales)
        assert M.device_status() == bits
        return cache.view(torch.uint8) != before
    assert not call([0], [16], [[9]], BAD_PAGE).any()
    assert not call([0], [16], [[-1]], BAD_PAGE).any()
    w = call([0], [20], [[1]], BAD_VBLOCK)                # the second page is past the table
    assert w[1].all() and not w[[0, 2, 3]].any()
    assert not call([-1], [5], [[1]], BAD_STEP).any()
    w = call([0], [9], [[2]], BAD_STEP, N=4)              # four rows are there, four are stored
    assert w[2, :4].all() and not w[2, 4:].any()
    assert not call([5, 7, 3], [5, 6, 0], [[0], [1], [2]], 0).any()   # nothing new


@pytest.mark.parametrize("N", [1, 3, 16, 100, 8200])
@pytest.mark.parametrize("total", [(1 << 31) - 1, (1 << 31) - 20])
def test_store_lengths_up_to_the_largest(N, total):
    """New tokens up to position 2^31 - 2.  A block behind a request's last group may have a group
    whose first key is 2^31 (3, 100 or 8,200 tokens up to the very end).  The table does not reach
    that far: flagged, nothing written."""
    ctx = total - N
    cache, scales = new_pool(4, 16)
    before = cache.view(torch.uint8).clone(), scales.view(torch.int32).clone()
    rows = torch.ones(2, N, 576, dtype=torch.bfloat16, device=DEV)
    M.cp_store_q8(rows, i32([ctx, 0]), i32([total, 0]), i32([[0, 1, 2, 3], [3, 2, 1, 0]]), cache, scales)
    assert M.device_status() == BAD_VBLOCK
    assert torch.equal(cache.view(torch.uint8), before[0]) and torch.equal(scales.view(torch.int32), before[1])
    # one of 2^26 ranks, whose tables do reach there
    cp = 1 << 26
    cache, scales = new_pool(4, 16, poison=False)
    M.cp_store_q8(rows[:1, :1].contiguous(), i32([ctx]), i32([ctx + 1]), i32([[0, 1, 2, 3]]), cache, scales,
                  cp, ctx // 16 % cp, interleave=16)
    assert M.device_status() == 0
    local = ctx // (cp * 16) * 16 + ctx % 16
    got = cache.view(4 * 16, 576)[local].float() * scales.view(-1)[local // 16]
    assert torch.equal(got, torch.ones_like(got))


def test_store_offsets_beyond_31_bits():
    """A pool of more than 2^31 bytes: pages behind byte 2^31 and 2^32."""
    bs = 64
    nb = (5 << 30) // (bs * 576)
    cache = torch.zeros(nb, bs, 576, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scales = torch.ones(nb, 4, device=DEV)
    table = i32([[nb - 1], [(3 << 30) // (bs * 576)], [0]])
    rows = torch.randn(3, 5, 576, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).to(DEV)
    M.cp_store_q8(rows, i32([0, 0, 0]), i32([5, 5, 5]), table, cache, scales)
    assert M.device_status() == 0
    for b in range(3):
        pg = int(table[b, 0])
        got = cache[pg, :5].float() * scales[pg, 0]
        x = rows[b].float()
        assert ((got - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * scales[pg, 0]).all()
    # and the decode reads them there
    q = torch.randn(3, 1, 16, 576, generator=torch.Generator().manual_seed(10)).to(torch.bfloat16).to(DEV)
    out, lse = M.mla_decode_q8(q, cache, scales, table, i32([5, 5, 5]), None, 1, 1, 0, SCALE)
    assert M.device_status() == 0
    for b in range(3):
        pg = int(table[b, 0])
        check_rows(q[b], out[b:b + 1], lse[b:b + 1], n64(cache[pg, :5].float()), n64(scales[pg, :1]).repeat(16)[:5],
                   [5], True)


# =============================================================================================
# decode
# =============================================================================================
def check_rows(q, out, lse, v8, sc, see, base_e):
    """One request: q [q_len, H, 576], its stored values v8 [n, 576] and each key's scale, see[i]
    the keys row i sees."""
    u = 2.0 ** -24
    worst = 0.0
    q, out, lse = n64(q), n64(out), n64(lse)
    err2 = ref2 = 0.0
    for i, n in enumerate(see):
        o, l = out[i], lse[i]
        if n == 0:
            assert np.all(o == 0) and np.all(np.isneginf(l))
            continue
        k = v8[:n] * sc[:n, None]
        s = SCALE * (q[i] @ k.T)
        top = s.max(1, keepdims=True)
        e = np.exp(s - top)
        z = e.sum(1, keepdims=True)
        w = e / z
        ref = w @ k[:, :512]
        A = w @ np.abs(k[:, :512])
        ws = w * sc[:n]
        qmax = np.abs(q[i]).max(1, keepdims=True)
        ka = np.abs(k)
        delta = SCALE * (2.0 ** -17 * qmax * ka.sum(1)[None] + 132 * u * (np.abs(q[i]) @ ka.T))
        delta = (delta + 8 * u * (np.abs(s) + np.abs(np.log2(sc[:n])) + 64) + 2.0 ** -22).max(1)[:, None]
        bound = (2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2 * np.expm1(2 * delta)) * A
                 + 2.0 ** -14 * ws.max(1)[:, None] * np.abs(v8[:n, :512]).sum(0)[None] + 1e-30)
        assert np.all(np.isfinite(o))
        worst = max(worst, float((np.abs(o - ref) / bound).max()))
        err2 += float(((o - ref) ** 2).sum())
        ref2 += float((ref ** 2).sum())
        ref_l = (top + np.log(z))[:, 0] / (1.0 if base_e else math.log(2.0))
        lb = (delta[:, 0] + 1e-6 * (1 + np.abs(ref_l))) / (1.0 if base_e else math.log(2.0))
        assert np.all(np.abs(l - ref_l) <= lb), (float((np.abs(l - ref_l) / lb).max()), n)
    assert worst <= 1.0, worst
    assert err2 <= 2.0 ** -14 * ref2, math.sqrt(err2 / max(ref2, 1e-300))
    return worst


def make_case(B, H, q_len, G, bs, cp, il, seed, spread=0, width_extra=1, pow2=True):
    """Queries, and every rank's pool filled by the oracle's store (unwritten slots and their
    scales NaN).  spread: rows' sizes vary by 2^+-spread."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    G = np.asarray(G)
    pages = -(-int(G.max()) // (bs * cp)) + width_extra
    nb = B * pages + 1
    table = random_table(rng, B, pages, nb)
    q = torch.randn(B, q_len, H, 576, generator=g).to(torch.bfloat16)
    pools = []
    for rank in range(cp):
        cache = np.full((nb, bs, 576), np.nan)
        scales = np.full((nb, bs // 16), np.nan)
        for b in range(B):
            n = int(R.ref_local_len(int(G[b]), cp, rank, il))
            if n == 0:
                continue
            x = torch.randn(n, 576, generator=g).numpy().astype(np.float64)
            x *= 2.0 ** rng.integers(-spread, spread + 1, (n, 1)) if spread else 1.0
            ng = -(-n // 16)
            xp = np.zeros((ng * 16, 576))
            xp[:n] = x
            s = np.array([Q.ref_scale(float(np.abs(t).max())) for t in xp.reshape(ng, -1)])
            if not pow2:
                s = np.float32(s * rng.uniform(0.7, 1.9, ng)).astype(np.float64)
            v = Q.ref_e4m3(xp / np.repeat(s, 16)[:, None])
            for j in range(-(-n // bs)):
                m = min(bs, n - j * bs)
                cache[table[b, j], :m] = v[j * bs:j * bs + m]
                mg = -(-m // 16)
                scales[table[b, j], :mg] = s[j * bs // 16:j * bs // 16 + mg]
        pools.append((cache, scales))
    return q, G, table, pools


def gpu_pool(pool):
    return f8(pool[0]), torch.tensor(pool[1], dtype=torch.float32, device=DEV)


def check_request(b, q, out, lse, G, table, pool, q_len, cp, rank, il, causal, base_e):
    n = int(R.ref_local_len(int(G[b]), cp, rank, il))
    bs = pool[0].shape[1]
    pg = table[b, :max(1, -(-n // bs))]
    v8 = pool[0][pg].reshape(-1, 576)[:n]
    sc = np.repeat(pool[1][pg].reshape(-1), 16)[:n]
    pre = R.ref_row_global_prefix(int(G[b]), q_len, causal)
    see = [min(n, int(R.ref_local_len(int(x), cp, rank, il))) for x in pre] if causal else [n] * q_len
    T = slice(b * q_len, (b + 1) * q_len)
    return check_rows(q[b], out[T], lse[T], v8, sc, see, base_e)


CASES = [
    # B, H, q_len, G, bs, cp, il, causal, base_e, spread
    (2, 16, 3, [37, 130], 16, 1, 1, True, True, 0),
    (1, 1, 1, [1], 16, 1, 1, True, True, 0),
    (3, 5, 2, [1, 16, 17], 16, 1, 1, True, False, 2),
    (4, 16, 4, [3, 1, 2, 4], 32, 1, 1, True, True, 0),        # rows that see no key
    (2, 64, 1, [127, 129], 64, 1, 1, True, True, 1),
    (2, 128, 1, [1000, 128], 64, 1, 1, True, True, 0),
    (2, 128, 4, [900, 257], 64, 2, 1, True, False, 3),
    (2, 24, 5, [300, 777], 48, 3, 4, True, True, 0),          # 48-slot pages, 120 rows
    (3, 64, 4, [1100, 64, 7], 64, 2, 1, True, False, 0),
    (2, 100, 3, [640, 65], 192, 1, 1, True, True, 2),
    (2, 96, 16, [400, 33], 128, 4, 16, True, True, 0),        # 1,536 rows
    (2, 16, 8, [700, 129], 32, 8, 2, False, True, 0),         # non-causal
    (1, 8, 1, [5000], 64, 1, 1, True, True, 4),               # split over many blocks
    (2, 128, 2, [3000, 1], 64, 16, 1, True, True, 0),         # ranks without a key
]


@pytest.mark.parametrize("B,H,q_len,G,bs,cp,il,causal,base_e,spread", CASES)
def test_decode_matches_oracle(B, H, q_len, G, bs, cp, il, causal, base_e, spread, kernel):
    q, G, table, pools = make_case(B, H, q_len, G, bs, cp, il, 700 + H + q_len, spread)
    worst = 0.0
    for rank in sorted({0, cp // 2, cp - 1}):
        cache, scales = gpu_pool(pools[rank])
        seq = R.ref_local_len(G, cp, rank, il)
        out = torch.full((B * q_len, H, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
        lse = torch.full((B * q_len, H), float("nan"), device=DEV)
        M.mla_decode_q8(q.to(DEV), cache, scales, bt32(table), i32(seq), i32(G), q_len, cp, rank, SCALE,
                        out=out, lse=lse, lse_base_e=base_e, causal=causal, interleave=il)
        assert M.device_status() == 0
        for b in range(B):
            worst = max(worst, check_request(b, q, out, lse, G, table, pools[rank], q_len, cp, rank, il,
                                             causal, base_e))
    print(f"[q8] {kernel} B{B} H{H} q{q_len}: bound used {worst:.3f}")


@pytest.mark.parametrize("H,q_len", [(32, 1), (33, 1), (13, 5), (64, 2), (129, 1), (7, 16)])
def test_decode_row_counts_around_a_unit(H, q_len, units):
    # 32, 33, 65, 128, 129 and 112 rows: whole units, one row past a unit, odd head counts
    q, G, table, pools = make_case(3, H, q_len, [129, 20, 256], 256, 1, 1, 60 + H)
    cache, scales = gpu_pool(pools[0])
    out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, bt32(table), i32(G), None, q_len, 1, 0, SCALE)
    assert M.device_status() == 0
    for b in range(3):
        check_request(b, q, out, lse, G, table, pools[0], q_len, 1, 0, 1, True, True)


@pytest.mark.parametrize("B,H,q_len,workspace", [(1500, 8, 1, True), (1300, 40, 1, True), (900, 8, 2, False),
                                                 (700, 70, 1, False)])
def test_decode_many_requests(B, H, q_len, workspace):
    """More requests than a block has threads, some without a key; every request is checked
    against attention over its pages (shared among requests here) in float64 on the GPU."""
    g = torch.Generator().manual_seed(B)
    rng = np.random.default_rng(B)
    bs, nb, pages = 32, 64, 12
    G = rng.integers(0, bs * pages + 1, B)
    G[rng.random(B) < 0.1] = 0
    G[rng.random(B) < 0.1] = 1
    wide = torch.full((B, pages + 5), -1, dtype=torch.int32, device=DEV)
    table = wide[:, 2:2 + pages]                          # a strided table
    table.copy_(torch.randint(0, nb, (B, pages), generator=g))
    x = torch.randn(nb, bs, 576, generator=g, device="cpu").numpy().astype(np.float64)
    s = np.array([[Q.ref_scale(float(np.abs(x[p, 16 * j:16 * j + 16]).max())) for j in range(bs // 16)] for p in range(nb)])
    v = Q.ref_e4m3(x / np.repeat(s, 16, 1)[..., None])
    cache, scales = gpu_pool((v, s))
    q = torch.randn(B, q_len, H, 576, generator=g).to(torch.bfloat16).to(DEV)
    ws = None if workspace else torch.empty(0, dtype=torch.uint8, device=DEV)
    out, lse = M.mla_decode_q8(q, cache, scales, table, i32(G), None, q_len, 1, 0, SCALE, workspace=ws)
    assert M.device_status() == 0
    keys = (cache.to(torch.float64) * torch.repeat_interleave(scales.double(), 16, 1)[..., None])
    n = torch.arange(bs * pages, device=DEV)
    Gt = torch.tensor(G, device=DEV)
    for b0 in range(0, B, 100):
        k = keys[table[b0:b0 + 100].long()].reshape(-1, bs * pages, 576)
        see = Gt[b0:b0 + 100, None] - (q_len - 1 - torch.arange(q_len, device=DEV))
        sc = SCALE * torch.einsum("bihd,bnd->bihn", q[b0:b0 + 100].double(), k)
        sc = sc.masked_fill((n >= see[..., None])[:, :, None], -math.inf)
        top = sc.amax(-1, keepdim=True)
        w = torch.exp(sc - torch.where(top == -math.inf, 0.0, top))
        z = w.sum(-1, keepdim=True)
        o = torch.where(z > 0, torch.einsum("bihn,bnd->bihd", w, k[..., :512]) / z, 0.0)
        l = (top + z.log())[..., 0]
        T = slice(b0 * q_len, (b0 + k.shape[0]) * q_len)
        go, gl = out[T].double().view_as(o), lse[T].double().view_as(l)
        A = torch.where(z > 0, torch.einsum("bihn,bnd->bihd", w, k[..., :512].abs()) / z, 0.0)
        # the docstring's bound, its terms in M and delta at most 2^-7 A for these values
        assert bool(((go - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -6 * A).all())
        assert torch.equal(torch.isneginf(gl), torch.isneginf(l))
        fin = torch.isfinite(l)
        assert bool(((gl - l)[fin].abs() <= 1e-3).all())


def test_decode_on_another_stream_than_the_current_one(units):
    q, G, table, pools = make_case(2, 64, 2, [300, 900], 64, 1, 1, 61)
    cache, scales = gpu_pool(pools[0])
    args = (q.to(DEV), cache, scales, bt32(table), i32(G), None, 2, 1, 0, SCALE)
    want = M.mla_decode_q8(*args)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append(M.mla_decode_q8(*args, stream=s))
        torch.full((1 << 20,), float("nan"), device=DEV)    # memory of the current stream, reused at once
    s.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    assert M.device_status() == 0


@pytest.mark.parametrize("B,H,q_len,G", [(2, 128, 2, [700, 2000]), (3, 16, 1, [100, 1, 515])])
def test_decode_without_workspace_and_without_lse(B, H, q_len, G, units):
    q, G, table, pools = make_case(B, H, q_len, G, 64, 1, 1, 41)
    cache, scales = gpu_pool(pools[0])
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    args = (q.to(DEV), cache, scales, bt32(table), i32(G), None, q_len, 1, 0, SCALE)
    out, lse = M.mla_decode_q8(*args, workspace=none)
    for b in range(B):
        check_request(b, q, out, lse, G, table, pools[0], q_len, 1, 0, 1, True, True)
    o2, l2 = M.mla_decode_q8(*args, workspace=none, return_lse=False)
    assert l2 is None and torch.equal(out, o2) and M.device_status() == 0


# How this file's bound covers a weight's second part as it is now.  In e4m3 with a dither it is off by
# up to a step, 2^-9, against a reference of 2^6 or more: 2^-15 M, inside the 2^-14 M there.  In
# e5m2 (tiles with a row whose largest of 16 weights is below 2^-9 of its reference, and tiles that
# move one) by 2^-7 of the weight, where 2^-8 and 2^-10 for partials and half precision are counted, and
# a step of 2^-16: the difference, 2^-8 of a weight, is inside 2^-14 M per key for weights below
# 2^-6 M, and for the few above it inside 2^-14 M of each of the 64 keys or more that there are (a
# request of fewer is one tile, whose rows' largest are put at 2^12 and have no error).
@pytest.mark.parametrize("n", [16384, 131072, 524288])
@pytest.mark.parametrize("where,big,raised", [(0, 1, 0), (0, 32, 0), (5000, 1, 0), (5000, 32, 0), (0, 1, 192),
                                              (5000, 32, 192), (0, 1, 384)])
def test_decode_many_small_weights_below_one_large(n, where, big, raised, kernel):
    """One key of value 0 above n - 1 equal ones, whose weights are e^-5 to e^-15 of its (336 rows,
    0.03 apart), in one block's hands (no workspace); the large key's 16 slots have the others'
    scale or 32 times that.  With `raised` every 32nd key is e^3.5 or e^6.9 above the others and of
    value 0.  Every rounding of the small weights is the same or follows the key's number, so
    nothing averages out that the kernel does not make average out.

    Bound, A = sum_l w_l S_l |v_l| = |ref| here, M the large key's weight times scale, Z all other
    weights' sum: the output 2^-8; a weight 2^-7 of itself; what the dithers leave of a sum of equal
    weights: a few steps (8) of 2^-16 against a reference of 2^6 or more: 2^-19 M, or, where 16 keys'
    largest is 2^-3 or more, 8 of 2^-9 over n / 32 such (2^-6 / (512 2^-3) = 2^-12 Z); the 31 keys
    beside the large one 2^-3 of themselves: 2^-3 31 / 16,384 < 2^-11; scores: below 2^-12.
    2^-8 + 2^-7 + 2^-11 + 2^-12 < 2^-6 of A, 2^-19 M, and with raised keys 2^-12 Z."""
    if kernel == "mma" and n > 16384:
        pytest.skip("the warp-level kernel rounds to bf16; one length is enough")
    rows, bs = 336, 64
    gap = torch.linspace(5.0, 15.0, rows)
    q = torch.zeros(1, 3, rows // 3, 576)
    q.view(rows, 576)[:, 575] = gap / (4 * SCALE)
    q[..., 574] = 16.0
    q = q.to(torch.bfloat16)
    c = (torch.arange(512) % 13 + 1) * 4.0 * (1 - 2 * (torch.arange(512) % 2))
    keys = torch.zeros(n, 576)
    keys[:, :512] = c
    high = n // 32 if raised else 0
    if raised:
        keys[16::32] = 0
        keys[16::32, 574] = raised
    keys[where // 16 * 16:where // 16 * 16 + 16] /= big
    keys[where] = 0
    keys[where, 575] = 256 / big
    cache = keys.to(torch.float8_e4m3fn).to(DEV).view(n // bs, bs, 576)
    assert torch.equal(cache.view(n, 576).float().cpu(), keys)
    scales = torch.full((n // bs, bs // 16), 2.0 ** -6, device=DEV)
    scales.view(-1)[where // 16] *= big
    table = bt32(np.arange(n // bs)[None])
    out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, table, i32([n]), None, 3, 1, 0, SCALE, causal=False,
                               workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    assert M.device_status() == 0
    s = SCALE * 4 * n64(q).reshape(rows, 576)[:, 575]
    low_w, high_w = (n - 1 - high) * np.exp(-s), high * np.exp(SCALE * 16 * raised / 64 - s)
    z = 1 + low_w + high_w
    ref = (low_w / z)[:, None] * c.double().numpy()[None] / 64
    cmax = float(c.abs().max())
    bound = 2.0 ** -6 * np.abs(ref) + (2.0 ** -19 * big / z)[:, None] * cmax / 64
    if raised:
        bound += 2.0 ** -12 * ((low_w + high_w) / z)[:, None] * cmax / 64
    err = np.abs(n64(out).reshape(rows, 512) - ref)
    print(f"[q8] {kernel} n {n} at {where} x{big} raised {raised}: {float((err / np.abs(ref)).max()):.5f} of the output, "
          f"bound used {float((err / bound).max()):.3f}")
    assert (err <= bound).all()
    # the LSE's sum: a thread adds twice a tile of 128 keys to a float that grows to its share of the
    # sum (2 n / 128 roundings of at most 2^-24 of it), and fewer than 16 more join the shares (the
    # warp-level kernel: 4 a tile of 32); scores up to 15 / ln 2 and reference as in this file's header
    # (8 u (22 + 64 + 6) < 5e-5), 1e-6 (1 + |lse|) of the logarithm and the result's rounding
    adds = (n / 8 if kernel == "mma" else n / 64) + 16
    assert np.abs(n64(lse).reshape(rows) - (s + np.log(z))).max() <= adds * 2.0 ** -24 + 5e-5 + 2e-5


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("gap,big", [(6.0, 1), (12.0, 1), (12.0, 16), (16.0, 1)])
def test_decode_values_beside_one_large_weight(gap, big, split, kernel):
    """A key of value 0 takes nearly all the weight (as first tokens do); the output is what the
    others make of the rest.  Their weights are used to within 2^-7 of themselves, however small
    against the large one: bound as in this file's header, but the term in M is two halves of a step
    of 2^-16 against a reference of 2^6, 2^-21 M; 12 units and more (2^17, and 2^13 above the others'
    largest) of 2^11 or more: 2^-26 M.  The norm of the error is at most 2^-7 of the output's, and the
    dithers' own: each is a step of 2^-16 or nothing, off by at most half a step in the mean square
    (p (1 - p) <= 1 / 4): 2^-17 against the reference, (sum_l |v_l|^2)^1/2 M, twice that for their
    dependence on one another."""
    n, rows, bs = 4096, 128, 64
    g = torch.Generator().manual_seed(int(gap) + big)
    q = torch.randn(1, 1, rows, 576, generator=g)
    q[..., 575] = 32.0
    q = q.to(torch.bfloat16)
    x = torch.randn(n, 576, generator=g).numpy().astype(np.float64) * 0.6
    x[:, 575] = 0
    at = 700
    x[at] = 0
    x[at, 575] = gap / (32 * SCALE)
    sc = np.array([Q.ref_scale(float(np.abs(t).max())) for t in x.reshape(-1, 16 * 576)])
    sc[at // 16] *= big
    v = Q.ref_e4m3(x / np.repeat(sc, 16)[:, None])
    cache, scales = gpu_pool((v.reshape(n // bs, bs, 576), sc.reshape(n // bs, bs // 16)))
    out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, bt32(np.arange(n // bs)[None]), i32([n]), None, 1, 1, 0, SCALE,
                               workspace=None if split else torch.empty(0, dtype=torch.uint8, device=DEV))
    assert M.device_status() == 0
    k = v * np.repeat(sc, 16)[:, None]
    s = SCALE * (n64(q)[0, 0] @ k.T)
    w = np.exp(s - s.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    ref, A = w @ k[:, :512], w @ np.abs(k[:, :512])
    Mx = (w * np.repeat(sc, 16)).max(1, keepdims=True)
    u = 2.0 ** -24
    delta = SCALE * (2.0 ** -17 * 32 * np.abs(k).sum(1)[None] + 132 * u * (np.abs(n64(q)[0, 0]) @ np.abs(k).T))
    delta = (delta + 8 * u * (np.abs(s) + 64) + 2.0 ** -22).max(1)[:, None]
    o = n64(out)[0]
    ref_at = 2.0 ** (6 if gap < 12 else 11)
    bound = (2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2.0 ** -10 + 2 * np.expm1(2 * delta)) * A
             + 2.0 ** -15 / ref_at * Mx * np.abs(v[:, :512]).sum(0)[None])
    noise = 2.0 ** -16 / ref_at * float(np.linalg.norm(Mx)) * math.sqrt(float((v[:, :512] ** 2).sum()))
    off, size = float(np.linalg.norm(o - ref)), float(np.linalg.norm(ref))
    print(f"[q8] {kernel} gap {gap} x{big}: error {off / size:.5f} of the output (dithers {noise / size:.5f}), bound used "
          f"{float((np.abs(o - ref) / bound).max()):.3f}")
    assert (np.abs(o - ref) <= bound).all()
    assert off <= 2.0 ** -7 * size + noise


def test_decode_any_scales(kernel):
    # scales that are no powers of two, from 2^-32 to 2^64
    q, G, table, pools = make_case(2, 16, 2, [200, 75], 32, 1, 1, 43, spread=3, pow2=False)
    cache, scales = gpu_pool(pools[0])
    pool = (pools[0][0], n64(scales))
    out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, bt32(table), i32(G), None, 2, 1, 0, SCALE)
    assert M.device_status() == 0
    for b in range(2):
        check_request(b, q, out, lse, G, table, pool, 2, 1, 0, 1, True, True)


@pytest.mark.parametrize("ends", ["large", "small", "both", "large, no power of two"])
@pytest.mark.parametrize("split", [True, False])
def test_decode_scales_at_the_ends_of_their_range(ends, split, kernel):
    """Scales of 2^64 and of 2^-32 over values that are not 0, queries of a size that gives ordinary
    scores; and both ends and 1 in turn in one request, the keys of 2^64 with weights about 2^-64 of
    the others', so that they matter as much in the output and nothing in the LSE."""
    q, G, table, pools = make_case(2, 40, 2, [300, 1203], 32, 1, 1, 47, pow2=ends != "large, no power of two")
    v, s = pools[0]
    if ends == "both":
        s[:] = np.array([2.0 ** 64, 1.0, 2.0 ** -32])[np.arange(s.size) % 3].reshape(s.shape)
        v[..., 512:] = 0
        rope = np.random.default_rng(5).choice([-36.0, -40.0, -44.0], v.shape[:2] + (64,))
        v[..., 575] = rope[..., 0]                                     # scores of -42, -46, -51 at 2^64
        q = torch.zeros_like(q)
        q[..., 575] = 2.0 ** -60
    else:
        top = float(np.nanmax(s))
        # (over powers of two: as they are, and up to 2^64 exactly)
        s *= (2.0 ** 64 if ends.startswith("large") else 2.0 ** -32) / (top if ends != "small" else float(np.nanmin(s)))
        s = np.float32(s).astype(np.float64)
        x = float(np.nanmedian(s)) * 150                               # about a key's size
        q = (q.double() / (SCALE * x * 24)).to(torch.bfloat16)
        assert np.nanmax(s) <= 2.0 ** 64 and np.nanmin(s) >= 2.0 ** -32
    cache, scales = gpu_pool((v, s))
    ws = None if split else torch.empty(0, dtype=torch.uint8, device=DEV)
    out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, bt32(table), i32(G), None, 2, 1, 0, SCALE, workspace=ws)
    assert M.device_status() == 0
    for b in range(2):
        check_request(b, q, out, lse, G, table, (v, s), 2, 1, 0, 1, True, True)


def test_decode_zero_blocks_and_growing_scores(kernel):
    """Blocks of zeros (smallest scale) among ordinary ones, and scores that grow along the
    context by far more than a weight's 8-bit range."""
    q, G, table, pools = make_case(1, 32, 2, [900], 64, 1, 1, 44)
    v, s = pools[0]
    s[table[0, 3]] = 2.0 ** -32
    v[table[0, 3]] = 0.0
    qs = q.double().numpy()[0, 1, 0]
    for l, x in ((200, 30.0), (500, 80.0), (501, 79.0), (800, 150.0)):   # scores, in log units
        k = qs * (x / SCALE / float(qs @ qs))
        pg, sl = table[0, l // 64], l % 64
        s[pg, sl // 16] = max(s[pg, sl // 16], Q.ref_scale(np.abs(k).max()))
        v[pg, sl] = Q.ref_e4m3(k / s[pg, sl // 16])
    cache, scales = gpu_pool((v, s))
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, bt32(table), i32(G), None, 2, 1, 0, SCALE, workspace=ws)
        assert M.device_status() == 0
        check_request(0, q, out, lse, G, table, (v, s), 2, 1, 0, 1, True, True)


@pytest.mark.parametrize("turn", [None, 140, 256])
def test_decode_scores_far_below_zero(kernel, turn):
    """Every key's score is about -150 (natural units; 2^-216 of a score of 0), or those of the keys
    before `turn`: a row's weights are relative to its own largest score."""
    q, G, table, pools = make_case(2, 48, 1, [300, 700], 64, 1, 1, 59)
    g = torch.Generator().manual_seed(59)
    base = torch.randn(576, generator=g).double().numpy()
    q = (torch.tensor(base) + 0.05 * torch.randn(q.shape, generator=g)).to(torch.bfloat16)
    away = -150.0 / SCALE / float(base @ base) * base
    v, s = pools[0]
    for b in range(2):
        for l in range(int(G[b])):
            x = 0.3 * torch.randn(576, generator=g).double().numpy() + (away if turn is None or l < turn else 0.0)
            pg, sl = table[b, l // 64], l % 64
            s[pg, sl // 16] = 0.125                          # (|x| is below 448 / 8)
            v[pg, sl] = Q.ref_e4m3(x / 0.125)
    cache, scales = gpu_pool((v, s))
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, bt32(table), i32(G), None, 1, 1, 0, SCALE, workspace=ws)
        assert M.device_status() == 0
        for b in range(2):
            check_request(b, q, out, lse, G, table, (v, s), 1, 1, 0, 1, True, True)


def test_decode_queries_of_any_size(kernel):
    # rows of q from 1e-30 to 1, one of zeros
    q, G, table, pools = make_case(2, 64, 1, [333, 64], 64, 1, 1, 45)
    q = q * (10.0 ** torch.linspace(-30, 0, 64))[None, None, :, None]
    q[:, :, 5] = 0
    q = q.to(torch.bfloat16)
    cache, scales = gpu_pool(pools[0])
    out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, bt32(table), i32(G), None, 1, 1, 0, SCALE)
    for b in range(2):
        check_request(b, q, out, lse, G, table, pools[0], 1, 1, 0, 1, True, True)
    assert M.device_status() == 0


def test_decode_nan_rows_and_nan_keys(units):
    """A NaN or an infinity in a row of q makes that row NaN, and only it; a NaN in a stored key
    makes the rows that see the key NaN, and only them."""
    for B, H, q_len, G in ((2, 64, 1, [333, 64]), (1, 16, 2, [4000])):
        q, G, table, pools = make_case(B, H, q_len, G, 64, 1, 1, 52)
        cache, scales = gpu_pool(pools[0])
        args = (cache, scales, bt32(table), i32(G), None, q_len, 1, 0, SCALE)
        out, lse = M.mla_decode_q8(q.to(DEV), *args)
        bad = q.clone()
        bad[0, 0, 7, 100] = float("nan")
        bad[0, 0, 9, 3] = -float("inf")
        o2, l2 = M.mla_decode_q8(bad.to(DEV), *args)
        hit = torch.zeros(B * q_len, H, dtype=torch.bool, device=DEV)
        hit[0, [7, 9]] = True
        assert torch.isnan(o2[hit]).all() and torch.isnan(l2[hit]).all()
        assert torch.equal(o2[~hit], out[~hit]) and torch.equal(l2[~hit], lse[~hit])
    # draft rows: the last key is NaN, which only the last row sees
    for G in (100, 128, 129, 700):
        q, Gs, table, pools = make_case(1, 16, 4, [G], 32, 1, 1, 53)
        v, s = pools[0]
        v[table[0, (G - 1) // 32], (G - 1) % 32, 5:576:70] = np.nan
        cache, scales = gpu_pool((v, s))
        out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, bt32(table), i32(Gs), None, 4, 1, 0, SCALE)
        assert torch.isnan(out[3]).all() and torch.isnan(lse[3]).all()
        pre = np.concatenate([v[table[0, j]] for j in range(-(-G // 32))])[:G - 1]
        sc = np.concatenate([np.repeat(s[table[0, j]], 16) for j in range(-(-G // 32))])[:G - 1]
        check_rows(q[0, :3], out[:3], lse[:3], pre, sc, [G - 3, G - 2, G - 1], True)
    assert M.device_status() == 0


def test_decode_timeout_reports_and_recovers(units):
    """One role of every block first waits for an arrival that never comes, with a limit of 200 us:
    the call returns, reports it, and the next call is right."""
    q, G, table, pools = make_case(2, 128, 2, [3000, 200], 64, 1, 1, 54)
    cache, scales = gpu_pool(pools[0])
    args = (q.to(DEV), cache, scales, bt32(table), i32(G), None, 2, 1, 0, SCALE)
    prev, stall = M.set_wait_limit_ns(200_000), M.set_test_stall(True)
    try:
        M.mla_decode_q8(*args)
        torch.cuda.synchronize()
        bits = M.device_status()
    finally:
        M.set_test_stall(stall)
        M.set_wait_limit_ns(prev)
    assert bits == 8, f"{bits:#x}"
    out, lse = M.mla_decode_q8(*args)
    assert M.device_status() == 0
    for b in range(2):
        check_request(b, q, out, lse, G, table, pools[0], 2, 1, 0, 1, True, True)


def test_decode_bad_scale_and_bad_page_are_flagged(kernel):
    q, G, table, pools = make_case(1, 16, 1, [100], 16, 1, 1, 46)
    v, s = pools[0]
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-12):
        s2 = s.copy()
        s2[table[0, 2]] = bad
        cache, scales = gpu_pool((v, s2))
        out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, bt32(table), i32(G), None, 1, 1, 0, SCALE)
        assert M.device_status() == BAD_SCALE
        s2[table[0, 2]] = 1.0
        check_request(0, q, out, lse, G, table, (v, s2), 1, 1, 0, 1, True, True)
    cache, scales = gpu_pool((v, s))
    for page in (-1, cache.shape[0], 2 ** 31 - 1, -2 ** 31):
        t2 = table.copy()
        t2[0, 2] = page
        out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, bt32(t2), i32(G), None, 1, 1, 0, SCALE)
        assert M.device_status() == BAD_PAGE
        v2, s2 = v.copy(), s.copy()                       # its keys are read as zeros
        v2[table[0, 2]], s2[table[0, 2]] = 0.0, 1.0
        check_request(0, q, out, lse, G, table, (v2, s2), 1, 1, 0, 1, True, True)


def test_decode_seq_lens_beyond_the_table_are_clamped(kernel):
    q, G, table, pools = make_case(1, 16, 1, [64], 16, 1, 1, 47, width_extra=0)
    cache, scales = gpu_pool(pools[0])
    out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, i32(table), i32([1000]), i32([1000]), 1, 1, 0, SCALE)
    assert M.device_status() == TOO_LONG
    check_request(0, q, out, lse, G, table, pools[0], 1, 1, 0, 1, True, True)
    out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, i32(table), i32([-5]), i32([64]), 1, 1, 0, SCALE)
    assert (out == 0).all() and torch.isneginf(lse).all() and M.device_status() == 0


@pytest.mark.parametrize("cp,il,causal", [(2, 1, True), (8, 2, True), (3, 1, False)])
def test_decode_shards_equals_rank_by_rank(cp, il, causal, kernel):
    B, H, q_len = 3, 64, 2
    q, G, table, pools = make_case(B, H, q_len, [700, 5, 260], 32, cp, il, 48)
    nb = pools[0][0].shape[0]
    cache = torch.cat([gpu_pool(p)[0].view(torch.uint8) for p in pools]).view(torch.float8_e4m3fn)
    scales = torch.cat([gpu_pool(p)[1] for p in pools])
    seq = np.concatenate([R.ref_local_len(G, cp, r, il) for r in range(cp)])
    bt = np.concatenate([table + r * nb for r in range(cp)])
    out, lse = M.mla_decode_shards_q8(q.to(DEV), cache, scales, bt32(bt), i32(seq), i32(G), q_len, cp, SCALE,
                                      causal=causal, interleave=il)
    for r in range(cp):
        for b in range(B):
            check_request(b, q, out[r], lse[r], G, table, pools[r], q_len, cp, r, il, causal, True)
    # merged, it is attention over every rank's keys
    mo, ml = R.ref_lse_merge(n64(out), n64(lse))
    go = torch.empty(B * q_len, H, device=DEV)
    go_out, _ = M.lse_merge(out, lse, out_lse=go)
    assert np.abs(n64(go_out) - mo).max() <= 2.0 ** -8 * np.abs(mo).max() + 1e-6
    assert np.nanmax(np.abs(n64(go) - ml)) <= 1e-4
    assert M.device_status() == 0


def test_decode_on_a_stream_and_in_a_graph():
    """Captured with its tables and its store, and replayed with other inputs."""
    B, H, q_len, bs = 2, 64, 2, 64
    g = torch.Generator().manual_seed(50)
    nb = 40
    cache, scales = new_pool(nb, bs)
    table = torch.full((B, 16), -1, dtype=torch.int32, device=DEV)
    ring, state = torch.randperm(nb, generator=g).to(torch.int32).to(DEV), i32([0, nb])
    prev, ctx, new = i32([0, 0]), i32([0, 0]), i32([2, 2])
    rows = torch.randn(B, q_len, 576, generator=g).to(torch.bfloat16).to(DEV)
    q = torch.randn(B, q_len, H, 576, generator=g).to(torch.bfloat16).to(DEV)
    ws = M.alloc_workspace_q8(B, H, q_len)
    t = M.cp_step_tables(prev, ctx, new, table, ring, state, bs, q_len)
    M.cp_store_q8(rows, ctx, t.total_lens, table, cache, scales)
    M.mla_decode_q8(q, cache, scales, table, t.seq_lens[0], t.total_lens, q_len, 1, 0, SCALE, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t = M.cp_step_tables(prev, ctx, new, table, ring, state, bs, q_len)
        M.cp_store_q8(rows, ctx, t.total_lens, table, cache, scales)
        out, lse = M.mla_decode_q8(q, cache, scales, table, t.seq_lens[0], t.total_lens, q_len, 1, 0, SCALE,
                                   workspace=ws)
        prev.copy_(t.total_lens)
        state.copy_(t.free_state)
    vc, vs = n64(cache.float()), n64(scales)
    held = np.zeros(B, np.int64)
    for step in range(40):
        n = np.array([2, 1 + step % 2])
        new.copy_(i32(n))
        ctx.copy_(i32(held))
        rows.copy_(torch.randn(B, q_len, 576, generator=g).to(torch.bfloat16))
        q.copy_(torch.randn(B, q_len, H, 576, generator=g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        tab = table.cpu().numpy()
        vc, vs = Q.ref_store_q8(n64(rows), held, held + n, np.maximum(tab, 0), vc, vs, 1, 0)
        held = held + n
        assert t.total_lens.tolist() == held.tolist()
    assert np.array_equal(n64(cache.float()), vc, equal_nan=True)
    for b in range(B):
        check_request(b, q.cpu(), out, lse, held, tab, (vc, vs), q_len, 1, 0, 1, True, True)
    assert M.device_status() == 0


def test_decode_is_repeatable_and_leaves_its_inputs(units):
    q, G, table, pools = make_case(4, 128, 2, [900, 33, 1500, 400], 64, 1, 1, 51)
    cache, scales = gpu_pool(pools[0])
    a = (q.to(DEV), cache, scales, bt32(table), i32(G), None, 2, 1, 0, SCALE)
    ws = M.alloc_workspace_q8(4, 128, 2)
    before = cache.view(torch.uint8).clone()
    o1, l1 = M.mla_decode_q8(*a, workspace=ws)
    ws.fill_(0xff)                                      # whatever the workspace holds
    for _ in range(5):
        o2, l2 = M.mla_decode_q8(*a, workspace=ws)
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    assert torch.equal(cache.view(torch.uint8), before) and M.device_status() == 0


def test_decode_most_rows_a_request_may_have():
    # as many row tiles of 64 as SMs; one head more is refused
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    q, G, table, pools = make_case(1, 4 * sms, 16, [150], 64, 1, 1, 55)
    cache, scales = gpu_pool(pools[0])
    args = (cache, scales, i32(table), i32(G), None, 16, 1, 0, SCALE)
    out, lse = M.mla_decode_q8(q.to(DEV), *args)
    assert M.device_status() == 0
    check_request(0, q, out, lse, G, table, pools[0], 16, 1, 0, 1, True, True)
    more = torch.zeros(1, 16, 4 * sms + 1, 576, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(RuntimeError, match="row tiles"):
        M.mla_decode_q8(more, *args)


def test_decode_pages_used_more_than_once(units):
    # the same page twice in a request, and in two requests
    q, G, table, pools = make_case(2, 64, 2, [330, 200], 32, 1, 1, 56)
    table[0, 4], table[0, 9], table[1, 3] = table[0, 1], table[0, 1], table[0, 0]
    cache, scales = gpu_pool(pools[0])
    out, lse = M.mla_decode_q8(q.to(DEV), cache, scales, bt32(table), i32(G), None, 2, 1, 0, SCALE)
    assert M.device_status() == 0
    for b in range(2):
        check_request(b, q, out, lse, G, table, pools[0], 2, 1, 0, 1, True, True)


def test_decode_two_streams_at_once(units):
    cases = []
    for seed, (H, G) in enumerate(((128, [3000, 500, 40]), (16, [2000, 7000, 900]))):
        q, G, table, pools = make_case(3, H, 2, G, 64, 1, 1, 57 + seed)
        a = (q.to(DEV), *gpu_pool(pools[0]), bt32(table), i32(G), None, 2, 1, 0, SCALE)
        cases.append((a, M.mla_decode_q8(*a), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for (a, _, s), g in zip(cases, got):
            g.append(M.mla_decode_q8(*a, stream=s))
    torch.cuda.synchronize()
    for (_, want, _), g in zip(cases, got):
        for o, l in g:
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    assert M.device_status() == 0


# =============================================================================================
# the wrappers' refusals: nothing is launched, the next call works
# =============================================================================================
def call_of(name):
    a, t2 = i32([0, 0]), i32([[0, 1], [2, 3]])
    cache, scales = new_pool(4, 16)
    tables = dict(prev_lens=a, ctx_lens=a.clone(), new_lens=i32([1, 1]), block_table=t2, free_pages=i32(range(4)),
                  free_state=i32([0, 4]), block_size=16, N=1)
    store = dict(kv_new=torch.zeros(2, 1, 576, dtype=torch.bfloat16, device=DEV), ctx_lens=a, total_lens=i32([1, 1]),
                 block_table=t2, kv_cache=cache, kv_scales=scales)
    decode = dict(q=torch.zeros(2, 1, 8, 576, dtype=torch.bfloat16, device=DEV), kv_cache=cache, kv_scales=scales,
                  block_table=t2, seq_lens=i32([0, 0]), causal_seqlens_global=None, q_len=1, scale=SCALE)
    return {"cp_step_tables": tables, "cp_store_q8": store, "mla_decode_q8": dict(decode, cp_world=1, cp_rank=0),
            "mla_decode_shards_q8": dict(decode, n_shards=1)}[name]


def long_rows(n=4):
    return torch.zeros(2, 2 * n, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("name,change,error", [
    ("cp_step_tables", lambda d: dict(prev_lens=d["prev_lens"].cpu()), ValueError),
    ("cp_step_tables", lambda d: dict(prev_lens=d["prev_lens"].long()), TypeError),
    ("cp_step_tables", lambda d: dict(prev_lens=[0, 0]), TypeError),
    ("cp_step_tables", lambda d: dict(ctx_lens=i32([0])), ValueError),
    ("cp_step_tables", lambda d: dict(new_lens=i32([1, 0, 1])[::2]), ValueError),
    ("cp_step_tables", lambda d: dict(block_table=long_rows()[:, ::2]), ValueError),
    ("cp_step_tables", lambda d: dict(block_table=d["block_table"][:1].expand(2, 2)), RuntimeError),
    ("cp_step_tables", lambda d: dict(block_table=d["block_table"][0]), TypeError),
    ("cp_step_tables", lambda d: dict(free_state=i32([0, 4, 0])), ValueError),
    ("cp_step_tables", lambda d: dict(free_pages=i32([[0, 1]])), ValueError),
    ("cp_step_tables", lambda d: dict(free_pages=i32([])), RuntimeError),
    ("cp_step_tables", lambda d: dict(N=1.5), TypeError),
    ("cp_step_tables", lambda d: dict(N=-1), ValueError),
    ("cp_step_tables", lambda d: dict(N=1 << 40), ValueError),
    ("cp_step_tables", lambda d: dict(N=1 << 30), ValueError),
    ("cp_step_tables", lambda d: dict(n_ranks=0), ValueError),
    ("cp_step_tables", lambda d: dict(n_ranks=2), RuntimeError),
    ("cp_step_tables", lambda d: dict(slots=torch.zeros(1, 2, 1, device=DEV)), TypeError),
    ("cp_step_tables", lambda d: dict(positions=torch.zeros(2, 2, dtype=torch.int64, device=DEV)), ValueError),
    ("cp_store_q8", lambda d: dict(kv_new=d["kv_new"].float()), TypeError),
    ("cp_store_q8", lambda d: dict(kv_new=d["kv_new"][..., :575]), ValueError),
    ("cp_store_q8", lambda d: dict(kv_new=d["kv_new"][0]), ValueError),
    ("cp_store_q8", lambda d: dict(kv_new=d["kv_new"].expand(2, 2, 576)), ValueError),
    ("cp_store_q8", lambda d: dict(kv_cache=d["kv_cache"].view(torch.uint8)), TypeError),
    ("cp_store_q8", lambda d: dict(kv_scales=d["kv_scales"][:3]), ValueError),
    ("cp_store_q8", lambda d: dict(kv_scales=None), TypeError),
    ("cp_store_q8", lambda d: dict(total_lens=i32([1])), ValueError),
    ("cp_store_q8", lambda d: dict(interleave=3), RuntimeError),
    ("mla_decode_q8", lambda d: dict(q=d["q"].float()), TypeError),
    ("mla_decode_q8", lambda d: dict(q_len=0), ValueError),
    ("mla_decode_q8", lambda d: dict(q_len=2), ValueError),
    ("mla_decode_q8", lambda d: dict(q=d["q"][0, 0]), ValueError),
    ("mla_decode_q8", lambda d: dict(q=d["q"].transpose(1, 2)), ValueError),
    ("mla_decode_q8", lambda d: dict(kv_cache=d["kv_cache"][:, :8].contiguous()), ValueError),
    ("mla_decode_q8", lambda d: dict(seq_lens=i32([0, 0, 0])), ValueError),
    ("mla_decode_q8", lambda d: dict(causal_seqlens_global=i32([1])), ValueError),
    ("mla_decode_q8", lambda d: dict(cp_world=2), RuntimeError),
    ("mla_decode_q8", lambda d: dict(scale=0.0), RuntimeError),
    ("mla_decode_q8", lambda d: dict(out=torch.zeros(2, 8, 512, device=DEV)), TypeError),
    ("mla_decode_q8", lambda d: dict(lse=torch.zeros(2, 7, device=DEV)), ValueError),
    ("mla_decode_q8", lambda d: dict(workspace=torch.zeros(1 << 20, device=DEV)[::2]), ValueError),
    ("mla_decode_q8", lambda d: dict(workspace=torch.zeros(8)), ValueError),
    ("mla_decode_q8", lambda d: dict(workspace=7), TypeError),
    ("mla_decode_shards_q8", lambda d: dict(n_shards=0), ValueError),
    ("mla_decode_shards_q8", lambda d: dict(n_shards=2), ValueError),
    ("mla_decode_shards_q8", lambda d: dict(block_table=d["block_table"].repeat(2, 1)), ValueError),
])
def test_wrappers_refuse(name, change, error):
    good = call_of(name)
    with pytest.raises(error):
        getattr(M, name)(**{**good, **change(good)})
    getattr(M, name)(**good)
    assert M.device_status() == 0


@pytest.mark.parametrize("change,message", [
    (dict(H=64 * 200), "row tiles of a request"),
    (dict(nb=(1 << 27) - 4096, bs=16), "num_blocks.block_size must stay below 2.31 - 65536"),
    (dict(maxb=(1 << 27) - 4096, bs=16), "max_blocks.block_size must stay below 2.31 - 65536"),
    (dict(B=1 << 20, maxb=1 << 14, bs=16), "times .max_blocks.block_size / 128 . 7. must stay below 2.31"),
    (dict(B=1 << 15, maxb=1 << 18, bs=16, shards=2), "2.31 .B=65536 over all shards"),
    (dict(B=1 << 28, H=1), "row tiles must stay below 2.28"),
])
def test_decode_limits_are_named(change, message):
    """What the tcgen05 kernel does not take is refused on the host, before the (made-up) addresses are
    used, by the limit that was passed."""
    a = dict(B=1, H=16, bs=16, nb=4, maxb=4, shards=1)
    a.update(change)
    head = [16, 16, 16, 16, a["maxb"], 16, 16, a["B"], a["H"], 1, 1, a["bs"], a["nb"], a["maxb"]]
    tail = [1, ctypes.c_float(0.1), 16, 16, 1, None, 0, None]
    lib = _lib.load()
    rc = (lib.mla_decode_shards_q8(*head, a["shards"], *tail) if a["shards"] > 1
          else lib.mla_decode_q8(*head, 1, 0, *tail))
    assert rc == _lib.MLA_ERR_UNSUPPORTED
    assert re.search(message, lib.mla_last_error().decode()), lib.mla_last_error()
    assert M.device_status() == 0


def test_wrappers_take_what_they_may():
    """A flat q, numpy and boolean numbers, empty batches, given outputs (returned as they are)."""
    d = call_of("mla_decode_q8")
    want = M.mla_decode_q8(**d)
    flat = M.mla_decode_q8(**dict(d, q=d["q"].view(2, 8, 576)))
    assert torch.equal(flat[0], want[0]) and torch.equal(flat[1], want[1])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    got = M.mla_decode_q8(**dict(d, q_len=np.int32(1), cp_world=True, scale=np.float64(SCALE), out=out, lse=lse))
    assert got[0] is out and got[1] is lse and torch.equal(out, want[0])
    assert M.mla_decode_q8(**dict(d, return_lse=False))[1] is None
    e = M.mla_decode_q8(**dict(d, q=d["q"][:0], block_table=d["block_table"][:0], seq_lens=d["seq_lens"][:0]))
    assert e[0].shape == (0, 8, 512) and e[1].shape == (0, 8)
    s = call_of("cp_store_q8")
    k = M.cp_store_q8(**dict(s, kv_new=s["kv_new"][:, :0]))
    assert k[0] is s["kv_cache"] and k[1] is s["kv_scales"]
    t = call_of("cp_step_tables")
    total = torch.empty(2, dtype=torch.int32, device=DEV)
    r = M.cp_step_tables(**dict(t, total_lens=total))
    assert isinstance(r, tuple) and r.total_lens is total and r[0] is total and len(r) == 5
    assert r.seq_lens.shape == (1, 2) and r.positions.shape == (2, 1) and r.slots.shape == (1, 2, 1)
    assert r.total_lens.tolist() == [1, 1] and r.free_state.tolist() == [2, 2]
    assert M.device_status() == 0


# =============================================================================================
# together
# =============================================================================================
@pytest.mark.parametrize("cp,il,bs,q_len,H", [(1, 1, 16, 4, 16), (2, 2, 16, 3, 64), (4, 1, 32, 1, 128)])
def test_serving_run(cp, il, bs, q_len, H):
    """Prompts, then draft blocks with rejections, a request that finishes and one that takes its
    place: tables, store and decode on every rank, against oracles fed with the same rows."""
    B = 3
    rng = np.random.default_rng(cp * 10 + bs)
    g = torch.Generator().manual_seed(cp)
    width, nb = 12, 60
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    ring, state = i32(rng.permutation(nb)), i32([0, nb])
    pools = [new_pool(nb, bs) for _ in range(cp)]
    ref = [(n64(c.float()), n64(s)) for c, s in pools]
    prev = i32([0] * B)
    held = np.zeros(B, np.int64)
    for step in range(7):
        if step == 0:
            N, new = 50, np.array([50, 17, 1])
        else:
            N, new = q_len, np.array([q_len] * B)
        if step == 4:
            held[1], new[1] = 0, 0                     # finished
        if step == 5:
            new[1] = min(q_len, 2)                     # another one begins
        ctx = i32(held)
        t = M.cp_step_tables(prev, ctx, i32(new), table, ring, state, bs, N, cp, 0, cp, il)
        rows = torch.randn(B, N, 576, generator=g).to(torch.bfloat16)
        tab = table.cpu().numpy()
        outs, lses = [], []
        G = held + new
        q = torch.randn(B, q_len, H, 576, generator=g).to(torch.bfloat16)
        for r in range(cp):
            M.cp_store_q8(rows.to(DEV), ctx, t.total_lens, table, *pools[r], cp, r, il)
            ref[r] = Q.ref_store_q8(n64(rows), held, G, np.maximum(tab, 0), *ref[r], cp, r, il)
            assert np.array_equal(n64(pools[r][0].float()), ref[r][0], equal_nan=True)
            assert np.array_equal(n64(pools[r][1]), ref[r][1], equal_nan=True)
            o, l = M.mla_decode_q8(q.to(DEV), *pools[r], table, t.seq_lens[r], t.total_lens, q_len, cp, r, SCALE,
                                   interleave=il)
            for b in range(B):
                check_request(b, q, o, l, G, tab, ref[r], q_len, cp, r, il, True, True)
            outs.append(o)
            lses.append(l)
        assert t.total_lens.tolist() == G.tolist()
        if cp > 1:
            M.lse_merge(torch.stack(outs), torch.stack(lses))
        prev, state = t.total_lens, t.free_state
        held = np.maximum(G - rng.integers(0, 2, B) * (new > 1), 0)    # a draft is rejected
    assert M.device_status() == 0

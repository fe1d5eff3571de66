"""Prompt processing on the GPU against its float64 oracle: the rotation, the append, the expanded
keys and values, the attention of chunks, the merge of shards, and a run of them together.

Tolerances (u = 2^-24; bf16's half step is 2^-8 of the value):
  * rotation: one rounding to bf16, 2^-8 |y|; the angle is exact to 2^-33 turns (2^-30 radians) and
    rounded to fp32 (2^-24 of at most pi), sincospi is within 2 ulp (2^-22), the two products and
    their sum are rounded (3 u): 2^-20 mscale (|x0| + |x1|) covers them; rows whose values are not
    computed (the latent, what is left) are equal bit for bit.
  * expanded: one rounding to bf16, 2^-8 |y|; the 512 exact products are summed by 32 instructions of
    16 products: (15 + 31) u, doubled for truncation: 92 u sum |w c|.  A scale that is no power of
    two rounds the row to bf16 first: 2^-8 sum |w c| more (and 2^-8 of the rope key).
  * attention, with w the weights, A = sum w |v|, D = the largest scale * sum |q_d k_d| of the keys:
    scores: 192 products in 12 instructions, (15 + 11) u doubled, 52 u D; the base-2 argument is
    rounded twice (the product and the difference: 2 u (|s| log2 e + 8 + |s|), at most 6 u (D + 8)
    in natural units), 2^x by 2^-22: delta = 60 u D + 2^-20.  A weight is rounded to bf16: 2^-8 A;
    the output: 2^-8 |out|.  Sums over n keys: P V adds 16 products an instruction, n/16 + 15 steps
    doubled, the row's sum n/4 + 8 steps: less than (n + 64) u in all.
    out: 2^-8 |out| + (2^-8 + 2 (e^{2 delta} - 1) + (n + 64) u) A;   lse: delta + (n/4 + 64) u +
    4 u (1 + |lse|).  Splitting the keys adds fp32 partials and their weights: 2^-20 A and 2^-20
    (1 + |lse|).
  * merge: one rounding, 2^-8 |out|, and fp32 weights: 2^-18 of sum w |partial|.
"""
import math

import numpy as np
import pytest
import torch

import mla_paged_decode_03_gb300 as M
import oracle.mla_ref as R
import oracle.prompt_ref as P
from mla_paged_decode_03_gb300.dcp import local_seq_lens

pytestmark = pytest.mark.gpu

DEV = "cuda"
U, BF = 2.0 ** -24, 2.0 ** -8
SCALE = 1.0 / math.sqrt(192.0)
BAD_PAGE, TOO_LONG, BAD_VBLOCK, BAD_SCALE, BAD_STEP = 1, 2, 4, 16, 64


@pytest.fixture(autouse=True)
def _clean():
    M.device_status()
    yield


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def i64(x):
    return torch.tensor(np.asarray(x), dtype=torch.int64, device=DEV)


def n64(t):
    return t.detach().cpu().to(torch.float64).numpy() if t.is_floating_point() else t.cpu().numpy()


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], float(np.max(err / (tol + 1e-300))))


# =============================================================================================
# rotation
# =============================================================================================
def pair_sum(x, half):
    a = np.abs(x)
    s = np.empty_like(a)
    if half:
        s[..., :32] = s[..., 32:] = a[..., :32] + a[..., 32:]
    else:
        s[..., 0::2] = s[..., 1::2] = a[..., 0::2] + a[..., 1::2]
    return s


FREQS = {"none": {}, "linear": dict(scaling="linear", factor=4.0), "ntk": dict(scaling="ntk", factor=8.0),
         "yarn": dict(scaling="yarn", factor=40.0)}


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("T,H,width,into,scaling,hi", [
    (1, 1, 64, 0, "none", 10), (3, 5, 192, 0, "linear", 5000), (7, 128, 192, 576, "yarn", 1 << 20),
    (70, 9, 576, 192, "ntk", 1 << 17), (300, 33, 192, 0, "yarn", 1 << 31), (2, 40, 192, 64, "none", 1 << 40),
])
def test_rope(T, H, width, into, scaling, hi, half):
    g = gen(T * 100 + H)
    freqs = M.rope_freqs(theta=10000.0, **FREQS[scaling])
    q = randn(g, T, H, width)
    pos = torch.randint(0, hi, (T,), generator=g)
    out = None
    if into:
        whole = randn(g, T, H, into)
        before = n64(whole)
        out = whole[..., into - 64:]
        pos[T // 2] = -1
    m = 1.25 if scaling == "yarn" else 1.0
    y = M.mla_rope(q[..., width - 64:], i64(pos), freqs, out=out, half=half, mscale=m)
    x = n64(q[..., width - 64:])
    start = n64(whole[..., into - 64:]) * 0 + before[..., into - 64:] if into else np.zeros_like(x)
    want = P.ref_rope(x, pos.numpy(), freqs.tolist(), half, m, start)
    within(n64(y), want, BF * np.abs(want) + 2.0 ** -20 * m * pair_sum(x, half), "rope")
    if into:
        assert y is out
        assert np.array_equal(n64(whole)[..., :into - 64], before[..., :into - 64])
        assert np.array_equal(n64(whole)[T // 2], before[T // 2])
    assert M.device_status() == 0


@pytest.mark.parametrize("half", [False, True])
def test_rope_in_place_and_batched(half):
    g = gen(1)
    freqs = M.rope_freqs()
    q = randn(g, 3, 5, 8, 192)
    pos = torch.randint(0, 4096, (3, 5), generator=g)
    pos[1, 4] = -1
    before = n64(q)
    y = M.mla_rope(q[..., 128:], i64(pos), freqs, out=q[..., 128:], half=half)
    want = P.ref_rope(before[..., 128:].reshape(15, 8, 64), pos.reshape(-1).numpy(), freqs.tolist(), half, 1.0,
                      before[..., 128:].reshape(15, 8, 64)).reshape(3, 5, 8, 64)
    within(n64(y), want, BF * np.abs(want) + 2.0 ** -20 * pair_sum(before[..., 128:], half), "rope")
    assert np.array_equal(n64(q)[..., :128], before[..., :128])


def test_rope_keeps_far_angles():
    """Two positions a whole number of turns of the slowest pair's unit apart differ as they should: the
    far one's angle is not rounded."""
    freqs = i64([1 << 40] * 32)                   # 2^-24 turns a position
    x = torch.ones(2, 1, 64, dtype=torch.bfloat16, device=DEV)
    y = n64(M.mla_rope(x, i64([(1 << 50) + (1 << 22), 1 << 22]), freqs))
    assert np.array_equal(y[0], y[1])
    assert np.allclose(y[1, 0, :2], [-1.0, 1.0])  # a quarter turn


# =============================================================================================
# append
# =============================================================================================
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("B,N,bs,cp,rank,il,hi", [
    (1, 1, 16, 1, 0, 1, 5), (5, 1, 64, 2, 1, 1, 300), (3, 40, 16, 3, 2, 2, 100), (2, 300, 192, 8, 5, 16, 1000),
    (70, 100, 64, 1, 0, 1, 64), (4, 7, 8, 2, 0, 4, 60), (2, 3, 1, 1, 0, 1, 4),
])
def test_rope_store(B, N, bs, cp, rank, il, hi, half):
    g = gen(B * 1000 + N)
    freqs = M.rope_freqs(**FREQS["yarn"])
    ctx = torch.randint(0, hi + 1, (B, 1), generator=g)
    pos = ctx + torch.arange(N)[None]
    pos[:, N - N // 4:] = -1
    width = (hi + N) // (bs * cp) + 1
    nb = B * width + 2
    table = torch.randperm(nb, generator=g)[:B * width].view(B, width).to(torch.int32)
    kv = randn(g, B, N, 576)
    cache = randn(g, nb, bs, 576)
    before = n64(cache)
    slots = torch.full((B, N), 77, dtype=torch.int64, device=DEV)
    r = M.cp_rope_store(kv[..., :512], kv[..., 512:], i64(pos), freqs, table.to(DEV), cache, cp, rank, il, half, 1.5,
                        slots=slots)
    assert r is cache
    x = n64(kv)
    want, written, ws = P.ref_rope_store(x[..., :512], x[..., 512:], pos.numpy(), freqs.tolist(), table.numpy(), before,
                                         cp, rank, il, half, 1.5)
    got = n64(cache)
    assert np.array_equal(n64(slots), ws)
    assert np.array_equal(got[..., :512], want[..., :512])
    flat_got, flat_want = got.reshape(-1, 576), want.reshape(-1, 576)
    left = np.ones(nb * bs, dtype=bool)
    left[written] = False
    assert np.array_equal(flat_got[left], before.reshape(-1, 576)[left])
    tol = BF * np.abs(flat_want[written][:, 512:]) + 2.0 ** -20 * 1.5 * 2 * 8.0    # |x| < 8
    within(flat_got[written][:, 512:], flat_want[written][:, 512:], tol, "rope key")
    assert M.device_status() == 0
    # the same rows through rotation and scatter
    again = torch.from_numpy(before).to(torch.bfloat16).to(DEV)
    kv2 = kv.clone()
    M.mla_rope(kv2[..., None, 512:], i64(pos), freqs, out=kv2[..., None, 512:], half=half, mscale=1.5)
    M.cp_local_slot_scatter(i64(pos), kv2, table.to(DEV), again, cp, rank, il)
    assert torch.equal(again, cache)


def test_rope_store_bad_pages():
    """Entries outside the cache and positions beyond the table write nothing and are reported."""
    freqs = M.rope_freqs()
    kv = torch.ones(1, 4, 576, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(3, 16, 576, dtype=torch.bfloat16, device=DEV)
    table = i32([[-1, 3, 2]])
    M.cp_rope_store(kv[..., :512], kv[..., 512:], i64([[0, 16, 32, -5]]), freqs, table, cache)
    assert M.device_status() == BAD_PAGE
    got = n64(cache)
    assert np.abs(got[:2]).sum() == 0 and np.abs(got[2, 1:]).sum() == 0 and (got[2, 0, :512] == 1).all()
    M.cp_rope_store(kv[..., :512], kv[..., 512:], i64([[48, 1 << 40, -1, -1]]), freqs, table, cache)
    assert M.device_status() == BAD_VBLOCK
    assert np.array_equal(n64(cache), got)


# =============================================================================================
# expanded keys and values
# =============================================================================================
def paged(g, lens, bs, spare=1, dtype=torch.bfloat16):
    width = max(1, max(-(-n // bs) for n in lens)) if lens else 1
    nb = len(lens) * width + spare
    table = torch.randperm(nb, generator=g)[:len(lens) * width].view(len(lens), width).to(torch.int32)
    for b, n in enumerate(lens):
        table[b, -(-n // bs):] = -1
    return table, nb


def starts_of(lens, gap=0):
    s, at = [], 0
    for n in lens:
        s.append(at)
        at += n + gap
    return s, at


@pytest.mark.parametrize("lens,H,bs,gap,extra", [
    ([1], 1, 16, 0, 0), ([5, 0, 130], 2, 16, 0, 0), ([128], 3, 64, 0, 5), ([257, 3], 1, 1, 0, 0),
    ([100, 300, 1, 77], 8, 48, 0, 0), ([0, 0], 2, 16, 0, 3), ([40, 50, 60], 5, 32, 7, 200), ([700], 20, 192, 0, 0),
    ([2000, 33], 33, 64, 0, 0),
])
@pytest.mark.parametrize("form", ["bf16", "q8", "q8 odd scales"])
def test_expand(lens, H, bs, gap, extra, form):
    if form != "bf16" and bs % 16:
        pytest.skip("pages of the 8-bit cache hold whole groups")
    g = gen(sum(lens) + H)
    table, nb = paged(g, lens, bs)
    starts, S = starts_of(lens, gap)
    S += extra
    w = randn(g, H, 256, 512, scale=512 ** -0.5)
    scales = None
    x = torch.randn(nb, bs, 576, generator=g)
    if form == "bf16":
        cache = x.to(torch.bfloat16).to(DEV)
        rows = n64(cache)
    else:
        s = torch.exp2(torch.randint(-12, 5, (nb, bs // 16), generator=g).float())
        if form == "q8 odd scales":
            s = s * (1 + torch.rand(nb, bs // 16, generator=g))
        cache = (x * 8).to(torch.float8_e4m3fn).to(DEV)
        scales = s.to(DEV)
        rows = n64(cache.float()) * np.repeat(n64(scales), 16, 1)[..., None]
    kv = torch.full((H, S, 256), 9.0, dtype=torch.bfloat16, device=DEV)
    kr = torch.full((S, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    k, v, r = M.mla_expand(cache, table.to(DEV), i32(lens), i32(starts), w, S, kv_scales=scales, kv=kv, k_rope=kr)
    assert k.shape == v.shape == (S, H, 128) and r is kr and (S == 0 or k.data_ptr() == kv.data_ptr())
    want, wr, mag, mine = P.ref_expand(lambda b: R.ref_gather_pages(rows, table[b].numpy(), lens[b]), lens, starts,
                                       n64(w), S)
    got = n64(kv)
    tol = BF * np.abs(want) + (92 * U + (BF if form == "q8 odd scales" else 0)) * mag
    within(got[:, mine], want[:, mine], tol[:, mine], "kv")
    assert (got[:, ~mine] == 9).all() and (n64(kr)[~mine] == 9).all()
    if form == "q8 odd scales":
        within(n64(kr)[mine], wr[mine], BF * np.abs(wr[mine]), "rope key")
    else:
        assert np.array_equal(n64(kr)[mine], wr[mine])
    assert np.array_equal(n64(k), got[..., :128].transpose(1, 0, 2)) and np.array_equal(n64(v), got[..., 128:].transpose(1, 0, 2))
    assert M.device_status() == 0
    # new outputs, on another stream: the same
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    k2, v2, r2 = M.mla_expand(cache, table.to(DEV), i32(lens), i32(starts), w, S, kv_scales=scales, stream=side)
    side.synchronize()
    m = torch.from_numpy(mine).to(DEV)
    assert torch.equal(k2[m], k[m]) and torch.equal(v2[m], v[m]) and torch.equal(r2[m], r[m])


def test_expand_many_requests():
    """More requests than a warp's lanes: the rows' requests are found by search."""
    g = gen(9)
    lens = [(7 * i) % 23 for i in range(70)]
    table, nb = paged(g, lens, 16)
    starts, S = starts_of(lens)
    cache, w = randn(g, nb, 16, 576), randn(g, 3, 256, 512, scale=512 ** -0.5)
    k, v, r = M.mla_expand(cache, table.to(DEV), i32(lens), i32(starts), w, S)
    want, wr, mag, mine = P.ref_expand(lambda b: R.ref_gather_pages(n64(cache), table[b].numpy(), lens[b]), lens, starts,
                                       n64(w), S)
    assert mine.all()
    got = np.concatenate([n64(k), n64(v)], -1).transpose(1, 0, 2)
    within(got, want, BF * np.abs(want) + 92 * U * mag, "kv")
    assert np.array_equal(n64(r), wr) and M.device_status() == 0


def test_expand_bad_inputs_are_bounded():
    g = gen(3)
    w = randn(g, 2, 256, 512, scale=0.05)
    cache = randn(g, 4, 16, 576)
    table = i32([[0, 9], [-3, 1]])
    k, v, r = M.mla_expand(cache, table, i32([20, 20]), i32([0, 20]), w, 40)
    assert M.device_status() == BAD_PAGE
    assert np.isfinite(n64(k)).all() and (n64(k)[16:20] == 0).all() and (n64(r)[20:36] == 0).all()
    # a length beyond the table, rows beyond S
    kv = torch.full((2, 50, 256), 9.0, dtype=torch.bfloat16, device=DEV)
    kr = torch.full((50, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    M.mla_expand(cache, i32([[0, 1]]), i32([1 << 30]), i32([3]), w, 50, kv=kv, k_rope=kr)
    assert M.device_status() == TOO_LONG
    assert (n64(kr)[:3] == 9).all() and (n64(kr)[35:] == 9).all() and np.array_equal(n64(kr)[3:35], n64(cache)[:2, :, 512:].reshape(32, 64))
    # starts out of order, negative lengths: nothing outside is touched
    M.mla_expand(cache, i32([[0, 1], [2, 3]]), i32([32, -7]), i32([40, -100]), w, 50, kv=kv, k_rope=kr)
    M.device_status()
    # a scale out of range reads as 1
    c8 = torch.ones(1, 16, 576, device=DEV).to(torch.float8_e4m3fn)
    _, _, r = M.mla_expand(c8, i32([[0]]), i32([16]), i32([0]), w, 16, kv_scales=torch.full((1, 1), math.nan, device=DEV))
    assert M.device_status() == BAD_SCALE and (n64(r) == 1).all()


# =============================================================================================
# attention of chunks
# =============================================================================================
def prefill_case(new, ctx, H, cp=1, rank=0, il=1, seed=0, gap=0, slack=0, outlier=0.0):
    g = gen(seed + 17 * sum(new) + sum(ctx) + H)
    G = [a + b for a, b in zip(new, ctx)]
    lens = [int(R.ref_local_len(x, cp, rank, il)) for x in G]
    starts, S = starts_of(lens, gap)
    S = max(S, 1) + slack
    T = sum(new)
    kv = randn(g, H, S, 256)
    if outlier:
        kv = torch.where(torch.rand(1, S, 1, generator=g).to(DEV) < outlier, kv * 12, kv)
    d = dict(q=randn(g, T, H, 192), k=kv[..., :128].transpose(0, 1), v=kv[..., 128:].transpose(0, 1), kr=randn(g, S, 64),
             cu=np.concatenate([[0], np.cumsum(new)]).astype(int).tolist(), starts=starts, lens=lens, G=G, H=H, T=T, S=S,
             cp=cp, rank=rank, il=il)
    return d


def call(d, causal=True, base_e=True, **kw):
    return M.mla_prefill(d["q"], d["k"], d["kr"], d["v"], i32(d["cu"]), i32(d["starts"]), i32(d["lens"]), i32(d["G"]), SCALE,
                         d["cp"], d["rank"], causal=causal, lse_base_e=base_e, interleave=d["il"], **kw)


def check(d, out, lse, causal=True, base_e=True, split=False):
    o, l, A, D, mine = P.ref_prefill(n64(d["q"]), n64(d["k"]), n64(d["kr"]), n64(d["v"]), d["cu"], d["starts"], d["lens"],
                                     d["G"], SCALE, d["cp"], d["rank"], d["il"], causal)
    n = max(d["lens"] + [0])
    delta = 60 * U * D + 2.0 ** -20
    extra = 2.0 ** -20 if split else 0.0
    tol = BF * np.abs(o) + (BF + 2 * (np.exp(2 * delta) - 1) + (n + 64) * U + extra)[..., None] * A
    got = n64(out)
    within(got[mine], o[mine], tol[mine], "out")
    gl = n64(lse) * (1.0 if base_e else math.log(2.0))
    empty = l == -np.inf
    assert (gl[mine] == -np.inf)[empty[mine]].all() and (got[mine][empty[mine]] == 0).all()
    seen = mine[:, None] & ~empty
    lt = delta + (n / 4 + 64) * U + (4 * U + extra) * (1 + np.abs(np.where(empty, 0, l)))
    within(gl[seen], l[seen], lt[seen], "lse")


CASES = [
    ([1], [0], 1), ([1], [300], 2), ([2, 1], [0, 127], 1), ([37, 130], [0, 0], 3), ([128], [0], 1), ([129], [128], 1),
    ([256], [0], 2), ([257], [1], 1), ([300, 0, 1, 5], [0, 40, 0, 700], 2), ([600], [0], 1), ([513, 20], [255, 1000], 1),
    ([0, 0, 3], [5, 0, 0], 2), ([1] * 40, list(range(0, 400, 10)), 2),
]


@pytest.mark.parametrize("new,ctx,H", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_prefill(new, ctx, H, causal):
    d = prefill_case(new, ctx, H)
    ws = torch.empty(0, dtype=torch.uint8, device=DEV)               # no split
    out, lse = call(d, causal, workspace=ws)
    check(d, out, lse, causal)
    assert M.device_status() == 0


@pytest.mark.parametrize("new,ctx,H", [([5], [2000], 1), ([300], [1300], 2), ([1, 130], [3000, 900], 1), ([64], [700], 3)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_split(new, ctx, H, causal):
    d = prefill_case(new, ctx, H)
    assert M.workspace_size_prefill(d["T"], len(new), H, d["S"]) > 0
    out, lse = call(d, causal, base_e=False)
    check(d, out, lse, causal, base_e=False, split=True)
    whole, l2 = call(d, causal, base_e=False, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    check(d, whole, l2, causal, base_e=False)
    assert M.device_status() == 0


@pytest.mark.parametrize("cp,il", [(2, 1), (3, 2), (8, 16)])
@pytest.mark.parametrize("new,ctx", [([1], [0]), ([37, 130], [0, 500]), ([300, 2], [5, 1])])
def test_prefill_shards_and_merge(new, ctx, cp, il):
    """Every shard against the oracle (early rows see nothing on some), and their merge against the
    attention over all keys."""
    H = 2
    g = gen(cp * 7 + sum(new))
    G = [a + b for a, b in zip(new, ctx)]
    T = sum(new)
    q = randn(g, T, H, 192)
    rows = [randn(g, H, x, 256) for x in G]
    ropes = [randn(g, x, 64) for x in G]
    outs, lses = [], []
    for r in range(cp):
        own = [torch.tensor([p for p in range(x) if p // il % cp == r], dtype=torch.int64, device=DEV) for x in G]
        lens = [len(o) for o in own]
        assert lens == local_seq_lens(torch.tensor(G), cp, r, il).tolist()
        starts, S = starts_of(lens)
        pad = torch.zeros(H, 1, 256, dtype=torch.bfloat16, device=DEV)
        kv = torch.cat([x[:, o] for x, o in zip(rows, own)] + [pad], 1)
        kr = torch.cat([x[o] for x, o in zip(ropes, own)] + [torch.zeros(1, 64, dtype=torch.bfloat16, device=DEV)])
        d = dict(q=q, k=kv[..., :128].transpose(0, 1), v=kv[..., 128:].transpose(0, 1), kr=kr, G=G, H=H, T=T, S=S + 1,
                 cu=np.concatenate([[0], np.cumsum(new)]).astype(int).tolist(), starts=starts, lens=lens, cp=cp, rank=r, il=il)
        out, lse = call(d)
        check(d, out, lse, split=True)
        outs.append(out)
        lses.append(lse)
    merged_lse = torch.empty(T, H, device=DEV)
    merged, _ = M.lse_merge(torch.stack(outs), torch.stack(lses), out_lse=merged_lse)
    kv = torch.cat(rows, 1)
    starts, S = starts_of(G)
    o, l, A, D, _ = P.ref_prefill(n64(q), n64(kv[..., :128].transpose(0, 1)), n64(torch.cat(ropes)),
                                  n64(kv[..., 128:].transpose(0, 1)), np.concatenate([[0], np.cumsum(new)]).astype(int).tolist(),
                                  starts, G, G, SCALE, 1, 0, 1, True)
    delta = 60 * U * D + 2.0 ** -20
    # a shard's weights and output are rounded to bf16 (2 x 2^-8 A), the merged output again
    tol = BF * np.abs(o) + (2 * BF + 4 * (np.exp(2 * delta) - 1) + (max(G) + 64) * U + 2.0 ** -18)[..., None] * A
    within(n64(merged), o, tol, "merged")
    within(n64(merged_lse), l, delta + 2.0 ** -18 * (1 + np.abs(l)), "merged lse")
    assert M.device_status() == 0


@pytest.mark.parametrize("n,T,H", [(1, 1, 1), (2, 3, 5), (7, 33, 2), (16, 1, 128), (40, 5, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("base_e", [True, False])
def test_merge_of_128_wide_rows(n, T, H, dtype, base_e):
    g = gen(n + T)
    parts = torch.randn(n, T, H, 128, generator=g).to(dtype).to(DEV)
    lses = (torch.randn(n, T, H, generator=g) * 4).to(DEV)
    lses[torch.rand(n, T, H, generator=g).to(DEV) < 0.2] = -math.inf
    lses[:, 0, 0] = -math.inf
    parts[:, 0, 0] = math.nan                                      # of empty shards: not read
    want, wl = R.ref_lse_merge(np.nan_to_num(n64(parts)), n64(lses), base_e)
    out_lse = torch.empty(T, H, device=DEV)
    out, _ = M.lse_merge(parts, lses, out_lse=out_lse, lse_base_e=base_e)
    mag, _ = R.ref_lse_merge(np.nan_to_num(np.abs(n64(parts))), n64(lses), base_e)
    within(n64(out), want, BF * np.abs(want) + 2.0 ** -18 * mag, "out")
    some = wl != -np.inf
    assert np.array_equal(n64(out_lse) == -np.inf, ~some)
    within(n64(out_lse)[some], wl[some], 2.0 ** -20 * (1 + np.abs(wl[some])), "lse")


def test_prefill_many_requests():
    """Several rounds of 32 requests, empty ones among them; heads in several groups."""
    new = [(5 * i) % 11 if i % 7 else 0 for i in range(150)] + [300] + [1] * 40
    ctx = [(13 * i) % 200 for i in range(len(new))]
    d = prefill_case(new, ctx, 2)
    out, lse = call(d)
    check(d, out, lse, split=True)
    assert M.device_status() == 0


def test_prefill_without_any_key():
    """A shard that holds no key yet: no row of memory for keys either."""
    d = prefill_case([3, 130], [0, 0], 2)
    e = dict(d, k=d["k"][:0], v=d["v"][:0], kr=d["kr"][:0], lens=[0, 0], starts=[0, 0], cp=300, rank=299)
    out, lse = call(e)
    assert (out == 0).all() and (lse == -math.inf).all() and M.device_status() == 0


def test_prefill_strided_inputs():
    """Token-major keys (a library product's layout), queries inside a wider tensor, rope keys inside
    cache rows, values in a tensor of their own."""
    d = prefill_case([40, 131], [3, 0], 3, gap=2, slack=9)
    ref, lref = call(d)
    wide = torch.zeros(d["T"], 5, 256, dtype=torch.bfloat16, device=DEV)
    wide[:, 1:4, 8:200] = d["q"]
    kv = torch.cat([d["k"], d["v"]], -1).contiguous()
    rows = torch.zeros(d["S"], 576, dtype=torch.bfloat16, device=DEV)
    rows[:, 512:] = d["kr"]
    e = dict(d, q=wide[:, 1:4, 8:200], k=kv[..., :128], v=d["v"].contiguous(), kr=rows[:, 512:])
    out, lse = call(e)
    assert torch.equal(out, ref) and torch.equal(lse, lref)
    check(d, out, lse, split=True)


def test_prefill_single_head_and_row_strides():
    d = prefill_case([1], [0], 1)
    out, lse = call(d)
    assert torch.equal(out[0, 0], d["v"][0, 0])
    check(d, out, lse)


def test_prefill_leaves_other_rows():
    """Rows behind the last request, and what lies between the requests' keys or behind them (here NaN),
    play no part; without an lse it is not written."""
    d = prefill_case([100, 30], [60, 7], 2, gap=5, slack=300)
    ws = torch.empty(M.workspace_size_prefill(d["T"], 2, 2, d["S"]), dtype=torch.uint8, device=DEV)
    mine = torch.zeros(d["S"], dtype=torch.bool)
    for s, n in zip(d["starts"], d["lens"]):
        mine[s:s + n] = True
    for name in ("k", "v", "kr"):
        d[name][~mine.to(DEV)] = math.nan
    extra = 20
    d["q"] = torch.cat([d["q"], torch.full((extra, 2, 192), math.nan, dtype=torch.bfloat16, device=DEV)])
    for w in (ws, ws[:0]):
        out = torch.full((d["T"] + extra, 2, 128), 9.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((d["T"] + extra, 2), 9.0, device=DEV)
        call(d, out=out, lse=lse, workspace=w)
        assert (out[d["T"]:] == 9).all() and (lse[d["T"]:] == 9).all()
        e = {k: v for k, v in d.items()}
        e["k"], e["v"], e["kr"] = (torch.nan_to_num(d[n]) for n in ("k", "v", "kr"))
        e["q"] = d["q"][:d["T"]]
        check(e, out[:d["T"]], lse[:d["T"]], split=True)
    o2, none = call(d, return_lse=False, workspace=ws)
    assert none is None and torch.equal(o2[:d["T"]], call(d, workspace=ws)[0][:d["T"]])


def test_prefill_nan_key_reaches_only_rows_that_see_it():
    """A key with NaN scores gives NaN to the rows that see it; rows in other blocks, and rows before it
    whose values are finite, keep theirs."""
    d = prefill_case([300], [0], 1)
    d["k"][140] = math.nan
    out, lse = call(d)
    o = n64(out)
    assert np.isfinite(o[:140]).all() and np.isnan(o[140:]).all() and np.isfinite(n64(lse)[:140]).all()


def test_merge_128_nan_lse():
    """A NaN among a row's LSEs, or nothing but NaN and empty shards, gives NaN; other rows keep theirs."""
    n, T, H = 3, 5, 2
    g = gen(5)
    parts, lses = randn(g, n, T, H, 128), torch.randn(n, T, H, generator=g).to(DEV)
    lses[:, 0, 0] = math.nan
    lses[1, 1, 1] = math.nan
    lses[0, 2, 0], lses[1:, 2, 0] = math.nan, -math.inf
    out_lse = torch.empty(T, H, device=DEV)
    out, _ = M.lse_merge(parts, lses, out_lse=out_lse)
    bad = torch.isnan(lses).any(0)
    assert torch.isnan(out[bad]).all() and torch.isnan(out_lse[bad]).all()
    assert torch.isfinite(out[~bad]).all() and torch.isfinite(out_lse[~bad]).all()



@pytest.mark.parametrize("new,ctx,cp,at", [
    ([300], [0], 1, [140]), ([300], [0], 1, [0, 5, 130, 299]), ([5], [2000], 1, [2001, 2004]), ([37, 130], [0, 500], 1, [36, 140, 600]),
    ([260, 3], [128, 700], 2, [150, 193, 540]), ([600], [0], 1, [127, 128, 383, 599]), ([2], [0], 1, [1]),
])
def test_prefill_values_that_are_not_finite(new, ctx, cp, at):
    """NaN and infinite values and keys reach the rows that see them and no others: rows before them in the
    same block keep their results within the usual bounds."""
    H = 2
    d = prefill_case(new, ctx, H, cp=cp)
    at = [x for x in at if x < d["S"]]
    for i, x in enumerate(at):
        d["v"][x, 0] = math.nan
        d["v"][x, 1, i:i + 9] = math.inf
        if i % 2:
            d["k"][x, 1] = math.nan
    for kw in ({}, {"workspace": torch.empty(0, dtype=torch.uint8, device=DEV)}):
        out, lse = call(d, **kw)
        with np.errstate(invalid="ignore"):
            o, l, A, D, mine = P.ref_prefill(n64(d["q"]), n64(d["k"]), n64(d["kr"]), n64(d["v"]), d["cu"], d["starts"],
                                             d["lens"], d["G"], SCALE, cp, 0, 1, True)
        assert mine.all()
        got, fin = n64(out), np.isfinite(o)
        assert np.array_equal(np.isnan(got), np.isnan(o)) and np.array_equal(got == np.inf, o == np.inf)
        assert fin.any() and (at == [] or not fin.all())
        n = max(d["lens"])
        D = np.where(np.isfinite(D), D, 0.0)
        delta = 60 * U * D + 2.0 ** -20
        A = np.where(fin, A, 0.0)
        tol = BF * np.abs(np.where(fin, o, 0)) + (BF + 2 * (np.exp(2 * delta) - 1) + (n + 64) * U + 2.0 ** -20)[..., None] * A
        within(got[fin], o[fin], tol[fin], "out")
    assert M.device_status() == 0


@pytest.mark.parametrize("new,ctx,H,cp", [([3, 300, 40, 1], [0, 10, 5000, 2500], 90, 1), ([260, 5, 17], [0, 6000, 900], 60, 2),
                                          ([2] * 31 + [600], [3000] + [4] * 31, 9, 1)])
def test_prefill_uneven_requests(new, ctx, H, cp):
    """More units than SMs, some of them long: every unit of every head is run, whatever runs first."""
    d = prefill_case(new, ctx, H, cp=cp)
    out, lse = call(d)
    # every row against the call with its request alone; a few heads against the oracle
    for b in range(len(new)):
        rows = slice(d["cu"][b], d["cu"][b + 1])
        e = dict(d, q=d["q"][rows], cu=[0, new[b]], starts=d["starts"][b:b + 1], lens=d["lens"][b:b + 1], G=d["G"][b:b + 1], T=new[b])
        o1, l1 = call(e, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
        assert torch.equal(o1, out[rows]) and torch.equal(l1, lse[rows])
    few = [0, H // 2, H - 1]
    e = dict(d, q=d["q"][:, few], k=d["k"][:, few], v=d["v"][:, few], H=3)
    check(e, out[:, few], lse[:, few])
    assert M.device_status() == 0


def test_prefill_many_units_with_a_short_rest():
    """Units of up to 128 rows take the two streams in turn: rows of the units beside them are not touched,
    whichever is written last."""
    d = prefill_case([300, 385, 70], [0, 3, 500], 128)
    outs = [call(d) for _ in range(4)]
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])
    few = [0, 41, 77, 127]
    for o, l in outs[:2]:
        check(dict(d, q=d["q"][:, few], k=d["k"][:, few], v=d["v"][:, few], H=4), o[:, few], l[:, few])


def test_prefill_large_scores():
    """Outlying keys: the reference maximum moves far and often."""
    for H, new, ctx in [(1, [200], [900]), (2, [130], [0])]:
        d = prefill_case(new, ctx, H, outlier=0.05)
        out, lse = call(d)
        check(d, out, lse, split=True)
    # maxima that grow from tile to tile by more than the threshold
    d = prefill_case([64], [1000], 1)
    ramp = torch.exp2(torch.arange(d["S"], device=DEV) / 128.0).to(torch.bfloat16)
    d["k"].mul_(ramp[:, None, None])
    out, lse = call(d, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    check(d, out, lse)


def test_prefill_bad_lengths_are_bounded():
    d = prefill_case([30, 30, 30], [0, 10, 0], 1)
    good, _ = call(d)
    for cu, lens, starts in [([0, 30, 20, 90], d["lens"], d["starts"]), ([0, 30, 60, 900], d["lens"], d["starts"]),
                             ([-5, 30, 60, 90], d["lens"], d["starts"]), (d["cu"], [30, 40, 3000], d["starts"]),
                             (d["cu"], [30, -40, 30], d["starts"]), (d["cu"], d["lens"], [0, 30, -70]),
                             (d["cu"], d["lens"], [0, 30, 1 << 30])]:
        out, lse = call(dict(d, cu=cu, lens=lens, starts=starts))
        assert M.device_status() == BAD_STEP
        if cu[1] == 30 and cu[0] == 0:
            assert torch.equal(out[:30], good[:30])


def test_prefill_in_a_graph_follows_new_lengths():
    """Lengths live on the GPU: a captured call takes what they hold when it is replayed."""
    a = prefill_case([100, 30], [60, 7], 2, slack=200)
    b = dict(a, cu=[0, 10, 130], lens=[40, 130], starts=[100, 200], G=[40, 130])
    bufs = {k: i32(a[k]) for k in ("cu", "starts", "lens", "G")}
    ws = M.alloc_workspace_prefill(a["T"], 2, 2, a["S"])
    out = torch.zeros(a["T"], 2, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(a["T"], 2, device=DEV)

    def step():
        M.mla_prefill(a["q"], a["k"], a["kr"], a["v"], bufs["cu"], bufs["starts"], bufs["lens"], bufs["G"], SCALE,
                      out=out, lse=lse, workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for d in (a, b):
        for k in bufs:
            bufs[k].copy_(i32(d[k]))
        graph.replay()
        torch.cuda.synchronize()
        check(d, out, lse, split=True)


def test_prompt_calls_on_two_streams():
    """Two layers' worth of calls at once, each on its own stream, with their own outputs and workspaces,
    queued behind one another without waiting: the same as one at a time."""
    freqs = M.rope_freqs()
    def step(seed):
        g = gen(seed)
        lens = [200 + seed, 33]
        table, nb = paged(g, lens, 16)
        cache, w = randn(g, nb, 16, 576), randn(g, 3, 256, 512, scale=512 ** -0.5)
        starts, S = starts_of(lens)
        args = (cache, table.to(DEV), i32(lens), i32(starts), w, S)
        q, cu, pos = randn(g, 70, 3, 192), i32([0, 60, 70]), i64(torch.arange(70))
        def run(stream=None):
            r = M.mla_rope(q[..., 128:], pos, freqs, stream=stream)
            k, v, kr = M.mla_expand(*args, stream=stream)
            o, l = M.mla_prefill(q, k, kr, v, cu, args[3], args[2], args[2], SCALE, stream=stream)
            return r, k, v, kr, o, l
        return run
    a, b = step(1), step(2)
    want = a(), b()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(a(s), b(t)) for _ in range(20)]
    torch.cuda.synchronize()
    for x, y in got:
        assert all(torch.equal(p, q) for p, q in zip(want[0], x)) and all(torch.equal(p, q) for p, q in zip(want[1], y))
    assert M.device_status() == 0


def test_prompt_calls_in_a_graph():
    """Rotation, append, expansion and attention captured once and replayed over other inputs."""
    g = gen(11)
    B, N, H, bs = 2, 40, 2, 16
    freqs, w = M.rope_freqs(**FREQS["yarn"]), randn(g, H, 256, 512, scale=512 ** -0.5)
    nb = 12
    table = i32([[3, 1, 7, 9], [0, 2, 5, 11]])
    cache = torch.zeros(nb, bs, 576, dtype=torch.bfloat16, device=DEV)
    kv, q = randn(g, B, N, 576), randn(g, B * N, H, 192)
    pos = torch.arange(N, device=DEV).repeat(B, 1)
    seq, starts, cu = i32([N, N]), i32([0, N]), i32([0, N, 2 * N])
    out = [torch.empty(B * N, H, 64, dtype=torch.bfloat16, device=DEV), torch.empty(H, B * N, 256, dtype=torch.bfloat16, device=DEV),
           torch.empty(B * N, 64, dtype=torch.bfloat16, device=DEV), torch.empty(B * N, H, 128, dtype=torch.bfloat16, device=DEV),
           torch.empty(B * N, H, device=DEV)]

    def step():
        M.mla_rope(q[..., 128:], pos.view(-1), freqs, out=out[0])
        M.cp_rope_store(kv[..., :512], kv[..., 512:], pos, freqs, table, cache)
        k, v, kr = M.mla_expand(cache, table, seq, starts, w, B * N, kv=out[1], k_rope=out[2])
        M.mla_prefill(q, k, kr, v, cu, starts, seq, None, SCALE, out=out[3], lse=out[4], workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (12, 13):
        h = gen(seed)
        kv.copy_(randn(h, B, N, 576))
        q.copy_(randn(h, B * N, H, 192))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out] + [cache.clone()]
        cache.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, out + [cache]))
    assert M.device_status() == 0


def test_tiny_wait_limit_returns():
    """As the decode's: with a limit of 1 ns a wait that is not satisfied at once may run out.  The calls
    return either way, the status holds at most that bit, and with the default limit all is well."""
    d = prefill_case([300, 40], [500, 0], 2)
    good = call(d)
    g = gen(3)
    lens = [300, 77]
    table, nb = paged(g, lens, 16)
    args = (randn(g, nb, 16, 576), table.to(DEV), i32(lens), i32([0, 300]), randn(g, 4, 256, 512, scale=0.04), 377)
    kv = M.mla_expand(*args)
    prev = M.set_wait_limit_ns(1)
    try:
        call(d)
        M.mla_expand(*args)
        torch.cuda.synchronize()
        bits = M.device_status()
    finally:
        M.set_wait_limit_ns(prev)
    assert bits & ~8 == 0
    again, kv2 = call(d), M.mla_expand(*args)
    torch.cuda.synchronize()
    assert M.device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(good + kv, again + kv2))


# =============================================================================================
# together
# =============================================================================================
@pytest.mark.parametrize("cp,il,q8", [(1, 1, False), (2, 4, False), (1, 1, True)])
def test_prompt_then_tokens(cp, il, q8):
    """A prompt in two chunks through the expanded form, then a token through the absorbed form (mla_decode),
    against plain attention over the exact keys: positions, pages, both caches, both forms and the merge
    agree.  The bound: keys and values of the expanded form are rounded to bf16 (2^-8 each), the 8-bit cache
    rounds the rows themselves, which the oracle takes from the cache."""
    g = gen(5 + cp)
    H, bs, chunks = 2, 16, ([150, 9], [61, 130])
    B = 2
    w = randn(g, H, 256, 512, scale=512 ** -0.5)
    freqs = M.rope_freqs(**FREQS["yarn"])
    width = -(-(211 + 140) // (bs * cp)) + 1
    nb = B * width + 1
    tables = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    ring = torch.randperm(nb, generator=g).to(torch.int32).to(DEV)
    state = i32([0, nb])
    caches = [torch.zeros(nb, bs, 576, dtype=torch.float8_e4m3fn if q8 else torch.bfloat16, device=DEV) for _ in range(cp)]
    scales = [torch.ones(nb, bs // 16, device=DEV) for _ in range(cp)]
    prev = i32([0, 0])
    total = np.zeros(B, dtype=int)
    ref_rows = [np.zeros((0, 576)) for _ in range(B)]      # the rows as the caches hold them
    for step, new in enumerate([chunks[0], chunks[1], [1, 1]]):
        N = max(new)
        t = M.cp_step_tables(prev, prev, i32(new), tables, ring, state, bs, N, cp, 0, cp, il)
        kv = randn(g, B, N, 576)
        for r in range(cp):
            if q8:
                rot = kv.clone()
                M.mla_rope(rot[..., None, 512:], t.positions, freqs, out=rot[..., None, 512:], mscale=1.2)
                M.cp_store_q8(rot, prev, t.total_lens, tables, caches[r], scales[r], cp, r, il)
            else:
                M.cp_rope_store(kv[..., :512], kv[..., 512:], t.positions, freqs, tables, caches[r], cp, r, il, mscale=1.2)
        total = total + np.asarray(new)
        assert t.total_lens.tolist() == total.tolist()
        # what the caches hold, position after position
        for b in range(B):
            rows = np.zeros((total[b], 576))
            for r in range(cp):
                own = R.ref_owned_positions(int(total[b]), cp, r, il)
                flat = n64(caches[r].float()) * (np.repeat(n64(scales[r]), 16, 1)[..., None] if q8 else 1.0)
                rows[own] = R.ref_gather_pages(flat, tables[b].cpu().numpy(), len(own))
            ref_rows[b] = rows
        # queries, packed, rotated in place
        T = sum(new)
        cu = [0, new[0], T]
        q = randn(g, T, H, 192)
        pos = torch.cat([t.positions[b, :new[b]] for b in range(B)])
        M.mla_rope(q[..., 128:], pos, freqs, out=q[..., 128:], mscale=1.2)
        parts, lses = [], []
        for r in range(cp):
            seq = t.seq_lens[r].contiguous()
            if step < 2:
                lens = seq.tolist()
                starts, S = starts_of(lens)
                k, v, kr = M.mla_expand(caches[r], tables, seq, i32(starts), w, max(S, 1), kv_scales=scales[r] if q8 else None)
                o, l = M.mla_prefill(q, k, kr, v, i32(cu), i32(starts), seq, t.total_lens, SCALE, cp, r, interleave=il)
            else:
                absorbed = torch.empty(B, 1, H, 576, dtype=torch.bfloat16, device=DEV)
                absorbed[:, 0, :, :512] = torch.einsum("thd,hdc->thc", q[..., :128].float(), w[:, :128].float()).to(torch.bfloat16)
                absorbed[:, 0, :, 512:] = q[..., 128:]
                if q8:
                    o, l = M.mla_decode_q8(absorbed, caches[r], scales[r], tables, seq, t.total_lens, 1, cp, r, SCALE, interleave=il)
                else:
                    o, l = M.mla_decode(absorbed, caches[r], tables, seq, t.total_lens, 1, cp, r, SCALE, interleave=il)
            parts.append(o)
            lses.append(l)
        out = parts[0] if cp == 1 else M.lse_merge(torch.stack(parts), torch.stack(lses))[0]
        got = n64(out)
        if step == 2:
            got = np.einsum("thc,hdc->thd", got, n64(w[:, 128:]))
        wn = n64(w)
        for b in range(B):
            key = np.einsum("sc,hdc->hsd", ref_rows[b][:, :512], wn[:, :128])
            val = np.einsum("sc,hdc->hsd", ref_rows[b][:, :512], wn[:, 128:])
            for i in range(new[b]):
                L = int(total[b]) - (new[b] - 1 - i)
                for h in range(H):
                    qr = n64(q[cu[b] + i, h])
                    s = SCALE * (key[h, :L] @ qr[:128] + ref_rows[b][:L, 512:] @ qr[128:])
                    e = np.exp(s - s.max())
                    o = (e / e.sum()) @ val[h, :L]
                    # norms: keys rounded by 2^-8 move a score by at most 2^-8 scale |q||k| ~ 2^-8 * 3 and the
                    # output by twice that of its spread; values, weights, output (and the absorbed query and
                    # 8-bit weights, 2^-6) by 2^-8 each: 2^-4 of the values' size in all
                    spread = np.sqrt(((e / e.sum()) ** 2).sum()) * np.abs(val[h, :L]).max() + np.abs(o).max()
                    assert np.abs(got[cu[b] + i, h] - o).max() <= 2.0 ** -4 * spread, (step, b, i, h)
        prev, state = t.total_lens, t.free_state
    assert M.device_status() == 0

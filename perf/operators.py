"""What is measured of the 8-bit paged cache: the step's tables, the store and the decode.

  tables   cp_step_tables: pages, lengths, positions and slots of a step, from request lengths
  store    cp_store_q8: new KV rows into the e4m3 cache with a scale for each 16 tokens
  decode   mla_decode_q8: MLA decode over that cache

With ``own`` false ``run`` computes the plain forms in elementary torch operations; with
``own`` true it calls the framework.
"""
import math

import torch

own = False

D_QK, D_V, GROUP = 576, 512, 16          # cache row, value part, tokens that share a scale
E4M3_MAX = 448.0
SCALE_MIN, SCALE_MAX = 2.0 ** -32, 2.0 ** 64


def listed():
    return [
        # one new token for each of a few requests: the smallest step, where latency counts
        dict(name="tables-token", op="tables", B=8, N=1, hi=4096, bs=64, cp=1, rank=0, ranks=1, il=1),
        # draft blocks of four tokens, every emulated shard's lengths and slots in one call
        dict(name="tables-draft", op="tables", B=256, N=4, hi=131072, bs=64, cp=8, rank=0, ranks=8, il=1),
        # a batch of prompts is admitted: thousands of pages and 262,144 positions
        dict(name="tables-prompt", op="tables", B=32, N=8192, hi=16384, bs=64, cp=1, rank=0, ranks=1, il=1),
        # one new row for each request, most of them into a block that is partly filled
        dict(name="store-token", op="store", B=64, N=1, hi=4096, bs=64, cp=1, rank=0, il=1),
        # draft rows on one of two ranks, small pages, segments of two positions
        dict(name="store-draft", op="store", B=256, N=4, hi=8192, bs=16, cp=2, rank=1, il=2),
        # prompts of up to 8,192 rows
        dict(name="store-prompt", op="store", B=16, N=8192, hi=2048, bs=64, cp=1, rank=0, il=1),
        # two short requests (the tiny workload's shape)
        dict(name="decode-tiny", op="decode", B=2, H=16, q_len=3, lo=37, hi=130, bs=16, cp=1, rank=0,
             il=1, causal=True, base_e=True, outlier=0.0),
        # a tensor-parallel share of the heads: few query rows, so the cache's bytes count
        dict(name="decode-heads16", op="decode", B=64, H=16, q_len=1, lo=1024, hi=16384, bs=64, cp=1,
             rank=0, il=1, causal=True, base_e=True, outlier=0.0),
        # one of two shards, draft blocks of four (the cp2 workload's shape)
        dict(name="decode-cp2", op="decode", B=8, H=64, q_len=4, lo=1024, hi=8192, bs=64, cp=2, rank=1,
             il=1, causal=True, base_e=False, outlier=0.0),
        # plain decode at 32k (the plain workload's shape)
        dict(name="decode-plain", op="decode", B=64, H=128, q_len=1, lo=32768, hi=32768, bs=64, cp=1,
             rank=0, il=1, causal=True, base_e=True, outlier=0.0),
        # one of eight shards under speculative decoding (the spec workload's shape)
        dict(name="decode-spec", op="decode", B=32, H=128, q_len=4, lo=8192, hi=131072, bs=64, cp=8,
             rank=3, il=1, causal=True, base_e=True, outlier=0.0),
        # few very long requests with outlying rows (the long workload's lengths, unsharded)
        dict(name="decode-long", op="decode", B=4, H=128, q_len=2, lo=262144, hi=524288, bs=64, cp=1,
             rank=0, il=1, causal=True, base_e=True, outlier=0.01),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["tables", "store", "decode", "decode"])
    bs = rng.choice([16, 32, 64, 64, 128, 192])
    cp = rng.choice([1, 1, 2, 3, 4, 8, 16])
    il = rng.choice([1, 1, 2, 16])
    rank = rng.randrange(cp)
    if op == "tables":
        N = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(2048, (1 << 17) // N)))
        every = rng.random() < 0.5 and cp * B * N <= 1 << 17
        return dict(op=op, B=B, N=N, hi=_log(rng, 64, 65536), bs=bs, cp=cp, rank=0 if every else rank,
                    ranks=cp if every else 1, il=il)
    if op == "store":
        N = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(1024, 98304 // N)))
        return dict(op=op, B=B, N=N, hi=_log(rng, 16, 4096), bs=bs, cp=cp, rank=rank, il=il)
    H = rng.choice([1, 5, 8, 16, 24, 32, 64, 96, 128, 128])
    q_len = rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
    hi = _log(rng, 16, min(262144, (5 << 26) // (H * q_len)))
    B = _log(rng, 1, max(1, min(256, (1 << 20) // hi, (1 << 28) // (hi * H * q_len))))
    return dict(op=op, B=B, H=H, q_len=q_len, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi, bs=bs, cp=cp,
                rank=rank, il=il, causal=rng.random() < 0.8, base_e=rng.random() < 0.7,
                outlier=rng.choice([0.0, 0.0, 0.01]))


# ---- what a step's inputs look like -----------------------------------------------------

def _lengths(c):
    """A decode case's context lengths: spread evenly over [lo, hi]; the seed orders them."""
    n = max(1, c["B"] - 1)
    return [c["lo"] + (c["hi"] - c["lo"]) * i // n for i in range(c["B"])] if c["B"] > 1 else [c["hi"]]


def _local(g, cp, rank, il):
    """Keys of a global prefix of g positions that a rank holds, segments of il dealt in turn."""
    span = cp * il
    if isinstance(g, torch.Tensor):
        return g // span * il + (g % span - rank * il).clamp(0, il)
    return g // span * il + min(max(g % span - rank * il, 0), il)


def _pages(x, vbs):
    return (x + vbs - 1) // vbs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _quantised(x):
    """Rows [pages, bs, 576] as e4m3 with one power-of-two scale for each 16 of them."""
    p, bs, d = x.shape
    g = x.view(p, bs // GROUP, GROUP * d)
    s = _pow2_scale(g.abs().amax(2))
    v = (g / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return v.view(p, bs, d), s.contiguous()


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, inside the cache's range of scales."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, -32).clamp(-32, 64)   # a block of zeros takes the smallest scale
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _table(g, need, width, num_blocks):
    """Random pages: row b's first need[b] entries are its own, the rest are -1."""
    perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(need, 0) - need
    j = torch.arange(width, device="cuda")[None]
    t = torch.where(j < need[:, None], perm[(first[:, None] + j).clamp(max=num_blocks - 1)], torch.tensor(-1, dtype=torch.int32, device="cuda"))
    return t.contiguous(), perm


def _new_tokens(c, g):
    """Cached lengths and new tokens: in blocks of up to four every request has a whole block,
    longer ones (prompts) differ in length."""
    B, N = c["B"], c["N"]
    ctx = torch.randint(0, c["hi"] + 1, (B,), generator=g, device="cuda")
    new = torch.full((B,), N, device="cuda") if N <= 4 else torch.randint(N // 2, N + 1, (B,), generator=g, device="cuda")
    return ctx, new


def prepare(c, seed):
    g = _gen(seed)
    vbs = c["bs"] * c["cp"]
    st = dict(c)
    if c["op"] == "tables":
        B, N = c["B"], c["N"]
        ctx, new = _new_tokens(c, g)
        # the last step had drafts rejected (its pages stay until this call), and one request
        # in eight has finished and gives its pages back
        prev = ctx + torch.randint(0, 4, (B,), generator=g, device="cuda")
        done = torch.rand(B, generator=g, device="cuda") < 0.125
        ctx, new = torch.where(done, 0, ctx), torch.where(done, 0, new)
        width = _pages(c["hi"] + N + 4, vbs) + 1
        cap = B * width + 8
        held = _pages(prev, vbs)
        st["table"], perm = _table(g, held, width, cap)
        total = held.sum()
        ring = torch.full_like(perm, -1)
        k = torch.arange(cap, device="cuda")
        head = cap // 3
        at = (head + k) % cap
        ring[at] = torch.where(k < cap - total, perm[(total + k).clamp(max=cap - 1)], -1)
        st["ring"] = ring
        st["state"] = torch.stack([torch.full_like(total, head), cap - total]).to(torch.int32)
        st["prev"], st["ctx"], st["new"] = (x.to(torch.int32) for x in (prev, ctx, new))
        return st
    if c["op"] == "store":
        B, N = c["B"], c["N"]
        ctx, new = _new_tokens(c, g)
        width = _pages(c["hi"] + N, vbs)
        nb = B * width + 1
        st["table"], _ = _table(g, _pages(ctx + new, vbs), width, nb)
        st["ctx"], st["total"] = ctx.to(torch.int32), (ctx + new).to(torch.int32)
        st["rows"] = torch.randn(B, N, D_QK, generator=g, device="cuda").to(torch.bfloat16)
        # rows of some tokens are larger, so that a partly filled block's scale has to grow
        st["rows"] *= torch.where(torch.rand(B, N, 1, generator=g, device="cuda") < 0.02, 8.0, 1.0).to(torch.bfloat16)
        st["cache"], st["scales"] = _quantised(torch.randn(nb, c["bs"], D_QK, generator=g, device="cuda"))
        return st
    lens = torch.tensor(_lengths(c), device="cuda")[torch.randperm(c["B"], generator=g, device="cuda")]
    local = _local(lens, c["cp"], c["rank"], c["il"])
    width = _pages(c["hi"], vbs)
    nb = c["B"] * width + 1
    st["table"], _ = _table(g, _pages(lens, vbs), width, nb)
    st["G"], st["seq"] = lens.to(torch.int32), local.to(torch.int32)
    x = torch.randn(nb, c["bs"], D_QK, generator=g, device="cuda")
    if c["outlier"]:
        x *= torch.where(torch.rand(nb, c["bs"], 1, generator=g, device="cuda") < c["outlier"], 20.0, 1.0)
    st["cache"], st["scales"] = _quantised(x)
    st["q"] = torch.randn(c["B"], c["q_len"], c["H"], D_QK, generator=g, device="cuda").to(torch.bfloat16)
    st["scale"] = 1.0 / math.sqrt(192.0)
    if own:
        import mla_paged_decode_03_gb300 as M
        st["workspace"] = M.alloc_workspace_q8(c["B"], c["H"], c["q_len"])
    return st


# ---- the plain forms --------------------------------------------------------------------

def _plain_tables(st):
    bs, cp, il, N = st["bs"], st["cp"], st["il"], st["N"]
    vbs, cap = bs * cp, st["ring"].numel()
    prev, ctx, new = (st[k].to(torch.int64) for k in ("prev", "ctx", "new"))
    head, count = st["state"][0].to(torch.int64), st["state"][1].to(torch.int64)
    table = st["table"]
    j = torch.arange(table.shape[1], device="cuda")[None]
    held, want = _pages(prev, vbs), _pages(ctx + new, vbs)
    fits = want <= table.shape[1]
    take = torch.where(fits, (want - held).clamp(min=0), 0)
    upto = torch.cumsum(take, 0)
    ok = fits & ((take == 0) | (upto <= count))
    total = torch.where(ok, ctx + new, torch.minimum(ctx, prev))
    keep = _pages(total, vbs)
    give = (held - keep).clamp(min=0)
    taken = torch.where(ok, take, 0)
    # released pages to the ring's end, new ones from its head
    end = (head + count + (torch.cumsum(give, 0) - give)[:, None] + (j - keep[:, None])) % cap
    out = (j >= keep[:, None]) & (j < held[:, None])
    pages_out, at_out = table[out], end[out]
    src = (head + (upto - take)[:, None] + (j - held[:, None])) % cap
    fresh = (j >= held[:, None]) & (j < (held + taken)[:, None])
    table.copy_(torch.where(fresh, st["ring"][src], table))
    st["ring"][at_out] = pages_out
    state = torch.stack([(head + taken.sum()) % cap, count - taken.sum() + give.sum()])
    n = torch.arange(N, device="cuda")[None]
    pos = torch.where(ok[:, None] & (n < new[:, None]), ctx[:, None] + n, -1)
    r = st["rank"] + torch.arange(st["ranks"], device="cuda")[:, None]
    seq = total // (cp * il) * il + (total % (cp * il) - r * il).clamp(0, il)
    page = torch.gather(table, 1, (pos.clamp(min=0) // vbs).clamp(max=table.shape[1] - 1)).to(torch.int64)
    off = pos.clamp(min=0) % vbs
    mine = (pos >= 0) & ((off // il) % cp == r[:, :, None])
    slots = torch.where(mine, page * bs + off // (il * cp) * il + off % il, -1)
    return dict(total=total.to(torch.int32), seq=seq.to(torch.int32), positions=pos, slots=slots, table=table,
                ring=st["ring"], state=state.to(torch.int32))


def _plain_store(st):
    bs, cp, il, rank = st["bs"], st["cp"], st["il"], st["rank"]
    vbs = bs * cp
    ctx, total = st["ctx"].to(torch.int64), st["total"].to(torch.int64)
    B, N = st["rows"].shape[:2]
    table = st["table"].to(torch.int64)
    cache = st["cache"].view(-1, D_QK)
    scales = st["scales"].view(-1)
    n = torch.arange(N, device="cuda")[None]
    pos = ctx[:, None] + n
    off = pos % vbs
    mine = (n < (total - ctx)[:, None]) & ((off // il) % cp == rank)
    page = torch.gather(table, 1, (pos // vbs).clamp(max=table.shape[1] - 1))
    slot = (page * bs + off // (il * cp) * il + off % il)[mine]
    x = st["rows"][mine].to(torch.float32)
    # the block a request's first new row lands in may hold earlier rows of it
    l0 = _local(ctx, cp, rank, il)
    has = (l0 % GROUP > 0) & (_local(total, cp, rank, il) > l0)
    base = (torch.gather(table, 1, (l0 // bs).clamp(max=table.shape[1] - 1)[:, None])[:, 0] * bs + l0 % bs // GROUP * GROUP)[has]
    group = slot // GROUP
    amax = torch.zeros(scales.numel(), device="cuda").scatter_reduce(0, group, x.abs().amax(1), "amax")
    grown = _pow2_scale(amax)
    old = scales[base // GROUP]
    grown[base // GROUP] = torch.maximum(grown[base // GROUP], old)
    k = torch.arange(GROUP, device="cuda")[None]
    rows = (base[:, None] + k)[k < (l0 % GROUP)[has][:, None]]
    ratio = (old / grown[base // GROUP])[:, None].expand(-1, GROUP)[k < (l0 % GROUP)[has][:, None]]
    bits = cache.view(torch.uint8)
    again = (bits[rows].view(torch.float8_e4m3fn).to(torch.float32) * ratio[:, None]).to(torch.float8_e4m3fn)
    bits[rows] = again.view(torch.uint8)
    v = (x / grown[group][:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    bits[slot] = v.view(torch.uint8)
    scales[group] = grown[group]
    return dict(cache=st["cache"], scales=st["scales"])


def _plain_decode(st):
    B, q_len, H, _ = st["q"].shape
    bs, dev = st["bs"], "cuda"
    G, seq = st["G"].to(torch.int64), st["seq"].to(torch.int64)
    L = st["table"].shape[1] * bs
    n = torch.arange(L, device=dev)
    page = st["table"].to(torch.int64).clamp(min=0)[:, n // bs]
    slot = page * bs + n % bs                                              # [B, L]
    k = st["cache"].view(torch.uint8).view(-1, D_QK)[slot].view(torch.float8_e4m3fn).to(torch.float32)
    k *= st["scales"].view(-1)[slot // GROUP][..., None]
    i = torch.arange(q_len, device=dev)[None]
    see = _local((G[:, None] - (q_len - 1 - i)).clamp(min=0), st["cp"], st["rank"], st["il"])
    see = torch.minimum(see, seq[:, None]) if st["causal"] else seq[:, None].expand(-1, q_len)
    s = torch.matmul(st["q"].view(B, q_len * H, D_QK).to(torch.float32) * st["scale"], k.transpose(1, 2))
    s = s.view(B, q_len, H, L).masked_fill_((n >= see[:, :, None])[:, :, None], -math.inf)
    m = s.amax(3, keepdim=True)
    s -= torch.where(m == -math.inf, 0.0, m)
    p = s.exp_()
    l = p.sum(3, keepdim=True)
    o = torch.matmul(p.view(B, q_len * H, L), k[..., :D_V]).view(B, q_len, H, D_V)
    o = torch.where(l > 0, o / l, 0.0)
    lse = (m + l.log())[..., 0] / (1.0 if st["base_e"] else math.log(2.0))
    return dict(out=o.to(torch.bfloat16).view(B * q_len, H, D_V), lse=lse.view(B * q_len, H))


def run(st):
    if not own:
        return {"tables": _plain_tables, "store": _plain_store, "decode": _plain_decode}[st["op"]](st)
    import mla_paged_decode_03_gb300 as M
    if st["op"] == "tables":
        t = M.cp_step_tables(st["prev"], st["ctx"], st["new"], st["table"], st["ring"], st["state"], st["bs"], st["N"],
                             cp_size=st["cp"], cp_rank=st["rank"], n_ranks=st["ranks"], interleave=st["il"])
        return dict(total=t.total_lens, seq=t.seq_lens, positions=t.positions, slots=t.slots, table=st["table"],
                    ring=st["ring"], state=t.free_state)
    if st["op"] == "store":
        M.cp_store_q8(st["rows"], st["ctx"], st["total"], st["table"], st["cache"], st["scales"], st["cp"], st["rank"],
                      interleave=st["il"])
        return dict(cache=st["cache"], scales=st["scales"])
    out, lse = M.mla_decode_q8(st["q"], st["cache"], st["scales"], st["table"], st["seq"], st["G"], st["q_len"], st["cp"],
                               st["rank"], st["scale"], lse_base_e=st["base_e"], workspace=st["workspace"],
                               causal=st["causal"], interleave=st["il"])
    return dict(out=out, lse=lse)


def work(c):
    vbs = c["bs"] * c["cp"]
    if c["op"] == "tables":
        # lengths in, lengths and slots out, the entries of the new tokens' pages read, and
        # (about) the pages that change hands
        pages = c["B"] * (c["N"] / vbs + (c["hi"] / 2 / vbs) / 8)
        return dict(bytes=12 * c["B"] + 4 * c["B"] * (1 + c["ranks"]) + 8 * c["B"] * c["N"] * (1 + c["ranks"]) + 8 * pages + 16,
                    flops=0)
    if c["op"] == "store":
        rows = c["B"] * (c["N"] if c["N"] <= 4 else 0.75 * c["N"]) / c["cp"]
        return dict(bytes=rows * (2 * D_QK + D_QK + 4 / GROUP) + 8 * c["B"] + 4 * max(c["B"], rows / c["bs"]), flops=2 * rows * D_QK)
    lens = _lengths(c)
    keys = sum(_local(g, c["cp"], c["rank"], c["il"]) for g in lens)
    seen = sum(_local(max(0, g - (c["q_len"] - 1 - i)) if c["causal"] else g, c["cp"], c["rank"], c["il"]) for g in lens for i in range(c["q_len"]))
    rows = c["B"] * c["q_len"] * c["H"]
    return dict(bytes=keys * (D_QK + 4 / GROUP + 4 / c["bs"]) + rows * (2 * D_QK + 2 * D_V + 4) + 8 * c["B"],
                flops=2 * (D_QK + D_V) * c["H"] * seen)


# ---- in 64 bits, from the definitions ---------------------------------------------------

def exact(c, seed):
    if c["op"] == "tables":
        return None                                 # whole numbers only
    st = prepare(c, seed)
    if c["op"] == "store":
        return _exact_store(st)
    return _exact_decode(st)


def _exact_store(st):
    """Token by token: its rank, its page, its block; then block by block the scale and rows."""
    import numpy as np
    bs, cp, il = st["bs"], st["cp"], st["il"]
    ctx, total, table = (st[k].cpu().numpy() for k in ("ctx", "total", "table"))
    cache = st["cache"].to(torch.float64).view(-1, D_QK).clone()
    scales = st["scales"].to(torch.float64).view(-1).clone()
    blocks = {}                                     # block -> ([(slot offset, row)], earlier rows)
    for b in range(len(ctx)):
        local = 0
        g = np.arange(int(total[b]))
        own_g = g[(g // il) % cp == st["rank"]]
        for local in np.nonzero(own_g >= ctx[b])[0]:
            slot = int(table[b, local // bs]) * bs + int(local % bs)
            got = blocks.setdefault(slot // GROUP, ([], slot % GROUP))
            got[0].append((slot, b, int(own_g[local] - ctx[b])))
    if not blocks:
        return dict(cache=cache.view(st["cache"].shape), scales=scales.view(st["scales"].shape))
    flat = [t for v, _ in blocks.values() for t in v]
    slot, b, n = (torch.tensor([t[i] for t in flat], device="cuda") for i in range(3))
    x = st["rows"].to(torch.float64)[b, n]
    peak = x.abs().amax(1).cpu().numpy()
    at, s_of = 0, {}
    for blk, (v, earlier) in blocks.items():
        top = float(peak[at:at + len(v)].max())
        at += len(v)
        s = SCALE_MIN if top == 0 else min(max(2.0 ** math.ceil(math.log2(top / E4M3_MAX)), SCALE_MIN), SCALE_MAX)
        if earlier:
            was = float(scales[blk])
            s = max(s, was)
            if s != was:
                cache[blk * GROUP:blk * GROUP + earlier] *= was / s
        s_of[blk] = s
    s = torch.tensor([s_of[t[0] // GROUP] for t in flat], dtype=torch.float64, device="cuda")
    cache[slot] = x / s[:, None]
    scales[slot // GROUP] = s
    return dict(cache=cache.view(st["cache"].shape), scales=scales.view(st["scales"].shape))


def _exact_decode(st):
    """Request by request, and each query position by itself."""
    import numpy as np
    B, q_len, H, _ = st["q"].shape
    bs = st["bs"]
    out = torch.zeros(B, q_len, H, D_V, dtype=torch.float64, device="cuda")
    lse = torch.full((B, q_len, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, (g, have) in enumerate(zip(st["G"].tolist(), st["seq"].tolist())):
        if have == 0:
            continue
        pages = st["table"][b, :_pages(have, bs)].to(torch.int64)
        held = np.arange(g)
        held = held[(held // st["il"]) % st["cp"] == st["rank"]]        # their global positions
        keys = st["cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).to(torch.float64).view(-1, GROUP, D_QK) * st["scales"][pages].to(torch.float64).view(-1, 1, 1)
        keys = keys.view(-1, D_QK)[:have]
        for i in range(q_len):
            see = have
            if st["causal"]:
                see = min(have, int(np.searchsorted(held, g - (q_len - 1 - i))))
            if see == 0:
                continue
            s = st["scale"] * (st["q"][b, i].to(torch.float64) @ keys[:see].T)
            top = s.max(1, keepdim=True).values
            w = torch.exp(s - top)
            z = w.sum(1, keepdim=True)
            out[b, i] = w @ keys[:see, :D_V] / z
            lse[b, i] = (top + torch.log(z))[:, 0]
    if not st["base_e"]:
        lse /= math.log(2.0)
    return dict(out=out.view(B * q_len, H, D_V), lse=lse.view(B * q_len, H))

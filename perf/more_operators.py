"""What is measured of prompt processing over the paged latent cache: the rotation of queries, the
append of new tokens, the heads' keys and values, and the attention of chunks of new tokens.

  rope     mla_rope: rotary positions of the queries' last 64 dims
  store    cp_rope_store: new tokens into the pages, their rope part rotated on the way
  expand   mla_expand: keys and values of all heads from the pages' latent rows
  prefill  mla_prefill: attention of ragged chunks of new tokens over those keys

With ``own`` false ``run`` computes the plain forms in elementary torch operations; with
``own`` true it calls the framework.
"""
import math

import torch

own = False

LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128      # cache row: latent | rope; a head's key: nope | rope
GROUP = 16                                        # slots of the 8-bit cache that share a scale


def listed():
    return [
        # queries of 64 requests with one new token, written beside the absorbed part of each query
        dict(name="rope-token", op="rope", T=64, H=128, width=192, into=576, hi=131072, half=False, scaling="yarn",
             factor=40.0),
        # a prompt's queries, halves layout
        dict(name="rope-prompt", op="rope", T=8192, H=128, width=192, into=0, hi=8192, half=True, scaling="none",
             factor=1.0),
        # one new token for each of 64 requests
        dict(name="store-token", op="store", B=64, N=1, hi=131072, bs=64, cp=1, rank=0, il=1, half=False,
             scaling="yarn", factor=40.0),
        # prompts on one of two ranks, small pages, segments of two positions
        dict(name="store-prompt", op="store", B=16, N=4096, hi=2048, bs=16, cp=2, rank=1, il=2, half=False,
             scaling="none", factor=1.0),
        # short prompts of a few requests on a tensor-parallel share of the heads
        dict(name="expand-short", op="expand", B=8, H=8, lo=16, hi=500, bs=16, q8=False),
        # one prompt, all heads
        dict(name="expand-prompt", op="expand", B=1, H=128, lo=8192, hi=8192, bs=64, q8=False),
        # long cached contexts in the 8-bit cache, a share of the heads
        dict(name="expand-q8", op="expand", B=4, H=32, lo=1024, hi=32768, bs=64, q8=True),
        # two short prompts: the smallest call
        dict(name="prefill-tiny", op="prefill", B=2, H=8, nlo=37, nhi=130, clo=0, chi=0, cp=1, rank=0, il=1,
             causal=True, base_e=True),
        # the next chunk of one long prompt, a share of the heads: few rows over many keys
        dict(name="prefill-chunk", op="prefill", B=1, H=8, nlo=512, nhi=512, clo=32256, chi=32256, cp=1, rank=0, il=1,
             causal=True, base_e=True),
        # a mixed batch: single tokens beside chunks, with and without cached tokens
        dict(name="prefill-mixed", op="prefill", B=24, H=32, nlo=1, nhi=700, clo=0, chi=4096, cp=1, rank=0, il=1,
             causal=True, base_e=True),
        # one of two shards of a few prompts, LSEs in base 2
        dict(name="prefill-cp2", op="prefill", B=4, H=64, nlo=1000, nhi=2048, clo=0, chi=2000, cp=2, rank=1, il=1,
             causal=True, base_e=False),
        # one prompt of 8,192 tokens, all heads
        dict(name="prefill-prompt", op="prefill", B=1, H=128, nlo=8192, nhi=8192, clo=0, chi=0, cp=1, rank=0, il=1,
             causal=True, base_e=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["rope", "store", "expand", "expand", "prefill", "prefill", "prefill"])
    H = rng.choice([1, 5, 8, 20, 32, 64, 128])
    scaling = rng.choice(["none", "linear", "yarn"])
    factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 40.0])
    cp = rng.choice([1, 1, 2, 3, 8])
    il = rng.choice([1, 1, 2, 16])
    rank = rng.randrange(cp)
    bs = rng.choice([16, 32, 64, 64, 192])
    if op == "rope":
        width = rng.choice([64, 192, 192, 576])
        into = rng.choice([0, 0, 192, 576])
        T = _log(rng, 1, (1 << 20) // max(H, 8) * 192 // max(width, into, 192))
        return dict(op=op, T=T, H=H, width=width, into=into, hi=_log(rng, 1024, 1 << 20), half=rng.random() < 0.5,
                    scaling=scaling, factor=factor)
    if op == "store":
        N = _log(rng, 1, 4096)
        return dict(op=op, B=_log(rng, 1, max(1, min(512, 65536 // N))), N=N, hi=_log(rng, 16, 4096), bs=bs, cp=cp,
                    rank=rank, il=il, half=rng.random() < 0.5, scaling=scaling, factor=factor)
    if op == "expand":
        hi = _log(rng, 8, min(65536, (1 << 20) // H))
        B = _log(rng, 1, max(1, min(64, (1 << 20) // (H * hi))))
        return dict(op=op, B=B, H=H, lo=rng.choice([1, (hi + 1) // 2, hi]), hi=hi, bs=bs, q8=rng.random() < 0.4)
    nhi = _log(rng, 1, 4096)
    total = _log(rng, nhi, max(nhi, min(32768, (1 << 32) // (H * nhi))))
    B = _log(rng, 1, max(1, min(48, (1 << 32) // (H * nhi * total), 131072 // total)))
    return dict(op=op, B=B, H=H, nlo=rng.choice([1, (nhi + 1) // 2, nhi]), nhi=nhi, clo=rng.choice([0, total - nhi]),
                chi=total - nhi, cp=cp, rank=rank, il=il, causal=rng.random() < 0.85, base_e=rng.random() < 0.7)


# ---- what a step's inputs look like -----------------------------------------------------

def _spread(lo, hi, n):
    """n lengths spread evenly over [lo, hi] (a single one is the largest)."""
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)] if n > 1 else [hi]


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


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def _table(g, need, width, num_blocks):
    """Random pages: row b's first need[b] entries are its own, the rest are -1."""
    perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(need, 0) - need
    j = torch.arange(width, device="cuda")[None]
    return torch.where(j < need[:, None], perm[(first[:, None] + j).clamp(max=num_blocks - 1)], torch.tensor(-1, dtype=torch.int32, device="cuda")).contiguous()


def _starts(lens):
    return torch.cumsum(lens, 0) - lens


def _rotation(st, c):
    """The rotation's frequencies (radians a position, 64 bits) and its factor on the values."""
    i = torch.arange(ROPE // 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-2.0 * i / ROPE)
    st["mscale"] = 1.0
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "yarn":
        # dims that turn often over the original 4,096 positions keep their frequency, those that turn
        # less than once are stretched by the factor, the others are between
        lo, hi = (ROPE * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0)) for turns in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), ROPE - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / c["factor"] * ramp + f * (1 - ramp)
        st["mscale"] = 0.1 * math.log(c["factor"]) + 1.0
    st["inv_freq"] = f
    if own:
        import mla_paged_decode_03_gb300 as M
        st["freqs"] = M.rope_freqs(theta=10000.0, scaling=c["scaling"], factor=c["factor"], original_max_position=4096)


def prepare(c, seed):
    g = _gen(seed)
    st = dict(c)
    if c["op"] == "rope":
        T, H = c["T"], c["H"]
        _rotation(st, c)
        st["q"] = _randn(g, T, H, c["width"])
        # a few new tokens at any place of their contexts; a prompt's are consecutive
        st["pos"] = torch.randint(0, c["hi"], (T,), generator=g, device="cuda") if T <= 256 else torch.arange(T, device="cuda") + torch.randint(0, c["hi"], (1,), generator=g, device="cuda")
        st["out"] = None
        if c["into"]:
            st["out"] = _randn(g, T, H, c["into"])[..., c["into"] - ROPE:]
            st["pos"][torch.rand(T, generator=g, device="cuda") < 0.03] = -1       # rejected: left as they were
        return st
    if c["op"] == "store":
        B, N, vbs = c["B"], c["N"], c["bs"] * c["cp"]
        _rotation(st, c)
        ctx = torch.randint(0, c["hi"] + 1, (B,), generator=g, device="cuda")
        new = torch.full((B,), N, device="cuda") if N <= 4 else torch.randint(N // 2, N + 1, (B,), generator=g, device="cuda")
        n = torch.arange(N, device="cuda")[None]
        st["pos"] = torch.where(n < new[:, None], ctx[:, None] + n, -1)
        held = _pages(ctx + new, vbs) - ctx // vbs         # pages that get new rows; the others are not touched
        nb = int(B * (_pages(N, vbs) + 1) + 1)
        part = _table(g, held, int(_pages(N, vbs) + 1), nb)
        width = int(_pages(c["hi"] + N, vbs)) + 1
        j = torch.arange(width, device="cuda")[None] - (ctx // vbs)[:, None]
        st["table"] = torch.where((j >= 0) & (j < part.shape[1]), torch.gather(part, 1, j.clamp(0, part.shape[1] - 1)), torch.tensor(-1, dtype=torch.int32, device="cuda")).contiguous()
        kv = _randn(g, B, N, LATENT + ROPE)                # the projection's output: latent and rope part side by side
        st["latent"], st["k_rope"] = kv[..., :LATENT], kv[..., LATENT:]
        st["cache"] = _randn(g, nb, c["bs"], LATENT + ROPE)
        return st
    if c["op"] == "expand":
        lens = torch.tensor(_spread(c["lo"], c["hi"], c["B"]), device="cuda")[torch.randperm(c["B"], generator=g, device="cuda")]
        need = _pages(lens, c["bs"])
        nb = c["B"] * _pages(c["hi"], c["bs"]) + 1
        st["table"] = _table(g, need, _pages(c["hi"], c["bs"]), nb)
        st["seq"], st["starts"] = lens.to(torch.int32), _starts(lens).to(torch.int32)
        st["total"] = sum(_spread(c["lo"], c["hi"], c["B"]))
        x = torch.randn(nb, c["bs"], LATENT + ROPE, generator=g, device="cuda")
        st["scales"] = None
        if c["q8"]:
            # values near the middle of the 8-bit range, a power-of-two scale for each 16 rows
            x = x.view(nb, c["bs"] // GROUP, GROUP, LATENT + ROPE)
            s = torch.exp2(torch.randint(-8, -4, (nb, c["bs"] // GROUP), generator=g, device="cuda").to(torch.float32))
            st["cache"] = (x / s[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(nb, c["bs"], -1)
            st["scales"] = s
        else:
            st["cache"] = x.to(torch.bfloat16)
        st["w"] = (torch.randn(c["H"], NOPE + VDIM, LATENT, generator=g, device="cuda") / math.sqrt(LATENT)).to(torch.bfloat16)
        return st
    new, ctx = _chunks(c)
    order = torch.randperm(c["B"], generator=g, device="cuda")
    new, ctx = torch.tensor(new, device="cuda")[order], torch.tensor(ctx, device="cuda")[order]
    G = ctx + new
    seq = _local(G, c["cp"], c["rank"], c["il"])
    T, S = sum(_chunks(c)[0]), sum(_local(n + x, c["cp"], c["rank"], c["il"]) for n, x in zip(*_chunks(c)))
    st["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(new, 0)]).to(torch.int32)
    st["starts"], st["seq"], st["G"] = _starts(seq).to(torch.int32), seq.to(torch.int32), G.to(torch.int32)
    st["q"] = _randn(g, T, c["H"], NOPE + ROPE)
    kv = _randn(g, c["H"], max(S, 1), NOPE + VDIM)          # head after head, as mla_expand lays them out
    st["k"], st["v"] = kv[..., :NOPE].transpose(0, 1), kv[..., NOPE:].transpose(0, 1)
    st["k_rope"] = _randn(g, max(S, 1), ROPE)
    st["scale"] = 1.0 / math.sqrt(192.0)
    if own:
        import mla_paged_decode_03_gb300 as M
        st["workspace"] = M.alloc_workspace_prefill(T, c["B"], c["H"], max(S, 1))
    return st


def _chunks(c):
    """A prefill case's new and cached tokens of each request: long chunks beside short contexts and the
    other way round."""
    return _spread(c["nlo"], c["nhi"], c["B"]), _spread(c["clo"], c["chi"], c["B"])[::-1]


# ---- the plain forms --------------------------------------------------------------------

def _rotated(x, pos, st):
    """x [..., 64] (32 bits) turned by its position; pos has x's leading shape, or broadcasts to it."""
    a = pos[..., None].to(torch.float64) * st["inv_freq"]
    cos, sin = (f(a).to(torch.float32) * st["mscale"] for f in (torch.cos, torch.sin))
    if st["half"]:
        x0, x1 = x[..., :ROPE // 2], x[..., ROPE // 2:]
        return torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2)


def _plain_rope(st):
    y = _rotated(st["q"][..., -ROPE:].to(torch.float32), st["pos"][:, None], st).to(torch.bfloat16)
    if st["out"] is None:
        return dict(q_rope=y)
    st["out"].copy_(torch.where((st["pos"] >= 0)[:, None, None], y, st["out"]))
    return dict(q_rope=st["out"])


def _plain_store(st):
    bs, cp, il = st["bs"], st["cp"], st["il"]
    vbs = bs * cp
    pos = st["pos"]
    off = pos.clamp(min=0) % vbs
    mine = (pos >= 0) & ((off // il) % cp == st["rank"])
    page = torch.gather(st["table"], 1, (pos.clamp(min=0) // vbs).clamp(max=st["table"].shape[1] - 1)).to(torch.int64)
    slot = (page * bs + off // (il * cp) * il + off % il)[mine]
    y = _rotated(st["k_rope"][mine].to(torch.float32), pos[mine], st).to(torch.bfloat16)
    st["cache"].view(-1, LATENT + ROPE)[slot] = torch.cat([st["latent"][mine], y], -1)
    return dict(cache=st["cache"])


def _rows(st, dtype):
    """Every request's cache rows, one after another."""
    r = torch.arange(st["total"], device="cuda")
    b = torch.searchsorted((st["starts"] + st["seq"]).to(torch.int64), r, right=True)
    l = r - st["starts"][b]
    slot = st["table"][b, l // st["bs"]].to(torch.int64) * st["bs"] + l % st["bs"]
    if st["scales"] is None:
        return st["cache"].view(-1, LATENT + ROPE)[slot].to(dtype)
    x = st["cache"].view(torch.uint8).view(-1, LATENT + ROPE)[slot].view(torch.float8_e4m3fn).to(dtype)
    return x * st["scales"].view(-1)[slot // GROUP][:, None].to(dtype)


def _plain_expand(st):
    x = _rows(st, torch.float32)
    kv = torch.matmul(x[:, :LATENT], st["w"].to(torch.float32).view(-1, LATENT).T).view(x.shape[0], -1, NOPE + VDIM).to(torch.bfloat16)
    return dict(k=kv[..., :NOPE], v=kv[..., NOPE:], k_rope=x[:, LATENT:].to(torch.bfloat16))


def _plain_prefill(st):
    """All requests at once, each padded to the longest chunk and the most keys."""
    cu, seq, G = (st[k].to(torch.int64) for k in ("cu", "seq", "G"))
    B, H, T, S = st["B"], st["H"], st["q"].shape[0], st["k"].shape[0]
    n, L = st["nhi"], max(1, max(_local(a + b, st["cp"], st["rank"], st["il"]) for a, b in zip(*_chunks(st))))
    i, l = torch.arange(n, device="cuda"), torch.arange(L, device="cuda")
    new = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i).clamp(max=T - 1)                                   # [B, n]
    key = (st["starts"].to(torch.int64)[:, None] + l).clamp(max=S - 1)           # [B, L]
    q = st["q"][row].permute(0, 2, 1, 3).to(torch.float32) * st["scale"]         # [B, H, n, 192]
    k = torch.cat([st["k"][key], st["k_rope"][key][:, :, None].expand(-1, -1, H, -1)], -1).permute(0, 2, 3, 1).to(torch.float32)
    s = torch.matmul(q, k)                                                       # [B, H, n, L]
    see = seq[:, None].expand(-1, n)
    if st["causal"]:
        see = torch.minimum(see, _local((G[:, None] - (new[:, None] - 1 - i)).clamp(min=0), st["cp"], st["rank"], st["il"]))
    s.masked_fill_((l >= see[:, :, None])[:, None], -math.inf)
    m = s.amax(3, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    z = p.sum(3, keepdim=True)
    v = st["v"][key].permute(0, 2, 1, 3).to(torch.float32)
    o = torch.where(z > 0, torch.matmul(p, v) / z, 0.0)
    lse = (m + z.log())[..., 0] / (1.0 if st["base_e"] else math.log(2.0))
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    return dict(out=o[b, :, t - cu[b]].to(torch.bfloat16), lse=lse[b, :, t - cu[b]])


def run(st):
    if not own:
        return {"rope": _plain_rope, "store": _plain_store, "expand": _plain_expand, "prefill": _plain_prefill}[st["op"]](st)
    import mla_paged_decode_03_gb300 as M
    if st["op"] == "rope":
        return dict(q_rope=M.mla_rope(st["q"][..., -ROPE:], st["pos"], st["freqs"], out=st["out"], half=st["half"], mscale=st["mscale"]))
    if st["op"] == "store":
        M.cp_rope_store(st["latent"], st["k_rope"], st["pos"], st["freqs"], st["table"], st["cache"], st["cp"], st["rank"],
                        interleave=st["il"], half=st["half"], mscale=st["mscale"])
        return dict(cache=st["cache"])
    if st["op"] == "expand":
        k, v, k_rope = M.mla_expand(st["cache"], st["table"], st["seq"], st["starts"], st["w"], st["total"], kv_scales=st["scales"])
        return dict(k=k, v=v, k_rope=k_rope)
    out, lse = M.mla_prefill(st["q"], st["k"], st["k_rope"], st["v"], st["cu"], st["starts"], st["seq"], st["G"], st["scale"],
                             st["cp"], st["rank"], lse_base_e=st["base_e"], workspace=st["workspace"], causal=st["causal"],
                             interleave=st["il"])
    return dict(out=out, lse=lse)


def work(c):
    if c["op"] == "rope":
        return dict(bytes=c["T"] * c["H"] * ROPE * 4 + 8 * c["T"], flops=c["T"] * c["H"] * ROPE * 3)
    if c["op"] == "store":
        rows = c["B"] * (c["N"] if c["N"] <= 4 else 0.75 * c["N"])
        return dict(bytes=rows / c["cp"] * 4 * (LATENT + ROPE) + 8 * c["B"] * c["N"] + 4 * max(c["B"], rows / c["bs"] / c["cp"]), flops=rows / c["cp"] * ROPE * 3)
    if c["op"] == "expand":
        keys = sum(_spread(c["lo"], c["hi"], c["B"]))
        row = LATENT + ROPE + 4 / GROUP if c["q8"] else 2 * (LATENT + ROPE)
        return dict(bytes=keys * (row + 4 / c["bs"] + c["H"] * 2 * (NOPE + VDIM) + 2 * ROPE) + c["H"] * (NOPE + VDIM) * LATENT * 2,
                    flops=2 * keys * LATENT * (NOPE + VDIM) * c["H"])
    keys, seen, rows = 0, 0, 0
    for n, x in zip(*_chunks(c)):
        have = _local(n + x, c["cp"], c["rank"], c["il"])
        keys, rows = keys + have, rows + n
        seen += sum(_local(x + i + 1, c["cp"], c["rank"], c["il"]) for i in range(n)) if c["causal"] else n * have
    return dict(bytes=rows * c["H"] * (2 * (NOPE + ROPE) + 2 * VDIM + 4) + keys * 2 * (c["H"] * (NOPE + VDIM) + ROPE) + 16 * c["B"],
                flops=2 * (NOPE + ROPE + VDIM) * c["H"] * seen)


# ---- in 64 bits, from the definitions ---------------------------------------------------

def exact(c, seed):
    st = prepare(c, seed)
    return {"rope": _exact_rope, "store": _exact_store, "expand": _exact_expand, "prefill": _exact_prefill}[c["op"]](st)


def _turned(x, pos, st):
    """Each pair as a complex number times e^(i pos f)."""
    x = x.to(torch.float64)
    z = torch.complex(x[..., :32], x[..., 32:]) if st["half"] else torch.view_as_complex(x.unflatten(-1, (32, 2)).contiguous())
    a = pos.to(torch.float64)[..., None] * st["inv_freq"]
    z = z * torch.polar(torch.full_like(a, st["mscale"]), a)
    return torch.cat([z.real, z.imag], -1) if st["half"] else torch.view_as_real(z).flatten(-2)


def _exact_rope(st):
    y = _turned(st["q"][..., -ROPE:], st["pos"][:, None].expand(-1, st["H"]), st)
    if st["out"] is not None:
        left = st["pos"] < 0
        y[left] = st["out"][left].to(torch.float64)
    return dict(q_rope=y)


def _exact_store(st):
    """Token by token: its owner, its page, its slot."""
    import numpy as np
    bs, cp, il, rank = st["bs"], st["cp"], st["il"], st["rank"]
    pos, table = st["pos"].cpu().numpy(), st["table"].cpu().numpy()
    cache = st["cache"].to(torch.float64)
    flat = cache.view(-1, LATENT + ROPE)
    for b in range(pos.shape[0]):
        n = np.nonzero(pos[b] >= 0)[0]
        n = n[(pos[b, n] // il) % cp == rank]
        p = pos[b, n]
        inside = p % (bs * cp)
        at = table[b, p // (bs * cp)].astype(np.int64) * bs + inside // (cp * il) * il + inside % il
        n, at, p = (torch.from_numpy(np.asarray(a, dtype=np.int64)).cuda() for a in (n, at, p))
        flat[at, :LATENT] = st["latent"][b, n].to(torch.float64)
        flat[at, LATENT:] = _turned(st["k_rope"][b, n], p, st)
    return dict(cache=cache)


def _exact_expand(st):
    """Request by request from its pages."""
    ks, vs, rs = [], [], []
    w = st["w"].to(torch.float64)
    for b, have in enumerate(st["seq"].tolist()):
        pages = st["table"][b, :_pages(have, st["bs"])].to(torch.int64)
        if st["scales"] is None:
            x = st["cache"][pages].to(torch.float64)
        else:
            x = st["cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).to(torch.float64).view(len(pages), -1, GROUP, LATENT + ROPE)
            x = x * st["scales"][pages].to(torch.float64)[..., None, None]
        x = x.reshape(-1, LATENT + ROPE)[:have]
        kv = torch.einsum("sc,hdc->shd", x[:, :LATENT], w)
        ks, vs, rs = ks + [kv[..., :NOPE]], vs + [kv[..., NOPE:]], rs + [x[:, LATENT:]]
    return dict(k=torch.cat(ks), v=torch.cat(vs), k_rope=torch.cat(rs))


def _exact_prefill(st):
    """Request by request and head by head; a query sees the keys that its rank holds of its prefix."""
    H, T = st["H"], st["q"].shape[0]
    out = torch.zeros(T, H, VDIM, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    cu, starts, seq, G = (st[k].tolist() for k in ("cu", "starts", "seq", "G"))
    for b in range(st["B"]):
        have, n = seq[b], cu[b + 1] - cu[b]
        if have == 0:
            continue
        held = torch.arange(G[b], device="cuda")
        held = held[(held // st["il"]) % st["cp"] == st["rank"]][:have]      # the keys' positions in the context
        hide = held[None] > torch.arange(G[b] - n, G[b], device="cuda")[:, None]
        rows, keys = slice(cu[b], cu[b + 1]), slice(starts[b], starts[b] + have)
        for h in range(H):
            s = st["q"][rows, h, :NOPE].to(torch.float64) @ st["k"][keys, h].to(torch.float64).T
            s += st["q"][rows, h, NOPE:].to(torch.float64) @ st["k_rope"][keys].to(torch.float64).T
            s *= st["scale"]
            if st["causal"]:
                s[hide] = -math.inf
            lse[rows, h] = torch.logsumexp(s, 1)
            top = lse[rows, h].clamp(min=-1e300)[:, None]                    # a row that sees nothing: weights 0
            out[rows, h] = torch.exp(s - top) @ st["v"][keys, h].to(torch.float64)
    if not st["base_e"]:
        lse /= math.log(2.0)
    return dict(out=out, lse=lse)

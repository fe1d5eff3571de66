"""Prompt processing without a GPU: what the C entry points and the Python wrappers refuse, the
frequencies of the rotation, and checks that pin its oracle."""
import math

import numpy as np
import pytest
import torch

import mla_paged_decode_03_gb300 as M
import oracle.mla_ref as R
import oracle.prompt_ref as P
from mla_paged_decode_03_gb300 import _lib

from test_abi_cpu import lib  # noqa: F401  (the built library)

E, U, OK = _lib.MLA_ERR_INVALID_ARGUMENT, _lib.MLA_ERR_UNSUPPORTED, _lib.MLA_OK


def _call(fn, names, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return fn(*[a[n] for n in names])


def _rope(lib, **kw):
    names = ["x", "xt", "xh", "pos", "freqs", "T", "H", "half", "m", "out", "ot", "oh", "stream"]
    return _call(lib.mla_rope, names, dict(x=16, xt=384, xh=192, pos=16, freqs=16, T=2, H=2, half=0, m=1.0, out=32, ot=128,
                                           oh=64, stream=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), E), (dict(H=0), E), (dict(m=math.nan), E), (dict(m=math.inf), E), (dict(xt=-8), E), (dict(xh=12), E),
    (dict(ot=4), E), (dict(oh=68), E), (dict(oh=56), E), (dict(ot=0), E), (dict(xt=1 << 40), E), (dict(x=None), E),
    (dict(pos=None), E), (dict(freqs=None), E), (dict(out=None), E), (dict(x=24), E), (dict(out=8), E), (dict(pos=12), E),
    (dict(freqs=20), E), (dict(ot=64, oh=64), E), (dict(ot=64, oh=120), E), (dict(T=3, ot=64, oh=184), E), (dict(T=0, x=None), OK),
])
def test_rope_refuses(lib, kw, code):  # noqa: F811
    assert _rope(lib, **kw) == code
    if code != OK:
        assert lib.mla_last_error().decode().startswith("mla_rope")


def _store(lib, **kw):
    names = ["latent", "ls", "k_rope", "rs", "pos", "freqs", "table", "stride", "maxb", "B", "N", "bs", "cp", "rank", "il",
             "half", "m", "cache", "nb", "slots", "stream"]
    return _call(lib.cp_rope_store, names, dict(latent=16, ls=576, k_rope=16, rs=576, pos=16, freqs=16, table=16, stride=4,
                                                maxb=4, B=1, N=8, bs=16, cp=2, rank=0, il=1, half=0, m=1.0, cache=16, nb=4,
                                                slots=None, stream=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), E), (dict(N=-1), E), (dict(bs=0), E), (dict(cp=0), E), (dict(rank=2), E), (dict(rank=-1), E), (dict(il=3), E),
    (dict(il=0), E), (dict(maxb=5), E), (dict(maxb=0), E), (dict(nb=0), E), (dict(m=math.nan), E), (dict(ls=-576), E),
    (dict(rs=4), E), (dict(latent=None), E), (dict(k_rope=None), E), (dict(pos=None), E), (dict(freqs=None), E),
    (dict(table=None), E), (dict(cache=None), E), (dict(latent=24), E), (dict(k_rope=8), E), (dict(cache=40), E),
    (dict(pos=12), E), (dict(slots=12), E), (dict(table=18), E), (dict(B=1 << 16, N=1 << 16), U),
    (dict(bs=1 << 16, cp=1 << 16), U), (dict(B=0, latent=None), OK), (dict(N=0, cache=None), OK),
])
def test_rope_store_refuses(lib, kw, code):  # noqa: F811
    assert _store(lib, **kw) == code
    if code != OK:
        assert lib.mla_last_error().decode().startswith("cp_rope_store")


def _expand(lib, **kw):
    names = ["cache", "sc", "table", "stride", "seq", "starts", "B", "bs", "nb", "maxb", "w", "H", "S", "kv", "kr", "stream"]
    return _call(lib.mla_expand, names, dict(cache=16, sc=None, table=16, stride=4, seq=16, starts=16, B=1, bs=16, nb=4, maxb=4,
                                             w=16, H=2, S=64, kv=16, kr=16, stream=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), E), (dict(S=-1), E), (dict(H=0), E), (dict(bs=0), E), (dict(nb=0), E), (dict(maxb=0), E), (dict(maxb=5), E),
    (dict(sc=16, bs=24), E), (dict(cache=None), E), (dict(table=None), E), (dict(seq=None), E), (dict(starts=None), E),
    (dict(w=None), E), (dict(kv=None), E), (dict(kr=None), E), (dict(cache=24), E), (dict(w=8), E), (dict(kv=8), E),
    (dict(kr=8), E), (dict(table=18), E), (dict(seq=18), E), (dict(starts=18), E), (dict(sc=18), E), (dict(H=1 << 30), U), (dict(S=2**31 - 1, H=1), U),
    (dict(bs=1 << 20, maxb=1 << 12, stride=1 << 12), U), (dict(B=0, cache=None), OK), (dict(S=0, kv=None), OK),
])
def test_expand_refuses(lib, kw, code):  # noqa: F811
    assert _expand(lib, **kw) == code
    if code != OK:
        assert lib.mla_last_error().decode().startswith("mla_expand")


def _prefill(lib, **kw):
    names = ["q", "qt", "qh", "k", "ks", "kh", "kr", "rs", "v", "vs", "vh", "cu", "starts", "seq", "gseq", "T", "B", "H", "S",
             "causal", "cp", "rank", "il", "scale", "out", "lse", "base_e", "ws", "ws_bytes", "stream"]
    return _call(lib.mla_prefill, names, dict(q=16, qt=384, qh=192, k=16, ks=256, kh=256 * 64, kr=16, rs=64, v=16, vs=256,
                                              vh=256 * 64, cu=16, starts=16, seq=16, gseq=16, T=8, B=1, H=2, S=64, causal=1,
                                              cp=1, rank=0, il=1, scale=0.1, out=16, lse=16, base_e=1, ws=None, ws_bytes=0,
                                              stream=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), E), (dict(B=-1), E), (dict(S=-1), E), (dict(H=0), E), (dict(cp=0), E), (dict(rank=1), E),
    (dict(rank=-1), E), (dict(il=0), E), (dict(scale=0.0), E), (dict(scale=-1.0), E), (dict(scale=math.nan), E),
    (dict(scale=math.inf), E), (dict(qt=4), E), (dict(qt=0), E), (dict(qh=-192), E), (dict(ks=12), E), (dict(ks=0), E),
    (dict(kh=0), E), (dict(rs=0), E), (dict(vs=0), E), (dict(vh=12), E), (dict(q=None), E), (dict(k=None), E),
    (dict(kr=None), E), (dict(v=None), E), (dict(cu=None), E), (dict(starts=None), E), (dict(seq=None), E),
    (dict(out=None), E), (dict(cp=2, gseq=None), E), (dict(q=24), E), (dict(k=24), E), (dict(kr=24), E), (dict(v=24), E),
    (dict(out=24), E), (dict(cu=18), E), (dict(lse=18), E), (dict(gseq=18), E), (dict(ws=272, ws_bytes=1 << 20), E),
    (dict(H=1 << 30, T=1 << 10), U), (dict(cp=1 << 16, il=1 << 16), U), (dict(T=0, q=None), OK), (dict(B=0, q=None), OK),
])
def test_prefill_refuses(lib, kw, code):  # noqa: F811
    assert _prefill(lib, **kw) == code
    if code != OK:
        assert lib.mla_last_error().decode().startswith("mla_prefill")


@pytest.mark.parametrize("kw,code", [
    (dict(dv=64), U), (dict(n=0), E), (dict(T=-1), E), (dict(H=0), E), (dict(parts=None), E), (dict(lses=None), E),
    (dict(out=None), E), (dict(parts=24), E), (dict(out=24), E), (dict(lse=18), E), (dict(T=0, out=None), OK),
    (dict(dv=512, n=0), E), (dict(dv=512, T=0, out=None), OK),
])
def test_merge_refuses(lib, kw, code):  # noqa: F811
    names = ["parts", "fp32", "lses", "n", "T", "H", "dv", "out", "lse", "base_e", "stream"]
    assert _call(lib.lse_merge_v, names, dict(parts=16, fp32=0, lses=16, n=2, T=1, H=1, dv=128, out=16, lse=None, base_e=1,
                                              stream=None), kw) == code


def test_prefill_workspace_size(lib):  # noqa: F811
    f = lib.mla_prefill_workspace_size
    assert f(0, 1, 1, 1, 152) == 0 and f(8, 0, 1, 1, 152) == 0
    assert f(8192, 1, 128, 8192, 152) == 0                      # enough blocks without a split
    n = f(64, 1, 8, 32768, 152)                                 # two row tiles at most, 8 heads: 16 blocks -> 9 parts
    assert n >= 9 * 64 * 8 * 129 * 4
    assert f(64, 1, 8, 100, 152) == 0                           # too few keys to cut


# ---- the wrappers --------------------------------------------------------------------------------
def test_wrappers_refuse_what_is_not_on_the_gpu(lib):  # noqa: F811
    bf = dict(dtype=torch.bfloat16)
    x, pos, freqs = torch.zeros(2, 1, 64, **bf), torch.zeros(2, dtype=torch.int64), M.rope_freqs(device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        M.mla_rope(x, pos, freqs)
    with pytest.raises(TypeError, match="x must be"):
        M.mla_rope(x.float(), pos, freqs)
    with pytest.raises(TypeError, match="x must be a torch.Tensor"):
        M.mla_rope(None, pos, freqs)
    with pytest.raises(ValueError, match="latent must be a CUDA tensor"):
        M.cp_rope_store(torch.zeros(1, 1, 512, **bf), torch.zeros(1, 1, 64, **bf), pos.view(1, 2), freqs, i.view(1, 2), x)
    with pytest.raises(ValueError, match="kv_cache must be a CUDA tensor"):
        M.mla_expand(torch.zeros(1, 16, 576, **bf), i.view(2, 1), i, i, torch.zeros(1, 256, 512, **bf), 4)
    with pytest.raises(TypeError, match="kv_cache must be"):
        M.mla_expand(torch.zeros(1, 16, 576, **bf), i.view(2, 1), i, i, torch.zeros(1, 256, 512, **bf), 4,
                     kv_scales=torch.ones(1, 1))
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        M.mla_prefill(torch.zeros(2, 1, 192, **bf), x, x, x, i, i, i, None, 0.1)


def test_rope_freqs():
    f = M.rope_freqs(theta=10000.0, device="cpu")
    assert f.dtype == torch.int64 and f.shape == (32,)
    want = 10000.0 ** (-np.arange(32) / 32.0) / (2 * math.pi)
    assert np.allclose(f.numpy().astype(np.float64) / 2.0 ** 64, want, rtol=1e-15, atol=0.5 / 2.0 ** 64)
    lin = M.rope_freqs(scaling="linear", factor=4.0, device="cpu").numpy()
    # (whole units: half of one for each of the two, the first times 4)
    assert np.allclose(lin.astype(np.float64) * 4, f.numpy().astype(np.float64), rtol=1e-15, atol=2.5)
    ntk = M.rope_freqs(scaling="ntk", factor=4.0, device="cpu").numpy().astype(np.float64)
    assert ntk[0] == f.numpy().astype(np.float64)[0] and np.allclose(ntk[31] * 4, f.numpy().astype(np.float64)[31], rtol=1e-12)
    yarn = M.rope_freqs(scaling="yarn", factor=40.0, original_max_position=4096, device="cpu").numpy().astype(np.float64)
    ratio = f.numpy().astype(np.float64) / yarn
    turns = 4096 * want
    assert np.allclose(ratio[turns > 40], 1.0) and np.allclose(ratio[turns < 0.75], 40.0) and (np.diff(ratio) > -1e-9).all()
    slow = M.rope_freqs(theta=1.0001, device="cpu").numpy()       # nearly a radian a position: no overflow
    assert (slow > 0).all() and np.allclose(slow.astype(np.float64) / 2.0 ** 64, 1 / (2 * math.pi), rtol=1e-3)
    for kw in (dict(theta=1.0), dict(theta=math.inf), dict(factor=0.0), dict(scaling="other"), dict(scaling="ntk", factor=1e-9),
               dict(scaling="yarn", original_max_position=0), dict(scaling="yarn", beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(ValueError):
            M.rope_freqs(device="cpu", **kw)


# ---- the oracle ------------------------------------------------------------------------------------
def test_oracle_rotation():
    """Lengths are kept, positions add up, and the product of two turned rows goes by their distance."""
    g = np.random.default_rng(0)
    f = M.rope_freqs(device="cpu").tolist()
    x, y = g.normal(size=64), g.normal(size=64)
    for half in (False, True):
        a = P.ref_rope_row(x, 1234567, f, half, 1.0)
        assert np.isclose(np.linalg.norm(a), np.linalg.norm(x))
        assert np.allclose(P.ref_rope_row(P.ref_rope_row(x, 70, f, half, 1.0), 30, f, half, 1.0), P.ref_rope_row(x, 100, f, half, 1.0))
        d = [P.ref_rope_row(x, p, f, half, 1.0) @ P.ref_rope_row(y, p - 9, f, half, 1.0) for p in (9, 100, 54321)]
        assert np.allclose(d, d[0])
    one = np.zeros(64)
    one[0] = 1.0
    assert np.allclose(P.ref_rope_row(one, 1, [1 << 62] * 32, False, 2.0)[:2], [0.0, 2.0])      # a quarter turn
    assert np.allclose(P.ref_rope_row(one, 1, [1 << 62] * 32, True, 2.0)[[0, 32]], [0.0, 2.0])


def test_oracle_expanded_attention_is_absorbed_attention():
    """The expanded form of a few rows equals the decode oracle on absorbed queries."""
    g = np.random.default_rng(1)
    H, G, n = 2, 9, 3
    w, rows, q = g.normal(size=(H, 256, 512)) * 0.05, g.normal(size=(G, 576)), g.normal(size=(n, H, 192))
    kv, kr, _, mine = P.ref_expand(lambda b: rows, [G], [0], w, G)
    assert mine.all()
    for cp, rank, il in [(1, 0, 1), (2, 1, 2)]:
        own = R.ref_owned_positions(G, cp, rank, il)
        out, lse, A, D, _ = P.ref_prefill(q, kv[:, own, :128].transpose(1, 0, 2), kr[own], kv[:, own, 128:].transpose(1, 0, 2),
                                          [0, n], [0], [len(own)], [G], 0.1, cp, rank, il, True)
        absorbed = np.concatenate([np.einsum("nhd,hdc->nhc", q[..., :128], w[:, :128]), q[..., 128:]], -1)
        pool = np.zeros((1, 16, 576))
        pool[0, :len(own)] = rows[own]
        o, l = R.ref_mla_decode(absorbed[None], pool, np.array([[0]]), [len(own)], [G], n, cp, rank, 0.1, interleave=il)
        assert np.allclose(out, np.einsum("thc,hdc->thd", o.reshape(n, H, 512), w[:, 128:]))
        assert np.allclose(lse, l.reshape(n, H)) and (A >= np.abs(out) - 1e-12).all()


def test_oracle_store_is_rotation_and_scatter():
    g = np.random.default_rng(2)
    f = M.rope_freqs(device="cpu").tolist()
    kv, cache = g.normal(size=(2, 5, 576)), g.normal(size=(6, 4, 576))
    table, pos = np.array([[3, 1], [5, 0]]), np.array([[0, 1, 2, -1, 7], [9, 10, 11, 12, -1]])
    got, written, slots = P.ref_rope_store(kv[..., :512], kv[..., 512:], pos, f, table, cache, 2, 1, 2, False, 1.0)
    rot = kv.copy()
    for b in range(2):
        for n in range(5):
            if pos[b, n] >= 0:
                rot[b, n, 512:] = P.ref_rope_row(kv[b, n, 512:], pos[b, n], f, False, 1.0)
    want = R.ref_scatter_kv(cache.copy(), pos, rot, table, 4, 2, 1, 2)
    assert np.allclose(got, want[0] if isinstance(want, tuple) else want) and len(written) == (slots >= 0).sum()

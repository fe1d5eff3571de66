"""The 8-bit paged cache without a GPU: what the C entry points and the Python wrappers
refuse, and checks that pin its oracle (torch's e4m3 conversion, hand-worked steps)."""
import ctypes
import os
import shutil

import numpy as np
import pytest
import torch

import mla_paged_decode_03_gb300 as M
import oracle.q8_ref as Q
from mla_paged_decode_03_gb300 import _lib, build

from test_abi_cpu import lib  # noqa: F401  (the built library)

E, U, OK = _lib.MLA_ERR_INVALID_ARGUMENT, _lib.MLA_ERR_UNSUPPORTED, _lib.MLA_OK


# ---- refusals of the C entry points (checked on the host before any CUDA call) ---------------
def _tables(lib, **kw):
    # distinct addresses 4 KB apart: outputs may not overlap inputs or one another
    names = ["prev", "ctx", "new", "B", "N", "table", "stride", "maxb", "ring", "cap", "state",
             "state_out", "bs", "cp", "rank", "ranks", "il", "total", "seq", "pos", "slots", "stream"]
    a = dict(prev=4096, ctx=8192, new=12288, B=4, N=2, table=16384, stride=8, maxb=8, ring=20480,
             cap=64, state=24576, state_out=28672, bs=16, cp=2, rank=0, ranks=2, il=1, total=32768,
             seq=36864, pos=40960, slots=45056, stream=None)
    a.update(kw)
    return lib.cp_step_tables(*[a[n] for n in names])


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), E), (dict(N=-1), E), (dict(bs=0), E), (dict(cp=0), E), (dict(rank=-1), E),
    (dict(rank=2), E), (dict(ranks=0), E), (dict(ranks=3), E), (dict(rank=1, ranks=2), E),
    (dict(il=0), E), (dict(il=3), E), (dict(maxb=0), E), (dict(maxb=9), E), (dict(cap=0), E),
    (dict(prev=None), E), (dict(ctx=None), E), (dict(new=None), E), (dict(table=None), E),
    (dict(ring=None), E), (dict(state=None), E), (dict(state_out=None), E), (dict(total=None), E),
    (dict(prev=4098), E), (dict(pos=40964), E), (dict(slots=45060), E), (dict(state=24578), E),
    (dict(total=4096), E),                  # over prev_lens
    (dict(total=4108), E),                  # its first entry is prev_lens' last
    (dict(total=8192), E), (dict(state_out=24576), E), (dict(state_out=24580), E),
    (dict(pos=16384), E), (dict(slots=40960), E), (dict(seq=32768), E), (dict(ring=16384), E),
    (dict(B=1 << 16, N=1 << 14, ranks=2, pos=None, slots=None), U),
    (dict(bs=1 << 16, cp=1 << 16), U),
])
def test_step_tables_refuses(lib, kw, code):  # noqa: F811
    assert _tables(lib, **kw) == code
    assert lib.mla_last_error().decode().startswith("cp_step_tables")


def _store(lib, **kw):
    names = ["rows", "ctx", "total", "table", "stride", "maxb", "B", "N", "bs", "cp", "rank", "il",
             "cache", "scales", "nb", "stream"]
    a = dict(rows=16, ctx=16, total=16, table=16, stride=4, maxb=4, B=1, N=8, bs=16, cp=2, rank=0,
             il=1, cache=16, scales=16, nb=4, stream=None)
    a.update(kw)
    return lib.cp_store_q8(*[a[n] for n in names])


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), E), (dict(N=-1), E), (dict(bs=8), E), (dict(bs=24), E), (dict(bs=0), E),
    (dict(cp=0), E), (dict(rank=2), E), (dict(il=3), E), (dict(maxb=5), E), (dict(nb=0), E),
    (dict(rows=None), E), (dict(ctx=None), E), (dict(total=None), E), (dict(table=None), E),
    (dict(cache=None), E), (dict(scales=None), E), (dict(rows=24), E), (dict(cache=40), E),
    (dict(scales=18), E), (dict(B=1 << 16, N=1 << 16), U), (dict(B=0, rows=None), OK),
    (dict(N=0, rows=None), OK),
])
def test_store_refuses(lib, kw, code):  # noqa: F811
    assert _store(lib, **kw) == code
    if code != OK:
        assert lib.mla_last_error().decode().startswith("cp_store_q8")


def _decode(lib, shards, **kw):
    names = ["q", "kv", "sc", "bt", "stride", "seq", "gseq", "B", "H", "q_len", "causal", "bs", "nb",
             "maxb"] + (["n"] if shards else ["cp", "rank"]) + [
             "il", "scale", "out", "lse", "base_e", "ws", "ws_bytes", "stream"]
    a = dict(q=16, kv=16, sc=16, bt=16, stride=4, seq=16, gseq=16, B=1, H=16, q_len=1, causal=1, bs=16,
             nb=4, maxb=4, n=2, cp=1, rank=0, il=1, scale=0.1, out=16, lse=16, base_e=1, ws=None,
             ws_bytes=0, stream=None)
    a.update(kw)
    f = lib.mla_decode_shards_q8 if shards else lib.mla_decode_q8
    return f(*[a[n] for n in names])


@pytest.mark.parametrize("shards", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), E), (dict(H=0), E), (dict(q_len=0), E), (dict(q_len=17), U), (dict(bs=8), E),
    (dict(bs=40), E), (dict(bs=0), E), (dict(nb=0), E), (dict(maxb=5), E), (dict(scale=0.0), E),
    (dict(scale=float("nan")), E), (dict(q=None), E), (dict(kv=None), E), (dict(sc=None), E),
    (dict(sc=18), E), (dict(bt=None), E), (dict(seq=None), E), (dict(out=None), E), (dict(q=24), E),
    (dict(kv=24), E), (dict(out=24), E), (dict(ws=272, ws_bytes=1024), E), (dict(il=3), E),
    (dict(B=1 << 20, H=1 << 8, q_len=16), U), (dict(B=0, q=None, out=None), OK),
])
def test_decode_refuses(lib, shards, kw, code):  # noqa: F811
    assert _decode(lib, shards, **kw) == code
    if code != OK:
        assert b"_q8" in lib.mla_last_error()


def test_shards_need_global_lengths(lib):  # noqa: F811
    assert _decode(lib, True, gseq=None) == E
    assert _decode(lib, True, n=0) == E
    assert _decode(lib, True, B=20000, n=16) == U
    assert _decode(lib, False, gseq=None, cp=2) == E


def test_workspace_size(lib):  # noqa: F811
    f = lib.mla_decode_q8_workspace_size
    assert f(0, 16, 1, 152) == 0 and f(1, 0, 1, 152) == 0 and f(1, 16, 0, 152) == 0
    assert f(8, 16, 1, 152) == f(8, 16, 1, 152) > 0


# ---- refusals of the Python wrappers ----------------------------------------------------------
def test_wrappers_refuse_cpu_tensors_and_wrong_types(lib):  # noqa: F811
    i32 = torch.zeros(2, dtype=torch.int32)
    bt = torch.zeros(2, 4, dtype=torch.int32)
    rows = torch.zeros(2, 1, 576, dtype=torch.bfloat16)
    cache = torch.zeros(8, 16, 576).to(torch.float8_e4m3fn)
    sc = torch.ones(8, 1)
    q = torch.zeros(2, 1, 16, 576, dtype=torch.bfloat16)
    bad = (ValueError, TypeError)
    with pytest.raises(bad):
        M.cp_step_tables(i32, i32, i32, bt, i32, i32, 16, 1)
    with pytest.raises(bad):
        M.cp_store_q8(rows, i32, i32, bt, cache, sc)
    with pytest.raises(bad):
        M.mla_decode_q8(q, cache, sc, bt, i32, i32, 1, 1, 0, 0.1)
    with pytest.raises(bad):
        M.mla_decode_shards_q8(q, cache.float(), sc, bt, i32, i32, 1, 1, 0.1)


# ---- the oracle -------------------------------------------------------------------------------
def test_oracle_e4m3_is_torchs():
    # every e4m3 value, every midpoint between neighbours, and what lies next to them
    every = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float()
    v = torch.sort(every[torch.isfinite(every)]).values.double()
    mid = (v[1:] + v[:-1]) / 2
    x = torch.cat([v, mid, mid * (1 + 2 ** -20), mid * (1 - 2 ** -20), torch.tensor([2.0 ** -12, 0.0])])
    want = x.float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(Q.ref_e4m3(x.numpy()), want)
    assert np.array_equal(Q.ref_e4m3([1e6, -465.0]), [448.0, -448.0]) and np.isnan(Q.ref_e4m3(np.nan))


def test_oracle_scale():
    for a, s in ((448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (225.0, 1.0), (0.0, 2.0 ** -32),
                 (2.0 ** -60, 2.0 ** -32), (2.0 ** 100, 2.0 ** 64), (1.75, 2.0 ** -8)):
        assert Q.ref_scale(a) == s


def test_oracle_step_by_hand():
    # pages of 2 x 2 positions; request 0 grows by one page, 1 gives two back, 2 does not fit
    # the supply, 3 needs nothing
    table = np.array([[7, -1, -1], [5, 6, 4], [3, -1, -1], [2, -1, -1]])
    total, seq, pos, slots, t, ring, state = Q.ref_step_tables(
        [4, 11, 4, 3], [4, 2, 4, 2], [2, 0, 5, 2], table, [9, 8, 0, 0, 0, 0], (0, 2), 2, 5, 2, [0, 1])
    assert total.tolist() == [6, 2, 4, 4]
    assert t[0].tolist() == [7, 9, -1] and t[2].tolist() == [3, -1, -1]
    assert ring.tolist() == [9, 8, 6, 4, 0, 0] and state.tolist() == [1, 3]
    assert pos[0].tolist() == [4, 5, -1, -1, -1] and pos[2].tolist() == [-1] * 5
    assert seq.tolist() == [[3, 1, 2, 2], [3, 1, 2, 2]]
    assert slots[0, 0].tolist() == [18, -1, -1, -1, -1] and slots[1, 0].tolist() == [-1, 18, -1, -1, -1]
    assert slots[0, 3].tolist() == [5, -1, -1, -1, -1] and slots[1, 3].tolist() == [-1, 5, -1, -1, -1]


def test_oracle_store_by_hand():
    cache, scales = np.zeros((2, 16, 576)), np.full((2, 1), 99.0)
    rows = np.zeros((1, 2, 576))
    rows[0, 0, :2] = [1.0, -1.75]           # scale 2^-8
    c, s = Q.ref_store_q8(rows[:, :1], [0], [1], [[1]], cache, scales, 1, 0)
    assert s[1, 0] == 2.0 ** -8 and s[0, 0] == 99 and c[1, 0, :2].tolist() == [256.0, -448.0]
    rows[0, 1, :3] = [7.0, np.inf, np.nan]  # scale 2^-6: the earlier row is stored again
    c, s = Q.ref_store_q8(rows[:, 1:], [1], [2], [[1]], c, s, 1, 0)
    assert s[1, 0] == 2.0 ** -6 and c[1, 0, :2].tolist() == [64.0, -112.0]
    assert c[1, 1, 0] == 448.0 and np.isnan(c[1, 1, 1:3]).all()
    assert np.allclose(Q.ref_dequantised(c, s)[1, 0, :2], [1.0, -1.75])


# ---- the library and its binding ---------------------------------------------------------------
def _use_objects(lib, monkeypatch, tmp_path):  # noqa: F811
    """build() into tmp_path, from the objects that the library was built of."""
    objs, here = build.OBJDIR, build._compile
    monkeypatch.setattr(build, "LIBDIR", str(tmp_path))
    monkeypatch.setattr(build, "OBJDIR", str(tmp_path / "obj"))

    def compiled(src, extra):
        obj = os.path.join(objs, os.path.basename(src)[:-3] + ".o")
        if not os.path.exists(obj):
            return here(src, extra)
        return shutil.copy(obj, build.OBJDIR)
    monkeypatch.setattr(build, "_compile", compiled)


def test_library_is_built_without_its_binding(lib, monkeypatch, tmp_path):  # noqa: F811
    """Where the binding does not compile (no C++ compiler here; no headers of Python or PyTorch) the
    C library is still built, no older binding stays beside it, and the failure is raised."""
    _use_objects(lib, monkeypatch, tmp_path)
    monkeypatch.setenv("CXX", "false")
    (tmp_path / "q8_binding.so").write_bytes(b"of an older build")
    with pytest.raises(RuntimeError, match="q8_binding"):
        build.build()
    assert ctypes.CDLL(build.lib_path()).mla_abi_version() == lib.mla_abi_version()
    assert not os.path.exists(build.binding_path())


def test_library_that_does_not_link_leaves_the_old_pair(lib, monkeypatch, tmp_path):  # noqa: F811
    _use_objects(lib, monkeypatch, tmp_path)
    monkeypatch.setattr(build, "_build_binding", lambda: str(tmp_path / "new"))
    monkeypatch.setattr(build, "ARCH", ["--no-such-option"])
    for f in (build.lib_path(), build.binding_path()):
        open(f, "w").write("old")
    with pytest.raises(RuntimeError, match="link failed"):
        build.build()
    for f in (build.lib_path(), build.binding_path()):
        assert open(f).read() == "old"


def test_binding_refuses_a_library_of_another_abi(lib):  # noqa: F811
    b = _lib.load_q8(M.StepTables)
    other = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: lib.mla_abi_version() + 1)
    address = [ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
               for f in ("cp_step_tables", "cp_store_q8", "mla_decode_q8", "mla_decode_shards_q8",
                         "mla_decode_q8_workspace_size")]
    with pytest.raises(ImportError, match="ABI version"):
        b.bind(*address, ctypes.cast(other, ctypes.c_void_p).value, _lib.check, M.StepTables)
    # and goes on with the one it was bound to
    with pytest.raises((ValueError, TypeError)):
        M.cp_store_q8(None, None, None, None, None, None)

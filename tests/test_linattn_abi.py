"""The entry points of kda_linattn.h are exported and refuse bad arguments on
the host before any HIP call (fake device addresses, never dereferenced)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = [0x10000000 * (i + 1) for i in range(16)]


def _fn(name):
    import gated_delta_rule_58_amd as kda
    if not os.path.exists(kda.lib_path()):
        from gated_delta_rule_58_amd.build import build_library
        build_library()
    from gated_delta_rule_58_amd import linattn
    return linattn._fn(name)


def _last():
    import gated_delta_rule_58_amd as kda
    return kda.lib().kda_last_error().decode()


def test_every_declared_entry_point_is_bound():
    import gated_delta_rule_58_amd as kda
    from gated_delta_rule_58_amd import linattn
    src = open(os.path.join(ROOT, "include", "kda_linattn.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"\b(kda_[a-z0-9_]+)\s*\(", src))
    assert names == set(linattn._SIGNATURES)
    assert names <= set(kda.exported_symbols())
    for n in names:
        _fn(n)


def _host(cu):
    a = np.ascontiguousarray(np.asarray(cu, dtype=np.int32))
    return a, a.ctypes.data


def _prefill(cu_host=(0, 20, 48), **kw):
    a = dict(q=DEV[0], qs=4 * 128, k=DEV[1], ks=4 * 128, v=DEV[2], vs=8 * 128, dt=1, g=DEV[3],
             g_len=48 * 8, cu=DEV[4], N=2, S0=None, Sf=DEV[5], S_dt=0, slots=2, idx=None, o=DEV[6],
             o_dt=1, T=48, H=8, Hk=4, dk=128, dv=128, scale=1.0, ws=None, ws_bytes=0)
    a.update(kw)
    keep, hp = _host(cu_host) if cu_host is not None else (None, None)
    return _fn("kda_linattn_chunk_prefill")(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["dt"], a["g"], a["g_len"], a["cu"],
        hp, a["N"], a["S0"], a["Sf"], a["S_dt"], a["slots"], a["idx"], a["o"], a["o_dt"], a["T"],
        a["H"], a["Hk"], a["dk"], a["dv"], a["scale"], a["ws"], a["ws_bytes"], None)


SHARED = [
    (dict(H=0), 1), (dict(Hk=0), 1), (dict(Hk=3, qs=4 * 128), 2), (dict(dt=7), 3),
    (dict(dk=96), 4), (dict(dv=256), 4), (dict(scale=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(g_len=7), 2), (dict(qs=4 * 128 - 8), 2),
    (dict(vs=8 * 128 - 8), 2), (dict(ks=(1 << 22) + 8), 4), (dict(ks=4 * 128 + 4), 5),
    (dict(q=DEV[0] + 8), 5), (dict(v=DEV[2] + 2), 5), (dict(g=DEV[3] + 2), 5), (dict(k=None), 1),
    (dict(g=None), 1), (dict(o=DEV[6] + 8), 5), (dict(o=DEV[0]), 1), (dict(o_dt=5), 3),
    (dict(S_dt=5), 3), (dict(slots=-1), 1), (dict(slots=1), 2), (dict(idx=DEV[7] + 2), 5),
    (dict(H=16385, Hk=16385, qs=16385 * 128, ks=16385 * 128, vs=16385 * 128, g_len=16385), 4),
]


@pytest.mark.parametrize("bad, status", SHARED + [
    (dict(N=0), 1), (dict(T=-1), 1), (dict(cu=None), 1), (dict(cu=DEV[4] + 2), 5),
    (dict(o=None), 1), (dict(Sf=DEV[2]), 1), (dict(S0=DEV[5] + 16), 1), (dict(S0=DEV[8] + 8), 5),
    (dict(ws=DEV[9] + 16, ws_bytes=1 << 20), 5), (dict(ws=DEV[0], ws_bytes=1 << 20), 1),
    (dict(Sf=DEV[4]), 1), (dict(T=1 << 31, g_len=8), 4),
])
def test_prefill_refusals(bad, status):
    assert _prefill(**bad) == status, _last()
    assert "kda_linattn_chunk_prefill" in _last()


@pytest.mark.parametrize("cu", [(1, 20, 48), (0, 30, 20), (0, 20, 47), (0, 49, 48)])
def test_prefill_refuses_bad_cu_seqlens(cu):
    assert _prefill(cu_host=cu) == 2


def test_prefill_equal_lengths_need_a_multiple():
    assert _prefill(cu_host=None, cu=None, N=5, slots=5) == 2
    assert "multiple" in _last()


def _decode(**kw):
    a = dict(q=DEV[0], qs=4 * 128, k=DEV[1], ks=4 * 128, v=DEV[2], vs=8 * 128, dt=1, g=DEV[3],
             g_len=48 * 8, S=DEV[5], S_dt=0, slots=48, idx=None, o=DEV[6], o_dt=1, T=48, H=8,
             Hk=4, dk=128, dv=128, scale=1.0)
    a.update(kw)
    return _fn("kda_linattn_recurrent_decode")(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["dt"], a["g"], a["g_len"], a["S"],
        a["S_dt"], a["slots"], a["idx"], a["o"], a["o_dt"], a["T"], a["H"], a["Hk"], a["dk"],
        a["dv"], a["scale"], None)


@pytest.mark.parametrize("bad, status", SHARED + [
    (dict(T=-1, g_len=8), 1), (dict(S=None), 1), (dict(S=DEV[2]), 1), (dict(S=DEV[5] + 4), 5),
    (dict(S=DEV[6]), 1), (dict(slots=47), 2), (dict(o=None), 1),
])
def test_decode_refusals(bad, status):
    assert _decode(**bad) == status, _last()
    assert "kda_linattn_recurrent_decode" in _last()


def test_decode_of_nothing_is_nothing():
    assert _decode(T=0, g_len=0, slots=0, q=None, k=None, v=None, g=None, S=None, o=None) == 0


def _backward(cu_host=(0, 20, 48), **kw):
    need = _fn("kda_linattn_chunk_prefill_backward_workspace_bytes")(48, 2, 8, 4, 128, 128)
    a = dict(q=DEV[0], qs=4 * 128, k=DEV[1], ks=4 * 128, v=DEV[2], vs=8 * 128, dt=1, g=DEV[3],
             g_len=48 * 8, cu=DEV[4], N=2, S0=None, do=DEV[5], do_dt=1, dS=None, dq=DEV[6],
             dk_=DEV[7], dv_=DEV[8], gdt=1, dg=DEV[9], dS0=DEV[10], T=48, H=8, Hk=4, dk=128,
             dv=128, scale=1.0, ws=DEV[11], ws_bytes=need)
    a.update(kw)
    keep, hp = _host(cu_host) if cu_host is not None else (None, None)
    return _fn("kda_linattn_chunk_prefill_backward")(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["dt"], a["g"], a["g_len"], a["cu"],
        hp, a["N"], a["S0"], a["do"], a["do_dt"], a["dS"], a["dq"], a["dk_"], a["dv_"], a["gdt"],
        a["dg"], a["dS0"], a["T"], a["H"], a["Hk"], a["dk"], a["dv"], a["scale"], a["ws"],
        a["ws_bytes"], None)


@pytest.mark.parametrize("bad, status", [
    (dict(H=0), 1), (dict(Hk=3), 2), (dict(dk=32), 4), (dict(do_dt=4), 3), (dict(gdt=4), 3),
    (dict(dq=None), 1), (dict(dg=None), 1), (dict(g=None), 1), (dict(do=DEV[5] + 8), 5),
    (dict(dS0=DEV[10] + 4), 5), (dict(dg=DEV[9] + 2), 5), (dict(ws=None), 6),
    (dict(ws_bytes=1024), 6), (dict(ws=DEV[11] + 64), 5), (dict(dq=DEV[0]), 1),
    (dict(dk_=DEV[6]), 1), (dict(dS0=DEV[5]), 1), (dict(N=0), 1), (dict(cu=None), 1),
    (dict(ws=DEV[2]), 1),
])
def test_backward_refusals(bad, status):
    assert _backward(**bad) == status, _last()
    assert "kda_linattn_chunk_prefill_backward" in _last()


def test_workspace_sizes_of_unsupported_shapes_are_zero():
    f = _fn("kda_linattn_chunk_prefill_workspace_bytes")
    b = _fn("kda_linattn_chunk_prefill_backward_workspace_bytes")
    assert f(4096, 1, 8, 96, 128) == 0 and f(4096, 0, 8, 128, 128) == 0
    assert f(64, 1, 8, 128, 128) == 0            # too short to be cut
    assert f(1 << 17, 1, 8, 128, 128) > 0
    assert b(4096, 1, 8, 3, 128, 128) == 0 and b(4096, 1, 8, 8, 128, 32) == 0
    assert b(4096, 1, 8, 8, 128, 128) > 0


def _ln(**kw):
    a = dict(x=DEV[0], x_dt=1, w=DEV[1], b=DEV[2], groups=4, y=DEV[3], y_dt=1, rows=40, d=128,
             eps=1e-5)
    a.update(kw)
    return _fn("kda_layernorm")(a["x"], a["x_dt"], a["w"], a["b"], a["groups"], a["y"], a["y_dt"],
                                a["rows"], a["d"], a["eps"], None)


@pytest.mark.parametrize("bad, status", [
    (dict(rows=-1), 1), (dict(groups=0), 1), (dict(d=0), 1), (dict(rows=41), 2),
    (dict(x_dt=3), 3), (dict(y_dt=3), 3), (dict(d=16385), 4), (dict(groups=65536, rows=65536), 4),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(x=None), 1), (dict(y=None), 1),
    (dict(x=DEV[0] + 1), 5), (dict(w=DEV[1] + 2), 5), (dict(y=DEV[0] + 2), 1),
    (dict(y=DEV[0], y_dt=0), 1), (dict(y=DEV[1]), 1),
])
def test_layernorm_refusals(bad, status):
    assert _ln(**bad) == status, _last()
    assert "kda_layernorm" in _last()


def test_layernorm_of_no_rows_is_nothing():
    assert _ln(rows=0, x=None, y=None) == 0


def _lnb(**kw):
    a = dict(dy=DEV[0], dy_dt=1, x=DEV[1], x_dt=1, w=DEV[2], groups=4, dx=DEV[3], dw=DEV[4],
             db=DEV[5], rows=40, d=128, eps=1e-5, ws=DEV[6], ws_bytes=1 << 26)
    a.update(kw)
    return _fn("kda_layernorm_backward")(
        a["dy"], a["dy_dt"], a["x"], a["x_dt"], a["w"], a["groups"], a["dx"], a["dw"], a["db"],
        a["rows"], a["d"], a["eps"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad, status", [
    (dict(rows=-4), 1), (dict(rows=42), 2), (dict(d=20000), 4), (dict(dy_dt=9), 3),
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(ws=None), 6), (dict(ws_bytes=16), 6),
    (dict(ws=DEV[6] + 8), 5), (dict(dw=DEV[4] + 1), 5), (dict(dx=DEV[1] + 2), 1),
    (dict(dx=DEV[0], dy_dt=0), 1), (dict(dw=DEV[5]), 1), (dict(dw=DEV[0]), 1), (dict(ws=DEV[1]), 1),
])
def test_layernorm_backward_refusals(bad, status):
    assert _lnb(**bad) == status, _last()
    assert "kda_layernorm_backward" in _last()


def test_binding_refuses_what_the_library_cannot_see():
    """Shapes, dtypes, devices and strides are checked before any pointer is taken."""
    import gated_delta_rule_58_amd as kda
    q, v, g = torch.zeros(4, 2, 128), torch.zeros(4, 4, 128), torch.zeros(4, 4)
    with pytest.raises(ValueError, match="GPU"):
        kda.linattn_chunk_prefill(q, q, v, g)
    with pytest.raises(ValueError, match="k must be"):
        kda.linattn_chunk_prefill(q, q[:3], v, g)
    with pytest.raises(TypeError, match="one dtype"):
        kda.linattn_chunk_prefill(q, q.bfloat16(), v, g)
    with pytest.raises(TypeError, match="g must be"):
        kda.linattn_recurrent_decode(q, q, v, g.bfloat16(), torch.zeros(4, 4, 128, 128))
    with pytest.raises(ValueError, match="g must be"):
        kda.linattn_chunk_prefill_backward(q, q, v, g[:, :3], None)
    with pytest.raises(ValueError, match="GPU"):
        kda.layernorm(v)
    with pytest.raises(ValueError, match="last two"):
        kda.layernorm(v, torch.ones(3, 128))
    with pytest.raises(TypeError, match="weight"):
        kda.layernorm(v, torch.ones(128).bfloat16())
    from gated_delta_rule_58_amd import linattn
    with pytest.raises(ValueError, match="dense"):
        linattn._row_stride("q", torch.zeros(4, 128, 2).transpose(1, 2))
    assert linattn._row_stride("q", torch.zeros(4, 6, 128)[:, 2:4]) == 6 * 128

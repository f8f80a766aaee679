"""The entry points of the norm and of the scaled tables without a GPU: what they refuse on the host, before touching
the device.  No call here launches work."""
import ctypes

import pytest
import torch

import rotary_position_embedding_rope_gb300 as R
from rotary_position_embedding_rope_gb300 import _build

A = 0x1000000  # fake, aligned "device" addresses: never dereferenced on these paths
INV, UNS = R.ROPE_ERR_INVALID_ARG, R.ROPE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return R.load_library()


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


NORM = dict(q=A, k=2 * A, qo=3 * A, ko=4 * A, wq=5 * A, wk=6 * A, cos=7 * A, sin=8 * A, pos=None, pbs=0, B=2, Hq=4, Hk=2, S=8,
            D=64, qs=None, ks=None, rd=64, layout=0, sbh=1, eps=1e-6, dtype=1, wdtype=1, rows=16)
BWD = dict(NORM, gq=9 * A, gk=10 * A, dq=11 * A, dk=12 * A, dwq=13 * A, dwk=14 * A, ws=15 * A, wsb=1 << 20)


def fwd(lib, **over):
    a = dict(NORM, **over)
    return lib.rope_norm_qk_fwd(*(a[x] for x in ("q", "k", "qo", "ko", "wq", "wk", "cos", "sin", "pos", "pbs", "B", "Hq", "Hk", "S",
                                                 "D", "qs", "ks", "rd", "layout", "sbh", "eps", "dtype", "wdtype", "rows")), None)


def bwd(lib, **over):
    a = dict(BWD, **over)
    return lib.rope_norm_qk_bwd(*(a[x] for x in ("q", "k", "gq", "gk", "dq", "dk", "wq", "wk", "dwq", "dwk", "cos", "sin", "pos",
                                                 "pbs", "B", "Hq", "Hk", "S", "D", "qs", "ks", "rd", "layout", "sbh", "eps", "dtype",
                                                 "wdtype", "rows", "ws", "wsb")), None)


SHARED = [
    (dict(dtype=3), UNS), (dict(wdtype=2), UNS), (dict(dtype=0), UNS), (dict(layout=2), UNS), (dict(D=72), UNS), (dict(D=8, rd=8), UNS),
    (dict(D=272), UNS), (dict(rd=80), UNS), (dict(rd=8), UNS), (dict(q=A + 8), UNS), (dict(wk=6 * A + 4), UNS), (dict(cos=7 * A + 4), UNS),
    (dict(qs=strides(8 * 4 * 64, 4 * 64 + 4, 64)), UNS), (dict(B=-1), INV), (dict(S=-1), INV), (dict(Hq=-1), INV), (dict(sbh=2), INV),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(rows=0), INV), (dict(rows=-1), INV),
    (dict(q=None), INV), (dict(k=None), INV), (dict(cos=None), INV), (dict(pos=20 * A, pbs=7), INV), (dict(pos=20 * A + 2), INV),
    (dict(pbs=-1), INV), (dict(B=1 << 20, S=1 << 20), INV), (dict(qs=strides(0, 256, 64)), INV), (dict(ks=strides(1024, -128, 64)), INV),
]


@pytest.mark.parametrize("over,status", SHARED + [
    (dict(qo=None), INV), (dict(ko=4 * A + 8), UNS), (dict(qo=2 * A), INV), (dict(ko=3 * A + 64), INV), (dict(ko=5 * A - 128), INV),
    (dict(qo=A + 1024), INV), (dict(qo=A, qs=strides(8 * 512, 512, 64)), INV), (dict(pos=3 * A), INV)])
def test_forward_refuses(lib, over, status):
    assert fwd(lib, **over) == status


@pytest.mark.parametrize("over,status", SHARED + [
    (dict(gq=None), INV), (dict(dk=None), INV), (dict(gk=10 * A + 8), UNS), (dict(dwq=13 * A + 2), UNS), (dict(ws=None), INV),
    (dict(wsb=100), INV), (dict(wsb=-1), INV), (dict(ws=15 * A + 8), UNS), (dict(dq=9 * A), INV), (dict(dq=A), INV), (dict(dwk=13 * A), INV),
    (dict(dwq=5 * A), INV), (dict(ws=11 * A), INV)])
def test_backward_refuses(lib, over, status):
    assert bwd(lib, **over) == status


def test_nothing_to_do(lib):
    none = dict(q=None, k=None, qo=None, ko=None, wq=None, wk=None)
    assert fwd(lib, S=0, **none) == fwd(lib, B=0, **none) == fwd(lib, Hq=0, Hk=0, **none) == R.ROPE_OK
    assert bwd(lib, S=0, dwq=None, dwk=None, ws=None, wsb=0) == R.ROPE_OK
    assert lib.rope_norm_qk_workspace(64) > 0 and lib.rope_norm_qk_workspace(72) == lib.rope_norm_qk_workspace(0) == -1


APPEND = dict(q=A, k=2 * A, v=3 * A, qo=4 * A, kp=5 * A, vp=6 * A, wq=7 * A, wk=8 * A, table=9 * A, cu=10 * A, lens=11 * A, cos=12 * A,
              sin=13 * A, pos=None, off=0, n=2, total=10, qs=256, ks=128, vs=128, Hq=4, Hk=2, D=64, rd=64, layout=0, eps=1e-6, page=16,
              n_pages=8, blocks=4, dtype=1, wdtype=0, rows=64)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=0), UNS), (dict(wdtype=2), UNS), (dict(layout=2), UNS), (dict(D=96), UNS), (dict(rd=8), UNS), (dict(page=8), UNS),
    (dict(qs=260), UNS), (dict(q=A + 8), UNS), (dict(qo=4 * A + 8), UNS), (dict(wq=7 * A + 8), UNS), (dict(n=-1), INV), (dict(total=-1), INV),
    (dict(Hq=-1), INV), (dict(qs=248), INV), (dict(ks=120), INV), (dict(off=-1), INV), (dict(eps=-1.0), INV), (dict(rows=0), INV),
    (dict(q=None), INV), (dict(qo=None), INV), (dict(kp=None), INV), (dict(v=None), INV), (dict(cu=None), INV), (dict(lens=11 * A + 1), INV),
    (dict(vp=5 * A), INV), (dict(qo=5 * A), INV), (dict(qo=2 * A), INV), (dict(kp=A), INV), (dict(q=4 * A, qs=264), INV),
    (dict(qo=7 * A - 128), INV), (dict(n_pages=0), INV), (dict(blocks=0), INV)])
def test_append_refuses(lib, over, status):
    a = dict(APPEND, **over)
    assert lib.rope_norm_cache_append(*(a[x] for x in (
        "q", "k", "v", "qo", "kp", "vp", "wq", "wk", "table", "cu", "lens", "cos", "sin", "pos", "off", "n", "total", "qs", "ks", "vs", "Hq",
        "Hk", "D", "rd", "layout", "eps", "page", "n_pages", "blocks", "dtype", "wdtype", "rows")), None) == status


TABLE = dict(kind=2, theta=1e4, rd=64, rows=10, off=0, factor=2.0, orig=100, low=1.0, high=4.0, scale=0.0, cos=A, sin=2 * A)


@pytest.mark.parametrize("over,status", [
    (dict(kind=4), UNS), (dict(kind=-1), UNS), (dict(rd=514), UNS), (dict(rd=63), INV), (dict(rd=0), INV), (dict(kind=1, rd=2), INV),
    (dict(rows=-1), INV), (dict(off=-1), INV), (dict(off=2 ** 31 - 1), INV), (dict(rows=2 ** 31), INV), (dict(theta=1.0), INV),
    (dict(theta=float("inf")), INV), (dict(factor=0.5), INV), (dict(factor=float("nan")), INV), (dict(scale=-1.0), INV),
    (dict(orig=0), INV), (dict(low=0.0), INV), (dict(high=1.0), INV), (dict(kind=3, high=float("inf")), INV), (dict(cos=None), INV),
    (dict(sin=A + 64), INV), (dict(sin=2 * A + 2), INV)])
def test_tables_refuse(lib, over, status):
    a = dict(TABLE, **over)
    assert lib.rope_tables_build_scaled(*(a[x] for x in ("kind", "theta", "rd", "rows", "off", "factor", "orig", "low", "high", "scale",
                                                         "cos", "sin")), None) == status


def test_python_refuses_host_tensors():
    x, w, t = torch.zeros(1, 4, 2, 64), torch.ones(64), torch.zeros(8, 32)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        R.norm_rotate_qk(x, x, w, w, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        R.norm_rotate_qk_backward(x, x, x, x, w, w, t, t)
    y, pool = x[0].bfloat16(), torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        R.norm_cache_append(y, y, y, w, w, pool, pool, i[:2].view(2, 1), i, i[:2], t, t)
    with pytest.raises(TypeError, match="expected a tensor"):
        R.norm_rotate_qk(None, None, w, w, t, t)
    with pytest.raises(KeyError):
        R.norm_rotate_qk(x, x, w, w, t, t, layout="pairs")


PAGED = dict(q=A, kp=2 * A, vp=3 * A, o=4 * A, table=5 * A, cu=6 * A, lens=7 * A, cos=8 * A, sin=9 * A, pq=None, n=3, tq=40, qs=512, Hq=4,
             Hk=2, D=128, rd=128, layout=0, causal=1, scale=-1.0, page=16, n_pages=20, blocks=4, dtype=1, rows=64, ws=10 * A, wsb=1 << 25)


def paged_args(**over):
    a = dict(PAGED, **over)
    return [a[x] for x in ("q", "kp", "vp", "o", "table", "cu", "lens", "cos", "sin", "pq", "n", "tq", "qs", "Hq", "Hk", "D", "rd",
                           "layout", "causal", "scale", "page", "n_pages", "blocks", "dtype", "rows", "ws", "wsb")] + [None]


@pytest.mark.parametrize("over,status", [
    (dict(dtype=0), UNS), (dict(layout=3), UNS), (dict(D=80), UNS), (dict(rd=24), UNS), (dict(page=24), UNS), (dict(page=256), UNS),
    (dict(n=4097), UNS), (dict(qs=516), UNS), (dict(q=A + 2), UNS), (dict(o=4 * A + 8), UNS), (dict(kp=2 * A + 8), UNS),
    (dict(sin=9 * A + 8), UNS), (dict(ws=10 * A + 16), UNS), (dict(n=-1), INV), (dict(tq=-1), INV), (dict(tq=1 << 31), INV),
    (dict(Hq=5, qs=640), INV), (dict(Hk=0), INV), (dict(qs=504), INV), (dict(causal=2), INV), (dict(blocks=-1), INV), (dict(n_pages=0), INV),
    (dict(n_pages=1 << 30), INV), (dict(blocks=1 << 40), INV), (dict(blocks=1 << 28), INV), (dict(scale=float("nan")), INV), (dict(rows=0), INV),
    (dict(cos=None), INV), (dict(sin=None), INV), (dict(q=None), INV), (dict(kp=None), INV), (dict(o=None), INV), (dict(table=None), INV),
    (dict(cu=None), INV), (dict(lens=None), INV), (dict(ws=None), INV), (dict(wsb=1000), INV), (dict(lens=7 * A + 1), INV), (dict(pq=A + 2), INV),
    (dict(o=A), INV), (dict(o=3 * A + 128), INV), (dict(ws=2 * A), INV), (dict(ws=6 * A - 128), INV), (dict(ws=4 * A), INV)])
def test_paged_refuses(lib, over, status):
    assert lib.rope_attention_paged_fwd(*paged_args(**over)) == status


def test_paged_workspace(lib):
    ws = lib.rope_attention_paged_workspace
    need = ws(3, 40, 4, 2, 128, 16, 4)
    assert need > 40 * 4 * 128 * 4 and need % 128 == 0
    assert lib.rope_attention_paged_fwd(*paged_args(wsb=need - 1)) == INV
    assert ws(0, 40, 4, 2, 128, 16, 4) == ws(3, 0, 4, 2, 128, 16, 4) == ws(3, 40, 0, 0, 128, 16, 4) == 0
    assert ws(3, 40, 4, 3, 128, 16, 4) == ws(3, 40, 4, 2, 96, 16, 4) == ws(3, 40, 4, 2, 128, 48, 4) == ws(4097, 5000, 4, 2, 128, 16, 4) == -1
    assert lib.rope_attention_paged_fwd(*paged_args(tq=0, q=None, o=None, ws=None, wsb=0)) == R.ROPE_OK
    assert ws(64, 64, 32, 8, 128, 64, 128) < 64 << 20

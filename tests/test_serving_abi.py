"""The serving entry points without a GPU: what they refuse on the host,
before touching the device.  No call here launches work."""
import pytest
import torch

import rotary_position_embedding_rope_gb300 as R
from rotary_position_embedding_rope_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return R.load_library()


A = 0x1000000  # fake, aligned "device" addresses: never dereferenced on these paths
INV, UNS = R.ROPE_ERR_INVALID_ARG, R.ROPE_ERR_UNSUPPORTED

APPEND = dict(k=A, v=2 * A, kp=3 * A, vp=4 * A, table=5 * A, cu=6 * A, lens=7 * A, cos=8 * A,
              sin=9 * A, pos=None, off=0, n=2, total=10, ks=128, vs=128, Hk=2, D=64, rd=64, layout=0,
              page=16, n_pages=8, blocks=4, dtype=1, rows=64)


def append_args(**over):
    a = dict(APPEND, **over)
    return [a[x] for x in ("k", "v", "kp", "vp", "table", "cu", "lens", "cos", "sin", "pos", "off",
                           "n", "total", "ks", "vs", "Hk", "D", "rd", "layout", "page", "n_pages",
                           "blocks", "dtype", "rows")] + [None]


@pytest.mark.parametrize("over,status", [
    (dict(dtype=0), UNS), (dict(dtype=3), UNS), (dict(layout=2), UNS), (dict(D=96, ks=192, vs=192), UNS),
    (dict(rd=8), UNS), (dict(rd=40), UNS), (dict(rd=80), UNS), (dict(page=8), UNS),
    (dict(page=48), UNS), (dict(page=256), UNS), (dict(ks=132), UNS), (dict(vs=130), UNS),
    (dict(k=A + 8), UNS), (dict(vp=4 * A + 2), UNS), (dict(cos=8 * A + 4), UNS),
    (dict(n=-1), INV), (dict(total=-1), INV), (dict(total=1 << 31), INV), (dict(Hk=-1), INV),
    (dict(ks=120), INV), (dict(vs=0), INV), (dict(off=-1), INV), (dict(rows=0), INV),
    (dict(n_pages=0), INV), (dict(blocks=0), INV), (dict(k=None), INV), (dict(v=None), INV),
    (dict(kp=None), INV), (dict(table=None), INV), (dict(cu=None), INV), (dict(lens=None), INV),
    (dict(sin=None), INV), (dict(table=5 * A + 2), INV),
    (dict(vp=3 * A + 64), INV),                 # the pools overlap
    (dict(k=3 * A + 128), INV),                 # a pool overlaps its input
    (dict(cu=4 * A + 64), INV),                 # a pool overlaps the offsets
    (dict(n_pages=1 << 31), INV), (dict(n=1 << 30, blocks=1 << 40), INV),
])
def test_append_refuses(lib, over, status):
    assert lib.rope_cache_append(*append_args(**over)) == status


@pytest.mark.parametrize("over", [dict(total=0, k=None, v=None), dict(n=0, table=None, cu=None, lens=None),
                                  dict(Hk=0, kp=None, vp=None)])
def test_append_of_nothing(lib, over):
    assert lib.rope_cache_append(*append_args(**over)) == R.ROPE_OK


def test_status_name(lib):
    assert R.rope_status_string(R.ROPE_ERR_BAD_INDEX) == "ROPE_ERR_BAD_INDEX"


def test_python_refuses_cpu_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pool = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    t = torch.zeros(8, 32)
    with pytest.raises(ValueError, match="CUDA"):
        R.cache_append(x, x, pool, pool, i[:2].view(2, 1), i, i[:2], t, t)


PACKED = dict(q=A, k=2 * A, v=3 * A, o=4 * A, cos=5 * A, sin=6 * A, pq=None, pk=None, cuq=7 * A, cuk=8 * A,
              n=2, tq=10, tk=12, qs=512, ks=256, vs=256, Hq=4, Hk=2, D=128, rd=128, layout=0, causal=1, scale=-1.0,
              dtype=1, rows=64, ws=9 * A, wsb=1 << 20)


def packed_args(**over):
    a = dict(PACKED, **over)
    return [a[x] for x in ("q", "k", "v", "o", "cos", "sin", "pq", "pk", "cuq", "cuk", "n", "tq", "tk", "qs", "ks",
                           "vs", "Hq", "Hk", "D", "rd", "layout", "causal", "scale", "dtype", "rows", "ws",
                           "wsb")] + [None]


@pytest.mark.parametrize("over,status", [
    (dict(dtype=0), UNS), (dict(dtype=3), UNS), (dict(layout=2), UNS), (dict(D=96), UNS), (dict(rd=8), UNS),
    (dict(rd=136), UNS), (dict(qs=516), UNS), (dict(ks=260), UNS), (dict(vs=258), UNS), (dict(q=A + 8), UNS),
    (dict(o=4 * A + 8), UNS), (dict(cos=5 * A + 4), UNS), (dict(ws=9 * A + 64), UNS),
    (dict(causal=2), INV), (dict(scale=float("nan")), INV), (dict(n=-1), INV), (dict(tq=-1), INV),
    (dict(tk=1 << 31), INV), (dict(Hq=3, qs=384), INV), (dict(Hk=0, ks=0, vs=0), INV), (dict(Hk=-1), INV),
    (dict(qs=504), INV), (dict(ks=128), INV), (dict(rows=0), INV), (dict(rows=-1), INV), (dict(q=None), INV),
    (dict(k=None), INV), (dict(v=None), INV), (dict(o=None), INV), (dict(cuq=None), INV), (dict(cuk=None), INV),
    (dict(ws=None), INV), (dict(wsb=100), INV), (dict(wsb=-1), INV), (dict(pq=7 * A + 2), INV),
    (dict(o=A + 1024), INV), (dict(o=2 * A), INV), (dict(ws=A), INV), (dict(ws=4 * A), INV), (dict(o=7 * A), INV),
])
def test_packed_refuses(lib, over, status):
    assert lib.rope_attention_packed_fwd(*packed_args(**over)) == status


@pytest.mark.parametrize("over", [dict(tq=0, q=None, o=None), dict(n=0, cuq=None, cuk=None),
                                  dict(Hq=0, Hk=0, qs=0, ks=0, vs=0, q=None, k=None, v=None, o=None)])
def test_packed_of_nothing(lib, over):
    assert lib.rope_attention_packed_fwd(*packed_args(ws=None, wsb=0, **over)) == R.ROPE_OK


def test_packed_workspace(lib):
    ws = lib.rope_attention_packed_workspace
    need = ws(2, 10, 12, 4, 2, 128)
    assert need >= 2 * 128 + 12 * 2 * 128 * 2 and need % 128 == 0
    assert lib.rope_attention_packed_fwd(*packed_args(wsb=need - 1)) == INV
    assert ws(0, 10, 12, 4, 2, 128) == ws(2, 0, 12, 4, 2, 128) == ws(2, 10, 12, 0, 0, 128) == 0
    assert ws(-1, 10, 12, 4, 2, 128) == ws(2, 10, 12, 4, 3, 128) == ws(2, 10, 12, 4, 2, 96) == -1
    assert ws(2, 10, 1 << 31, 4, 2, 128) == -1


DECODE = dict(q=A, kp=2 * A, vp=3 * A, o=4 * A, table=5 * A, lens=6 * A, pt=7 * A, P=40, cos=8 * A, sin=9 * A, pq=None,
              B=3, qs=512, Hq=4, Hk=2, D=128, rd=128, layout=0, scale=-1.0, page=16, n_pages=20, blocks=4, dtype=1,
              rows=64, ws=10 * A, wsb=1 << 23)


def decode_args(**over):
    a = dict(DECODE, **over)
    return [a[x] for x in ("q", "kp", "vp", "o", "table", "lens", "pt", "P", "cos", "sin", "pq", "B", "qs", "Hq", "Hk",
                           "D", "rd", "layout", "scale", "page", "n_pages", "blocks", "dtype", "rows", "ws",
                           "wsb")] + [None]


@pytest.mark.parametrize("over,status", [
    (dict(dtype=0), UNS), (dict(layout=3), UNS), (dict(D=80), UNS), (dict(rd=24), UNS), (dict(page=24), UNS),
    (dict(page=256), UNS), (dict(B=4097), UNS), (dict(qs=516), UNS), (dict(q=A + 2), UNS), (dict(o=4 * A + 8), UNS),
    (dict(kp=2 * A + 8), UNS), (dict(sin=9 * A + 8), UNS), (dict(ws=10 * A + 16), UNS),
    (dict(B=-1), INV), (dict(Hq=5, qs=640), INV), (dict(Hk=0), INV), (dict(qs=504), INV), (dict(P=-1), INV),
    (dict(P=0x7fffffff), INV), (dict(blocks=-1), INV), (dict(n_pages=0), INV), (dict(n_pages=1 << 30), INV),
    (dict(blocks=1 << 40), INV), (dict(scale=float("nan")), INV), (dict(rows=0), INV), (dict(q=None), INV),
    (dict(kp=None), INV), (dict(vp=None), INV), (dict(o=None), INV), (dict(table=None), INV), (dict(lens=None), INV),
    (dict(pt=None), INV), (dict(cos=None), INV), (dict(ws=None), INV), (dict(wsb=1000), INV), (dict(lens=6 * A + 1), INV),
    (dict(o=A), INV), (dict(o=3 * A + 128), INV), (dict(ws=2 * A), INV), (dict(ws=6 * A - 128), INV), (dict(ws=4 * A), INV),
])
def test_decode_refuses(lib, over, status):
    assert lib.rope_attention_decode_fwd(*decode_args(**over)) == status


@pytest.mark.parametrize("over", [dict(B=0, q=None, o=None, lens=None, table=None),
                                  dict(Hq=0, Hk=0, qs=0, q=None, o=None)])
def test_decode_of_nothing(lib, over):
    assert lib.rope_attention_decode_fwd(*decode_args(ws=None, wsb=0, **over)) == R.ROPE_OK


def test_decode_workspace(lib):
    ws = lib.rope_attention_decode_workspace
    need = ws(3, 4, 2, 128, 16, 4, 40)
    assert need > 3 * 4 * 128 * 4 and need % 128 == 0
    assert lib.rope_attention_decode_fwd(*decode_args(wsb=need - 1)) == INV
    assert ws(0, 4, 2, 128, 16, 4, 40) == ws(3, 0, 0, 128, 16, 4, 40) == 0
    assert ws(3, 4, 3, 128, 16, 4, 40) == ws(3, 4, 2, 96, 16, 4, 40) == ws(3, 4, 2, 128, 48, 4, 40) == -1
    assert ws(4097, 4, 2, 128, 16, 4, 40) == ws(3, 4, 2, 128, 16, 4, -1) == -1
    # nothing but a prefix, nothing but suffixes
    assert 0 < ws(3, 4, 2, 128, 16, 0, 40) < need and 0 < ws(3, 4, 2, 128, 16, 4, 0) < need

"""build_tables_scaled against the rules in 64 bits.

Bound: 5 * 2^-24 of the value (the conversion of the phase, sincospif's one unit, the factor and its product), and
the phase's own: p 2^-64 turns for the fraction, and what the reference's product p w in 64 bits may be off, 2^-52 of
the angle."""
import math

import pytest
import torch

import norm_ref as N
from gpu_util import lib, require_gpu

pytestmark = pytest.mark.gpu


def check(R, kind, rd, rows, factor, original, theta=1e4, offset=0, **more):
    cos, sin = R.build_tables_scaled(kind, rd, rows, factor, original, theta=theta, pos_offset=offset, **more)
    assert cos.shape == sin.shape == (rows, rd // 2) and cos.is_contiguous() and sin.is_contiguous()
    w, scale = N.frequencies(kind, rd, factor, original, theta, more.get("low_turns"), more.get("high_turns"))
    scale = more.get("value_scale") or scale
    p = torch.arange(offset, offset + rows, dtype=torch.float64)[:, None]
    angle = p * torch.tensor(w, dtype=torch.float64)
    off = scale * (p * 2.0 ** -64 * 2 * math.pi + angle * 2.0 ** -51 + 2.0 ** -52)
    for got, want in ((cos, scale * angle.cos()), (sin, scale * angle.sin())):
        d = (got.cpu().double() - want).abs()
        bound = 5 * N.U * want.abs() + off
        assert (d <= bound).all(), "%s: %.3f of the bound" % (kind, (d / bound).max())


@pytest.mark.parametrize("kind", ["linear", "ntk", "smooth", "yarn"])
@pytest.mark.parametrize("rd,rows,factor,original,offset", [
    (128, 1, 8.0, 8192, 0), (64, 513, 4.0, 4096, 20011), (16, 3001, 1.0, 2048, 0), (34, 77, 2.5, 512, 1), (6, 9, 32.0, 64, 5),
    (512, 700, 20.0, 32768, 1 << 20), (2, 5, 2.0, 100, 3), (128, 40, 32.0, 32768, (1 << 31) - 100)])
def test_rules(kind, rd, rows, factor, original, offset):
    require_gpu()
    R = lib()
    if kind == "ntk" and rd == 2:
        with pytest.raises(R.RopeError):
            R.build_tables_scaled(kind, rd, rows, factor, original)
        return
    check(R, kind, rd, rows, factor, original, theta=5e5 if rd == 128 else 1e4, offset=offset)


def test_own_turns_and_scale():
    require_gpu()
    R = lib()
    check(R, "smooth", 128, 300, 8.0, 8192, low_turns=0.5, high_turns=7.0, value_scale=1.5)
    check(R, "yarn", 96, 300, 8.0, 4096, low_turns=2.0, high_turns=20.0, value_scale=0.75)
    check(R, "smooth", 128, 70000, 8.0, 8192, theta=5e5)


def test_linear_is_the_interpolated_table():
    """Within one unit of fp32 besides the bound, build_tables with the same factor."""
    require_gpu()
    R = lib()
    a = R.build_tables(1e4, 64, 500, 4.0)
    b = R.build_tables_scaled("linear", 64, 500, 4.0)
    for x, y in zip(a, b):
        assert ((x.double() - y.double()).abs() <= 6 * N.U * x.abs().double() + 2.0 ** -40).all()


def test_the_tables_rotate():
    """A run as a program makes it: tables, rotation, and what is left of a score depends on the distance alone."""
    require_gpu()
    R = lib()
    cos, sin = R.build_tables_scaled("smooth", 64, 300, 8.0, 128)
    g = torch.Generator().manual_seed(4)
    q, k = (torch.randn(1, 1, 1, 64, generator=g).cuda().expand(1, 1, 300, 64).contiguous() for _ in range(2))
    R.apply_qk(q, k, cos, sin)
    s = (q[0, 0].double() @ k[0, 0].double().T).cpu()
    size = (q[0, 0, 0].norm() * k[0, 0, 0].norm()).item()
    for d in (0, 1, 17, 200):
        line = torch.diagonal(s, -d)
        # two tables' values and two rotations of 64 elements: 2^-20 of the vectors' sizes
        assert (line - line[0]).abs().max() <= size * 2.0 ** -20


def test_streams_and_refusals():
    require_gpu()
    R = lib()
    s = torch.cuda.Stream()
    a = R.build_tables_scaled("yarn", 128, 4096, 8.0, 8192, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, R.build_tables_scaled("yarn", 128, 4096, 8.0, 8192)))
    graph = torch.cuda.CUDAGraph()
    cos, sin = (torch.zeros(50, 64, device="cuda") for _ in range(2))
    with torch.cuda.graph(graph):
        R.rope_tables_build_scaled(R.ROPE_SCALE_NTK, 1e4, 128, 50, 0, 2.0, 0, 1, 4, 0, cos, sin)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cos, R.build_tables_scaled("ntk", 128, 50, 2.0)[0])
    # an output whose rows are no whole 16-byte vectors' start
    flat = torch.zeros(2, 50 * 64 + 1, device="cuda")
    R.rope_tables_build_scaled(R.ROPE_SCALE_NTK, 1e4, 128, 50, 0, 2.0, 0, 1, 4, 0, flat[0, 1:], flat[1, 1:])
    assert torch.equal(flat[1, 1:].view(50, 64), sin)
    with pytest.raises(KeyError):
        R.build_tables_scaled("other", 64, 10, 2.0)
    with pytest.raises(ValueError):
        R.rope_tables_build_scaled(0, 1e4, 128, 60, 0, 2.0, 0, 1, 4, 0, cos, sin)
    assert R.build_tables_scaled("linear", 64, 0, 2.0)[0].shape == (0, 32)
    assert R.rope_check_errors() == R.ROPE_OK

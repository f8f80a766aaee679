"""Weight gradients of the norm: of tensors without heads, at the lengths of a training step, and of weights that lie
anywhere in a buffer of parameters."""
import pytest
import torch

import norm_ref as N
import serving_ref as S
from gpu_util import lib, require_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.mark.parametrize("wtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,S_,Hq,Hk", [(2, 5, 0, 3), (2, 5, 3, 0), (2, 5, 0, 0), (2, 0, 0, 3), (0, 5, 0, 0)])
def test_a_tensor_without_heads_has_zero_weight_gradients(B, S_, Hq, Hk, wtype):
    require_gpu()
    R = lib()
    from rotary_position_embedding_rope_gb300 import autograd

    D = 64
    cos, sin = (x.cuda() for x in S.tables(1e4, D, 8))
    x = lambda H: torch.randn(B, S_, H, D, device="cuda", dtype=torch.bfloat16)
    q, k, gq, gk = x(Hq), x(Hk), x(Hq), x(Hk)
    w = torch.ones(D, device="cuda", dtype=wtype)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dw = [torch.full((D,), float("nan"), device="cuda", dtype=wtype) for _ in range(2)]
    need = R.rope_norm_qk_workspace(D)
    R.rope_norm_qk_bwd(q, k, gq, gk, dq, dk, w, w, dw[0], dw[1], cos, sin, None, 0, B, Hq, Hk, S_, D, None, None, D,
                       R.ROPE_SPLIT_HALF, 1, EPS, R.ROPE_BF16, R.ROPE_F32 if wtype == torch.float32 else R.ROPE_BF16, 8,
                       torch.empty(need, device="cuda", dtype=torch.uint8), need)
    rows = B * S_
    for d, H in zip(dw, (Hq, Hk)):
        assert d.isfinite().all() and (rows * H > 0 or not d.any())
    # one gradient alone is wanted
    one = torch.full((D,), float("nan"), device="cuda", dtype=wtype)
    R.rope_norm_qk_bwd(q, k, gq, gk, dq, dk, w, w, one if Hq == 0 else None, None if Hq == 0 else one, cos, sin, None, 0, B,
                       Hq, Hk, S_, D, None, None, D, R.ROPE_SPLIT_HALF, 1, EPS, R.ROPE_BF16,
                       R.ROPE_F32 if wtype == torch.float32 else R.ROPE_BF16, 8,
                       torch.empty(need, device="cuda", dtype=torch.uint8), need)
    assert torch.equal(one, dw[0 if Hq == 0 else 1])
    got = R.norm_rotate_qk_backward(gq, gk, q, k, w, w, cos, sin, EPS, seq_before_head=True)
    assert torch.equal(got[2], dw[0]) and torch.equal(got[3], dw[1])
    leaves = [t.requires_grad_() for t in (q, k, w.clone(), w.clone())]
    out = autograd.norm_rotary_qk(*leaves, cos, sin, EPS, seq_before_head=True)
    grads = torch.autograd.grad(out, leaves, (gq, gk))
    assert torch.equal(grads[2], dw[0]) and torch.equal(grads[3], dw[1])
    assert R.rope_check_errors() == R.ROPE_OK


def weight_gradient(x, g, cos, sin, chain):
    """(dw, bound) of rows x [1, S, H, D] and their outputs' gradients g, split halves, in 64 bits, some tokens at a time.

    An element's terms: its root 11 u, the rotation back 2 u of its size, two products 2 u; then `chain` additions in
    its thread, 5 of its warp's groups, 4 of the CTA's warps, 6 of a warp's rows of partial sums, 5 of those warps and 8
    of the cluster: 15 + 28 + chain roundings of at most u of the sum of the sizes."""
    D = x.shape[-1]
    dw = torch.zeros(D, dtype=torch.float64, device=x.device)
    size = torch.zeros_like(dw)
    step = max(1, (1 << 24) // (x.shape[2] * D))
    for s in range(0, x.shape[1], step):
        rows = x[:, s:s + step].double()
        c, sn = N.angles(torch.arange(s, s + rows.shape[1], device=x.device), cos, sin)
        c, sn = c[None, :, None], sn[None, :, None]
        n = rows / torch.sqrt(rows.square().mean(-1, keepdim=True) + EPS)
        up = g[:, s:s + step].double()
        wide = lambda t: t.expand(*rows.shape[:-1], -1)
        dw += (N.turn(up, wide(c), wide(-sn), "split_half") * n).sum((0, 1, 2))
        size += (N.turn_size(up, wide(c), wide(sn), "split_half") * n.abs()).sum((0, 1, 2))
    return dw, (43 + chain) * N.U * size


def longest_chain(tokens, heads, D, U):
    """Additions of a thread at most: its CTA's tiles, of at least three CTAs an SM, U rows of each."""
    groups = 128 // (2 if D <= 32 else 4 if D <= 64 else 8 if D <= 128 else 16)
    tiles = -(-tokens // groups) * -(-heads // U)
    ctas = 3 * torch.cuda.get_device_properties(0).multi_processor_count
    return (-(-tiles // ctas) + 1) * U, tiles, ctas


@pytest.mark.parametrize("dtype,U", [(torch.bfloat16, 2), (torch.float32, 1)])
def test_at_training_length(dtype, U):
    """Several waves of CTAs, and as many as there are rows of partial sums; q's tiles and k's."""
    require_gpu()
    R = lib()
    S_, Hq, Hk, D = 8201, 64, 65, 64
    chain, tiles, ctas = longest_chain(S_, Hq + Hk, D, U)
    assert tiles >= 36 * ctas
    g = torch.Generator("cuda").manual_seed(8)
    cos, sin = (x.cuda() for x in S.tables(1e4, D, S_))
    w = torch.rand(D, device="cuda", generator=g) + 0.5
    q, k = (torch.randn(1, S_, H, D, device="cuda", generator=g).to(dtype) for H in (Hq, Hk))
    # gradients along the outputs, so that every row's share counts
    gq, gk = R.norm_rotate_qk(q, k, w, w, cos, sin, EPS, seq_before_head=True)
    gq, gk = gq + 0.25 * torch.randn_like(gq), gk + 0.25 * torch.randn_like(gk)
    _, _, dwq, dwk = R.norm_rotate_qk_backward(gq, gk, q, k, w, w, cos, sin, EPS, seq_before_head=True)
    for got, x, up in ((dwq, q, gq), (dwk, k, gk)):
        want, bound = weight_gradient(x, up, cos, sin, chain)
        assert ((got.double() - want).abs() <= bound).all()
    assert R.rope_check_errors() == R.ROPE_OK


def test_past_32_bit_offsets():
    require_gpu()
    R = lib()
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    S_, H, D = 8300, 2048, 128
    assert S_ * H * D > 1 << 31
    chain, tiles, ctas = longest_chain(S_, H, D, 2)
    cos, sin = (x.cuda() for x in S.tables(1e4, D, S_))
    w = torch.rand(D, device="cuda") + 0.5
    q = torch.randn(1, S_, H, D, device="cuda", dtype=torch.bfloat16)
    up, _ = R.norm_rotate_qk(q, None, w, None, cos, sin, EPS, seq_before_head=True)
    dw = R.norm_rotate_qk_backward(up, None, q, None, w, None, cos, sin, EPS, seq_before_head=True)[2]
    want, bound = weight_gradient(q, up, cos, sin, chain)
    assert ((dw.double() - want).abs() <= bound).all()
    assert R.rope_check_errors() == R.ROPE_OK


@pytest.mark.parametrize("wtype", [torch.float32, torch.bfloat16])
def test_weights_anywhere_in_a_buffer(wtype):
    """Views of a flat buffer that start at any element, as dense copies of them."""
    require_gpu()
    R = lib()
    from rotary_position_embedding_rope_gb300 import autograd

    D = 64
    cos, sin = (x.cuda() for x in S.tables(1e4, D, 16))
    flat = (torch.rand(2 * D + 3, device="cuda") + 0.5).to(wtype).requires_grad_()
    wq, wk = flat[1:1 + D], flat[D + 2:2 * D + 2]
    q, k = (torch.randn(2, 9, H, D, device="cuda", dtype=torch.bfloat16, requires_grad=True) for H in (4, 2))
    out = autograd.norm_rotary_qk(q, k, wq, wk, cos, sin, EPS, seq_before_head=True)
    up = [torch.randn_like(o) for o in out]
    dense = [w.detach().clone().requires_grad_() for w in (wq, wk)]
    same = autograd.norm_rotary_qk(q, k, *dense, cos, sin, EPS, seq_before_head=True)
    assert all(torch.equal(a, b) for a, b in zip(out, same))
    got = torch.autograd.grad(out, (q, k, flat), up)
    want = torch.autograd.grad(same, (q, k, *dense), up)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(got[2][1:1 + D], want[2]) and torch.equal(got[2][D + 2:2 * D + 2], want[3])
    assert not got[2][[0, D + 1, -1]].any()
    with pytest.raises(R.RopeError):
        R.norm_rotate_qk(q.detach(), None, wq.detach(), None, cos, sin, EPS, seq_before_head=True)
    assert R.rope_check_errors() == R.ROPE_OK

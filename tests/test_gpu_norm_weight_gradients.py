"""Weight gradients of the norm: of tensors without heads."""
import pytest
import torch

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

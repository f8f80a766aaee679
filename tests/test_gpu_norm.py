"""norm_rotate_qk, its gradients and norm_cache_append against the plain forms in 64 bits, within bounds that
norm_ref derives, at the sizes, strides and positions where they can go wrong."""
import pytest
import torch

import norm_ref as N
import serving_ref as S
from gpu_util import lib, require_gpu
from test_gpu_cache_append import same_bits, scattered_tables, starts

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def near(got, want, bound, what):
    got = got.detach().cpu()
    d = (got.double() - want).abs()
    worst = (d / (bound + N.half_step(want, got.dtype))).max().item() if d.numel() else 0.0
    assert got.isfinite().all() and worst <= 1, "%s: %.3f of the bound" % (what, worst)


def make(B, S_, Hq, Hk, D, dtype, wtype, seq_first, seed=5):
    g = torch.Generator().manual_seed(seed)
    dt, wt = TYPES[dtype], TYPES[wtype]
    x = lambda H: (2 * torch.randn(*((B, S_, H, D) if seq_first else (B, H, S_, D)), generator=g)).to(dt)
    w = lambda: (1 + 0.3 * torch.randn(D, generator=g)).to(wt)
    return dict(q=x(Hq), k=x(Hk), wq=w(), wk=w(), gq=x(Hq), gk=x(Hk))


def rows_of(pos, B, S_):
    r = torch.arange(S_).expand(B, S_) if pos is None else pos.expand(B, -1)[:, :S_] if pos.dim() == 1 else pos[:, :S_]
    return r


def reference(t, pos, cos, sin, layout, seq_first, grads=True):
    B, S_ = t["q"].shape[0], t["q"].shape[1 if seq_first else 2]
    c, s = N.angles(rows_of(pos, B, S_), cos, sin)
    head = 2 if seq_first else 1
    c, s = c.unsqueeze(head), s.unsqueeze(head)
    out = {}
    for n in "qk":
        out[n] = N.forward(t[n], t["w" + n], c, s, layout, EPS)
        if grads:
            dx, bx, dw, bw = N.backward(t[n], t["w" + n], t["g" + n], c, s, layout, EPS)
            out["d" + n], out["dw" + n] = (dx, bx), (dw, bw)
    return out


CASES = [
    # B, S, Hq, Hk, D, rd, type, weights, layout, sequence first
    (1, 1, 1, 1, 128, 128, "bf16", "bf16", "split_half", False),
    (2, 37, 32, 8, 128, 128, "bf16", "f32", "split_half", True),
    (3, 129, 5, 1, 64, 32, "f16", "f16", "interleaved", False),
    (1, 200, 6, 3, 96, 48, "bf16", "bf16", "split_half", True),
    (2, 33, 3, 2, 80, 80, "f32", "f32", "interleaved", True),
    (2, 65, 4, 4, 256, 64, "f32", "f32", "split_half", False),
    (1, 19, 2, 7, 16, 16, "f16", "f32", "interleaved", True),
    (4, 50, 9, 2, 32, 16, "bf16", "bf16", "split_half", False),
    (1, 1500, 16, 4, 240, 16, "f16", "f16", "split_half", True),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "_".join(map(str, c)))
@pytest.mark.parametrize("positions", ["none", "shared", "own"])
def test_norm_and_gradients(c, positions):
    require_gpu()
    R = lib()
    from rotary_position_embedding_rope_gb300 import autograd

    B, S_, Hq, Hk, D, rd, dtype, wtype, layout, seq_first = c
    t = make(*c[:5], dtype, wtype, seq_first)
    cos, sin = S.tables(1e4, rd, 1600)
    g = torch.Generator().manual_seed(2)
    pos = None
    if positions != "none":
        pos = torch.randint(-1, 1600, (S_,) if positions == "shared" else (B, S_ + 3), generator=g, dtype=torch.int32)
    want = reference(t, pos, cos, sin, layout, seq_first)
    d = {n: x.cuda() for n, x in t.items()}
    args = dict(cos=cos.cuda(), sin=sin.cuda(), eps=EPS, pos_idx=None if pos is None else pos.cuda(), layout=layout,
                seq_before_head=seq_first)
    q, k = R.norm_rotate_qk(d["q"], d["k"], d["wq"], d["wk"], **args)
    near(q, *want["q"], "q")
    near(k, *want["k"], "k")
    for n in ("q", "k", "wq", "wk"):
        d[n].requires_grad_()
    out = autograd.norm_rotary_qk(d["q"], d["k"], d["wq"], d["wk"], **args)
    assert same(out[0], q) and same(out[1], k)
    got = torch.autograd.grad(out, (d["q"], d["k"], d["wq"], d["wk"]), (d["gq"], d["gk"]))
    for x, n in zip(got, ("dq", "dk", "dwq", "dwk")):
        near(x, *want[n], n)
    again = R.norm_rotate_qk_backward(d["gq"], d["gk"], *(d[n].detach() for n in ("q", "k", "wq", "wk")), **args)
    assert all(same(a, b) for a, b in zip(again, got))
    assert R.rope_check_errors() == R.ROPE_OK


def same(a, b):
    return a.dtype == b.dtype and torch.equal(a, b)


def test_gradients_against_differences():
    """The directional derivative of a weighted sum of the outputs, by central differences of the 64-bit form."""
    require_gpu()
    lib()
    from rotary_position_embedding_rope_gb300 import autograd

    B, S_, Hq, Hk, D, rd = 1, 9, 2, 1, 64, 32
    t = make(B, S_, Hq, Hk, D, "f32", "f32", True)
    cos, sin = S.tables(1e4, rd, 16)
    c, s = (x[:, :S_, None] for x in N.angles(rows_of(None, B, S_), cos, sin))
    leaves = [t[n].cuda().requires_grad_() for n in ("q", "k", "wq", "wk")]
    out = autograd.norm_rotary_qk(*leaves, cos.cuda(), sin.cuda(), EPS, seq_before_head=True)
    grads = [x.cpu().double() for x in torch.autograd.grad(out, leaves, (t["gq"].cuda(), t["gk"].cuda()))]
    g = torch.Generator().manual_seed(8)
    for i, n in enumerate(("q", "k", "wq", "wk")):
        v = torch.randn(t[n].shape, generator=g).double()

        def total(h):
            m = {a: t[a].double() + (h * v if a == n else 0) for a in ("q", "k", "wq", "wk")}
            return sum((N.forward(m[a], m["w" + a], c, s, "split_half", EPS)[0] * t["g" + a].double()).sum() for a in "qk")

        h = 1e-5
        want = (total(h) - total(-h)) / (2 * h)
        # differences: h^2 of a third derivative of order one per element and 1e-16 / h of the sum's sizes; the kernel's
        # gradient is within 1e-5 of each element
        size = (grads[i].abs() * v.abs()).sum()
        assert abs((grads[i] * v).sum() - want) <= 1e-4 * size, n


def test_strided_views_and_one_tensor():
    """Parts of a fused projection, a transposed view and an expanded one give what dense copies do."""
    require_gpu()
    R = lib()
    from rotary_position_embedding_rope_gb300 import autograd

    B, S_, Hq, Hk, D = 3, 41, 6, 2, 128
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(B, S_, Hq + 2 * Hk, D, generator=g).bfloat16().cuda()
    wq, wk = (torch.randn(D, generator=g).cuda() for _ in range(2))
    cos, sin = (x.cuda() for x in S.tables(1e4, D, 64))
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    a = R.norm_rotate_qk(q, k, wq, wk, cos, sin, seq_before_head=True)
    b = R.norm_rotate_qk(q.contiguous(), k.contiguous(), wq, wk, cos, sin, seq_before_head=True)
    assert same(a[0], b[0]) and same(a[1], b[1]) and a[0].is_contiguous()
    # the same memory with the heads first
    t = R.norm_rotate_qk(q.transpose(1, 2), k.transpose(1, 2), wq, wk, cos, sin)
    assert same(t[0].transpose(1, 2).contiguous(), b[0])
    # one tensor alone, without a weight
    only, none = R.norm_rotate_qk(None, k, None, wk, cos, sin, seq_before_head=True)[::-1]
    assert none is None and same(only, b[1])
    bare, _ = R.norm_rotate_qk(q, None, None, None, cos, sin, seq_before_head=True)
    ones, _ = R.norm_rotate_qk(q, None, torch.ones_like(wq), None, cos, sin, seq_before_head=True)
    assert same(bare, ones)
    # in place
    x, y = q.contiguous(), k.contiguous()
    R.norm_rotate_qk(x, y, wq, wk, cos, sin, seq_before_head=True, q_out=x, k_out=y)
    assert same(x, b[0]) and same(y, b[1])
    # gradients of an expanded input and of an odd offset, which is copied
    base = torch.randn(1, S_, 1, D, generator=g).cuda().requires_grad_()
    odd = torch.randn(B * S_ * D + 1, generator=g).cuda()[1:].view(B, S_, 1, D)
    out = autograd.norm_rotary_qk(base.expand(B, S_, Hq, D), odd, wq, None, cos, sin, seq_before_head=True)
    up = torch.randn(B, S_, Hq, D, generator=g).cuda()
    got, = torch.autograd.grad(out[0], base, up)
    dense = base.detach().expand(B, S_, Hq, D).contiguous()
    dq = R.norm_rotate_qk_backward(up, None, dense, None, wq, None, cos, sin, seq_before_head=True)[0]
    assert torch.equal(got, dq.sum((0, 2), keepdim=True))
    assert R.rope_check_errors() == R.ROPE_OK


def test_graphs_of_parts():
    """Outputs without a part in the loss, inputs and weights that need no gradient."""
    require_gpu()
    R = lib()
    from rotary_position_embedding_rope_gb300 import autograd

    host = make(2, 20, 4, 2, 64, "f32", "f32", True)
    t = {n: x.cuda() for n, x in host.items()}
    cos, sin = (x.cuda() for x in S.tables(1e4, 64, 32))
    exact = reference(host, None, cos.cpu(), sin.cpu(), "split_half", True)
    full = R.norm_rotate_qk_backward(t["gq"], t["gk"], t["q"], t["k"], t["wq"], t["wk"], cos, sin, seq_before_head=True)
    want = dict(zip(("q", "k", "wq", "wk"), full))
    for used in ("q", "k", "qk"):
        for need in (("q",), ("wk",), ("k", "wq"), ("q", "k", "wq", "wk")):
            leaves = {n: t[n].detach().clone().requires_grad_(n in need) for n in ("q", "k", "wq", "wk")}
            out = autograd.norm_rotary_qk(*leaves.values(), cos, sin, seq_before_head=True)
            loss = sum((o * t["g" + n]).sum() for o, n in zip(out, "qk") if n in used and o.requires_grad)
            if not torch.is_tensor(loss):
                continue
            loss.backward()
            for n in leaves:
                g = leaves[n].grad
                if n in need and n[-1] in used:
                    # (a weight's gradient is summed in an order that the sizes of the call give: queries alone, keys
                    # alone and both are three orders, each within the bound)
                    if n[0] == "w":
                        near(g, *exact["d" + n], n)
                    else:
                        assert same(g, want[n])
                else:
                    assert g is None or not g.any()
    assert R.rope_check_errors() == R.ROPE_OK


def test_graph_rules():
    """What autograd promises of any node: saved tensors that changed are an error, so is a second backward pass or a second
    derivative; without a graph there is no node; leaves on several calls add up."""
    require_gpu()
    lib()
    from rotary_position_embedding_rope_gb300 import autograd

    t = {n: x.cuda() for n, x in make(1, 12, 2, 1, 64, "f32", "f32", True).items()}
    cos, sin = (x.cuda() for x in S.tables(1e4, 64, 16))
    leaves = [t[n].clone().requires_grad_() for n in ("q", "k", "wq", "wk")]
    call = lambda: autograd.norm_rotary_qk(*leaves, cos, sin, seq_before_head=True)
    with torch.no_grad():
        assert not any(o.requires_grad for o in call())
    assert not any(o.requires_grad for o in autograd.norm_rotary_qk(*(x.detach() for x in leaves), cos, sin, seq_before_head=True))
    out = call()
    assert all(o.requires_grad and not o.is_leaf for o in out)
    out[0].sum().backward()
    once = leaves[0].grad.clone()
    with pytest.raises(RuntimeError, match="second time"):
        out[0].sum().backward()
    call()[0].sum().backward()
    assert torch.equal(leaves[0].grad, 2 * once)
    out = call()
    with torch.no_grad():
        leaves[2].add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        out[0].sum().backward()
    g, = torch.autograd.grad(call()[0].square().sum(), leaves[0], create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated"):
        g.sum().backward()
    # a graph behind the inputs, and hooks on the way
    seen = []
    x = leaves[0] * 3
    x.register_hook(lambda d: seen.append(d.shape))
    o, _ = autograd.norm_rotary_qk(x, None, leaves[2], None, cos, sin, seq_before_head=True)
    d, = torch.autograd.grad(o.sum(), leaves[0])
    assert seen == [x.shape] and d.isfinite().all()
    # saved tensors may be packed elsewhere
    with torch.autograd.graph.save_on_cpu():
        o, _ = autograd.norm_rotary_qk(x.detach().requires_grad_(), None, leaves[2], None, cos, sin, seq_before_head=True)
    o.sum().backward()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** 50, 2.0 ** -46])
def test_rows_of_extreme_size(dtype, size):
    """Rows whose squares still fit fp32 while the third power of 1 / |x| does not; eps 0, as the formula allows."""
    require_gpu()
    R = lib()
    B, S_, Hq, Hk, D = 1, 40, 3, 2, 64
    t = make(B, S_, Hq, Hk, D, dtype, "f32", True)
    t["q"], t["k"] = t["q"] * size, t["k"] * size
    assert t["q"].isfinite().all() and t["q"].dtype == TYPES[dtype]
    cos, sin = S.tables(1e4, D, S_)
    d = {n: x.cuda() for n, x in t.items()}
    out = R.norm_rotate_qk(d["q"], d["k"], d["wq"], d["wk"], cos.cuda(), sin.cuda(), 0.0, seq_before_head=True)
    grads = R.norm_rotate_qk_backward(d["gq"], d["gk"], d["q"], d["k"], d["wq"], d["wk"], cos.cuda(), sin.cuda(), 0.0,
                                      seq_before_head=True)
    c, s = (x[:, :, None] for x in N.angles(rows_of(None, B, S_), cos, sin))
    for i, n in enumerate("qk"):
        near(out[i], *N.forward(t[n], t["w" + n], c, s, "split_half", 0.0), n)
        dx, bx, dw, bw = N.backward(t[n], t["w" + n], t["g" + n], c, s, "split_half", 0.0)
        near(grads[i], dx, bx, "d" + n)
        near(grads[2 + i], dw, bw, "dw" + n)


def test_forward_mode_is_refused():
    """A tangent would be dropped without a word."""
    require_gpu()
    lib()
    from rotary_position_embedding_rope_gb300 import autograd

    t = {n: x.cuda() for n, x in make(1, 12, 2, 1, 64, "f32", "f32", True).items()}
    cos, sin = (x.cuda() for x in S.tables(1e4, 64, 16))
    with torch.autograd.forward_ad.dual_level():
        w = torch.autograd.forward_ad.make_dual(t["wq"], torch.ones_like(t["wq"]))
        with pytest.raises(RuntimeError, match="forward-mode"):
            autograd.norm_rotary_qk(t["q"], t["k"], w, t["wk"], cos, sin, seq_before_head=True)


def test_empty_and_zero_rows():
    require_gpu()
    R = lib()
    cos, sin = (x.cuda() for x in S.tables(1e4, 64, 8))
    w = torch.ones(64, device="cuda")
    z = torch.zeros(2, 0, 3, 64, device="cuda", dtype=torch.bfloat16)
    q, k = R.norm_rotate_qk(z, z, w, w, cos, sin, seq_before_head=True)
    assert q.shape == z.shape and k.shape == z.shape
    _, _, dw, dwk = R.norm_rotate_qk_backward(z, z, z, z, w, w, cos, sin, seq_before_head=True)
    assert not dw.any() and not dwk.any()
    # rows of zeros stay zeros
    x = torch.zeros(1, 5, 2, 64, device="cuda")
    q, _ = R.norm_rotate_qk(x, None, w, None, cos, sin, seq_before_head=True)
    assert not q.any()
    # a NaN or infinity stays in its row
    x = torch.randn(1, 5, 2, 64, device="cuda")
    clean, _ = R.norm_rotate_qk(x, None, w, None, cos, sin, seq_before_head=True)
    x[0, 2, 1, 7] = float("nan")
    q, _ = R.norm_rotate_qk(x, None, w, None, cos, sin, seq_before_head=True)
    clean[0, 2, 1], q[0, 2, 1] = 0, 0
    assert torch.equal(q, clean)
    assert R.rope_check_errors() == R.ROPE_OK


def test_positions_outside_the_table():
    require_gpu()
    R = lib()
    t = make(1, 12, 2, 1, 64, "f32", "f32", True)
    cos, sin = S.tables(1e4, 64, 10)
    pos = torch.tensor([0, 3, -1, 9, 10, -2, 2 ** 31 - 1, 1, 2, 4, 5, 6], dtype=torch.int32)
    want = reference(t, pos, cos, sin, "split_half", True, grads=False)
    q, k = R.norm_rotate_qk(t["q"].cuda(), t["k"].cuda(), t["wq"].cuda(), t["wk"].cuda(), cos.cuda(), sin.cuda(), EPS,
                            pos.cuda(), seq_before_head=True)
    assert R.rope_check_errors() == R.ROPE_ERR_POS_OUT_OF_RANGE
    near(q, *want["q"], "q")
    near(k, *want["k"], "k")


def test_captured_forward_and_backward():
    require_gpu()
    R = lib()
    from rotary_position_embedding_rope_gb300 import autograd

    t = {n: x.cuda() for n, x in make(2, 33, 4, 2, 128, "bf16", "bf16", False).items()}
    cos, sin = (x.cuda() for x in S.tables(1e4, 128, 64))
    leaves = [t[n].requires_grad_() for n in ("q", "k", "wq", "wk")]
    eager = autograd.norm_rotary_qk(*leaves, cos, sin)     # an eager graph of the same leaves that lives on

    def step():
        out = autograd.norm_rotary_qk(*leaves, cos, sin)
        return tuple(x.detach() for x in out) + torch.autograd.grad(out, leaves, (t["gq"], t["gk"]))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    # it would make the captured backward pass wait for another stream
    with pytest.raises(RuntimeError, match="alive"), torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
        step()
    del eager
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for n, x in make(2, 33, 4, 2, 128, "bf16", "bf16", False, seed=77).items():
        t[n].data.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got, step()))
    assert R.rope_check_errors() == R.ROPE_OK


def test_another_stream():
    require_gpu()
    R = lib()
    t = {n: x.cuda() for n, x in make(2, 700, 8, 2, 128, "bf16", "bf16", False).items()}
    cos, sin = (x.cuda() for x in S.tables(1e4, 128, 700))
    x = (t["q"], t["k"], t["wq"], t["wk"], cos, sin)
    want = R.norm_rotate_qk(*x), R.norm_rotate_qk_backward(t["gq"], t["gk"], *x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = R.norm_rotate_qk(*x, stream=s), R.norm_rotate_qk_backward(t["gq"], t["gk"], *x, stream=s)
    s.synchronize()
    assert all(same(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_rows_past_32_bit_offsets():
    require_gpu()
    R = lib()
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    S_, H, D = 8300, 2048, 128
    assert S_ * H * D > 1 << 31
    cos, sin = (x.cuda() for x in S.tables(1e4, D, S_))
    w = torch.rand(D, device="cuda") + 0.5
    q = torch.randn(1, S_, H, D, device="cuda", dtype=torch.bfloat16)
    out, _ = R.norm_rotate_qk(q, None, w, None, cos, sin, seq_before_head=True)
    tail = q[:, -3:].contiguous()
    pos = torch.arange(S_ - 3, S_, device="cuda", dtype=torch.int32)
    small, _ = R.norm_rotate_qk(tail, None, w, None, cos, sin, pos_idx=pos, seq_before_head=True)
    assert same(out[:, -3:].contiguous(), small)
    dq = R.norm_rotate_qk_backward(out, None, q, None, w, None, cos, sin, seq_before_head=True)[0]
    ds = R.norm_rotate_qk_backward(out[:, -3:].contiguous(), None, tail, None, w, None, cos, sin, pos_idx=pos,
                                   seq_before_head=True)[0]
    assert same(dq[:, -3:].contiguous(), ds)
    assert R.rope_check_errors() == R.ROPE_OK


def test_norm_refusals():
    require_gpu()
    R = lib()
    t = {n: x.cuda() for n, x in make(2, 8, 4, 2, 64, "bf16", "bf16", True).items()}
    cos, sin = (x.cuda() for x in S.tables(1e4, 64, 8))
    ok = dict(q=t["q"], k=t["k"], wq=t["wq"], wk=t["wk"], cos=cos, sin=sin, seq_before_head=True)
    for bad, err, says in [
            (dict(q=None, k=None), TypeError, "expected a tensor"), (dict(k=t["k"].float()), ValueError, "k must be"),
            (dict(k=t["k"][:, :7]), ValueError, "agree"), (dict(q=t["q"][0]), ValueError, "4-dimensional"),
            (dict(q=t["q"].double()), TypeError, "bf16 or fp16"), (dict(q=t["q"].cpu()), ValueError, "CUDA"),
            (dict(wq=t["wq"][:32]), ValueError, "wq must be"), (dict(wk=t["wk"].half()), ValueError, "fp32 or of the rows"),
            (dict(wk=t["wk"].float()), ValueError, "one type"), (dict(cos=cos.double(), sin=sin.double()), ValueError, "cos"),
            (dict(rotary_dim=32), ValueError, "rotary_dim"), (dict(pos_idx=torch.zeros(7, dtype=torch.int32, device="cuda")), ValueError, "pos_idx"),
            (dict(pos_idx=torch.zeros(8, device="cuda")), ValueError, "pos_idx"),
            (dict(q=t["q"].transpose(2, 3)), ValueError, "dense"), (dict(q_out=t["q"][:1]), ValueError, "q_out"),
            (dict(q_out=t["q"].reshape(-1)[:t["k"].numel()].view_as(t["k"]), q=t["k"].clone(), k=t["k"].clone(),
                  k_out=t["q"].reshape(-1)[64:t["k"].numel() + 64].view_as(t["k"])), R.RopeError, None),
            (dict(eps=-1.0), R.RopeError, None), (dict(eps=float("nan")), R.RopeError, None),
            (dict(q=torch.zeros(2, 8, 4, 72, device="cuda", dtype=torch.bfloat16), k=None, wq=None, wk=None), R.RopeError, None),
            (dict(q=t["q"][:1].expand(2, -1, -1, -1)), R.RopeError, None)]:
        with pytest.raises(err, match=says):
            R.norm_rotate_qk(**dict(ok, **bad))
    with pytest.raises(ValueError, match="gq must be"):
        R.norm_rotate_qk_backward(t["gq"][:, :4].contiguous(), t["gk"], **ok)
    with pytest.raises(ValueError, match="contiguous"):
        R.norm_rotate_qk_backward(t["gq"].transpose(0, 1).contiguous().transpose(0, 1), t["gk"], **ok)
    assert R.rope_check_errors() == R.ROPE_OK


# ---------------------------------------------------------------------------------------------------------------------
# into the cache

APPEND = [
    dict(new=[1, 1, 1], old=[0, 15, 16], Hq=32, Hk=8, D=128, rd=128, page=16, dtype="bf16", wtype="bf16", layout="split_half"),
    dict(new=[5, 0, 33, 1], old=[3, 9, 0, 63], Hq=6, Hk=2, D=64, rd=64, page=32, dtype="f16", wtype="f32", layout="interleaved"),
    dict(new=[70, 129], old=[0, 100], Hq=5, Hk=5, D=128, rd=96, page=64, dtype="f16", wtype="f16", layout="split_half"),
    dict(new=[17], old=[120], Hq=7, Hk=1, D=64, rd=16, page=128, dtype="bf16", wtype="f32", layout="interleaved"),
    dict(new=[1 + i % 3 for i in range(1100)], old=[i % 40 for i in range(1100)], Hq=2, Hk=1, D=64, rd=32, page=16, dtype="bf16",
         wtype="bf16", layout="split_half"),
]


def append_inputs(c, first=2, behind=3, seed=3):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[c["dtype"]]
    T, D, Hq, Hk = first + sum(c["new"]) + behind, c["D"], c["Hq"], c["Hk"]
    qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g).to(dt)
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).to(TYPES[c["wtype"]]) for _ in range(2))
    table, n = scattered_tables([a + b for a, b in zip(c["new"], c["old"])], c["page"], g)
    kp, vp = (torch.randn(n, Hk, c["page"], D, generator=g).to(dt) for _ in range(2))
    return qkv, wq, wk, kp, vp, table, starts(c["new"], first), torch.tensor(c["old"], dtype=torch.int32)


@pytest.mark.parametrize("c", APPEND, ids=lambda c: "n%d_Hk%d_D%d_p%d_%s" % (len(c["new"]), c["Hk"], c["D"], c["page"], c["dtype"]))
@pytest.mark.parametrize("own_positions", [False, True])
def test_norm_append(c, own_positions):
    """Queries and keys have norm_rotate_qk's bits at the tokens' rows, values are copied, the rest stays."""
    require_gpu()
    R = lib()
    qkv, wq, wk, kp, vp, table, cu, old = (x.cuda() for x in append_inputs(c))
    Hq, Hk, page, T = c["Hq"], c["Hk"], c["page"], qkv.shape[0]
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    cos, sin = (x.cuda() for x in S.tables(1e4, c["rd"], 400))
    seq = torch.repeat_interleave(torch.arange(len(c["new"])), torch.tensor(c["new"]))
    tok = torch.arange(seq.numel()) + 2
    slot = old.cpu().long()[seq] + tok - cu.cpu().long()[seq]
    rows = torch.full((T,), -1, dtype=torch.int32)
    rows[tok] = (slot + 7).int()
    if own_positions:
        rows[tok] = torch.randint(-1, 400, (tok.numel(),), generator=torch.Generator().manual_seed(6), dtype=torch.int32)
    want_q, want_k = (x[0] for x in R.norm_rotate_qk(q[None], k[None], wq, wk, cos, sin, EPS, rows.cuda(), layout=c["layout"],
                                                     seq_before_head=True))
    gk, gv = kp.clone(), vp.clone()
    mark = torch.full_like(want_q, 3.0)
    out = R.norm_cache_append(q, k, v, wq, wk, gk, gv, table, cu, old, cos, sin, EPS, pos=rows.cuda() if own_positions else None,
                              pos_offset=7, layout=c["layout"], q_out=mark)
    assert out is mark and R.rope_check_errors() == R.ROPE_OK
    t = tok.cuda()
    assert same_bits(out[t], want_q[t]) and bool((out[:2] == 3).all()) and bool((out[-3:] == 3).all())
    at = table.cpu().long()[seq, slot // page].cuda(), slot.cuda() % page
    wk_, wv_ = kp.clone(), vp.clone()
    wk_[at[0], :, at[1]], wv_[at[0], :, at[1]] = want_k[t], v[t]
    assert same_bits(gk, wk_) and same_bits(gv, wv_)


def test_norm_append_bad_indices_and_in_place():
    require_gpu()
    R = lib()
    c = APPEND[1]
    qkv, wq, wk, kp, vp, table, cu, old = (x.cuda() for x in append_inputs(c, 0, 0))
    Hq, Hk = c["Hq"], c["Hk"]
    k, v = qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    cos, sin = (x.cuda() for x in S.tables(1e4, c["rd"], 400))

    def call(tb, o, cu_=cu, **more):
        q = qkv[:, :Hq].contiguous()
        gk, gv = kp.clone(), vp.clone()
        out = R.norm_cache_append(q, k, v, wq, wk, gk, gv, tb, cu_, o, cos, sin, layout=c["layout"], q_out=q, **more)
        assert out.data_ptr() == q.data_ptr()
        return R.rope_check_errors(), out, gk, gv

    st, q0, k0, v0 = call(table, old)
    assert st == R.ROPE_OK
    bad = table.clone()
    bad[0, 0] = kp.shape[0]
    st, q1, k1, v1 = call(bad, old)
    assert st == R.ROPE_ERR_BAD_INDEX and torch.equal(q1, q0)
    p = int(table[0, 0])
    k0[p], v0[p] = kp[p], vp[p]                            # that sequence's keys alone are missing
    assert torch.equal(k1, k0) and torch.equal(v1, v0)
    neg = old.clone()
    neg[2] = -5
    assert call(table, neg)[0] == R.ROPE_ERR_BAD_INDEX
    disorder = cu.clone()
    disorder[1], disorder[2] = 6, 2
    assert call(table, old, disorder)[0] == R.ROPE_ERR_BAD_INDEX
    assert call(table, old, pos_offset=390)[0] == R.ROPE_ERR_POS_OUT_OF_RANGE


def test_norm_append_refusals_and_versions():
    require_gpu()
    R = lib()
    c = APPEND[0]
    qkv, wq, wk, kp, vp, table, cu, old = (x.cuda() for x in append_inputs(c, 0, 0))
    q, k, v = qkv[:, :32], qkv[:, 32:40], qkv[:, 40:]
    cos, sin = (x.cuda() for x in S.tables(1e4, c["rd"], 64))
    ok = dict(q=q, k=k, v=v, wq=wq, wk=wk, k_pages=kp, v_pages=vp, block_table=table, cu_seqlens=cu, cache_lens=old, cos=cos,
              sin=sin)
    for bad, err, says in [
            (dict(q=q.float()), TypeError, "bf16 or fp16"), (dict(q=q[:2]), ValueError, "same tokens"), (dict(wq=wq[:1]), ValueError, "wq"),
            (dict(wq=wq.float()), ValueError, "one type"), (dict(k=k[:, :4]), ValueError, "k must be"),
            (dict(q_out=torch.empty_like(k)), ValueError, "q_out must be"), (dict(v_pages=kp), R.RopeError, None),
            (dict(eps=float("inf")), R.RopeError, None), (dict(q=kp[0].transpose(0, 1)[:3]), ValueError, "dense")]:
        with pytest.raises(err, match=says):
            R.norm_cache_append(**dict(ok, **bad))
    before = kp._version
    R.norm_cache_append(**ok)
    assert kp._version == before + 1 and vp._version >= 1
    assert R.rope_check_errors() == R.ROPE_OK

"""The norm, table and paged attention calls as a program makes them beside the ordinary way: through the thin wrappers of
the C entry points, and from several threads at once."""
import threading

import pytest
import torch

import serving_ref as S
from gpu_util import lib, require_gpu
from test_gpu_cache_append import scattered_tables, starts

pytestmark = pytest.mark.gpu


def step(seed=3, n=9, Hq=8, Hk=2, D=128, page=32):
    """A step's tensors: three sequences of one token, some of a few and a chunk, with a cache behind them."""
    g = torch.Generator().manual_seed(seed)
    new = [1, 1, 1, 2, 4, 40, 0, 3, 70][:n]
    old = [(i * 83) % 500 for i in range(n)]
    lens = [a + b for a, b in zip(new, old)]
    table, pages = scattered_tables(lens, page, g)
    x = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    t = dict(q=x(sum(new), Hq, D), k=x(sum(new), Hk, D), v=x(sum(new), Hk, D), kp=x(pages, Hk, page, D), vp=x(pages, Hk, page, D),
             wq=1 + 0.1 * torch.randn(D, generator=g), wk=1 + 0.1 * torch.randn(D, generator=g), table=table, cu=starts(new, 0),
             old=torch.tensor(old, dtype=torch.int32), lens=torch.tensor(lens, dtype=torch.int32))
    return {n: v.cuda() for n, v in t.items()}


def serve(R, t, cos, sin):
    kp, vp = t["kp"].clone(), t["vp"].clone()
    q = R.norm_cache_append(t["q"], t["k"], t["v"], t["wq"], t["wk"], kp, vp, t["table"], t["cu"], t["old"], cos, sin)
    return [R.attention_paged(q, kp, vp, t["table"], t["cu"], t["lens"]), q, kp, vp]


def test_thin_wrappers_do_the_same():
    require_gpu()
    R = lib()
    t = step()
    D, page = 128, 32
    cos, sin = R.build_tables_scaled("smooth", D, 700, 4.0, 256)
    c, s = torch.empty_like(cos), torch.empty_like(sin)
    R.rope_tables_build_scaled(R.ROPE_SCALE_SMOOTH, 10000.0, D, 700, 0, 4.0, 256, 1.0, 4.0, 1.0, c, s)
    assert torch.equal(c, cos) and torch.equal(s, sin)

    want = serve(R, t, cos, sin)
    T, Hq, Hk = t["q"].shape[0], t["q"].shape[1], t["k"].shape[1]
    n, blocks = t["table"].shape
    q, kp, vp, o = torch.empty_like(t["q"]), t["kp"].clone(), t["vp"].clone(), torch.empty_like(t["q"])
    R.rope_norm_cache_append(t["q"], t["k"], t["v"], q, kp, vp, t["wq"], t["wk"], t["table"], t["cu"], t["old"], cos, sin, None, 0, n, T,
                             Hq * D, Hk * D, Hk * D, Hq, Hk, D, D, R.ROPE_SPLIT_HALF, 1e-6, page, kp.shape[0], blocks, R.ROPE_BF16,
                             R.ROPE_F32, 700)
    size = R.rope_attention_paged_workspace(n, T, Hq, Hk, D, page, blocks)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    R.rope_attention_paged_fwd(q, kp, vp, o, t["table"], t["cu"], t["lens"], None, None, None, n, T, Hq * D, Hq, Hk, D, D,
                               R.ROPE_SPLIT_HALF, 1, 0.0, page, kp.shape[0], blocks, R.ROPE_BF16, 0, ws, size)
    for a, b in zip((o, q, kp, vp), want):
        assert torch.equal(a, b)

    x, y = t["q"][None], t["k"][None]
    args = (x, y, t["wq"], t["wk"], cos, sin)
    want = [*R.norm_rotate_qk(*args, seq_before_head=True),
            *R.norm_rotate_qk_backward(x, y, x, y, *args[2:], seq_before_head=True)]
    got = [torch.empty_like(w) for w in want]
    shape = (None, 0, 1, Hq, Hk, T, D, None, None, D, R.ROPE_SPLIT_HALF, 1, 1e-6, R.ROPE_BF16, R.ROPE_F32, 700)
    R.rope_norm_qk_fwd(x, y, got[0], got[1], *args[2:], *shape)
    size = R.rope_norm_qk_workspace(D)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    R.rope_norm_qk_bwd(x, y, x, y, got[2], got[3], t["wq"], t["wk"], got[4], got[5], cos, sin, *shape, ws, size)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert R.rope_check_errors() == R.ROPE_OK


def test_threads_with_streams_of_their_own():
    """Four threads serve and train at once; each finds what a call alone gives, bit for bit."""
    require_gpu()
    R = lib()
    from rotary_position_embedding_rope_gb300 import autograd

    steps = [step(seed=i, n=9 - i) for i in range(4)]
    cos, sin = S.tables(1e4, 128, 700)
    cos, sin = cos.cuda(), sin.cuda()

    def work(t):
        leaves = [t["q"][None].clone().requires_grad_(), t["k"][None].clone().requires_grad_(), t["wq"].clone().requires_grad_(),
                  t["wk"].clone().requires_grad_()]
        out = autograd.norm_rotary_qk(*leaves, cos, sin, seq_before_head=True)
        return serve(R, t, cos, sin) + list(out) + list(torch.autograd.grad(out, leaves, [x.detach() for x in out]))

    want = [work(t) for t in steps]
    torch.cuda.synchronize()
    bad, gate = [], threading.Barrier(len(steps))

    def thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait(60)
                for _ in range(25):
                    got = work(steps[i])
                    torch.cuda.current_stream().synchronize()
                    bad.extend((i, j) for j, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))
        except BaseException as e:     # noqa: B036 -- reported below
            bad.append((i, repr(e)))

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(len(steps))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:5]
    assert R.rope_check_errors() == R.ROPE_OK

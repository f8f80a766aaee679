"""rope_attention_packed_fwd against the plain form in 64 bits, sequence by
sequence, under the rule of the dense attention's tests (attention_check.py:
P is rounded to the element type before P V, o once)."""
import pytest
import torch

import attention_check as AC
import serving_ref as S
from gpu_util import lib, require_gpu

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def starts(lens, first=0):
    return torch.tensor([first] + [first + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)


def make(c, seed=5, first=0, behind=0):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[c["dtype"]]
    kl = c.get("k", c["q"])
    Tq, Tk = first + sum(c["q"]) + behind, first + sum(kl) + behind
    q = torch.randn(Tq, c["Hq"], c["D"], generator=g).to(dt)
    k = torch.randn(Tk, c["Hk"], c["D"], generator=g).to(dt)
    v = torch.randn(Tk, c["Hk"], c["D"], generator=g).to(dt)
    return q, k, v, starts(c["q"], first), starts(kl, first)


def run(R, c, q, k, v, cuq, cuk, cos, sin, **more):
    out = R.attention_packed(q.cuda(), k.cuda(), v.cuda(), cuq.cuda(), cos.cuda(), sin.cuda(), cu_seqlens_k=cuk.cuda(),
                             layout=c["layout"], causal=c["causal"], **more)
    assert R.rope_check_errors() == R.ROPE_OK
    return out.cpu()


def check(got, ref, c, what):
    """The rows of the sequences under the rule; the others untouched is the caller's."""
    o, w, a = ref
    live = ~torch.isnan(o[:, 0, 0])
    AC.check(got[live].float().numpy(), o[live].numpy(), w[live].numpy(), a[live].numpy(), c["dtype"], what)


CASES = [
    dict(q=[1], Hq=4, Hk=1, D=128, rd=128, dtype="bf16", layout="split_half", causal=True),
    dict(q=[17, 64, 1, 130, 0, 65], Hq=8, Hk=2, D=128, rd=128, dtype="bf16", layout="split_half", causal=True),
    dict(q=[300, 5, 257], Hq=6, Hk=2, D=128, rd=96, dtype="f16", layout="interleaved", causal=True),      # groups of 3: one head a row
    dict(q=[129, 40], Hq=12, Hk=2, D=64, rd=32, dtype="f16", layout="split_half", causal=False),           # groups of 6: two
    dict(q=[33, 200], Hq=16, Hk=1, D=64, rd=64, dtype="bf16", layout="interleaved", causal=True),          # sixteen heads, 16 tokens a tile
    dict(q=[70, 3], Hq=32, Hk=1, D=128, rd=16, dtype="bf16", layout="split_half", causal=False),           # 32 heads: two units of 16
    # fewer queries than keys (the last tokens), more queries than keys (rows that see none), no keys at all
    dict(q=[10, 100, 260], k=[300, 513, 260], Hq=8, Hk=4, D=128, rd=128, dtype="bf16", layout="split_half", causal=True),
    dict(q=[200, 90, 7], k=[70, 0, 7], Hq=4, Hk=2, D=128, rd=64, dtype="f16", layout="split_half", causal=True),
    dict(q=[150, 90, 0], k=[70, 0, 30], Hq=2, Hk=2, D=64, rd=64, dtype="bf16", layout="split_half", causal=False),
    # many tiles: several units per cluster, uneven rounds
    dict(q=[700, 31, 1300, 64, 256, 1] * 3, Hq=8, Hk=8, D=64, rd=32, dtype="f16", layout="interleaved", causal=True),
    dict(q=[1025, 513, 90, 1800], Hq=16, Hk=4, D=128, rd=128, dtype="bf16", layout="split_half", causal=True),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "n%d_q%d_Hq%d_Hk%d_D%d_rd%d_%s_c%d" % (
    len(c["q"]), sum(c["q"]), c["Hq"], c["Hk"], c["D"], c["rd"], c["dtype"], c["causal"]))
def test_packed(c):
    require_gpu()
    R = lib()
    first, behind = 3, 5
    q, k, v, cuq, cuk = make(c, first=first, behind=behind)
    cos, sin = S.tables(1e4, c["rd"], max(c["q"] + c.get("k", [0])) + 2)
    ref = S.packed(q, k, v, cuq, cuk, cos, sin, layout=c["layout"], causal=c["causal"])
    out = torch.full_like(q, 7.0).cuda()
    got = run(R, c, q, k, v, cuq, cuk, cos, sin, out=out)
    check(got, ref, c, "packed %s" % c)
    assert (got[:first] == 7).all() and (got[-behind:] == 7).all()       # rows of no sequence


def test_strided_views_positions_and_scale():
    """A fused projection's views, positions of their own (-1 among them), another scale: the bits of the dense call."""
    require_gpu()
    R = lib()
    c = dict(q=[150, 31, 200], Hq=8, Hk=2, D=128, rd=64, dtype="bf16", layout="split_half", causal=True)
    q, k, v, cu, _ = make(c)
    cos, sin = S.tables(1e4, 64, 1000)
    pos = torch.randint(0, 1000, (q.shape[0],), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    pos[::7] = -1
    ref = S.packed(q, k, v, cu, cu, cos, sin, pos, pos, causal=True, scale=0.05)
    fused = torch.cat([q, k, v], 1).cuda()
    out = R.attention_packed(fused[:, :8], fused[:, 8:10], fused[:, 10:], cu.cuda(), cos.cuda(), sin.cuda(),
                             pos_q=pos.cuda(), pos_k=pos.cuda(), causal=True, scale=0.05)
    assert R.rope_check_errors() == R.ROPE_OK
    check(out.cpu(), ref, c, "packed strided")
    dense = run(R, c, q, k, v, cu, cu, cos, sin, pos_q=pos.cuda(), pos_k=pos.cuda(), scale=0.05)
    assert torch.equal(out.cpu(), dense)


@pytest.mark.parametrize("D", [64, 128])
def test_neighbours_do_not_leak(D):
    """Infinities and NaN in the other sequences, and in the rows of none, change no bit of a sequence."""
    require_gpu()
    R = lib()
    c = dict(q=[130, 77, 64, 200], Hq=4, Hk=2, D=D, rd=D, dtype="bf16", layout="split_half", causal=False)
    q, k, v, cu, _ = make(c, behind=4)
    cos, sin = S.tables(1e4, D, 256)
    clean = run(R, c, q, k, v, cu, cu, cos, sin)
    for bad in (float("nan"), float("inf")):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for x in (q2, k2, v2):
            x[130:207] = bad
            x[-4:] = bad
        got = run(R, c, q2, k2, v2, cu, cu, cos, sin)
        for a, b in ((0, 130), (207, 471)):
            assert torch.equal(got[a:b], clean[a:b])


def test_agrees_with_the_dense_call():
    """Sequences of one length: the dense attention's result (the same rounding points)."""
    require_gpu()
    R = lib()
    B, Hq, Hk, L, D = 3, 8, 2, 320, 128
    c = dict(q=[L] * B, Hq=Hq, Hk=Hk, D=D, rd=D, dtype="bf16", layout="split_half", causal=True)
    q, k, v, cu, _ = make(c)
    cos, sin = S.tables(1e4, D, L)
    got = run(R, c, q, k, v, cu, cu, cos, sin).view(B, L, Hq, D).transpose(1, 2)
    dense = R.attention(*(x.view(B, L, -1, D).transpose(1, 2).contiguous().cuda() for x in (q, k, v)), cos.cuda(),
                        sin.cuda(), causal=True).cpu()
    assert torch.equal(got, dense)


def test_bad_offsets_and_short_tables_write_nothing():
    require_gpu()
    R = lib()
    c = dict(q=[40, 30], Hq=4, Hk=2, D=64, rd=64, dtype="f16", layout="split_half", causal=True)
    q, k, v, cu, _ = make(c)
    cos, sin = S.tables(1e4, 64, 40)
    args = [x.cuda() for x in (q, k, v)]
    for bad_q, bad_k, rows, status in (([0, 40, 71], [0, 40, 70], 40, R.ROPE_ERR_BAD_INDEX),
                                       ([0, 40, 30], [0, 40, 70], 40, R.ROPE_ERR_BAD_INDEX),
                                       ([-1, 40, 70], [0, 40, 70], 40, R.ROPE_ERR_BAD_INDEX),
                                       ([0, 40, 70], [5, 3, 70], 40, R.ROPE_ERR_BAD_INDEX),
                                       ([0, 40, 70], [0, 40, 70], 39, R.ROPE_ERR_POS_OUT_OF_RANGE)):
        out = torch.full_like(args[0], 7.0)
        R.attention_packed(*args, torch.tensor(bad_q, dtype=torch.int32).cuda(), cos[:rows].cuda(), sin[:rows].cuda(),
                           cu_seqlens_k=torch.tensor(bad_k, dtype=torch.int32).cuda(), causal=True, out=out)
        assert R.rope_check_errors() == status
        assert (out == 7).all()


def test_position_out_of_the_table_is_not_rotated():
    require_gpu()
    R = lib()
    c = dict(q=[40, 30], Hq=4, Hk=2, D=64, rd=64, dtype="bf16", layout="split_half", causal=True)
    q, k, v, cu, _ = make(c)
    cos, sin = S.tables(1e4, 64, 64)
    pq = torch.arange(70, dtype=torch.int32) % 60
    pq[3], pk = 64, pq.clone()
    pk[50] = -5
    ref = S.packed(q, k, v, cu, cu, cos, sin, pq, pk, causal=True)
    out = R.attention_packed(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), cos.cuda(), sin.cuda(), pos_q=pq.cuda(),
                             pos_k=pk.cuda(), causal=True)
    assert R.rope_check_errors() == R.ROPE_ERR_POS_OUT_OF_RANGE
    check(out.cpu(), ref, c, "packed positions")


def test_captured_replayed_and_on_another_stream():
    """A captured call follows new lengths and data; two calls share a workspace one after the other."""
    require_gpu()
    R = lib()
    c = dict(q=[90, 120, 46], Hq=8, Hk=2, D=128, rd=128, dtype="bf16", layout="split_half", causal=True)
    q, k, v, cu, _ = make(c)
    cos, sin = S.tables(1e4, 128, 256)
    ins = [x.cuda() for x in (q, k, v, cu, cos, sin)]
    ws = torch.empty(R.rope_attention_packed_workspace(3, 256, 256, 8, 2, 128), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(ins[0])
    R.attention_packed(*ins, causal=True, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        R.attention_packed(*ins, causal=True, out=out, workspace=ws)
        free = R.attention_packed(*ins, causal=False)
    q2, k2, v2, _, _ = make(c, seed=9)
    cu2 = torch.tensor([0, 1, 200, 256], dtype=torch.int32)
    for dst, src in zip(ins[:4], (q2, k2, v2, cu2)):
        dst.copy_(src)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert R.rope_check_errors() == R.ROPE_OK
    for got, causal in ((out, True), (free, False)):
        check(got.cpu(), S.packed(q2, k2, v2, cu2, cu2, cos, sin, causal=causal), c, "packed graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = R.attention_packed(*ins, causal=True, stream=side)
    side.synchronize()
    assert torch.equal(again, out)
    # raw handles, the default stream's among them, from another current stream
    with torch.cuda.stream(side):
        for handle in (0, s.cuda_stream):
            again = R.attention_packed(*ins, causal=True, stream=handle)
            torch.cuda.synchronize()
            assert torch.equal(again, out)


def test_thousands_of_sequences():
    """More sequences than the planner's CTA has threads, map CTAs have warps or offsets are cached for."""
    require_gpu()
    R = lib()
    n = 2500
    c = dict(q=[(i * 7) % 4 for i in range(n)], Hq=2, Hk=1, D=64, rd=32, dtype="bf16", layout="split_half", causal=True)
    q, k, v, cu, _ = make(c)
    cos, sin = S.tables(1e4, 32, 4)
    ref = S.packed(q, k, v, cu, cu, cos, sin, causal=True)
    check(run(R, c, q, k, v, cu, cu, cos, sin), ref, c, "packed thousands")


def test_no_keys_at_all_and_nothing_at_all():
    require_gpu()
    R = lib()
    cos, sin = (x.cuda() for x in S.tables(1e4, 64, 64))
    q = torch.randn(50, 4, 64, device="cuda").bfloat16()
    none = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    cu, zero = torch.tensor([0, 20, 50], dtype=torch.int32).cuda(), torch.zeros(3, dtype=torch.int32).cuda()
    out = R.attention_packed(q, none, none, cu, cos, sin, cu_seqlens_k=zero, causal=False)
    assert R.rope_check_errors() == R.ROPE_OK and torch.count_nonzero(out) == 0
    assert R.attention_packed(q[:0], none, none, zero, cos, sin).shape == (0, 4, 64)
    keep = torch.full_like(q, 3.0)
    # rows that see no key stay zeros beside infinite values that other rows see
    inf = torch.full((30, 2, 64), float("inf"), device="cuda", dtype=torch.bfloat16)
    one = torch.tensor([0, 50], dtype=torch.int32).cuda()
    out = R.attention_packed(q, torch.zeros_like(inf), inf, one, cos, sin, causal=True,
                             cu_seqlens_k=torch.tensor([0, 30], dtype=torch.int32).cuda())
    assert torch.count_nonzero(out[:20]) == 0 and not out[20:].isfinite().any()
    R.attention_packed(q, none, none, cu[:1], cos, sin, cu_seqlens_k=zero[:1], out=keep)
    assert R.rope_check_errors() == R.ROPE_OK and (keep == 3).all()


def test_large_scores_and_infinities():
    """Scores hundreds apart; an infinite key gives what the formula gives (NaN where it is seen)."""
    require_gpu()
    R = lib()
    c = dict(q=[140, 260], Hq=4, Hk=2, D=128, rd=128, dtype="bf16", layout="split_half", causal=True)
    q, k, v, cu, _ = make(c)
    q = (q.float() * torch.linspace(0.1, 12, 400)[:, None, None]).bfloat16()
    cos, sin = S.tables(1e4, 128, 300)
    o, w, a = S.packed(q, k, v, cu, cu, cos, sin, causal=True)
    # A rotated element in the middle of two neighbours may be rounded to either, which moves scores of this size by
    # up to d = score_slack.  Every p_j = e^(s_j) / sum e^(s) then changes by a factor within e^(+-2d), and o by at
    # most (e^(2d) - 1) sum p_j |v_j| = (e^(2d) - 1) W; the rule's (u + 2^-14) W is widened by that.
    d = S.score_slack(q, k, cu, cos, sin)
    w = w * (1 + torch.expm1(2 * d) / (AC.U["bf16"] + AC.ARITH))[..., None]
    check(run(R, c, q, k, v, cu, cu, cos, sin), (o, w, a), c, "packed large scores")
    k2 = k.clone()
    k2[139] = float("nan")                                 # the last key of the first sequence
    got = run(R, c, q, k2, v, cu, cu, cos, sin)
    clean = run(R, c, q, k, v, cu, cu, cos, sin)
    assert torch.equal(got[:139], clean[:139]) and torch.equal(got[140:], clean[140:]) and got[139].isnan().all()


def test_refusals():
    require_gpu()
    R = lib()
    c = dict(q=[40, 30], Hq=4, Hk=2, D=64, rd=64, dtype="f16", layout="split_half", causal=True)
    q, k, v, cu, _ = (x.cuda() for x in make(c))
    cos, sin = (x.cuda() for x in S.tables(1e4, 64, 64))
    ok = dict(q=q, k=k, v=v, cu_seqlens_q=cu, cos=cos, sin=sin)
    for bad, err in [(dict(q=q.float()), TypeError), (dict(k=k.bfloat16()), ValueError), (dict(v=v[:60]), ValueError),
                     (dict(q=q[:, :3]), R.RopeError), (dict(q=q[..., ::2]), ValueError), (dict(v=v.cpu()), ValueError),
                     (dict(q=q.transpose(0, 1)), ValueError), (dict(cu_seqlens_q=cu.long()), ValueError),
                     (dict(cu_seqlens_k=cu[:2].contiguous()), ValueError), (dict(pos_q=cu), ValueError),
                     (dict(out=q[:, :2]), ValueError), (dict(out=q), R.RopeError), (dict(rotary_dim=32), ValueError),
                     (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), R.RopeError)]:
        with pytest.raises(err):
            R.attention_packed(**dict(ok, **bad))
    assert R.rope_check_errors() == R.ROPE_OK


@pytest.mark.parametrize("D, Hq, Hk, causal", [(128, 8, 2, True), (64, 4, 4, False), (128, 32, 1, False)])
def test_what_neighbours_hold_stays_with_them(D, Hq, Hk, causal):
    """Sequences whose queries, keys and values are infinities and NaN, between others of every kind of length."""
    require_gpu()
    R = lib()
    lens = [5, 130, 1, 7, 300, 64, 33, 129, 2, 256, 90]
    c = dict(q=lens, Hq=Hq, Hk=Hk, D=D, rd=D, dtype="bf16", layout="split_half", causal=causal)
    q, k, v, cu, _ = make(c)
    cos, sin = S.tables(1e4, D, 300)
    clean = run(R, c, q, k, v, cu, cu, cos, sin)
    for x in (q, k, v):
        for b in range(1, len(lens), 2):
            rows = x[int(cu[b]):int(cu[b + 1])]
            rows[:, :, ::2], rows[:, :, 1::2] = float("nan"), float("inf")
    got = run(R, c, q, k, v, cu, cu, cos, sin)
    for b in range(0, len(lens), 2):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        assert torch.equal(got[rows], clean[rows])


def test_positions_of_no_sequence_are_not_looked_at():
    """A padded batch: whatever stands at the tokens before the first and behind the last sequence raises nothing."""
    require_gpu()
    R = lib()
    c = dict(q=[40, 30], Hq=4, Hk=2, D=64, rd=64, dtype="bf16", layout="split_half", causal=True)
    q, k, v, cu, _ = make(c, first=3, behind=9)
    cos, sin = S.tables(1e4, 64, 64)
    pos = torch.full((82,), 10 ** 6, dtype=torch.int32)
    pos[3:43], pos[43:73] = torch.arange(40), torch.arange(30)
    plain = run(R, c, q, k, v, cu, cu, cos, sin)
    got = run(R, c, q, k, v, cu, cu, cos, sin, pos_q=pos.cuda(), pos_k=pos.cuda())
    assert torch.equal(got[3:73], plain[3:73])

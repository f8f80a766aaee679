"""rope_cache_append against the plain form in 64 bits: keys within one unit
in the last place of the rotation rounded once (the rule of the rotation
kernels), values and everything not written bit for bit."""
import pytest
import torch

import serving_ref as S
import workloads as W
from gpu_util import lib, require_gpu, ulp_distance16

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def scattered_tables(counts, page, g, spare=2):
    """Block lists on scattered pages for the given numbers of keys; unused entries -1."""
    need = [-(-c // page) for c in counts]
    order = torch.randperm(sum(need) + spare, generator=g)
    table = torch.full((len(counts), max([1] + need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].int()
        at += n
    return table, sum(need) + spare


def starts(lens, first=0):
    return torch.tensor([first] + [first + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def check_pools(got_k, got_v, want_k, want_v, wrote, k_pages):
    assert same_bits(got_v, want_v)
    m = wrote[:, None, :, None].expand_as(k_pages)
    assert same_bits(torch.where(m, 0, got_k), torch.where(m, 0, k_pages))
    d = ulp_distance16(W.bits(got_k), W.bits(want_k))
    assert d.max(initial=0) <= 1


CASES = [
    # new tokens, keys already cached
    dict(new=[1, 1, 1], old=[0, 15, 16], Hk=8, D=128, rd=128, page=16, dtype="bf16", layout="split_half"),
    dict(new=[5, 0, 33, 1], old=[3, 9, 0, 63], Hk=2, D=64, rd=64, page=32, dtype="f16", layout="interleaved"),
    dict(new=[70, 129], old=[0, 100], Hk=5, D=128, rd=96, page=64, dtype="f16", layout="split_half"),
    dict(new=[17], old=[120], Hk=1, D=64, rd=16, page=128, dtype="bf16", layout="interleaved"),
    dict(new=[2] * 40, old=list(range(40)), Hk=3, D=64, rd=32, page=16, dtype="bf16", layout="split_half"),
]


def make(c, seed=3, first=0, behind=0):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[c["dtype"]]
    T = first + sum(c["new"]) + behind
    k = torch.randn(T, c["Hk"], c["D"], generator=g).to(dt)
    v = torch.randn(T, c["Hk"], c["D"], generator=g).to(dt)
    table, n_pages = scattered_tables([a + b for a, b in zip(c["new"], c["old"])], c["page"], g)
    kp = torch.randn(n_pages, c["Hk"], c["page"], c["D"], generator=g).to(dt)
    vp = torch.randn(n_pages, c["Hk"], c["page"], c["D"], generator=g).to(dt)
    return k, v, kp, vp, table, starts(c["new"], first), torch.tensor(c["old"], dtype=torch.int32)


@pytest.mark.parametrize("c", CASES, ids=lambda c: "n%d_Hk%d_D%d_rd%d_p%d_%s" % (
    len(c["new"]), c["Hk"], c["D"], c["rd"], c["page"], c["dtype"]))
def test_append(c):
    require_gpu()
    R = lib()
    k, v, kp, vp, table, cu, old = make(c, first=2, behind=3)
    cos, sin = S.tables(1e4, c["rd"], 400)
    want = S.append(k, v, kp, vp, table, cu, old, cos, sin, pos_offset=11, layout=c["layout"])
    gk, gv = kp.cuda(), vp.cuda()
    R.cache_append(k.cuda(), v.cuda(), gk, gv, table.cuda(), cu.cuda(), old.cuda(), cos.cuda(), sin.cuda(),
                   pos_offset=11, layout=c["layout"])
    assert R.rope_check_errors() == R.ROPE_OK
    check_pools(gk.cpu(), gv.cpu(), want[0], want[1], want[2], kp)


def test_append_bits_are_the_rotation_kernels():
    """The keys have the bits that rotate_qk gives, from strided views and positions of their own."""
    require_gpu()
    R = lib()
    c = CASES[2]
    k, v, kp, vp, table, cu, old = make(c)
    cos, sin = (x.cuda() for x in S.tables(1e4, c["rd"], 300))
    T, Hk, D = k.shape
    pos = torch.randint(0, 300, (T,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    pos[7] = -1
    fused = torch.cat([k, v, k], 1).cuda()                # token stride 3 Hk D
    gk, gv = kp.cuda(), vp.cuda()
    R.cache_append(fused[:, :Hk], fused[:, Hk:2 * Hk], gk, gv, table.cuda(), cu.cuda(), old.cuda(), cos, sin,
                   pos=pos.cuda())
    assert R.rope_check_errors() == R.ROPE_OK
    turned, _ = R.rotate_qk(k.cuda()[None], None, cos, sin, pos.cuda(), seq_before_head=True)
    turned = turned[0].cpu()
    gk, gv = gk.cpu(), gv.cpu()
    for b in range(len(c["new"])):
        for i in range(c["new"][b]):
            s, t = c["old"][b] + i, int(cu[b]) + i
            p = int(table[b, s // c["page"]])
            assert same_bits(gk[p, :, s % c["page"]], turned[t]) and same_bits(gv[p, :, s % c["page"]], v[t])


def test_append_bad_indices_write_nothing_else():
    """Pages, blocks, lengths and positions out of range: flagged, everything else written."""
    require_gpu()
    R = lib()
    c = CASES[1]
    k, v, kp, vp, table, cu, old = make(c)
    cos, sin = S.tables(1e4, c["rd"], 400)
    for change in ("page", "negative page", "block", "length"):
        tb, o = table.clone(), old.clone()
        if change == "page":
            tb[0, 0] = kp.shape[0]
        elif change == "negative page":
            tb[2, 1] = -7
        elif change == "block":
            o[3] = tb.shape[1] * c["page"]
        else:
            o[0] = -3
        want = S.append(k, v, kp, vp, tb, cu, o, cos, sin, layout=c["layout"])
        gk, gv = kp.cuda(), vp.cuda()
        R.cache_append(k.cuda(), v.cuda(), gk, gv, tb.cuda(), cu.cuda(), o.cuda(), cos.cuda(), sin.cuda(),
                       layout=c["layout"])
        assert R.rope_check_errors() == R.ROPE_ERR_BAD_INDEX, change
        check_pools(gk.cpu(), gv.cpu(), *want, kp)
    # a table too short for the positions: those keys are written unrotated
    want = S.append(k, v, kp, vp, table, cu, old, cos[:20], sin[:20], layout=c["layout"])
    gk, gv = kp.cuda(), vp.cuda()
    R.cache_append(k.cuda(), v.cuda(), gk, gv, table.cuda(), cu.cuda(), old.cuda(), cos[:20].cuda(),
                   sin[:20].cuda(), layout=c["layout"])
    assert R.rope_check_errors() == R.ROPE_ERR_POS_OUT_OF_RANGE
    check_pools(gk.cpu(), gv.cpu(), *want, kp)
    # offsets out of order
    bad = cu.clone()
    bad[2], bad[3] = cu[3], cu[2]
    R.cache_append(k.cuda(), v.cuda(), kp.cuda(), vp.cuda(), table.cuda(), bad.cuda(), old.cuda(), cos.cuda(),
                   sin.cuda(), layout=c["layout"])
    assert R.rope_check_errors() == R.ROPE_ERR_BAD_INDEX


def test_append_many_sequences_search_in_global_memory():
    """More sequences than the kernel keeps offsets for, empty ones among them."""
    require_gpu()
    R = lib()
    c = dict(new=[(i * 7) % 3 for i in range(1500)], old=[i % 5 for i in range(1500)], Hk=1, D=64, rd=32, page=16,
             dtype="bf16", layout="split_half")
    k, v, kp, vp, table, cu, old = make(c)
    cos, sin = S.tables(1e4, c["rd"], 16)
    want = S.append(k, v, kp, vp, table, cu, old, cos, sin)
    gk, gv = kp.cuda(), vp.cuda()
    R.cache_append(k.cuda(), v.cuda(), gk, gv, table.cuda(), cu.cuda(), old.cuda(), cos.cuda(), sin.cuda())
    assert R.rope_check_errors() == R.ROPE_OK
    check_pools(gk.cpu(), gv.cpu(), *want, kp)


def test_append_refusals():
    require_gpu()
    R = lib()
    c = CASES[0]
    k, v, kp, vp, table, cu, old = (x.cuda() for x in make(c))
    cos, sin = (x.cuda() for x in S.tables(1e4, c["rd"], 64))
    ok = dict(k=k, v=v, k_pages=kp, v_pages=vp, block_table=table, cu_seqlens=cu, cache_lens=old, cos=cos, sin=sin)
    for bad, err in [(dict(k=k.float()), TypeError), (dict(v=v.half()), ValueError), (dict(v=v[:, :4]), ValueError),
                     (dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                     (dict(k_pages=kp.half()), ValueError), (dict(cu_seqlens=cu.long()), ValueError),
                     (dict(cu_seqlens=cu[:-1].contiguous()), ValueError), (dict(cache_lens=old[:1]), ValueError),
                     (dict(block_table=table[:, ::2] if table.shape[1] > 1 else table.t()[::1, ::2]), ValueError),
                     (dict(rotary_dim=64), ValueError), (dict(pos=old), ValueError) if k.shape[0] != 3 else
                     (dict(pos=old[:2]), ValueError),
                     (dict(k_pages=torch.empty(4, 8, 48, 128, dtype=k.dtype, device="cuda"),
                           v_pages=torch.empty(4, 8, 48, 128, dtype=k.dtype, device="cuda")), R.RopeError)]:
        with pytest.raises(err):
            R.cache_append(**dict(ok, **bad))
    assert R.rope_check_errors() == R.ROPE_OK


def test_append_captured_and_on_another_stream():
    require_gpu()
    R = lib()
    c = CASES[4]
    k, v, kp, vp, table, cu, old = make(c)
    cos, sin = S.tables(1e4, c["rd"], 64)
    args = [x.cuda() for x in (k, v, kp, vp, table, cu, old, cos, sin)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        R.cache_append(*args)
    # new data in the same buffers, then a replay
    k2, v2 = torch.randn_like(k), torch.randn_like(v)
    args[0].copy_(k2)
    args[1].copy_(v2)
    args[6].add_(1)
    graph.replay()
    torch.cuda.synchronize()
    want = S.append(k2, v2, kp, vp, table, cu, old + 1, cos, sin)
    flagged = any((int(o) + 1 + n - 1) // c["page"] >= table.shape[1] or
                  int(table[b, (int(o) + n) // c["page"]]) < 0 for b, (o, n) in enumerate(zip(c["old"], c["new"])))
    assert R.rope_check_errors() == (R.ROPE_ERR_BAD_INDEX if flagged else R.ROPE_OK)
    check_pools(args[2].cpu(), args[3].cpu(), *want, kp)

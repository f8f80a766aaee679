"""rope_attention_decode_fwd against the plain form in 64 bits, under the rule
of the dense attention's tests (attention_check.py: P is rounded to the element
type before P V, o once).  Every row of a page that holds no key holds NaN."""
import pytest
import torch

import attention_check as AC
import serving_ref as S
from gpu_util import lib, require_gpu
from test_gpu_cache_append import scattered_tables, starts

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def make(c, seed=5, poison=True):
    """q, pools, block lists, lengths and prefix list of a case; pages lie scattered."""
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[c["dtype"]]
    lens, P, page = c["lens"], c["prefix"], c["page"]
    table, n_pages = scattered_tables(lens + [P], page, g)
    q = torch.randn(len(lens), c["Hq"], c["D"], generator=g).to(dt)
    kp = torch.randn(n_pages, c["Hk"], page, c["D"], generator=g).to(dt)
    vp = torch.randn(n_pages, c["Hk"], page, c["D"], generator=g).to(dt)
    if poison:
        for row, n in zip(table, lens + [P]):
            if n % page:
                p = int(row[n // page])
                kp[p, :, n % page:] = float("nan")
                vp[p, :, n % page:] = float("nan")
                vp[p, :, n % page:, ::2] = float("inf")
        used = set(table.flatten().tolist())
        for p in range(n_pages):
            if p not in used:
                kp[p] = float("nan")
                vp[p] = float("nan")
    need = max([0] + [-(-n // page) for n in lens])
    return q, kp, vp, table[:-1, :max(need, 1)].contiguous(), torch.tensor(lens, dtype=torch.int32), \
        table[-1, :-(-P // page)].contiguous()


def run(R, c, q, kp, vp, table, lens, ptable, cos, sin, **more):
    out = R.attention_shared_prefix(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), ptable.cuda(), c["prefix"],
                                    cos.cuda(), sin.cuda(), layout=c["layout"], **more)
    assert R.rope_check_errors() == R.ROPE_OK
    return out.cpu()


def check(got, ref, c, what):
    o, w, a = ref
    AC.check(got.float().numpy(), o.numpy(), w.numpy(), a.numpy(), c["dtype"], what)


CASES = [
    dict(lens=[1], prefix=0, Hq=4, Hk=1, D=128, rd=128, page=16, dtype="bf16", layout="split_half"),
    dict(lens=[0], prefix=1, Hq=2, Hk=2, D=64, rd=64, page=64, dtype="f16", layout="split_half"),
    dict(lens=[33, 1, 0, 64, 17, 16, 100], prefix=300, Hq=8, Hk=2, D=128, rd=128, page=64, dtype="bf16", layout="split_half"),
    dict(lens=[40, 0, 129], prefix=127, Hq=6, Hk=2, D=128, rd=96, page=16, dtype="f16", layout="interleaved"),       # groups of 3
    dict(lens=[15, 31, 47, 63], prefix=128, Hq=4, Hk=4, D=64, rd=32, page=32, dtype="f16", layout="split_half"),      # groups of 1
    dict(lens=[200, 7], prefix=1000, Hq=16, Hk=2, D=64, rd=16, page=128, dtype="bf16", layout="interleaved"),         # groups of 8
    dict(lens=[70, 0, 130], prefix=77, Hq=48, Hk=2, D=128, rd=128, page=64, dtype="bf16", layout="split_half"),       # 24: rows of 16 and 8
    dict(lens=[5] * 3, prefix=0, Hq=32, Hk=1, D=64, rd=64, page=16, dtype="f16", layout="split_half"),                # 32
    dict(lens=[0, 0, 5, 0, 0], prefix=0, Hq=4, Hk=2, D=128, rd=64, page=32, dtype="bf16", layout="split_half"),       # rows without keys
    dict(lens=[(i * 37) % 90 for i in range(150)], prefix=513, Hq=8, Hk=2, D=64, rd=64, page=16, dtype="bf16", layout="split_half"),
    # more rows than a cluster's tile, long enough for many splits and runs over several pairs
    dict(lens=[(i * 61) % 400 for i in range(70)], prefix=3000, Hq=16, Hk=4, D=128, rd=128, page=64, dtype="bf16", layout="split_half"),
    dict(lens=[3000, 1, 700], prefix=5000, Hq=4, Hk=1, D=128, rd=128, page=128, dtype="f16", layout="interleaved"),
    # rows between the merge's forms, with and without many parts; one sequence in more than 300 parts
    dict(lens=[(i * 29) % 200 for i in range(40)], prefix=0, Hq=16, Hk=2, D=128, rd=128, page=32, dtype="bf16", layout="split_half"),
    dict(lens=[(i * 29) % 70 for i in range(33)], prefix=2000, Hq=16, Hk=2, D=64, rd=32, page=64, dtype="f16", layout="interleaved"),
    dict(lens=[500] * 32, prefix=0, Hq=32, Hk=8, D=64, rd=64, page=16, dtype="bf16", layout="split_half"),
    dict(lens=[25000], prefix=0, Hq=4, Hk=1, D=64, rd=64, page=64, dtype="bf16", layout="split_half"),
    dict(lens=[100], prefix=21000, Hq=8, Hk=1, D=128, rd=128, page=128, dtype="f16", layout="split_half"),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "B%d_P%d_n%d_Hq%d_Hk%d_D%d_p%d_%s" % (
    len(c["lens"]), c["prefix"], sum(c["lens"]), c["Hq"], c["Hk"], c["D"], c["page"], c["dtype"]))
def test_decode(c):
    require_gpu()
    R = lib()
    q, kp, vp, table, lens, ptable = make(c)
    cos, sin = S.tables(1e4, c["rd"], c["prefix"] + max(c["lens"]) + 1)
    ref = S.shared_prefix(q, kp, vp, table, lens, ptable, c["prefix"], cos, sin, layout=c["layout"])
    got = run(R, c, q, kp, vp, table, lens, ptable, cos, sin)
    check(got, ref, c, "decode %s" % {k: v for k, v in c.items() if k != "lens"})
    again = run(R, c, q, kp, vp, table, lens, ptable, cos, sin)
    assert torch.equal(got, again)


def test_prefix_and_suffix_are_one_softmax():
    """The same keys with the border between prefix and suffix elsewhere: the same attention."""
    require_gpu()
    R = lib()
    c = dict(lens=[320], prefix=0, Hq=8, Hk=2, D=128, rd=128, page=32, dtype="bf16", layout="split_half")
    q, kp, vp, table, lens, _ = make(c)
    cos, sin = S.tables(1e4, 128, 400)
    ref = S.shared_prefix(q, kp, vp, table, lens, table[0, :0], 0, cos, sin)
    for blocks in range(0, 11):
        n = 32 * blocks
        d = dict(c, prefix=n)
        got = run(R, d, q, kp, vp, table[:, blocks:].contiguous() if blocks < 10 else table[:, :1], lens - n,
                  table[0, :blocks].contiguous(), cos, sin)
        check(got, ref, c, "decode border")


def test_large_scores_positions_scale_and_strides():
    """Scores far apart (the running maximum moves by hundreds), positions of their own, a strided query."""
    require_gpu()
    R = lib()
    c = dict(lens=[150, 31, 290, 4], prefix=700, Hq=8, Hk=2, D=128, rd=64, page=16, dtype="bf16", layout="split_half")
    q, kp, vp, table, lens, ptable = make(c)
    ramp = torch.linspace(-3, 3, kp.shape[0])[torch.randperm(kp.shape[0], generator=torch.Generator().manual_seed(1))]
    kp = (kp.float() * torch.exp(ramp)[:, None, None, None]).to(kp.dtype)
    cos, sin = S.tables(1e4, 64, 50)
    pos = torch.tensor([3, -1, 49, 0], dtype=torch.int32)
    ref = S.shared_prefix(q, kp, vp, table, lens, ptable, 700, cos, sin, pos_q=pos, scale=0.4)
    fused = torch.cat([q, q, q], 1).cuda()
    got = R.attention_shared_prefix(fused[:, 8:16], kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), ptable.cuda(), 700,
                                    cos.cuda(), sin.cuda(), pos_q=pos.cuda(), scale=0.4)
    assert R.rope_check_errors() == R.ROPE_OK
    check(got.cpu(), ref, c, "decode large scores")


def test_sequences_share_pages():
    """Forked sequences: the same pages in several block lists."""
    require_gpu()
    R = lib()
    c = dict(lens=[60, 60, 60], prefix=40, Hq=4, Hk=2, D=64, rd=64, page=16, dtype="f16", layout="split_half")
    q, kp, vp, table, lens, ptable = make(c)
    table[1] = table[0]
    table[2, :2] = table[0, :2]
    cos, sin = S.tables(1e4, 64, 128)
    ref = S.shared_prefix(q, kp, vp, table, lens, ptable, 40, cos, sin)
    check(run(R, c, q, kp, vp, table, lens, ptable, cos, sin), ref, c, "decode shared pages")


def test_bad_indices_spoil_only_their_sequences():
    require_gpu()
    R = lib()
    c = dict(lens=[33, 50, 64], prefix=40, Hq=4, Hk=2, D=64, rd=64, page=16, dtype="bf16", layout="split_half")
    q, kp, vp, table, lens, ptable = make(c)
    cos, sin = S.tables(1e4, 64, 128)
    clean = run(R, c, q, kp, vp, table, lens, ptable, cos, sin)
    for what in ("page", "negative page", "length", "negative length"):
        tb, n = table.clone(), lens.clone()
        if what == "page":
            tb[1, 2] = kp.shape[0]
        elif what == "negative page":
            tb[1, 0] = -1
        else:
            n[1] = 65 if what == "length" else -4
        got = R.attention_shared_prefix(q.cuda(), kp.cuda(), vp.cuda(), tb.cuda(), n.cuda(), ptable.cuda(), 40, cos.cuda(),
                                        sin.cuda()).cpu()
        assert R.rope_check_errors() == R.ROPE_ERR_BAD_INDEX, what
        # the split of the work, and so the last bit, may follow the lengths
        for b in (0, 2):
            assert torch.allclose(got[b].float(), clean[b].float(), rtol=2 ** -7, atol=2 ** -9), what
    bad = ptable.clone()
    bad[1] = 1 << 30
    R.attention_shared_prefix(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), bad.cuda(), 40, cos.cuda(),
                              sin.cuda())
    assert R.rope_check_errors() == R.ROPE_ERR_BAD_INDEX
    # a query past the table is not rotated
    ref = S.shared_prefix(q, kp, vp, table, lens, ptable, 40, cos[:100], sin[:100])
    got = R.attention_shared_prefix(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), ptable.cuda(), 40,
                                    cos[:100].cuda(), sin[:100].cuda())
    assert R.rope_check_errors() == R.ROPE_ERR_POS_OUT_OF_RANGE
    check(got.cpu(), ref, c, "decode position past the table")


def test_a_serving_step():
    """Prompts attended packed and appended, then decode steps over a shared prefix, against one plain softmax."""
    require_gpu()
    R = lib()
    Hq, Hk, D, page, P = 8, 2, 128, 16, 50
    g = torch.Generator().manual_seed(11)
    prompts, steps = [21, 1, 40], 3
    B = len(prompts)
    cos, sin = (x.cuda() for x in S.tables(5e5, D, 128))
    n_pages = 40
    kp = torch.full((n_pages, Hk, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    ptable = torch.arange(4, dtype=torch.int32, device="cuda")
    table = (4 + torch.arange(B * 4, dtype=torch.int32).view(B, 4)).cuda()

    def new(n):
        return [torch.randn(n, h, D, generator=g).bfloat16().cuda() for h in (Hq, Hk, Hk)]

    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, kx, vx = new(P)
    R.cache_append(kx, vx, kp, vp, ptable.view(1, 4), torch.tensor([0, P], dtype=torch.int32, device="cuda"), zero, cos, sin)
    cu = starts(prompts).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q, k, v = new(sum(prompts))
    # the prompts attend among themselves here (a model without the prefix in this layer)
    packed = R.attention_packed(q, k, v, cu, cos, sin, causal=True)
    check(packed.cpu(), S.packed(q.cpu(), k.cpu(), v.cpu(), cu.cpu(), cu.cpu(), cos.cpu(), sin.cpu(), causal=True),
          dict(dtype="bf16"), "serving prompts")
    R.cache_append(k, v, kp, vp, table, cu, lens, cos, sin, pos_offset=P)
    lens += torch.tensor(prompts, dtype=torch.int32, device="cuda")
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    for _ in range(steps):
        q, k, v = new(B)
        R.cache_append(k, v, kp, vp, table, one, lens, cos, sin, pos_offset=P)
        lens += 1
        got = R.attention_shared_prefix(q, kp, vp, table, lens, ptable, P, cos, sin)
        assert R.rope_check_errors() == R.ROPE_OK
        ref = S.shared_prefix(q.cpu(), kp.cpu(), vp.cpu(), table.cpu(), lens.cpu(), ptable.cpu(), P, cos.cpu(), sin.cpu())
        check(got.cpu(), ref, dict(dtype="bf16"), "serving step")


def test_captured_replayed_and_on_another_stream():
    """A captured step follows lengths, pages and data; the workspace is shared by two captured calls."""
    require_gpu()
    R = lib()
    c = dict(lens=[33, 50, 64, 0], prefix=200, Hq=8, Hk=2, D=128, rd=128, page=16, dtype="bf16", layout="split_half")
    q, kp, vp, table, lens, ptable = make(c)
    cos, sin = S.tables(1e4, 128, 300)
    ins = [x.cuda() for x in (q, kp, vp, table, lens, ptable)]
    ct = [x.cuda() for x in (cos, sin)]
    ws = torch.empty(R.rope_attention_decode_workspace(4, 8, 2, 128, 16, table.shape[1], 200), dtype=torch.uint8,
                     device="cuda")
    out, out2 = torch.zeros_like(ins[0]), torch.zeros_like(ins[0])
    R.attention_shared_prefix(*ins, 200, *ct, out=out, workspace=ws)
    torch.cuda.synchronize()
    graphs, s = [], torch.cuda.Stream()
    for o, p in ((out, 200), (out2, 199)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            R.attention_shared_prefix(*ins, p, *ct, out=o, workspace=ws)
    q2 = torch.randn_like(q)
    n2 = torch.tensor([1, 64, 0, 20], dtype=torch.int32)
    tb2 = table.clone()
    tb2[3, :2] = table[2, :2]
    for dst, src in ((ins[0], q2), (ins[4], n2), (ins[3], tb2)):
        dst.copy_(src)
    kc, vc = kp.clone(), vp.clone()
    kc[kc.isnan()], vc[~vc.isfinite()] = 0.5, 0.25                     # row 1 grew into rows that held nothing
    ins[1].copy_(kc)
    ins[2].copy_(vc)
    for _ in range(2):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert R.rope_check_errors() == R.ROPE_OK
    for o, p in ((out, 200), (out2, 199)):
        check(o.cpu(), S.shared_prefix(q2, kc, vc, tb2, n2, ptable, p, cos, sin), c, "decode graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = R.attention_shared_prefix(*ins, 200, *ct, stream=side)
    side.synchronize()
    assert torch.equal(again, out)


@pytest.mark.parametrize("prefix", [0, 33])
def test_the_largest_batch(prefix):
    """4096 sequences, most with few keys, some with none."""
    require_gpu()
    R = lib()
    c = dict(lens=[(i * 5) % 7 for i in range(4096)], prefix=prefix, Hq=2, Hk=1, D=64, rd=32, page=16, dtype="f16",
             layout="split_half")
    q, kp, vp, table, lens, ptable = make(c)
    cos, sin = S.tables(1e4, 32, 64)
    ref = S.shared_prefix(q, kp, vp, table, lens, ptable, prefix, cos, sin)
    check(run(R, c, q, kp, vp, table, lens, ptable, cos, sin), ref, c, "decode largest batch")


def test_prefix_alone_and_nothing_at_all():
    """No suffix blocks; no keys of either kind; no sequences."""
    require_gpu()
    R = lib()
    for B in (2, 20):                                      # the prefix with the suffix kernel, and its own
        c = dict(lens=[0] * B, prefix=300, Hq=8, Hk=2, D=128, rd=128, page=64, dtype="bf16", layout="split_half")
        q, kp, vp, table, lens, ptable = make(c)
        cos, sin = S.tables(1e4, 128, 301)
        ref = S.shared_prefix(q, kp, vp, table, lens, ptable, 300, cos, sin)
        check(run(R, c, q, kp, vp, table[:, :0].contiguous(), lens, ptable, cos, sin), ref, c, "decode prefix alone")
        c["prefix"] = 0
        for blocks in (0, 1):
            got = run(R, c, q, kp, vp, table[:, :blocks].contiguous(), lens, ptable, cos, sin)
            assert torch.count_nonzero(got) == 0
        assert run(R, c, q[:0], kp, vp, table[:0], lens[:0], ptable, cos, sin).shape == (0, 8, 128)


def test_nan_keys_reach_their_sequence_only():
    require_gpu()
    R = lib()
    c = dict(lens=[33, 50, 64], prefix=40, Hq=4, Hk=2, D=64, rd=64, page=16, dtype="bf16", layout="split_half")
    q, kp, vp, table, lens, ptable = make(c, poison=False)
    cos, sin = S.tables(1e4, 64, 128)
    clean = run(R, c, q, kp, vp, table, lens, ptable, cos, sin)
    kp[int(table[1, 3]), :, 1] = float("nan")              # the last key of sequence 1
    got = run(R, c, q, kp, vp, table, lens, ptable, cos, sin)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2]) and got[1].isnan().all()


def test_refusals():
    require_gpu()
    R = lib()
    c = dict(lens=[33, 50], prefix=40, Hq=4, Hk=2, D=64, rd=64, page=16, dtype="bf16", layout="split_half")
    q, kp, vp, table, lens, ptable = (x.cuda() for x in make(c))
    cos, sin = (x.cuda() for x in S.tables(1e4, 64, 128))
    ok = dict(q=q, k_pages=kp, v_pages=vp, block_table=table, seq_lens=lens, prefix_table=ptable, prefix_len=40, cos=cos,
              sin=sin)
    for bad, err in [(dict(q=q.float()), TypeError), (dict(q=q.half()), ValueError), (dict(v_pages=vp[:2]), ValueError),
                     (dict(block_table=table[:1]), ValueError), (dict(seq_lens=lens.long()), ValueError),
                     (dict(prefix_len=49), ValueError), (dict(prefix_table=None), ValueError), (dict(prefix_len=-1), R.RopeError),
                     (dict(q=q[:, :3]), R.RopeError), (dict(out=q), R.RopeError), (dict(pos_q=table), ValueError),
                     (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), R.RopeError)]:
        with pytest.raises(err):
            R.attention_shared_prefix(**dict(ok, **bad))
    assert R.rope_check_errors() == R.ROPE_OK

"""attention_paged against the plain form in 64 bits, under the rule of the dense attention's tests
(attention_check.py: P is rounded to the element type before P V, o once).  Every row of a page that holds no
key holds NaN or infinities."""
import pytest
import torch

import attention_check as AC
import serving_ref as S
from gpu_util import lib, require_gpu
from test_gpu_cache_append import scattered_tables, starts

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def reference(q, kp, vp, table, cu, lens, cos, sin, pos_q=None, layout="split_half", causal=True, scale=None, rounded=False):
    """(o, w, a) [Tq, Hq, D] in fp64; rows of no sequence are NaN.  cos None: queries as they are.

    Rotated queries are rounded to their type, but for sequences of at most eight rows (token, head) per key head, whose
    products take them in two parts (rounded: those too, as the other attentions do)."""
    Tq, Hq, D = q.shape
    _, Hk, page, _ = kp.shape
    scale = D ** -0.5 if scale is None else scale
    out = [torch.full((Tq, Hq, D), torch.nan, dtype=torch.float64) for _ in range(3)]
    for b in range(len(lens)):
        q0, q1, n = int(cu[b]), int(cu[b + 1]), int(lens[b])
        Lq = q1 - q0
        if Lq == 0:
            continue
        blocks = table[b, :-(-n // page)].long()
        k, v = (x[blocks].double().transpose(0, 1).reshape(Hk, -1, D)[:, :n] for x in (kp, vp))
        if cos is None:
            qr = q[q0:q1].double()
        else:
            rows = range(n - Lq, n) if pos_q is None else [int(x) for x in pos_q[q0:q1]]
            if Lq * (Hq // Hk) <= 8 and not rounded:
                qr = torch.stack([S.rotate(q[q0 + i], r, cos, sin, layout) for i, r in enumerate(rows)])
            else:
                qr = S._rotated_rounded(q[q0:q1], rows, cos, sin, layout)
        seen = torch.ones(Lq, n, dtype=torch.bool)
        if causal:
            seen = torch.arange(n)[None] <= torch.arange(Lq)[:, None] + (n - Lq)
        for h in range(Hq):
            g = h // (Hq // Hk)
            for o, x in zip(out, S.softmax_rows(qr[:, h], k[g], v[g], seen, scale)):
                o[q0:q1, h] = x
    return out


def make(c, seed=5, first=0, behind=0):
    g = torch.Generator().manual_seed(seed)
    dt, page, kl = TYPES[c["dtype"]], c["page"], c["k"]
    table, n_pages = scattered_tables(kl, page, g)
    q = torch.randn(first + sum(c["q"]) + behind, c["Hq"], c["D"], generator=g).to(dt)
    kp = torch.randn(n_pages, c["Hk"], page, c["D"], generator=g).to(dt)
    vp = torch.randn(n_pages, c["Hk"], page, c["D"], generator=g).to(dt)
    for row, n in zip(table, kl):
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
    return q, kp, vp, table, starts(c["q"], first), torch.tensor(kl, dtype=torch.int32)


def run(R, q, kp, vp, table, cu, lens, cos, sin, status=0, **more):
    dev = lambda x: x.cuda() if isinstance(x, torch.Tensor) else x
    out = R.attention_paged(*(dev(x) for x in (q, kp, vp, table, cu, lens, cos, sin)), **{n: dev(x) for n, x in more.items()})
    assert R.rope_check_errors() == status
    return out.cpu()


def check(got, ref, c, what):
    AC.check(got.float().numpy(), *(x.numpy() for x in ref), c["dtype"], what)


def case(q, k, Hq, Hk, D, rd, page, dtype="bf16", layout="split_half"):
    return dict(q=q, k=k, Hq=Hq, Hk=Hk, D=D, rd=rd, page=page, dtype=dtype, layout=layout)


CASES = [
    case([1], [1], 4, 1, 128, 128, 16),
    case([1], [130], 2, 2, 64, 64, 64, "f16"),
    case([5], [5], 8, 2, 128, 128, 64),                                       # 20 rows: a tile
    case([2, 4, 3], [700, 4, 129], 16, 4, 128, 128, 32, "f16", "interleaved"),    # rows of up to 16, several tokens
    case([1, 0, 70, 1, 0, 16], [33, 64, 300, 0, 5, 16], 8, 2, 128, 128, 64),  # both kinds, empty ones, no keys
    case([9, 40], [3, 40], 6, 2, 64, 32, 32, "f16", "interleaved"),           # groups of 3, more tokens than keys
    case([300], [300], 4, 4, 64, 64, 16),                                     # a whole prompt, groups of 1
    case([129, 255, 257, 31], [129, 513, 300, 31], 8, 1, 128, 96, 128, "f16"),    # groups of 8
    case([1, 2, 3], [70, 40, 130], 48, 2, 128, 128, 64),                      # groups of 24: rows of 16 and 8, tiles
    case([1] * 5, [5, 17, 0, 64, 3], 32, 1, 64, 64, 16, "f16"),               # groups of 32
    case([40], [5000], 8, 2, 128, 128, 64),                                   # one long context: many pieces a unit
    case([33, 1, 1, 7, 60], [3000, 2500, 1, 900, 4000], 4, 1, 128, 64, 128, "f16", "interleaved"),
    case([(i * 7) % 5 for i in range(150)], [(i * 37) % 200 + 5 for i in range(150)], 8, 2, 64, 64, 16),
    case([(i * 53) % 90 for i in range(40)], [(i * 53) % 90 + (i * 31) % 300 for i in range(40)], 4, 2, 128, 128, 32),
    case([1] * 40, [(i * 61) % 400 + 1 for i in range(40)], 16, 2, 128, 128, 64, "f16"),
    case([8, 2, 9, 1, 5], [900, 2, 40, 1500, 70], 3, 3, 64, 48, 16, "f16", "interleaved"),     # rows up to eight and past
    case([1] * 30, [(i * 67) % 500 for i in range(30)], 24, 2, 64, 64, 16),   # groups of 12: 16-row pairs
    case([1] * 33, [(i * 67) % 500 for i in range(33)], 28, 2, 128, 128, 32, "f16"),          # groups of 14
    case([700], [2200], 3, 1, 64, 48, 64),                                    # groups of 3, many query tiles
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "n%d_q%d_k%d_Hq%d_Hk%d_D%d_p%d_%s" % (
    len(c["q"]), sum(c["q"]), sum(c["k"]), c["Hq"], c["Hk"], c["D"], c["page"], c["dtype"]))
@pytest.mark.parametrize("causal", [True, False])
def test_paged(c, causal):
    require_gpu()
    R = lib()
    x = make(c, first=2, behind=3)
    cos, sin = S.tables(1e4, c["rd"], max(c["k"]) + 1)
    status = R.ROPE_OK
    if not causal and any(a > b + 1 for a, b in zip(c["q"], c["k"])):
        # rows before the sequence's first key have no table row
        status = R.ROPE_ERR_POS_OUT_OF_RANGE
    ref = reference(*x, cos, sin, layout=c["layout"], causal=causal)
    dt = TYPES[c["dtype"]]
    out = torch.full(x[0].shape, 3.0, dtype=dt, device="cuda")
    got = run(R, *x, cos, sin, status, layout=c["layout"], causal=causal, out=out)
    n = got.shape[0]
    assert bool((got[:2] == 3).all()) and bool((got[n - 3:] == 3).all())
    check(got[2:n - 3], [r[2:n - 3] for r in ref], c, "paged %s %s" % ({k: v for k, v in c.items() if k not in "qk"}, causal))
    again = run(R, *x, cos, sin, status, layout=c["layout"], causal=causal)
    assert torch.equal(got[2:n - 3], again[2:n - 3])


def test_rotated_queries_positions_scale_and_strides():
    """Large scores, table rows of their own, queries rotated before, a strided view, a scale."""
    require_gpu()
    R = lib()
    c = case([3, 50, 1, 1], [150, 310, 290, 4], 8, 2, 128, 64, 16)
    q, kp, vp, table, cu, lens = make(c)
    ramp = torch.linspace(-3, 3, kp.shape[0])[torch.randperm(kp.shape[0], generator=torch.Generator().manual_seed(1))]
    kp = (kp.float() * torch.exp(ramp)[:, None, None, None]).to(kp.dtype)
    cos, sin = S.tables(1e4, 64, 60)
    pos = torch.randint(-1, 60, (q.shape[0],), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    fused = torch.cat([q, q, q], 1).cuda()
    ref = reference(q, kp, vp, table, cu, lens, cos, sin, pos_q=pos, scale=0.4)
    got = run(R, fused[:, 8:16], kp, vp, table, cu, lens, cos, sin, pos_q=pos, scale=0.4)
    check(got, ref, c, "paged positions")
    ref = reference(q, kp, vp, table, cu, lens, None, None, scale=0.4)
    got = run(R, fused[:, 8:16], kp, vp, table, cu, lens, None, None, scale=0.4)
    check(got, ref, c, "paged rotated before")
    # rows outside the table are not rotated, and reported
    bad = pos.clone()
    bad[1], bad[20], bad[54] = 60, -2, 2 ** 31 - 1
    as_is = bad.clone()
    as_is[[1, 20, 54]] = -1
    ref = reference(q, kp, vp, table, cu, lens, cos, sin, pos_q=as_is)
    check(run(R, q, kp, vp, table, cu, lens, cos, sin, R.ROPE_ERR_POS_OUT_OF_RANGE, pos_q=bad), ref, c, "paged bad positions")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_few_rows_lose_nothing_before_the_output(dtype):
    """At most eight rows a key head: rotated queries and P go into the products in two parts, so an output is within its
    one rounding of the exact one.  Besides: each part's own rounding, 2^-16 of a probability (fp16 2^-22, or 2^-25 of the
    largest where that is more) and of a score's terms, and fp32 arithmetic, 2^-14 in all of sum |p v| for scores below 30."""
    require_gpu()
    R = lib()
    c = case([1, 2, 1, 1], [2000, 700, 33, 129], 8, 2, 128, 128, 64, dtype)
    x = make(c)
    cos, sin = S.tables(1e4, 128, 2048)
    o, w, a = reference(*x, cos, sin)
    got = run(R, *x, cos, sin).double()
    half = torch.finfo(TYPES[dtype]).eps / 2
    bound = half * o.abs() * (1 + 2.0 ** -10) + 2.0 ** -14 * w + (2.0 ** -25 * a if dtype == "f16" else 0)
    assert ((got - o).abs() <= bound + 2.0 ** -25).all()


def test_shared_pages_and_the_other_attentions():
    """Forked sequences share pages; single tokens agree with attention_shared_prefix's, each within the rule."""
    require_gpu()
    R = lib()
    c = case([60, 1, 20], [60, 60, 60], 4, 2, 64, 64, 16, "f16")
    q, kp, vp, table, cu, lens = make(c)
    table[1] = table[0]
    table[2, :2] = table[0, :2]
    cos, sin = S.tables(1e4, 64, 128)
    check(run(R, q, kp, vp, table, cu, lens, cos, sin), reference(q, kp, vp, table, cu, lens, cos, sin), c, "paged shared pages")
    c = case([1] * 6, [5, 100, 37, 64, 1, 300], 8, 2, 128, 128, 64)
    q, kp, vp, table, cu, lens = make(c)
    cos, sin = S.tables(1e4, 128, 320)
    a = run(R, q, kp, vp, table, cu, lens, cos, sin)
    b = R.attention_shared_prefix(*(x.cuda() for x in (q, kp, vp, table, lens)), None, 0, cos.cuda(), sin.cuda()).cpu()
    ref = reference(q, kp, vp, table, cu, lens, cos, sin)
    check(a, ref, c, "paged single tokens")
    check(b, reference(q, kp, vp, table, cu, lens, cos, sin, rounded=True), c, "decode single tokens")


def test_bad_offsets_lengths_and_pages():
    require_gpu()
    R = lib()
    c = case([70, 1, 3], [300, 64, 129], 8, 2, 128, 128, 64)
    q, kp, vp, table, cu, lens = make(c)
    cos, sin = S.tables(1e4, 128, 400)
    want = run(R, q, kp, vp, table, cu, lens, cos, sin)
    for what in ("order", "end", "negative", "length", "long"):
        cb, lb = cu.clone(), lens.clone()
        if what == "order":
            cb[1], cb[2] = 72, 70
        elif what == "end":
            cb[3] = q.shape[0] + 1
        elif what == "negative":
            cb[0] = -1
        elif what == "length":
            lb[2] = -1
        else:
            lb[0] = table.shape[1] * 64 + 1
        out = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
        got = run(R, q, kp, vp, table, cb, lb, cos, sin, R.ROPE_ERR_BAD_INDEX, out=out)
        assert bool((got == 3).all()), what
    for b in range(3):
        for bad in (kp.shape[0], -5, 2 ** 31 - 1):
            tb = table.clone()
            tb[b, 0] = bad
            got = run(R, q, kp, vp, tb, cu, lens, cos, sin, R.ROPE_ERR_BAD_INDEX)
            for o in range(3):
                if o != b:
                    assert torch.equal(got[cu[o]:cu[o + 1]], want[cu[o]:cu[o + 1]])
    # entries behind a sequence's last page may be anything
    tb = torch.cat([table, torch.full((3, 2), 2 ** 31 - 1, dtype=torch.int32)], 1)
    for b in range(3):
        tb[b, -(-int(lens[b]) // 64):] = 12345678
    assert torch.equal(run(R, q, kp, vp, tb, cu, lens, cos, sin), want)


def test_nothing_to_attend():
    require_gpu()
    R = lib()
    c = case([3, 20], [0, 0], 4, 2, 64, 64, 16)
    q = torch.randn(23, 4, 64).bfloat16()
    cos, sin = S.tables(1e4, 64, 32)
    for pages in (0, 2):
        kp = torch.full((pages, 2, 16, 64), float("nan")).bfloat16()
        table = torch.zeros(2, 1 if pages else 0, dtype=torch.int32)
        got = run(R, q, kp, kp.clone(), table, starts(c["q"]), torch.zeros(2, dtype=torch.int32), cos, sin)
        assert not got.any()
    assert R.attention_paged(q[:0].cuda(), kp.cuda(), kp.cuda(), table[:0].cuda(), starts([]).cuda(), torch.zeros(0, dtype=torch.int32).cuda(),
                             cos.cuda(), sin.cuda()).shape == (0, 4, 64)


@pytest.mark.parametrize("c", CASES, ids=lambda c: "n%d_Hq%d_Hk%d_D%d_p%d" % (len(c["q"]), c["Hq"], c["Hk"], c["D"], c["page"]))
def test_nothing_behind_the_workspace(c):
    """A workspace of exactly the size asked for: what lies behind it stays, what lies in it beforehand does not matter."""
    require_gpu()
    R = lib()
    q, kp, vp, table, cu, lens = make(c)
    cos, sin = S.tables(1e4, c["rd"], max(c["k"]) + 8)
    size = R.rope_attention_paged_workspace(len(lens), q.shape[0], c["Hq"], c["Hk"], c["D"], c["page"], table.shape[1])
    more = dict(rotary_dim=c["rd"], layout=c["layout"])
    want = run(R, q, kp, vp, table, cu, lens, cos, sin, **more)
    for fill in (0, 0xff):
        big = torch.full((size + (1 << 20),), fill, dtype=torch.uint8, device="cuda")
        got = run(R, q, kp, vp, table, cu, lens, cos, sin, workspace=big[:size], **more)
        assert torch.equal(got, want) and bool((big[size:] == fill).all())


def test_many_sequences():
    """The most sequences a call takes, a few tokens each, chunks among them; one more is refused."""
    require_gpu()
    R = lib()
    n = 4096
    c = case([1 + (i % 97 == 0) * 6 for i in range(n)], [7 + (i * 11) % 12 for i in range(n)], 4, 1, 64, 64, 16)
    x = make(c)
    cos, sin = S.tables(1e4, 64, 32)
    check(run(R, *x, cos, sin), reference(*x, cos, sin), c, "paged 4096 sequences")
    q, kp, vp, table, cu, lens = x
    with pytest.raises(R.RopeError):
        run(R, q, kp, vp, torch.cat([table, table[:1]]), torch.cat([cu, cu[-1:]]), torch.cat([lens, lens[:1]]), cos, sin)


@pytest.mark.parametrize("Hq,Hk,D,page", [(8, 2, 128, 16), (6, 6, 64, 32), (16, 2, 128, 128), (3, 1, 64, 16)])
def test_short_sequences_among_long_ones(Hq, Hk, D, page):
    """Pairs of no, one and two chunks, of one to 16 rows, between long ones: runs that begin and end everywhere."""
    require_gpu()
    R = lib()
    G = Hq // Hk
    k = [(0, 1, 15, 16, 17, 700, 33, 2, 64, 3, 31, 1500)[i * 5 % 12] + (i % 3 == 0) for i in range(120)]
    q = [min(n, 1 + i * 7 % max(16 // G, 1)) if n else i % 2 for i, n in enumerate(k)]
    c = case(q, k, Hq, Hk, D, D, page)
    t = make(c)
    cos, sin = S.tables(1e4, D, 1600)
    want = reference(*t, cos, sin)
    got = run(R, *t, cos, sin)
    check(got, want, c, "short sequences")
    assert torch.equal(got, run(R, *t, cos, sin))


@pytest.mark.parametrize("normed", [False, True])
def test_prompt_in_chunks_then_single_tokens(normed):
    """A run as a program makes it: the tokens of two sequences appended and attended in steps of ragged chunks, then one by
    one; every step against the plain attention over what the cache holds, and the cache against one append of everything."""
    require_gpu()
    R = lib()
    Hq, Hk, D, page = 8, 2, 128, 16
    g = torch.Generator().manual_seed(9)
    lens = [0, 0]
    steps = [[100, 37], [0, 130], [90, 1], [1, 1], [1, 0], [1, 1]]
    total = [sum(s[b] for s in steps) for b in range(2)]
    c = dict(dtype="bf16")
    table, n_pages = scattered_tables(total, page, g)
    cos, sin = S.tables(1e4, D, 300)
    qkv = [torch.randn(t, Hq + 2 * Hk, D, generator=g).bfloat16() for t in total]
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
    kp, vp = (torch.full((n_pages, Hk, page, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dev = [x.cuda() for x in (cos, sin, table, wq, wk)]

    def step(new, kp, vp, old):
        x = torch.cat([qkv[b][old[b]:old[b] + new[b]] for b in range(2)]).cuda()
        cu = starts(new).cuda()
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
        have = torch.tensor(old, dtype=torch.int32).cuda()
        now = have + cu.diff()
        if normed:
            q = R.norm_cache_append(q, k, v, dev[3], dev[4], kp, vp, dev[2], cu, have, dev[0], dev[1])
            return q, R.attention_paged(q, kp, vp, dev[2], cu, now), cu, now
        R.cache_append(k, v, kp, vp, dev[2], cu, have, dev[0], dev[1])
        return q, R.attention_paged(q, kp, vp, dev[2], cu, now, dev[0], dev[1]), cu, now

    for new in steps:
        q, o, cu, now = step(new, kp, vp, lens)
        lens = [a + b for a, b in zip(lens, new)]
        ref = reference(q.cpu(), kp.cpu(), vp.cpu(), table, cu.cpu(), now.cpu(), *((None, None) if normed else (cos, sin)))
        check(o.cpu(), ref, c, "paged step")
    k2, v2 = (torch.full_like(x, float("nan")) for x in (kp, vp))
    step(total, k2, v2, [0, 0])
    assert torch.equal(kp.nan_to_num(7.0), k2.nan_to_num(7.0)) and torch.equal(vp.nan_to_num(7.0), v2.nan_to_num(7.0))
    assert R.rope_check_errors() == R.ROPE_OK


def test_captured_and_replayed():
    """Two captured calls that share a workspace, replayed with other lengths: the plan is made anew."""
    require_gpu()
    R = lib()
    c = case([1, 50, 2], [200, 130, 90], 8, 2, 128, 128, 32)
    x = make(c)
    cos, sin = S.tables(1e4, 128, 300)
    d = [t.cuda() for t in (*x, cos, sin)]
    ws = torch.empty(R.rope_attention_paged_workspace(3, 53, 8, 2, 128, 32, x[3].shape[1]), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs, graphs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            outs.append(R.attention_paged(*d, workspace=ws))
    for cu, lens in (([0, 1, 51, 53], [200, 130, 90]), ([0, 30, 33, 53], [64, 100, 20]), ([0, 0, 0, 1], [0, 0, 90])):
        d[4].copy_(torch.tensor(cu))
        d[5].copy_(torch.tensor(lens))
        for o, gr in zip(outs, graphs):
            o.fill_(5.0)
            gr.replay()
        torch.cuda.synchronize()
        ref = reference(*x[:4], cu, lens, cos, sin)
        for o in outs:
            check(o[:cu[-1]].cpu(), [r[:cu[-1]] for r in ref], c, "paged replay")
            assert bool((o[cu[-1]:] == 5).all())
    assert R.rope_check_errors() == R.ROPE_OK


def test_streams_threads_of_work():
    """Calls on another stream, and calls of two streams at once, each with its own workspace."""
    require_gpu()
    R = lib()
    c = case([1, 150, 2], [2000, 1300, 900], 8, 2, 128, 128, 32)
    d = [t.cuda() for t in (*make(c), *S.tables(1e4, 128, 2048))]
    want = R.attention_paged(*d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        a, b = R.attention_paged(*d), R.attention_paged(*d, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want)
    assert R.rope_check_errors() == R.ROPE_OK


def test_pages_at_the_end_of_a_large_pool():
    require_gpu()
    R = lib()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    c = case([1, 60, 3], [200, 130, 90], 8, 8, 128, 128, 64)
    q, kp, vp, table, cu, lens = make(c)
    cos, sin = S.tables(1e4, 128, 300)
    want = run(R, q, kp, vp, table, cu, lens, cos, sin)
    big = [torch.empty(40000, 8, 64, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert big[0].numel() > 1 << 31
    for b, s in zip(big, (kp, vp)):
        b[-s.shape[0]:] = s.cuda()
    tb = torch.where(table >= 0, table + 40000 - kp.shape[0], table)
    got = run(R, q, big[0], big[1], tb, cu, lens, cos, sin)
    assert torch.equal(got, want)


def test_refusals():
    require_gpu()
    R = lib()
    c = case([1, 20], [30, 40], 4, 2, 64, 64, 16)
    q, kp, vp, table, cu, lens = (t.cuda() for t in make(c))
    cos, sin = (t.cuda() for t in S.tables(1e4, 64, 64))
    ok = dict(q=q, k_pages=kp, v_pages=vp, block_table=table, cu_seqlens_q=cu, seq_lens=lens, cos=cos, sin=sin)
    for bad, err, says in [
            (dict(q=q.float()), TypeError, "bf16 or fp16"), (dict(q=q.cpu()), ValueError, "CUDA"), (dict(q=q[:, :, :32]), ValueError, "features"),
            (dict(v_pages=vp[:1]), ValueError, "one shape"), (dict(k_pages=kp.half(), v_pages=vp.half()), ValueError, "k_pages"),
            (dict(block_table=table[0]), ValueError, "block_table"), (dict(block_table=table.long()), ValueError, "block_table"),
            (dict(cu_seqlens_q=cu[:2]), ValueError, "cu_seqlens_q"), (dict(seq_lens=lens[:1]), ValueError, "seq_lens"),
            (dict(sin=None), ValueError, "together"), (dict(cos=cos[:0], sin=sin[:0]), ValueError, "rows"), (dict(rotary_dim=32), ValueError, "rotary_dim"),
            (dict(pos_q=lens), ValueError, "pos_q"), (dict(out=q[:3]), ValueError, "out must be"), (dict(out=q), R.RopeError, None),
            (dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")), R.RopeError, None),
            (dict(scale=float("nan")), R.RopeError, None), (dict(q=q[:, :3]), R.RopeError, None)]:
        with pytest.raises(err, match=says):
            R.attention_paged(**dict(ok, **bad))
    out = torch.empty_like(q)
    v = out._version
    assert R.attention_paged(**ok, out=out) is out and out._version == v + 1
    assert not R.attention_paged(**dict(ok, q=q.clone().requires_grad_())).requires_grad
    assert R.rope_check_errors() == R.ROPE_OK

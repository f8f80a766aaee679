"""More operators of the rotary framework: what they compute, in plain torch, and the cases they are timed on.

Four operators that a model with normalised queries and keys trains and serves with: the RMS norm of every query and key head with
the rotation in the same pass, forward and backward (``norm_rotate_qk`` and its autograd form), the same before new keys and values
enter a paged cache (``norm_cache_append``), the attention of each sequence's new tokens -- one, or a chunk of a prompt -- over its
paged cache (``attention_paged``), and the cos/sin tables of contexts longer than those trained on (``build_tables_scaled``).
With ``own`` false every operator is computed from elementary torch operations in 32 bits (angles and sums over all tokens in 64),
rounded once at the end.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
THETA = 5e5
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------------------
# cases


def _lens(text):
    return [int(x) for x in text.split(",")]


def _text(lens):
    return ",".join(str(int(x)) for x in lens)


def _norm(name, B, S, Hq, Hk, D, rd, dtype, wtype, layout, seq_first, fused, positions, train):
    return {"name": name, "op": "norm", "B": B, "S": S, "Hq": Hq, "Hk": Hk, "D": D, "rd": rd, "dtype": dtype, "wtype": wtype,
            "layout": layout, "seq_first": seq_first, "fused": fused, "positions": positions, "train": train}


def _append(name, new, old, Hq, Hk, D, rd, page, dtype, wtype, layout, fused):
    return {"name": name, "op": "append", "new": _text(new), "old": _text(old), "Hq": Hq, "Hk": Hk, "D": D, "rd": rd, "page": page,
            "dtype": dtype, "wtype": wtype, "layout": layout, "fused": fused}


def _paged(name, q_lens, k_lens, Hq, Hk, D, rd, page, dtype, layout, rotate, fused):
    return {"name": name, "op": "paged", "q_lens": _text(q_lens), "k_lens": _text(k_lens), "Hq": Hq, "Hk": Hk, "D": D, "rd": rd,
            "page": page, "dtype": dtype, "layout": layout, "rotate": rotate, "fused": fused}


def _table(name, kind, rows, rd, factor, original, offset):
    return {"name": name, "op": "table", "kind": kind, "rows": rows, "rd": rd, "factor": factor, "original": original, "offset": offset}


def _spread(n, lo, hi, step):
    """n lengths spread over lo .. hi in a fixed, unsorted order."""
    return [lo + (i * step) % (hi - lo + 1) for i in range(n)]


def listed():
    return [
        # a short prompt, read from its fused projection: the latency of one small call
        _norm("norm_prompt_37", 1, 37, 32, 8, 128, 128, "bf16", "bf16", "split_half", True, True, False, False),
        # a training step of a Llama-3-8B-shaped layer, gradients of the inputs and of both weights
        _norm("norm_train_4x4096", 4, 4096, 32, 8, 128, 128, "bf16", "bf16", "split_half", False, False, False, True),
        # training in fp32 on padded batches of odd length: equal heads of width 64, a partial rotary span, positions of its own for
        # every sequence
        _norm("norm_train_f32_d64", 6, 1027, 16, 16, 64, 32, "f32", "f32", "interleaved", True, False, True, True),
        # one decode step of 64 sequences: one token each
        _append("norm_append_step_b64", [1] * 64, _spread(64, 1, 4000, 1237), 32, 8, 128, 128, 64, "bf16", "bf16", "split_half", True),
        # the prompts that arrived since the last step
        _append("norm_append_prompts_16k", [4096, 1333, 2048, 777, 3500, 96, 2900, 1634], [0, 5, 0, 100, 33, 0, 1, 64], 32, 8, 128, 128,
                64, "f16", "f32", "split_half", True),
        # a handful of users, one of them with the rest of a prompt: latency
        _paged("paged_few", [1, 1, 21, 1], [533, 64, 300, 1025], 32, 8, 128, 128, 64, "bf16", "split_half", True, True),
        # the ordinary decode step: single tokens after contexts of up to 8k
        _paged("paged_step_b64", [1] * 64, _spread(64, 100, 8192, 2533), 32, 8, 128, 128, 64, "bf16", "split_half", True, False),
        # drafted tokens checked five at a time: equal heads of width 64, small pages, in fp16; some sequences wait
        _paged("paged_draft_d64_f16", [5, 5, 0, 5, 3, 5, 5, 1] * 5, _spread(40, 8, 3000, 1171), 16, 16, 64, 32, 16, "f16", "interleaved", True,
               False),
        # the step that a scheduler fills up: the rest of two prompts and a question about a long document beside 48 decoding
        # sequences, queries rotated before
        _paged("paged_mixed", [1] * 24 + [1500] + [1] * 24 + [547, 60],
               _spread(24, 100, 4096, 1531) + [9001] + _spread(24, 50, 5000, 977) + [547, 65536], 32, 8, 128, 128, 64, "bf16", "split_half",
               False, True),
        # a large chunk in the middle of a long document
        _paged("paged_chunk_8k", [8192], [24576], 32, 8, 128, 128, 128, "bf16", "split_half", True, False),
        # the rows of the next few steps, of a table that grows with the text: latency
        _table("table_ntk_64_rows", "ntk", 64, 64, 4.0, 4096, 20011),
        # the table of a context of 128k for a model trained on 8k
        _table("table_smooth_128k", "smooth", 131072, 128, 8.0, 8192, 0),
    ]


_MOST = {"norm": (1e12, 2.4e9), "append": (1e12, 6e8), "paged": (3.6e12, 1.1e9), "table": (1e12, 5.4e8)}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        D = rng.choice([64, 128, 128])
        rd = rng.choice([16, 32, 48, 64] if D == 64 else [32, 64, 96, 128, 128])
        Hk = rng.choice([1, 2, 4, 8, 8, 16])
        Hq = Hk * rng.choice([1, 2, 3, 4, 4, 5, 8])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        common = {"Hq": Hq, "Hk": Hk, "D": D, "rd": rd, "dtype": dtype, "layout": rng.choice(["split_half", "split_half", "interleaved"])}
        op = rng.choice(["norm", "append", "paged", "paged", "table"])
        if op == "norm":
            if rng.random() < 0.4:
                D = common["D"] = rng.choice([32, 80, 96, 256])
                common["rd"] = rng.choice([16, 32, D])
            common["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
            seq_first = rng.random() < 0.5
            case = _norm("", _log(rng, 1, 16), _log(rng, 1, 16384), wtype=rng.choice([common["dtype"], "f32"]), seq_first=seq_first,
                         fused=seq_first and rng.random() < 0.5, positions=rng.random() < 0.3, train=rng.random() < 0.6, **common)
        elif op == "append":
            n, top = _log(rng, 1, 256), _log(rng, 1, 16384)
            case = _append("", [_log(rng, 1, top) for _ in range(n)], [rng.randrange(0, 300) for _ in range(n)], page=rng.choice([16, 32, 64, 128]),
                           wtype=rng.choice([dtype, "f32"]), fused=rng.random() < 0.5, **common)
        elif op == "paged":
            n, top = _log(rng, 1, 128), _log(rng, 16, 65536)
            k_lens = [_log(rng, 1, top) for _ in range(n)]
            some = rng.choice([0.0, 0.1, 1.0])                        # how many of the sequences have more than one new token
            longest = _log(rng, 1, 4096)
            q_lens = [min(k, _log(rng, 1, longest)) if rng.random() < some else 1 for k in k_lens]
            if n > 1 and rng.random() < 0.3:
                q_lens[rng.randrange(n)] = 0
            if sum(q_lens) == 0:
                continue
            case = _paged("", q_lens, k_lens, page=rng.choice([16, 32, 64, 128]), rotate=rng.random() < 0.7, fused=rng.random() < 0.5, **common)
        else:
            case = _table("", rng.choice(["linear", "ntk", "smooth", "yarn"]), _log(rng, 1, 1048576), rng.choice([16, 32, 64, 96, 128, 128, 256]),
                          rng.choice([2.0, 4.0, 8.0, 20.0, 32.0]), rng.choice([2048, 4096, 8192, 32768]), rng.choice([0, 0, _log(rng, 1, 1000000)]))
        w = work(case)
        if w["flops"] <= _MOST[op][0] and w["bytes"] <= _MOST[op][1]:
            del case["name"]
            return case


def work(case):
    if case["op"] == "table":
        n = case["rows"] * case["rd"] // 2
        return {"bytes": 8 * n, "flops": 40 * n}
    D, Hq, Hk = case["D"], case["Hq"], case["Hk"]
    wide = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n = case["B"] * case["S"] * (Hq + Hk) * D
        # forward: a row read, a row written; backward: the row and its gradient read, a gradient written
        return {"bytes": wide * n * (5 if case["train"] else 2) + 4 * case["S"] * case["rd"], "flops": n * (24 if case["train"] else 8)}
    if case["op"] == "append":
        t = sum(_lens(case["new"]))
        return {"bytes": wide * D * t * (2 * Hq + 4 * Hk), "flops": 8 * D * (Hq + Hk) * t}
    ql, kl = _lens(case["q_lens"]), _lens(case["k_lens"])
    keys = sum(b for a, b in zip(ql, kl) if a > 0)
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(ql, kl))       # row i sees b - a + i + 1 keys
    return {"bytes": 2 * D * (2 * Hk * keys + 2 * Hq * sum(ql)), "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------------------------------------------------------------
# what a program has in hand


def _tables(rd, rows):
    """cos and sin [rows, rd / 2] in fp32, from angles in 64 bits."""
    w = THETA ** (-2.0 * torch.arange(rd // 2, dtype=torch.float64, device="cuda") / rd)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * w
    return a.cos().float(), a.sin().float()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(lens):
    return _ints([0] + list(torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist()))


def _pages(gen, counts, page):
    """Block lists for sequences of the given numbers of tokens, on scattered pages: [n, most] (unused entries -1), and the pages in all."""
    need = [-(-c // page) for c in counts]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(counts), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def prepare(case, seed):
    s = dict(case)
    if case["op"] == "table":
        # a table has no input but its numbers: the base varies a little with the seed
        s["theta"] = THETA * (1 + (seed % 1009) / 4096)
        return s
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, wt, D, Hq, Hk = TYPES[case["dtype"]], TYPES[case.get("wtype", "f32")], case["D"], case["Hq"], case["Hk"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    if case["op"] in ("norm", "append"):
        # trained weights lie about one
        s["wq"], s["wk"] = ((1 + 0.25 * torch.randn(D, generator=gen, device="cuda")).to(wt) for _ in range(2))
    if case["op"] == "norm":
        B, S = case["B"], case["S"]
        if case["fused"]:
            # one projection's output: a token's query heads, key heads and value heads lie side by side
            qkv = 2 * normal(B, S, Hq + 2 * Hk, D)
            q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        elif case["seq_first"]:
            q, k = 2 * normal(B, S, Hq, D), 2 * normal(B, S, Hk, D)
        else:
            q, k = 2 * normal(B, Hq, S, D), 2 * normal(B, Hk, S, D)
        s["q"], s["k"] = q, k
        s["pos"], rows = None, S
        if case["positions"]:
            # left-padded batches: the padding (-1) is not rotated, the rest counts from zero
            pad = torch.randint(0, S // 4 + 1, (B, 1), generator=gen, device="cuda")
            s["pos"] = (torch.arange(S, device="cuda") - pad).clamp(min=-1).to(torch.int32)
        s["cos"], s["sin"] = _tables(case["rd"], rows)
        if case["train"]:
            s["gq"], s["gk"] = normal(*q.shape), normal(*k.shape)
            for n in ("q", "k", "wq", "wk"):
                s[n].requires_grad_(True)
    elif case["op"] == "append":
        new, old = _lens(case["new"]), _lens(case["old"])
        table, total = _pages(gen, [a + b for a, b in zip(new, old)], case["page"])
        if case["fused"]:
            qkv = normal(sum(new), Hq + 2 * Hk, D)
            s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        else:
            s["q"], s["k"], s["v"] = normal(sum(new), Hq, D), normal(sum(new), Hk, D), normal(sum(new), Hk, D)
        s["k_pages"], s["v_pages"] = normal(total, Hk, case["page"], D), normal(total, Hk, case["page"], D)
        s |= {"table": table, "cu": _starts(new), "old": _ints(old)}
        s["cos"], s["sin"] = _tables(case["rd"], max(a + b for a, b in zip(new, old)))
    else:
        ql, kl = _lens(case["q_lens"]), _lens(case["k_lens"])
        s["table"], total = _pages(gen, kl, case["page"])
        s["k_pages"], s["v_pages"] = normal(total, Hk, case["page"], D), normal(total, Hk, case["page"], D)
        s["q"] = normal(sum(ql), Hq + 2 * Hk, D)[:, :Hq] if case["fused"] else normal(sum(ql), Hq, D)
        s |= {"cu": _starts(ql), "lens": _ints(kl), "q_lens": ql, "k_lens": kl, "cos": None, "sin": None}
        if case["rotate"]:
            s["cos"], s["sin"] = _tables(case["rd"], max(kl))
    return s


# ---------------------------------------------------------------------------------------------------------------------
# the plain forms


def _rotate(x, cos, sin, layout):
    """x [..., D] in 32 bits, cos and sin [..., rd / 2]: the first rd features rotated, the rest as they are."""
    h = cos.shape[-1]
    out = x.clone()
    if layout == "split_half":
        a, b = x[..., :h], x[..., h:2 * h]
        out[..., :h], out[..., h:2 * h] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        out[..., 0:2 * h:2], out[..., 1:2 * h:2] = a * cos - b * sin, a * sin + b * cos
    return out


def _at_rows(cos, sin, row):
    """Values of the given table rows; row -1 turns nothing."""
    none = (row < 0)[..., None]
    row = row.long().clamp(min=0)
    return torch.where(none, 1.0, cos[row]), torch.where(none, 0.0, sin[row])


def _plain_norm(s):
    S = s["S"]
    row = torch.arange(S, device="cuda") if s["pos"] is None else s["pos"]
    cos, sin = _at_rows(s["cos"], s["sin"], row)                      # [S, h] or [B, S, h]
    if row.dim() == 1:
        cos, sin = cos[None], sin[None]
    head = 2 if s["seq_first"] else 1
    cos, sin = cos.unsqueeze(head), sin.unsqueeze(head)
    outs, grads, weights = [], [], []
    with torch.no_grad():
        for x, w, g in ((s["q"], s["wq"], s.get("gq")), (s["k"], s["wk"], s.get("gk"))):
            xf, wf = x.float(), w.float()
            r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
            n = xf * r
            outs.append(_rotate(n * wf, cos, sin, s["layout"]).to(x.dtype))
            if s["train"]:
                gy = _rotate(g.float(), cos, -sin, s["layout"])       # the rotation's transpose is the one by the negated angle
                weights.append((gy * n).flatten(0, 2).sum(0, dtype=torch.float64).to(w.dtype))
                gn = gy * wf
                grads.append((r * (gn - n * (gn * n).mean(-1, keepdim=True))).to(x.dtype))
    return tuple(outs + grads + weights)


def _plain_append(s):
    cu = s["cu"].long()
    tok = torch.arange(s["k"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:], tok, right=True)
    slot = s["old"].long()[seq] + tok - cu[seq]
    cos, sin = s["cos"][slot][:, None], s["sin"][slot][:, None]

    def norm(x, w):
        x = x.float()
        return _rotate(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float(), cos, sin, s["layout"]).to(s["v"].dtype)

    page = s["k_pages"].shape[2]
    where = s["table"].long()[seq, slot // page]
    s["k_pages"][where, :, slot % page] = norm(s["k"], s["wk"])
    s["v_pages"][where, :, slot % page] = s["v"]
    return norm(s["q"], s["wq"]), s["k_pages"], s["v_pages"]


def _plain_paged(s):
    Tq, Hq, D = s["q"].shape
    _, Hk, page, _ = s["k_pages"].shape
    G = Hq // Hk
    cu, lens = s["cu"].long(), s["lens"].long()
    out = torch.empty((Tq, Hq, D), dtype=s["q"].dtype, device="cuda")
    for a in sorted(set(s["q_lens"]) - {0}):                          # sequences with equally many new tokens, padded to the longest of them
        some = [b for b, n in enumerate(s["q_lens"]) if n == a]
        ids = torch.tensor(some, device="cuda")
        most = max(1, -(-max(s["k_lens"][b] for b in some) // page))
        i = torch.arange(a, device="cuda")
        at = cu[ids][:, None] + i                                     # [n, a]
        q = s["q"][at].float()
        if s["cos"] is not None:
            row = (lens[ids] - a)[:, None] + i
            q = _rotate(q, s["cos"][row][:, :, None], s["sin"][row][:, :, None], s["layout"])
        seen = torch.arange(most * page, device="cuda") <= (lens[ids] - a)[:, None, None] + i[:, None]      # [n, a, keys]
        pages = s["table"][ids, :most].long().clamp(min=0)
        live = torch.arange(most * page, device="cuda") < lens[ids][:, None]
        for h in range(Hk):                                           # a key head at a time: the scores of all would be tens of GB
            k = s["k_pages"][:, h][pages].float().flatten(1, 2)
            v = s["v_pages"][:, h][pages].float().flatten(1, 2).masked_fill(~live[..., None], 0.0)
            x = q[:, :, h * G:(h + 1) * G].transpose(1, 2) @ k[:, None].transpose(-1, -2) / math.sqrt(D)    # [n, G, a, keys]
            x = x.masked_fill(~seen[:, None], -math.inf)
            p = torch.exp(x - x.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            out[at, h * G:(h + 1) * G] = (p @ v[:, None]).transpose(1, 2).to(out.dtype)
    return out


def _plain_table(s):
    rd, theta, factor, first = s["rd"], s["theta"], s["factor"], s["original"]
    i = torch.arange(rd // 2, dtype=torch.float64, device="cuda")
    w, scale = theta ** (-2.0 * i / rd), 1.0
    if s["kind"] == "linear":
        w = w / factor
    elif s["kind"] == "ntk":
        w = (theta * factor ** (rd / (rd - 2))) ** (-2.0 * i / rd)
    elif s["kind"] == "smooth":
        turns = first * w / (2 * math.pi)                             # of a pair over the trained context
        mix = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        w = (1 - mix) * w / factor + mix * w
    else:
        def pair(turns):
            return rd * math.log(first / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rd - 1)
        mix = ((i - lo) / (hi - lo if hi > lo else 0.001)).clamp(0, 1)
        w = w / factor * mix + w * (1 - mix)
        scale = 0.1 * math.log(factor) + 1.0
    angle = (s["offset"] + torch.arange(s["rows"], dtype=torch.float64, device="cuda"))[:, None] * w
    return (scale * angle.cos()).float(), (scale * angle.sin()).float()


def run(state):
    s = state
    if own:
        import rotary_position_embedding_rope_gb300 as R
        from rotary_position_embedding_rope_gb300 import autograd

        if s["op"] == "norm":
            args = (s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"])
            more = {"eps": EPS, "pos_idx": s["pos"], "layout": s["layout"], "seq_before_head": s["seq_first"]}
            if not s["train"]:
                return R.norm_rotate_qk(*args, **more)
            out = autograd.norm_rotary_qk(*args, **more)
            return tuple(x.detach() for x in out) + torch.autograd.grad(out, args[:4], (s["gq"], s["gk"]))
        if s["op"] == "append":
            q = R.norm_cache_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["old"],
                                    s["cos"], s["sin"], eps=EPS, layout=s["layout"])
            return q, s["k_pages"], s["v_pages"]
        if s["op"] == "paged":
            return R.attention_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"], s["cos"], s["sin"],
                                     layout=s["layout"])
        return R.build_tables_scaled(s["kind"], s["rd"], s["rows"], s["factor"], s["original"], theta=s["theta"], pos_offset=s["offset"])
    return {"norm": _plain_norm, "append": _plain_append, "paged": _plain_paged, "table": _plain_table}[s["op"]](s)


# ---------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits


def _turn(x, z, rd, layout):
    """x [..., D] in 64 bits as complex pairs, multiplied by z [..., rd / 2]."""
    r = x[..., :rd]
    pair = r.unflatten(-1, (2, rd // 2)).transpose(-1, -2) if layout == "split_half" else r.unflatten(-1, (rd // 2, 2))
    y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    y = (y.transpose(-1, -2) if layout == "split_half" else y).flatten(-2)
    return torch.cat([y, x[..., rd:]], -1)


def _unit(x, w):
    """x over the root of its mean square, weighted."""
    return w * x / torch.sqrt(torch.linalg.vecdot(x, x)[..., None] / x.shape[-1] + EPS)


def _exact_norm(case, s):
    z = torch.complex(s["cos"].double(), s["sin"].double())
    row = torch.arange(case["S"], device="cuda").expand(case["B"], -1) if s["pos"] is None else s["pos"]
    outs, grads, weights = [], [], []
    for x, w, g in ((s["q"], s["wq"], s.get("gq")), (s["k"], s["wk"], s.get("gk"))):
        H = x.shape[2 if case["seq_first"] else 1]
        out, dx = torch.empty(x.shape, dtype=torch.float64, device="cuda"), torch.empty(x.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(case["D"], dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            zb = z[row[b].long().clamp(min=0)].clone()
            zb[row[b] < 0] = 1
            for h in range(H):
                at = (b, slice(None), h) if case["seq_first"] else (b, h)
                xs, ws = x[at].detach().double().requires_grad_(case["train"]), w.detach().double().requires_grad_(case["train"])
                y = _turn(_unit(xs, ws), zb, case["rd"], case["layout"])
                out[at] = y.detach()
                if case["train"]:
                    gx, gw = torch.autograd.grad(y, (xs, ws), g[at].double())
                    dx[at] = gx
                    dw += gw
        outs.append(out)
        grads.append(dx)
        weights.append(dw)
    return tuple(outs + grads + weights) if case["train"] else tuple(outs)


def _exact_append(case, s):
    z = torch.complex(s["cos"].double(), s["sin"].double())
    q_out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    k_out, v_out, at, page = s["k_pages"].double(), s["v_pages"].double(), 0, case["page"]
    for b, (n, old) in enumerate(zip(_lens(case["new"]), _lens(case["old"]))):
        p = torch.arange(old, old + n, device="cuda")
        mine = slice(at, at + n)
        q_out[mine] = _turn(_unit(s["q"][mine].double(), s["wq"].double()), z[p][:, None], case["rd"], case["layout"])
        blocks = s["table"][b].long()[torch.div(p, page, rounding_mode="floor")]
        k_out[blocks, :, p % page] = _turn(_unit(s["k"][mine].double(), s["wk"].double()), z[p][:, None], case["rd"], case["layout"])
        v_out[blocks, :, p % page] = s["v"][mine].double()
        at += n
    return q_out, k_out, v_out


def _exact_paged(case, s):
    Hk, G, D, page = case["Hk"], case["Hq"] // case["Hk"], case["D"], case["page"]
    out, at = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b, (a, n) in enumerate(zip(s["q_lens"], s["k_lens"])):
        blocks = s["table"][b, :-(-n // page)].long()
        k, v = (x[blocks].double().transpose(0, 1).reshape(Hk, -1, D)[:, :n] for x in (s["k_pages"], s["v_pages"]))
        for r in range(0, a, 512):
            m = min(512, a - r)
            i = torch.arange(r, r + m, device="cuda")
            q = s["q"][at + r:at + r + m].double()
            if case["rotate"]:
                z = torch.complex(s["cos"][n - a + i].double(), s["sin"][n - a + i].double())
                q = _turn(q, z[:, None], case["rd"], case["layout"])
            e = n - a + r + m                                         # keys that the last of these rows sees
            x = torch.einsum("mhgd,hkd->hgmk", q.view(m, Hk, G, D), k[:, :e]) * D ** -0.5
            x = torch.where(torch.arange(e, device="cuda") <= n - a + i[:, None], x, -math.inf)
            out[at + r:at + r + m] = torch.einsum("hgmk,hkd->mhgd", torch.softmax(x, -1), v[:, :e]).reshape(m, -1, D)
        at += a
    return out


def _exact_table(case, s):
    rd, base, stretch = case["rd"], math.log(s["theta"]), case["factor"]
    speeds, scale = [], 1.0
    for i in range(rd // 2):
        w = math.exp(-2 * i * base / rd)
        if case["kind"] == "linear":
            w /= stretch
        elif case["kind"] == "ntk":
            w = math.exp(-2 * i / rd * (base + rd / (rd - 2) * math.log(stretch)))
        elif case["kind"] == "smooth":
            wave = 2 * math.pi / w
            if wave > case["original"]:
                w /= stretch
            elif wave >= case["original"] / 4:
                part = (case["original"] / wave - 1) / 3
                w = w * part + w / stretch * (1 - part)
        else:
            lo, hi = (rd / 2 * math.log(case["original"] / (2 * math.pi * t)) / base for t in (32, 1))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rd - 1)
            part = min(max((i - lo) / (hi - lo if hi > lo else 0.001), 0), 1)
            w = w * (1 - part) + w / stretch * part
            scale = 1 + math.log(stretch) / 10
        speeds.append(w)
    p = torch.arange(case["offset"], case["offset"] + case["rows"], dtype=torch.float64, device="cuda")
    z = torch.polar(torch.full((), scale, dtype=torch.float64, device="cuda"),
                    torch.outer(p, torch.tensor(speeds, dtype=torch.float64, device="cuda")))
    return z.real.contiguous(), z.imag.contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    if work(case)["flops"] > 5e12:
        return None
    return {"norm": _exact_norm, "append": _exact_append, "paged": _exact_paged, "table": _exact_table}[case["op"]](case, s)

"""Serving operators of the rotary framework: what they compute, in plain torch, and the cases they are timed on.

Three operators that a serving program runs one after the other: attention over packed prompts of different lengths
(``attention_packed``), writing new keys, rotated, and values into a paged cache (``cache_append``), and the attention of one
new token per sequence over a prefix that all sequences share and a suffix of their own (``attention_shared_prefix``).
With ``own`` false every operator is computed from elementary torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
THETA = 5e5


# ---------------------------------------------------------------------------------------------------------------------
# cases


def _lens(text):
    return [int(x) for x in text.split(",")]


def _text(lens):
    return ",".join(str(int(x)) for x in lens)


def _packed(name, q_lens, k_lens, Hq, Hk, D, rd, dtype, layout, causal, fused):
    return {"name": name, "op": "packed", "q_lens": _text(q_lens), "k_lens": _text(k_lens), "Hq": Hq, "Hk": Hk, "D": D, "rd": rd,
            "dtype": dtype, "layout": layout, "causal": causal, "fused": fused}


def _append(name, new, old, Hk, D, rd, page, dtype, layout, offset, fused):
    return {"name": name, "op": "append", "new": _text(new), "old": _text(old), "Hk": Hk, "D": D, "rd": rd, "page": page,
            "dtype": dtype, "layout": layout, "offset": offset, "fused": fused}


def _decode(name, prefix, lens, Hq, Hk, D, rd, page, dtype, layout):
    return {"name": name, "op": "decode", "prefix": prefix, "lens": _text(lens), "Hq": Hq, "Hk": Hk, "D": D, "rd": rd, "page": page,
            "dtype": dtype, "layout": layout}


def _spread(n, lo, hi, step):
    """n lengths spread over lo .. hi in a fixed, unsorted order."""
    return [lo + (i * step) % (hi - lo + 1) for i in range(n)]


def listed():
    return [
        # a few chat turns that arrive together: the latency of one small call
        _packed("packed_short_chat", [17, 301, 1, 128, 64, 5, 211, 90], [17, 301, 1, 128, 64, 5, 211, 90], 32, 8, 128, 128, "bf16",
                "split_half", True, True),
        # an ordinary prompt batch of a Llama-3-8B-shaped layer, read from its fused projection
        _packed("packed_prompts_16k", [4096, 1333, 2048, 777, 3500, 96, 2900, 1634], [4096, 1333, 2048, 777, 3500, 96, 2900, 1634], 32, 8,
                128, 128, "bf16", "split_half", True, True),
        # long documents among short prompts, the last third of each given (the first two thirds were seen earlier)
        _packed("packed_long_chunked", [5461, 200, 3001, 1024, 50], [16384, 600, 9003, 4096, 150], 32, 8, 128, 128, "bf16", "split_half",
                True, False),
        # equal heads of width 64 with a partial rotary span, no causal mask: encoder-like batches, in fp16
        _packed("packed_d64_f16", _spread(24, 300, 1026, 331), _spread(24, 300, 1026, 331), 16, 16, 64, 32, "f16", "interleaved", False,
                False),
        # one decode step of 64 sequences: one token each
        _append("append_step_b64", [1] * 64, _spread(64, 1, 4000, 1237), 8, 128, 128, 64, "bf16", "split_half", 8192, True),
        # the packed prompts above
        _append("append_prompts_16k", [4096, 1333, 2048, 777, 3500, 96, 2900, 1634], [0, 5, 0, 100, 33, 0, 1, 64], 8, 128, 128, 64,
                "bf16", "split_half", 0, True),
        # equal heads, interleaved pairs, small pages, many sequences
        _append("append_f16_mha_32k", _spread(40, 1, 1640, 701), _spread(40, 0, 50, 7), 32, 128, 96, 16, "f16", "interleaved", 100, False),
        # a handful of users of one system prompt: latency
        _decode("decode_b4_prefix_500", 500, [33, 1, 120, 64], 32, 8, 128, 128, 64, "bf16", "split_half"),
        # the ordinary step: 64 sequences after a long instruction
        _decode("decode_b64_prefix_8k", 8192, _spread(64, 100, 1500, 533), 32, 8, 128, 128, 64, "bf16", "split_half"),
        # questions about one very long document
        _decode("decode_b32_prefix_128k", 131072, _spread(32, 1, 600, 211), 32, 8, 128, 128, 128, "bf16", "split_half"),
        # a full batch: the prefix is a matrix product of 1024 rows for each key head, the suffixes are 2 GB
        _decode("decode_b256_prefix_4k", 4001, _spread(256, 64, 4096, 1531), 32, 8, 128, 128, 64, "bf16", "split_half"),
        # equal heads of width 64, small pages, short suffixes with empty ones among them, in fp16
        _decode("decode_b48_d64_f16", 1026, _spread(48, 0, 900, 337), 16, 16, 64, 32, 16, "f16", "interleaved"),
    ]


_MOST = {"packed": (2.6e12, 6e8), "append": (1e9, 1.2e9), "decode": (3.5e10, 2.3e9)}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        D = rng.choice([64, 128, 128])
        rd = rng.choice([16, 32, 48, 64] if D == 64 else [32, 64, 96, 128, 128])
        common = {"D": D, "rd": rd, "dtype": rng.choice(["bf16", "bf16", "f16"]), "layout": rng.choice(["split_half", "split_half", "interleaved"])}
        Hk = rng.choice([1, 2, 4, 8, 8, 16])
        Hq = Hk * rng.choice([1, 2, 3, 4, 4, 8])
        op = rng.choice(["packed", "append", "decode"])
        if op == "packed":
            n, top = _log(rng, 1, 64), _log(rng, 16, 16384)
            k_lens = [_log(rng, 1, top) for _ in range(n)]
            q_lens = [max(1, x // rng.choice([1, 1, 2, 5])) for x in k_lens] if rng.random() < 0.4 else k_lens
            case = dict(_packed("", q_lens, k_lens, Hq, Hk, causal=rng.random() < 0.8, fused=q_lens is k_lens and rng.random() < 0.5, **common))
            if n * max(q_lens) * max(k_lens) * (Hq // Hk) * 4 > 8e9:
                continue
        elif op == "append":
            n = _log(rng, 1, 256)
            top = _log(rng, 1, 16384)
            case = dict(_append("", [_log(rng, 1, top) for _ in range(n)], [rng.randrange(0, 300) for _ in range(n)], Hk, page=rng.choice([16, 32, 64, 128]),
                                offset=rng.choice([0, _log(rng, 1, 16384)]), fused=rng.random() < 0.5, **common))
        else:
            n = _log(rng, 1, 256)
            top = _log(rng, 16, 8192)
            case = dict(_decode("", rng.choice([0, _log(rng, 1, 131072), _log(rng, 256, 131072)]), [rng.randrange(0, top + 1) for _ in range(n)], Hq, Hk,
                                page=rng.choice([16, 32, 64, 128]), **common))
        w = work(case)
        if w["flops"] <= _MOST[op][0] and w["bytes"] <= _MOST[op][1] and w["bytes"] > 0:
            del case["name"]
            return case


def work(case):
    D = case["D"]
    if case["op"] == "packed":
        ql, kl = _lens(case["q_lens"]), _lens(case["k_lens"])
        pairs = 0
        for a, b in zip(ql, kl):
            # row i sees min(b, i + 1 + b - a) keys under the causal mask
            pairs += sum(max(0, min(b, i + 1 + b - a)) for i in range(a)) if case["causal"] else a * b
        return {"bytes": 2 * D * (2 * sum(ql) * case["Hq"] + 2 * sum(kl) * case["Hk"]) + 4 * case["rd"] * max(kl), "flops": 4 * D * case["Hq"] * pairs}
    if case["op"] == "append":
        t = sum(_lens(case["new"]))
        return {"bytes": 2 * D * case["Hk"] * t * 4, "flops": 3 * case["rd"] * case["Hk"] * t}
    lens = _lens(case["lens"])
    return {"bytes": 2 * D * (2 * case["Hk"] * (case["prefix"] + sum(lens)) + 2 * case["Hq"] * len(lens)),
            "flops": 4 * D * case["Hq"] * (case["prefix"] * len(lens) + sum(lens))}


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
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, D = TYPES[case["dtype"]], case["D"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    s = {"op": case["op"], "rd": case["rd"], "layout": case["layout"]}
    if case["op"] == "packed":
        ql, kl, Hq, Hk = _lens(case["q_lens"]), _lens(case["k_lens"]), case["Hq"], case["Hk"]
        if case["fused"]:
            # one projection's output: a token's query heads, key heads and value heads lie side by side
            qkv = normal(sum(ql), Hq + 2 * Hk, D)
            s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        else:
            s["q"], s["k"], s["v"] = normal(sum(ql), Hq, D), normal(sum(kl), Hk, D), normal(sum(kl), Hk, D)
        s["cu_q"], s["cu_k"], s["causal"] = _starts(ql), _starts(kl), case["causal"]
        s["q_lens"], s["k_lens"] = ql, kl
        # the queries of a sequence are its last tokens
        s["pos_q"] = torch.cat([torch.arange(b - a, b, dtype=torch.int32, device="cuda") for a, b in zip(ql, kl)])
        if ql == kl:
            s["pos_q"] = None
        s["cos"], s["sin"] = _tables(case["rd"], max(kl))
    elif case["op"] == "append":
        new, old, Hk = _lens(case["new"]), _lens(case["old"]), case["Hk"]
        table, total = _pages(gen, [a + b for a, b in zip(new, old)], case["page"])
        if case["fused"]:
            kv = normal(sum(new), 2 * Hk, D)
            s["k"], s["v"] = kv[:, :Hk], kv[:, Hk:]
        else:
            s["k"], s["v"] = normal(sum(new), Hk, D), normal(sum(new), Hk, D)
        s["k_pages"], s["v_pages"] = normal(total, Hk, case["page"], D), normal(total, Hk, case["page"], D)
        s |= {"table": table, "cu": _starts(new), "old": _ints(old), "offset": case["offset"]}
        s["cos"], s["sin"] = _tables(case["rd"], case["offset"] + max(a + b for a, b in zip(new, old)))
    else:
        lens, prefix = _lens(case["lens"]), case["prefix"]
        table, total = _pages(gen, lens + [prefix], case["page"])
        n = -(-prefix // case["page"])
        s["prefix_table"] = table[-1, :n].contiguous()
        s["table"] = table[:-1, :max(1, -(-max(lens) // case["page"]))].contiguous()
        s["k_pages"], s["v_pages"] = normal(total, case["Hk"], case["page"], D), normal(total, case["Hk"], case["page"], D)
        s["q"] = normal(len(lens), case["Hq"], D)
        s |= {"lens": _ints(lens), "prefix": prefix}
        s["cos"], s["sin"] = _tables(case["rd"], prefix + max(lens) + 1)
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


def _softmax(scores):
    """Softmax of the last axis; a row that is -inf throughout gives zeros."""
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total)


def _plain_packed(s):
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    Lq, Lk = max(s["q_lens"]), max(s["k_lens"])                       # a program knows its prompts' lengths
    Tq, Hq, D = s["q"].shape
    Tk, Hk, _ = s["k"].shape
    iq, ik = torch.arange(Lq, device="cuda"), torch.arange(Lk, device="cuda")
    live_q, live_k = iq < nq[:, None], ik < nk[:, None]
    at_q, at_k = (cu_q[:-1, None] + iq).clamp(max=Tq - 1), (cu_k[:-1, None] + ik).clamp(max=Tk - 1)
    tok_q, tok_k = torch.arange(Tq, device="cuda"), torch.arange(Tk, device="cuda")
    seq_q, seq_k = torch.searchsorted(cu_q[1:], tok_q, right=True), torch.searchsorted(cu_k[1:], tok_k, right=True)
    pos_q = tok_q - cu_q[seq_q] if s["pos_q"] is None else s["pos_q"].long()
    pos_k = tok_k - cu_k[seq_k]
    q = _rotate(s["q"].float(), s["cos"][pos_q][:, None], s["sin"][pos_q][:, None], s["layout"])
    k = _rotate(s["k"].float(), s["cos"][pos_k][:, None], s["sin"][pos_k][:, None], s["layout"])
    v = s["v"].float()
    seen = live_k[:, None, :]
    if s["causal"]:
        seen = seen & (ik[None, None, :] <= iq[None, :, None] + (nk - nq)[:, None, None])
    G = Hq // Hk
    out = torch.empty((Tq, Hq, D), dtype=s["q"].dtype, device="cuda")
    for h in range(Hk):                                               # a key head at a time: the scores of all would be tens of GB
        qh = q[:, h * G:(h + 1) * G][at_q].transpose(1, 2)            # [n, G, Lq, D], padded to the longest prompt
        scores = (qh @ k[:, h][at_k].transpose(1, 2)[:, None]) / math.sqrt(D)
        p = _softmax(scores.masked_fill(~seen[:, None], -math.inf))
        out[:, h * G:(h + 1) * G] = (p @ v[:, h][at_k][:, None]).transpose(1, 2)[live_q].to(out.dtype)
    return out


def _plain_append(s):
    cu = s["cu"].long()
    T = s["k"].shape[0]
    tok = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu[1:], tok, right=True)
    slot = s["old"].long()[seq] + tok - cu[seq]
    row = s["offset"] + slot
    k = _rotate(s["k"].float(), s["cos"][row][:, None], s["sin"][row][:, None], s["layout"])
    page = s["k_pages"].shape[2]
    where = s["table"].long()[seq, slot // page]
    s["k_pages"][where, :, slot % page] = k.to(s["k_pages"].dtype)
    s["v_pages"][where, :, slot % page] = s["v"]
    return s["k_pages"], s["v_pages"]


def _plain_decode(s):
    B, Hq, D = s["q"].shape
    _, Hk, page, _ = s["k_pages"].shape
    G = Hq // Hk
    lens, P = s["lens"].long(), s["prefix"]
    row = (P + lens - 1).clamp(min=0)                                 # the new token is the last one of its sequence
    q = _rotate(s["q"].float(), s["cos"][row][:, None], s["sin"][row][:, None], s["layout"]).view(B, Hk, G, D)

    def gather(pool, table):                                          # [..., blocks] -> [..., Hk, blocks * page, D]
        x = pool[table.long().clamp(min=0)].float()
        return x.transpose(-4, -3).reshape(*table.shape[:-1], Hk, -1, D)

    k, v = gather(s["k_pages"], s["table"]), gather(s["v_pages"], s["table"])
    own_scores = q @ k.transpose(-1, -2) / math.sqrt(D)
    seen = torch.arange(k.shape[2], device="cuda") < lens[:, None]
    own_scores = own_scores.masked_fill(~seen[:, None, None], -math.inf)
    kp, vp = gather(s["k_pages"], s["prefix_table"])[:, :P], gather(s["v_pages"], s["prefix_table"])[:, :P]
    rows = q.transpose(0, 1).reshape(Hk, B * G, D)                    # all sequences' queries meet the prefix's keys at once
    pre = (rows @ kp.transpose(-1, -2) / math.sqrt(D)).view(Hk, B, G, P).transpose(0, 1)
    p = _softmax(torch.cat([pre, own_scores], -1))
    o = (p[..., :P].transpose(0, 1).reshape(Hk, B * G, P) @ vp).view(Hk, B, G, D).transpose(0, 1)
    return (o + p[..., P:] @ v.masked_fill(~seen[:, None, :, None], 0.0)).reshape(B, Hq, D).to(s["q"].dtype)


def run(state):
    s = state
    if own:
        import rotary_position_embedding_rope_gb300 as R

        if s["op"] == "packed":
            return R.attention_packed(s["q"], s["k"], s["v"], s["cu_q"], s["cos"], s["sin"], cu_seqlens_k=s["cu_k"], pos_q=s["pos_q"],
                                      layout=s["layout"], causal=s["causal"])
        if s["op"] == "append":
            R.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["old"], s["cos"], s["sin"],
                           pos_offset=s["offset"], layout=s["layout"])
            return s["k_pages"], s["v_pages"]
        return R.attention_shared_prefix(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["prefix_table"], s["prefix"],
                                         s["cos"], s["sin"], layout=s["layout"])
    return {"packed": _plain_packed, "append": _plain_append, "decode": _plain_decode}[s["op"]](s)


# ---------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence


def _turn(x, row, rd, layout, cos, sin):
    """x [H, n, D] in 64 bits as complex pairs, multiplied by exp(i angle) of its table rows."""
    z = torch.complex(cos[row].double(), sin[row].double())[None]
    r = x[..., :rd]
    pair = r.unflatten(-1, (2, rd // 2)).transpose(-1, -2) if layout == "split_half" else r.unflatten(-1, (rd // 2, 2))
    y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    y = (y.transpose(-1, -2) if layout == "split_half" else y).flatten(-2)
    return torch.cat([y, x[..., rd:]], -1)


def _attend(q, k, v, shift):
    """[H, a, D] against [H, b, D]: row i sees the keys j <= i + shift (all of them for None). A block of rows at a time."""
    a, b, D = q.shape[1], k.shape[1], q.shape[2]
    out = torch.zeros(q.shape[0], a, v.shape[2], dtype=torch.float64, device=q.device)
    for r in range(0, a, 1024):
        n = min(1024, a - r)
        e = b if shift is None else max(0, min(b, r + n + shift))
        if e == 0:
            continue
        x = torch.einsum("had,hbd->hab", q[:, r:r + n], k[:, :e]) * D ** -0.5
        if shift is not None:
            i = torch.arange(r, r + n, device=q.device)[:, None]
            x = torch.where(torch.arange(e, device=q.device)[None] <= i + shift, x, -math.inf)
        lse = torch.logsumexp(x, -1, keepdim=True)
        w = torch.where(lse == -math.inf, 0.0, torch.exp(x - lse))
        out[:, r:r + n] = torch.einsum("hab,hbd->had", w, v[:, :e])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if work(case)["flops"] > 5e12:
        return None
    args = (case["rd"], case["layout"], s["cos"], s["sin"])
    if case["op"] == "packed":
        G = case["Hq"] // case["Hk"]
        outs, iq, ik = [], 0, 0
        for a, b in zip(s["q_lens"], s["k_lens"]):
            rows = torch.arange(b, device="cuda")
            q = _turn(s["q"][iq:iq + a].double().transpose(0, 1), rows[:a] if s["pos_q"] is None else rows[b - a:], *args)
            k = _turn(s["k"][ik:ik + b].double().transpose(0, 1), rows, *args)
            v = s["v"][ik:ik + b].double().transpose(0, 1)
            heads = [_attend(q[h * G:(h + 1) * G].reshape(1, G * a, -1) if not case["causal"] else q[h * G:(h + 1) * G],
                             k[h:h + 1] if not case["causal"] else k[h:h + 1].expand(G, -1, -1),
                             v[h:h + 1] if not case["causal"] else v[h:h + 1].expand(G, -1, -1),
                             b - a if case["causal"] else None).reshape(G, a, -1) for h in range(case["Hk"])]
            outs.append(torch.cat(heads).transpose(0, 1))
            iq, ik = iq + a, ik + b
        return torch.cat(outs)
    if case["op"] == "append":
        k_out, v_out, at, page = s["k_pages"].double(), s["v_pages"].double(), 0, case["page"]
        for b, (n, old) in enumerate(zip(_lens(case["new"]), _lens(case["old"]))):
            p = torch.arange(old, old + n, device="cuda")
            k = _turn(s["k"][at:at + n].double().transpose(0, 1), p + case["offset"], *args).transpose(0, 1)
            blocks = s["table"][b].long()[torch.div(p, page, rounding_mode="floor")]
            k_out[blocks, :, p % page], v_out[blocks, :, p % page] = k, s["v"][at:at + n].double()
            at += n
        return k_out, v_out
    outs, G, Hk, page = [], case["Hq"] // case["Hk"], case["Hk"], case["page"]

    def keys(pool, blocks, n):
        return pool[blocks.long()].double().transpose(0, 1).reshape(Hk, -1, case["D"])[:, :n]

    P = case["prefix"]
    kp, vp = keys(s["k_pages"], s["prefix_table"], P), keys(s["v_pages"], s["prefix_table"], P)
    for b, n in enumerate(_lens(case["lens"])):
        mine = s["table"][b, :-(-n // page)]
        k, v = torch.cat([kp, keys(s["k_pages"], mine, n)], 1), torch.cat([vp, keys(s["v_pages"], mine, n)], 1)
        row = torch.full((1,), max(0, P + n - 1), device="cuda")
        q = _turn(s["q"][b].double()[:, None], row, *args)
        outs.append(_attend(q.view(Hk, G, -1), k, v, None).reshape(case["Hq"], -1))
    return torch.stack(outs)

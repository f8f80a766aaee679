"""Plain 64-bit forms of the serving operators, token by token or sequence by
sequence on the CPU, for the tests.  Table values are the fp32 ones the
library reads (they are part of the method's input)."""
from __future__ import annotations

import torch


def tables(theta: float, rd: int, rows: int):
    w = theta ** (-2.0 * torch.arange(rd // 2, dtype=torch.float64) / rd)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * w
    return a.cos().float(), a.sin().float()


def rotate(x, row, cos, sin, layout):
    """x [..., D] in fp64 at table row `row`; None, or a row outside the table: as it is."""
    y = x.double().clone()
    if row is None or row < 0 or row >= cos.shape[0]:
        return y
    c, s = cos[row].double(), sin[row].double()
    h = c.numel()
    if layout == "split_half":
        a, b = y[..., :h].clone(), y[..., h:2 * h].clone()
        y[..., :h], y[..., h:2 * h] = a * c - b * s, a * s + b * c
    else:
        a, b = y[..., 0:2 * h:2].clone(), y[..., 1:2 * h:2].clone()
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = a * c - b * s, a * s + b * c
    return y


def append(k, v, k_pages, v_pages, table, cu, lens, cos, sin, pos=None, pos_offset=0,
           layout="split_half"):
    """The pools after the call (new tensors), and the rows written, as a mask [pages, page]."""
    kp, vp = k_pages.clone(), v_pages.clone()
    page = kp.shape[2]
    wrote = torch.zeros(kp.shape[0], page, dtype=torch.bool)
    for b in range(len(lens)):
        for t in range(int(cu[b]), int(cu[b + 1])):
            slot = int(lens[b]) + t - int(cu[b])
            if slot < 0 or int(lens[b]) < 0 or slot // page >= table.shape[1]:
                continue
            p = int(table[b, slot // page])
            if p < 0 or p >= kp.shape[0]:
                continue
            row = pos_offset + slot if pos is None else int(pos[t])
            kp[p, :, slot % page] = rotate(k[t], row, cos, sin, layout).to(kp.dtype)
            vp[p, :, slot % page] = v[t]
            wrote[p, slot % page] = True
    return kp, vp, wrote


def softmax_rows(q, k, v, seen, scale):
    """q [R, D], k, v [N, D] in fp64, seen [R, N]: (o, w, a) [R, D]: the
    attention and its two error weights, sum_j p_j |v_j| / l and
    sum_j seen_j |v_j| / l; zeros for rows that see nothing."""
    s = (q @ k.T) * scale
    s = torch.where(seen, s, -torch.inf)
    m = s.amax(1, keepdim=True) if s.shape[1] else torch.full((q.shape[0], 1), -torch.inf).double()
    p = torch.where(seen, torch.exp(s - torch.where(m == -torch.inf, 0.0, m)), 0.0)
    l = p.sum(1, keepdim=True)
    inv = torch.where(l > 0, 1.0 / torch.where(l > 0, l, 1.0), 0.0)
    vis = torch.where(seen.any(0)[:, None], v, 0.0)      # what no row sees may hold anything
    return p @ vis * inv, p @ vis.abs() * inv, seen.double() @ vis.abs() * inv


def _rotated_rounded(x, rows, cos, sin, layout):
    """x [n, H, D] at table rows `rows`, rounded to its type, in fp64."""
    y = torch.stack([rotate(x[i], rows[i], cos, sin, layout) for i in range(x.shape[0])]) \
        if x.shape[0] else x.double()
    return y.to(x.dtype).double()


def tie_slack(x, rows, cos, sin, layout):
    """Per element of x [n, H, D]: one unit of its type where the rotated value, exact, lies so near the middle of
    two neighbours (2^-21 of it; the fp32 rotation is within 2^-22) that a correct kernel may round to the other
    one, else 0."""
    y = torch.stack([rotate(x[i], rows[i], cos, sin, layout) for i in range(x.shape[0])])
    r = y.to(x.dtype).double()
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1e-30)))) * torch.finfo(x.dtype).eps
    return torch.where((unit / 2 - (y - r).abs()).abs() <= y.abs() * 2.0 ** -21, unit, 0.0)


def score_slack(q, k, cu, cos, sin, layout="split_half", scale=None):
    """[T, Hq]: how far a score of a row of packed causal self-attention can lie from the reference's because of such
    elements: max_j scale sum_d (|dq_d| |k_jd| + |q_d| |dk_jd|), elements a unit larger than they are."""
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(T, Hq, dtype=torch.float64)
    for b in range(len(cu) - 1):
        a, e = int(cu[b]), int(cu[b + 1])
        dq, dk = (tie_slack(x[a:e], range(e - a), cos, sin, layout) for x in (q, k))
        qa, ka = (_rotated_rounded(x[a:e], range(e - a), cos, sin, layout).abs() + d for x, d in ((q, dq), (k, dk)))
        for h in range(Hq):
            g = h // (Hq // k.shape[1])
            s = (dq[:, h] @ ka[:, g].T + qa[:, h] @ dk[:, g].T) * scale
            out[a:e, h] = torch.tril(s).amax(1)
    return out


def packed(q, k, v, cu_q, cu_k, cos, sin, pos_q=None, pos_k=None, layout="split_half",
           causal=False, scale=None):
    """(o, w, a) [Tq, Hq, D] in fp64; rows of no sequence are NaN."""
    Tq, Hq, D = q.shape
    Hk = k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out = [torch.full((Tq, Hq, D), torch.nan, dtype=torch.float64) for _ in range(3)]
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        Lq, Lk = q1 - q0, k1 - k0
        pq = range(Lq) if pos_q is None else [int(x) for x in pos_q[q0:q1]]
        pk = range(Lk) if pos_k is None else [int(x) for x in pos_k[k0:k1]]
        qr = _rotated_rounded(q[q0:q1], pq, cos, sin, layout)
        kr = _rotated_rounded(k[k0:k1], pk, cos, sin, layout)
        vr = v[k0:k1].double()
        seen = torch.ones(Lq, Lk, dtype=torch.bool)
        if causal:
            seen = torch.arange(Lk)[None] <= torch.arange(Lq)[:, None] + (Lk - Lq)
        for h in range(Hq):
            g = h // (Hq // Hk)
            r = softmax_rows(qr[:, h], kr[:, g], vr[:, g], seen, scale)
            for o, x in zip(out, r):
                o[q0:q1, h] = x
    return out


def shared_prefix(q, k_pages, v_pages, table, lens, prefix_table, prefix, cos, sin, pos_q=None,
                  layout="split_half", scale=None):
    """(o, w, a) [B, Hq, D] in fp64."""
    B, Hq, D = q.shape
    _, Hk, page, _ = k_pages.shape
    scale = D ** -0.5 if scale is None else scale
    out = [torch.zeros(B, Hq, D, dtype=torch.float64) for _ in range(3)]

    def keys(pool, blocks, n):
        m = -(-n // page)
        x = pool[blocks[:m].long()].double()              # [m, Hk, page, D]
        return x.transpose(0, 1).reshape(Hk, m * page, D)[:, :n]

    for b in range(B):
        n = int(lens[b])
        k = torch.cat([keys(k_pages, prefix_table, prefix), keys(k_pages, table[b], n)], 1)
        v = torch.cat([keys(v_pages, prefix_table, prefix), keys(v_pages, table[b], n)], 1)
        row = prefix + n - 1 if pos_q is None else int(pos_q[b])
        qr = rotate(q[b], row, cos, sin, layout).to(q.dtype).double()
        for h in range(Hq):
            g = h // (Hq // Hk)
            seen = torch.ones(1, prefix + n, dtype=torch.bool)
            r = softmax_rows(qr[h:h + 1], k[g], v[g], seen, scale)
            for o, x in zip(out, r):
                o[b, h] = x[0]
    return out

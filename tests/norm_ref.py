"""Plain 64-bit forms of the norm of query and key heads with the rotation, of its gradients and of the long-context
tables, on the CPU, with the bounds that the fp32 kernels' errors obey.

u = 2^-24 is fp32's rounding.  A lane adds 16 squares in chains of at most eight and the lanes of a row theirs: at most 13
roundings on a sum of positive terms, 1 for the mean and eps, so the root is off by 7 u, and 1 / sqrt by 11 u (rsqrtf: two
units, 4 u); a normalised, weighted element by 13 u.  The rotation's product and fma add at most 2 u of their sizes.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24


def half_step(y, dtype):
    """Rounding once to dtype: half a step of a normal value, or of the subnormal ones."""
    f = torch.finfo(dtype)
    return y.abs() * (f.eps / 2) * (1 + 2.0 ** -10) + f.smallest_normal * f.eps / 2


def angles(rows, cos, sin):
    """cos and sin in 64 bits of table rows (any shape); rows outside the table turn nothing."""
    ok = (rows >= 0) & (rows < cos.shape[0])
    r = rows.long().clamp(0, max(cos.shape[0] - 1, 0))
    c, s = cos.double()[r], sin.double()[r]
    return torch.where(ok[..., None], c, 1.0), torch.where(ok[..., None], s, 0.0)


def turn(x, c, s, layout):
    h = c.shape[-1]
    y = x.clone()
    if layout == "split_half":
        a, b = x[..., :h], x[..., h:2 * h]
        y[..., :h], y[..., h:2 * h] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = a * c - b * s, a * s + b * c
    return y


def turn_size(x, c, s, layout):
    """What the products of a rotation amount to: |a c| + |b s| (|b c| + |a s|)."""
    c, s = c.abs(), s.abs()
    h = c.shape[-1]
    x = x.abs()
    y = x.clone()
    if layout == "split_half":
        a, b = x[..., :h], x[..., h:2 * h]
        y[..., :h], y[..., h:2 * h] = a * c + b * s, a * s + b * c
    else:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = a * c + b * s, a * s + b * c
    return y


def forward(x, w, c, s, layout, eps):
    """(y, bound before rounding) for rows x [..., D]; c, s broadcast against them."""
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w
    c, s = c.expand(*x.shape[:-1], -1), s.expand(*x.shape[:-1], -1)
    return turn(n, c, s, layout), 16 * U * turn_size(n, c, s, layout)


def backward(x, w, g, c, s, layout, eps):
    """(dx, bound, dw, bound) of rows x [..., D] and their outputs' gradients g, before rounding.

    dx = r (w g - n m): w g within 5 u of its products, n within 11 u, m a sum of D products in chains of 16 and a
    tree: 16 + 5 roundings, n's and w g's errors, 40 u of the sum of its sizes; their product and difference 4 u more.
    dw: at most 128 additions on an element's way (the tests' sizes), n's and g's errors: 150 u of the sum of sizes."""
    x, g = x.double(), g.double()
    one = w is None
    w = torch.ones(x.shape[-1], dtype=torch.float64) if one else w.double()
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    n = x * r
    c, s = c.expand(*x.shape[:-1], -1), s.expand(*x.shape[:-1], -1)
    t, size = turn(g, c, -s, layout), turn_size(g, c, s, layout)
    dx = r * (w * t - n * (w * t * n).mean(-1, keepdim=True))
    bound = U * r * (24 * w.abs() * size + 64 * n.abs() * (w.abs() * size * n.abs()).mean(-1, keepdim=True))
    dims = tuple(range(x.dim() - 1))
    return dx, bound, (t * n).sum(dims), 150 * U * (size * n.abs()).sum(dims)


def frequencies(kind, rd, factor, original, theta, low=None, high=None):
    """(w_i, scale of all values), with 64-bit numbers one by one."""
    low = 1.0 if low is None else low
    high = (32.0 if kind == "yarn" else 4.0) if high is None else high
    out = []
    for i in range(rd // 2):
        w = theta ** (-2 * i / rd)
        if kind == "linear":
            w = w / factor
        elif kind == "ntk":
            w = (theta * factor ** (rd / (rd - 2))) ** (-2 * i / rd)
        elif kind == "smooth":
            n = original * w / (2 * math.pi)
            m = min(max((n - low) / (high - low), 0.0), 1.0)
            w = (1 - m) * w / factor + m * w
        else:
            def pair(n):
                return rd * math.log(original / (n * 2 * math.pi)) / (2 * math.log(theta))
            a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rd - 1)
            m = min(max((i - a) / (b - a if b > a else 0.001), 0.0), 1.0)
            w = w / factor * m + w * (1 - m)
        out.append(w)
    return out, (0.1 * math.log(factor) + 1.0 if kind == "yarn" and factor > 1 else 1.0)

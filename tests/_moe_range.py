"""The experts' layer in 64 bits with the bounds of its products for rows of any
size and spread (tests/_moe.py's hold where a row's values lie within 2^-20 of
its largest, and its largest above 2^-86).

A row of activations enters the MMAs as fp16, times 2^up, which puts its largest
magnitude into [2^14, 2^15), or 2^126 where that is more; up to 2^-pre of that
where a code lies pre bits up in its fp16.  So a value is off by 2^-11 of itself
(not at all where it came from 16 bits) or by half of fp16's smallest step:
    spread = 2^(pre - 25 - up) <= max(2^(pre - 39) * largest, 2^(pre - 151)),
in its code's product and in its group's sum alike, so times its weight.
A group's sum enters times 2^-8 in two such parts: off by 2^-22 of itself, which
is in the sums' own bound, or by
    floor = 2^(8 - 25 - up) <= max(2^-31 * largest, 2^-143)."""
from __future__ import annotations

import torch

from . import _moe


def pre(bits: int, group: int) -> int:
    """The highest first bit of a code in its fp16."""
    return {2: 6 if group == 32 else 8, 3: 6, 4: 4, 5: 5, 6: 0, 8: 0}[bits]


def _parts(stack, bits, group):
    v, mag = _moe.values(stack, bits, group)
    return v, mag, stack[2].double().abs().sum(-1)


def _off(x, part, bits, group, own):
    """Bound of a product of x [n, K] with a matrix; own: the rounding of x's
    own values, relative."""
    v, mag, biases = part
    peak = x.abs().amax(1, keepdim=True)
    spread = torch.clamp(2.0 ** (pre(bits, group) - 39) * peak, min=2.0 ** (pre(bits, group) - 151))
    floor = torch.clamp(2.0 ** -31 * peak, min=2.0 ** -143)
    off = _moe.steps(x.shape[1]) * (x.abs() @ mag.T) + spread * v.abs().sum(1) + floor * biases
    return off + own * (x.abs() @ v.abs().T) + 2.0 ** -149


def experts(x, ids, weights, gate, up, down, bits, group) -> tuple:
    """(y, bound of |y - y_kernel| before the output's rounding), float64."""
    x64 = x.double()
    y, bound, mag = (torch.zeros_like(x64) for _ in range(3))
    for e in range(gate[0].shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        g_, u_, d_ = (_parts([p[e] for p in m], bits, group) for m in (gate, up, down))
        g, u = x64[t] @ g_[0].T, x64[t] @ u_[0].T
        tg, tu = _off(x64[t], g_, bits, group, 0.0), _off(x64[t], u_, bits, group, 0.0)
        sg = g * torch.sigmoid(g)
        h = sg * u
        # |silu'| <= 1.1; exp, the quotient and the product round 8 times at most
        th = 1.1 * tg * (u.abs() + tu) + (sg.abs() + 1.1 * tg) * tu + 8 * 2.0 ** -24 * h.abs()
        th = th + 2.0 ** -149 * (2 + u.abs())
        top = h.abs() + th
        d = h @ d_[0].T
        td = th @ d_[0].abs().T + _off(top, d_, bits, group, 2.0 ** -11)
        w = weights.double()[t, j, None]
        y.index_add_(0, t, w * d)
        bound.index_add_(0, t, w.abs() * td)
        mag.index_add_(0, t, w.abs() * (d.abs() + td))
    return y, bound + (ids.shape[1] + 1) * 2.0 ** -24 * mag


def tolerance(want, bound, dtype):
    return bound + _moe.HALF_STEP[dtype] * (want.abs() + bound) + _moe.SMALLEST[dtype]

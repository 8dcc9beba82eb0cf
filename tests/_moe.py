"""Plain models in 64 bits of the mixture-of-experts layer and of the embedding
lookup, with the error bounds that the kernels' arithmetic allows."""
from __future__ import annotations

import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SMALLEST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half of the smallest subnormal


def codes(words: torch.Tensor, bits: int) -> torch.Tensor:
    """int64 codes of packed rows [..., K * bits / 32], bit by bit."""
    K = words.shape[-1] * 32 // bits
    wide = words.to(torch.int64) & 0xFFFFFFFF
    at = torch.arange(K, device=words.device) * bits
    out = torch.zeros((*words.shape[:-1], K), dtype=torch.int64, device=words.device)
    for i in range(bits):
        out += (wide[..., (at + i) // 32] >> ((at + i) % 32) & 1) << i
    return out


def values(stack, bits: int, group: int) -> tuple:
    """(values, |scale| * code + |bias|) of packed rows, float64."""
    words, s, b = stack
    c = codes(words, bits).double()
    s, b = (t.double().repeat_interleave(group, -1) for t in (s, b))
    return s * c + b, s.abs() * c + b.abs()


def stack(E, rows, cols, bits, group, gen, device):
    """Random words; scales and biases of centred rows of about unit norm, some
    groups with a scale of zero and some negative."""
    words = torch.randint(-2 ** 31, 2 ** 31, (E, rows, cols * bits // 32), dtype=torch.int32,
                          generator=gen)
    size = (E, rows, cols // group)
    s = (torch.rand(size, generator=gen) + 0.5) * (3.4 / 2 ** bits) * cols ** -0.5
    b = -(2 ** bits - 1) / 2 * s + 0.1 * cols ** -0.5 * torch.randn(size, generator=gen)
    pick = torch.rand(size, generator=gen)
    s = torch.where(pick < 0.03, torch.zeros_like(s), torch.where(pick > 0.97, -s, s))
    return words.to(device), s.half().to(device), b.half().to(device)


def steps(K: int) -> float:
    """Rounding of a row's fp32 sum of K products, relative to the sum of
    magnitudes: a group's four MMA steps and two fused products, K / 64 groups
    one after the other, the slots of 8 warps and the chunks, each 2^-23 (a
    step of the MMA truncates, a fused product rounds by half of that)."""
    return (K / 64 * 2 + 4 + 8 + K / 512) * 2.0 ** -23


def experts(x, ids, weights, gate, up, down, bits, group) -> tuple:
    """(y, bound of |y - y_kernel| before the output's rounding), float64."""
    x64, T = x.double(), x.shape[0]
    E = gate[0].shape[0]
    y = torch.zeros_like(x64)
    bound, mag = torch.zeros_like(x64), torch.zeros_like(x64)
    K, inner = x.shape[1], gate[1].shape[1]
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        (wg, ag), (wu, au), (wd, ad) = (values([p[e] for p in m], bits, group)
                                        for m in (gate, up, down))
        xt, peak = x64[t], x64[t].abs().amax(1, keepdim=True)
        g, u = xt @ wg.T, xt @ wu.T
        # small values of a row lose 2^-39 of its largest when they become fp16
        tg = steps(K) * (xt.abs() @ ag.T) + 2.0 ** -39 * peak * ag.sum(1)
        tu = steps(K) * (xt.abs() @ au.T) + 2.0 ** -39 * peak * au.sum(1)
        sg = g * torch.sigmoid(g)
        h = sg * u
        # |silu'| <= 1.1; exp, the quotient and the product round 8 times at most
        th = 1.1 * tg * (u.abs() + tu) + (sg.abs() + 1.1 * tg) * tu + 8 * 2.0 ** -24 * h.abs()
        th = th + 2.0 ** -11 * (h.abs() + th) + 2.0 ** -39 * (h.abs() + th).amax(1, keepdim=True)
        d = h @ wd.T
        td = th @ wd.abs().T + steps(inner) * ((h.abs() + th) @ ad.T)
        w = weights.double()[t, j, None]
        y.index_add_(0, t, w * d)
        bound.index_add_(0, t, w.abs() * td)
        mag.index_add_(0, t, w.abs() * (d.abs() + td))
    bound = bound + (ids.shape[1] + 1) * 2.0 ** -24 * mag
    return y, bound


def check(y, want, bound, dtype, what=""):
    tol = bound + HALF_STEP[dtype] * (want.abs() + bound) + SMALLEST[dtype]
    bad = ~((y.double() - want).abs() <= tol)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, at {i}: "
                             f"{float(y[tuple(i)])} for {float(want[tuple(i)])}, "
                             f"tolerance {float(tol[tuple(i)]):.3g}")


def route(x, weight, top_k, bias=None, score="softmax", normalize=True, scale=1.0) -> tuple:
    """(ids ascending int64, weights float64, relative bound of the weights)."""
    x64, w64 = x.double(), weight.double()
    logits = x64 @ w64.T
    p = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    likes = logits if bias is None else p + bias.double()
    order = torch.sort(likes, dim=1, descending=True, stable=True).indices
    ids = order[:, :top_k].sort(1).values
    picked = logits.gather(1, ids)
    if score == "softmax":
        over = picked if normalize else logits
        w = torch.exp(picked - torch.logsumexp(over, 1, keepdim=True))
    else:
        low = torch.nn.functional.logsigmoid(picked)
        w = torch.exp(low - torch.logsumexp(low, 1, keepdim=True)) if normalize else torch.exp(low)
    # a logit is off by its sum's rounding; a weight by twice that (itself and
    # the sum over which it is taken), and by a few roundings of exp and sum
    K = x.shape[1]
    off = (K / 32 + 24) * 2.0 ** -22 * (x64.abs() @ w64.abs().T).amax(1, keepdim=True)
    return ids, w * scale, torch.expm1(2 * off) + (weight.shape[0] + 32) * 2.0 ** -23


def embed(ids, table, bits, group, scale) -> tuple:
    words, s, b = table
    n = words.shape[0]
    ok = (ids >= 0) & (ids < n)
    rows = torch.where(ok, ids, torch.zeros_like(ids)).long()
    v, _ = values((words[rows], s[rows], b[rows]), bits, group)
    v = torch.where(ok[..., None], v * scale, torch.zeros_like(v))
    return v, 2.0 ** -23 * v.abs()

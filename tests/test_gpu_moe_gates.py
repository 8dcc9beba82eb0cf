"""Gates far below zero: silu(g) = g exp(g) / (1 + exp(g)) goes on where exp(-g)
has passed the largest float."""
import pytest
import torch

import quantized_matmul_affine_gb300 as aq

from . import _moe, _moe_range

pytestmark = pytest.mark.gpu
K, INNER = 128, 128


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 12, 40])
@pytest.mark.parametrize("low,high", [(-79.9, -60.0), (-81.0, -79.0), (-88.5, -80.1), (-100.0, -88.8), (-130.0, -100.0)])
def test_low_gates(low, high, T, dtype):
    g = torch.Generator().manual_seed(T)
    words = torch.zeros(1, INNER, K // 8, dtype=torch.int32)
    zero = torch.zeros(1, INNER, K // 64)
    biases = (low + (high - low) * torch.rand(1, INNER, 1, generator=g)) / K
    gate = tuple(t.cuda() for t in (words, zero.half(), biases.expand(1, INNER, 2).half().contiguous()))
    up, down = (_moe.stack(1, r, c, 4, 64, g, "cuda") for r, c in ((INNER, K), (K, INNER)))
    up = (up[0], up[1] * 8, up[2] * 8 + 8)  # about 1000 for x of ones
    x = torch.ones(T, K, dtype=dtype, device="cuda")
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")

    (vg, ag, sg), (vu, au, su), (vd, ad, sd) = (_moe_range._parts([p[0] for p in m], 4, 64) for m in (gate, up, down))
    x64 = x.double()
    a, u = x64 @ vg.T, x64 @ vu.T
    ta, tu = (_moe_range._off(x64, p, 4, 64, 0.0) for p in ((vg, ag, sg), (vu, au, su)))
    assert (a > low - 0.1).all() and (a < high + 0.1).all()
    h = a * torch.sigmoid(a) * u
    # |silu'(a)| <= (1 + |a|) exp(a) below zero; two exps of two places each, six roundings
    th = ta * (1 + a.abs() + ta) * torch.exp(a + ta) * (u.abs() + tu) + h.abs() / u.abs() * tu + 16 * 2.0 ** -24 * h.abs()
    th = th + 2.0 ** -149 * (2 + u.abs())
    lift = float(1 / (h @ vd.T).square().mean().sqrt())
    weights = torch.full((T, 1), min(lift, 3e38), device="cuda")
    w = weights.double()
    want = w * (h @ vd.T)
    bound = w * (th @ vd.abs().T + _moe_range._off(h.abs() + th, (vd, ad, sd), 4, 64, 2.0 ** -11))
    tol = _moe_range.tolerance(want, bound + 2.0 ** -23 * (want.abs() + bound), dtype)
    got = aq.aq_moe_experts(x, aq.AqExperts(gate, up, down, 4, 64), ids, weights)
    assert ((got.double() - want).abs() <= tol).all(), float(((got.double() - want).abs() / tol).max())
    if high >= -100:  # zeros would not pass
        assert (want.abs() > tol).double().mean() > 0.6

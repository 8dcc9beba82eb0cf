"""Experts' products of rows whose largest value has no weight: what is left of
the small ones decides the outputs."""
import pytest
import torch

import quantized_matmul_affine_gb300 as aq

from . import _moe, _moe_range

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
SHAPES = [(3, 256, 128, 2), (3, 8192, 128, 2), (14, 640, 128, 3), (50, 384, 256, 2)]  # as in test_gpu_moe_scale
FORMATS = [(2, 32), (2, 64), (3, 32), (3, 64), (4, 32), (4, 64), (5, 32), (5, 128), (6, 64), (8, 64)]


def _pack(codes, bits):
    """int32 words of codes [..., K], bit by bit."""
    K = codes.shape[-1]
    one = (codes[..., None] >> torch.arange(bits)) & 1
    one = one.reshape(*codes.shape[:-1], K * bits // 32, 32)
    words = (one << torch.arange(32)).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def _near_zero(E, rows, cols, bits, group, g, up):
    """Weights of half a step either way, a part `up` of them up: their codes'
    part, scale * code, is many times as large."""
    mid = (2 ** bits - 1) // 2
    codes = mid + (torch.rand(E, rows, cols, generator=g) < up).long()
    s = 2.0 ** torch.randint(-7, -4, (E, rows, cols // group), generator=g).float()
    if up < 1:
        s[..., 0] = 0  # x's largest value has no weight
    return tuple(t.cuda() for t in (_pack(codes, bits), s.half(), (-(mid + 0.5) * s).half()))


def _check(x, mats, bits, group, ids, dtype):
    weights = torch.ones(x.shape[0], 1, device="cuda")
    y, _ = _moe_range.experts(x, ids, weights, *mats, bits, group)
    weights[:, 0] = (1 / y.square().mean(1).sqrt()).clamp(max=3e38).float()
    want, bound = _moe_range.experts(x, ids, weights, *mats, bits, group)
    tol = _moe_range.tolerance(want, bound, dtype)
    got = aq.aq_moe_experts(x, aq.AqExperts(*mats, bits, group), ids, weights)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), float(got[bad][0]), float(want[bad][0]),
                           float(tol[bad][0]))
    return want, tol, weights


def _codes_rounded(x, expert, bits, group):
    """A token's output where the codes' products see it rounded, the group sums not."""
    up = 14 - int(x.abs().max().log2())
    down = 2.0 ** (up - _moe_range.pre(bits, group))
    rounded = (x * down).half().double() / down

    def times(m):
        v, _ = _moe.values(m, bits, group)
        b = m[2].double().repeat_interleave(group, -1)
        return (v - b) @ rounded + b @ x

    g, u = times(expert[0]), times(expert[1])
    return _moe.values(expert[2], bits, group)[0] @ (g * torch.sigmoid(g) * u)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,K,inner,E", SHAPES)
@pytest.mark.parametrize("bits,group", FORMATS)
def test_halves_of_a_step(T, K, inner, E, bits, group, dtype):
    """All small values half a step of their fp16 off, one way: the rounding
    counts by the weights, which are small, not by scale * code."""
    g = torch.Generator().manual_seed(T + bits)
    mats = [_near_zero(E, r, c, bits, group, g, p) for r, c, p in ((inner, K, 0.75), (inner, K, 0.75), (K, inner, 1))]
    x = torch.randn(T, K, generator=g)
    peak = 2.0 ** 15 if dtype == F16 else 2.0 ** -3
    up = 14 - (15 if dtype == F16 else -3)
    x[1] = 61 * 2.0 ** (_moe_range.pre(bits, group) - 25 - up)
    x[1, 5] = peak
    assert torch.equal(x[1].to(dtype).float(), x[1])
    ids = torch.randint(0, E, (T, 1), generator=g, dtype=torch.int32).cuda()
    x = x.to(dtype).cuda()
    want, tol, weights = _check(x, mats, bits, group, ids, dtype)
    # rounded for the codes alone, the outputs would not pass (with groups of 32 the
    # bound of the group sums hides it in part)
    if _moe_range.pre(bits, group) and group > 32:
        wrong = _codes_rounded(x[1].double(), [[p[ids[1, 0]] for p in m] for m in mats], bits, group)
        assert ((weights[1].double() * wrong - want[1]).abs() > tol[1]).double().mean() > 0.5


@pytest.mark.parametrize("below", [16, 20, 24, 28])
@pytest.mark.parametrize("T,K,inner,E", SHAPES)
@pytest.mark.parametrize("bits,group", FORMATS)
def test_small_values_decide(T, K, inner, E, bits, group, below):
    """Values at 2^-below of the row's largest, random weights."""
    g = torch.Generator().manual_seed(T + bits + below)
    mats = [_moe.stack(E, r, c, bits, group, g, "cuda") for r, c in ((inner, K), (inner, K), (K, inner))]
    for m in mats[:2]:
        m[1][..., 0], m[2][..., 0] = 0, 0
    x = torch.randn(T, K, generator=g)
    x[1] *= 2.0 ** -below / x[1].abs().max()
    x[1, 3], x[1, 7] = 1.0, -1.0
    ids = torch.randint(0, E, (T, 1), generator=g, dtype=torch.int32).cuda()
    _check(x.to(BF16).cuda(), mats, bits, group, ids, BF16)

"""Experts' products of tokens of every size: outputs of about 1 (the weights of
the sum bring them there), so that a row that lost its bits shows."""
import pytest
import torch

import quantized_matmul_affine_gb300 as aq

from . import _moe, _moe_range

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
# the kernels by tokens: 8 columns from rows as they are, 8 packed, 16, 32
SHAPES = [(3, 128, 128, 2), (3, 8192, 128, 2), (14, 640, 128, 3), (50, 384, 256, 2)]


@pytest.mark.parametrize("dtype,size", [(BF16, 1e18), (BF16, 1e9), (F16, 6e4), (F16, 1e-6), (BF16, 1e-9),
                                        (BF16, 1e-14), (BF16, 1e-17), (BF16, 1e-18), (BF16, 1e-19), (BF16, 2e-20)])
@pytest.mark.parametrize("T,K,inner,E", SHAPES)
@pytest.mark.parametrize("bits,group", [(2, 64), (3, 32), (4, 64), (5, 128), (8, 32)])
def test_sizes(T, K, inner, E, bits, group, dtype, size):
    """One token of `size` among ordinary ones."""
    g = torch.Generator().manual_seed(T + bits)
    mats = [_moe.stack(E, r, c, bits, group, g, "cuda") for r, c in ((inner, K), (inner, K), (K, inner))]
    x = torch.randn(T, K, generator=g)
    x[1] *= size / x[1].abs().max()
    x = x.to(dtype).cuda()
    ids = torch.randint(0, E, (T, 1), generator=g, dtype=torch.int32).cuda()
    weights = torch.ones(T, 1, device="cuda")
    y, _ = _moe_range.experts(x, ids, weights, *mats, bits, group)
    weights[:, 0] = (1 / y.square().mean(1).sqrt()).clamp(max=3e38).float()
    want, bound = _moe_range.experts(x, ids, weights, *mats, bits, group)
    tol = _moe_range.tolerance(want, bound, dtype)
    got = aq.aq_moe_experts(x, aq.AqExperts(*mats, bits, group), ids, weights)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (bad.nonzero()[0].tolist(), float(got[bad][0]), float(want[bad][0]), float(tol[bad][0]))
    # zeros would not pass
    assert (want[1].abs() > tol[1]).double().mean() > 0.6

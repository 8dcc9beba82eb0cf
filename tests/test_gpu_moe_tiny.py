"""The router's choice among logits that 32 bits hardly hold: products of two
small bf16 numbers, below 2^-126 and below 2^-149."""
import pytest
import torch

import quantized_matmul_affine_gb300 as aq

from . import _moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [1e-34, 1e-37, 1e-39, 1e-41, 1e-43, 1e-45, 1e-50, 1e-60])
@pytest.mark.parametrize("T,K,E,top", [(1, 256, 64, 4), (5, 2048, 128, 8), (70, 576, 33, 3), (3, 64, 512, 16)])
def test_small_logits(T, K, E, top, size):
    """Logits of about `size`: weights alike, the choice theirs."""
    g = torch.Generator().manual_seed(T + E)
    x = (torch.randn(T, K, generator=g) * size ** 0.5).bfloat16().cuda()
    w = (torch.randn(E, K, generator=g) * size ** 0.5 * K ** -0.5).bfloat16().cuda()
    logits = x.double() @ w.double().T
    ids, p = aq.aq_moe_route(x, aq.AqRouter(w, top))
    want, _, _ = _moe.route(x, w, top)
    assert torch.equal(ids.long(), want)
    assert ((p.double() * top - 1).abs() <= (E + 32) * 2.0 ** -23).all()
    assert logits.abs().max() < 1e2 * size


@pytest.mark.parametrize("size", [1e-39, 1e-43, 1e-50])
def test_small_among_large(size):
    """The border among small logits, others far above and far below it."""
    T, K, E, top = 6, 512, 96, 8
    g = torch.Generator().manual_seed(7)
    x = torch.zeros(T, K)
    x[:, :256] = torch.randn(T, 256, generator=g) * size ** 0.5
    x[:, 256] = 1.0
    w = torch.zeros(E, K)
    w[:, :256] = torch.randn(E, 256, generator=g) * size ** 0.5
    w[::32, 256], w[1::4, 256] = 3.0, -3.0  # 3 certain, 24 not
    x, w = x.bfloat16().cuda(), w.bfloat16().cuda()
    ids, _ = aq.aq_moe_route(x, aq.AqRouter(w, top))
    # (one sum of all would not tell the small from each other beside 3)
    small = x[:, :256].double() @ w[:, :256].double().T
    large = w[:, 256].double()
    order = torch.sort(small, dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(large[order], dim=1, descending=True, stable=True).indices)
    assert torch.equal(ids.long(), order[:, :top].sort(1).values)
    assert (large[ids.long()] > 0).sum(1).eq(3).all()

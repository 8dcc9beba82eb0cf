"""Padded batches: rows of zeros, and of whatever was in memory, cost a call
nothing that its tokens do not."""
import pytest
import torch

import quantized_matmul_affine_gb300 as aq

from . import _moe

pytestmark = pytest.mark.gpu


def _time(x, router):
    ids, weights = aq.aq_moe_route(x, router)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(10):
            aq.aq_moe_route(x, router, out=(ids, weights))
    best = float("inf")
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("pad", [0.0, float("nan")])
@pytest.mark.parametrize("T,K,E,top", [(4, 2048, 128, 8), (64, 1024, 512, 16), (200, 5120, 256, 8)])
def test_padding(T, K, E, top, pad, bias):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    w = (torch.randn(E, K, generator=g) * K ** -0.5).bfloat16().cuda()
    kw = dict(score="sigmoid", bias=torch.zeros(E, device="cuda")) if bias else {}
    router = aq.AqRouter(w, top, **kw)
    padded = x.clone()
    padded[T // 2:] = pad
    ids, p = aq.aq_moe_route(padded, router)
    want, exact, rel = _moe.route(padded[:T // 2], w, top, **kw)
    assert torch.equal(ids[:T // 2].long(), want)
    assert (ids[:, 1:] > ids[:, :-1]).all() and (ids >= 0).all() and (ids < E).all()
    if pad == 0:  # all experts alike: the lowest, with like weights
        assert (ids[T // 2:] == torch.arange(top, device="cuda")).all()
        assert ((p[T // 2:].double() * top - 1).abs() <= (E + 32) * 2.0 ** -23).all()
    # 512 experts one after the other are milliseconds, a call is 6 to 35 us
    assert _time(padded, router) < 5 * _time(x, router)


def test_zeros_against_biases():
    """Of zeros the choice is the biases', to the last bit that 64 bits have."""
    E = 70
    bias = torch.full((E,), 0.25)
    bias[[3, 60]] += 2.0 ** -24
    bias[69] += 2.0 ** -25  # half a step in the sum with 0.5, a quarter in fp32's
    w = torch.randn(E, 128, generator=torch.Generator().manual_seed(1)).half().cuda()
    ids, _ = aq.aq_moe_route(torch.zeros(2, 128, dtype=torch.float16, device="cuda"),
                             aq.AqRouter(w, 4, score="sigmoid", bias=bias.cuda()))
    assert (ids == torch.tensor([0, 3, 60, 69], dtype=torch.int32, device="cuda")).all()

"""What an MMA step of the router may lose: the error bound under the choice
takes each of a step's 16 products to be cut at 2^-24 of the largest, 4.5 * 2^-22
of the sum of magnitudes with the roundings after it.  Logits are read back from
the weights of a softmax over all experts, beside an expert whose logit is 0."""
import pytest
import torch

import quantized_matmul_affine_gb300 as aq

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
BOUND = 4.5 * 2.0 ** -22


def _steps(K):
    """The products of each MMA step: [K / 16, 16] positions."""
    k = torch.arange(K).view(-1, 4, 2, 4)  # 32 values: four lanes' eight, two steps' four of each
    return k.transpose(1, 2).reshape(-1, 16)


def _error(x, w):
    """|logit - exact| over the sum of magnitudes, and what of it the weights'
    own roundings allow, for every expert but the first."""
    E = w.shape[0]
    ids, p = aq.aq_moe_route(x, aq.AqRouter(w, E, normalize=False))
    assert (ids == torch.arange(E, device="cuda")).all()
    got = (p.double() / p[:, :1].double()).log()[:, 1:]
    exact = (x.double() @ w.double().T)[:, 1:]
    mag = (x.double().abs() @ w.double().abs().T)[:, 1:]
    assert p.isfinite().all() and (p > 0).all()
    # a logit and its distance from the largest are rounded; exp is good to two
    # places, the quotients to a half
    high = exact.abs().amax(1, keepdim=True)
    own = 2.0 ** -24 * (exact.abs() + 2 * high + 2 * BOUND * mag) + 6 * 2.0 ** -23
    return (got - exact).abs(), own, mag


def _dominated(K, low, T, dtype):
    """Steps of one product of 2^18 and 15 about 2^-low of it, of one sign; the
    next step has -2^18, so that the small ones are the logit."""
    g = torch.Generator().manual_seed(K + low)
    E, steps = 16, _steps(K)
    # (as many steps as leave the logits within what exp holds)
    steps = steps[: max(2, min(len(steps), 2 << max(0, low - 24)))]
    x, w = torch.ones(T, K), torch.zeros(E, K)
    for i, at in enumerate(steps):
        big = at[int(torch.randint(0, 16, (1,), generator=g))]
        small = 2.0 ** (18 - low) * (1 + torch.rand(E - 1, 16, generator=g))
        small[::3] *= 2.0 ** torch.randint(-3, 2, (E - 1, 16), generator=g)[::3]  # of different sizes
        w[1:, at] = small * (1 - 2 * (torch.arange(E - 1) % 2))[:, None]
        x[:, big], w[1:, big] = 2.0 ** 9, 2.0 ** 9 * (-1) ** i
    return x.to(dtype).cuda(), w.to(dtype).cuda()


def _cancelling(K, T, dtype):
    """Products of all sizes from 2^-12 to 2^12 that cancel in pairs, half of a
    pair in another step; a few small ones are left."""
    g = torch.Generator().manual_seed(K)
    E, n = 16, K // 2
    order = torch.randperm(K, generator=g)
    a, b = order[:n], order[n:]
    x, w = torch.zeros(T, K), torch.zeros(E, K)
    x[:, a] = 2.0 ** torch.randint(-6, 7, (T, n), generator=g) * (1 + torch.rand(T, n, generator=g))
    w[1:, a] = 2.0 ** torch.randint(-6, 7, (E - 1, n), generator=g) * torch.randn(E - 1, n, generator=g)
    x[:, b], w[:, b] = x[:, a], -w[:, a]
    w[1:, b[:4]] = 0
    w[1:, a[:4]] = torch.randn(E - 1, 4, generator=g) / 64
    return x.to(dtype).cuda(), w.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("K,low", [(64, 23), (64, 24), (64, 25), (512, 24), (512, 27), (4096, 26), (5120, 22)])
def test_one_term_dominates(K, low, T, dtype):
    off, own, mag = _error(*_dominated(K, low, T, dtype))
    assert (off <= BOUND * mag + own).all(), float(((off - own) / mag).max())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,K", [(1, 64), (9, 320), (70, 512), (8, 2048)])
def test_sums_that_cancel(T, K, dtype):
    off, own, mag = _error(*_cancelling(K, T, dtype))
    assert (off <= BOUND * mag + own).all(), float(((off - own) / mag).max())

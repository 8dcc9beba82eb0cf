"""The router's choice where sums in 32 bits end: products that pass their
range and cancel, rows that are not finite.  Each row has top_k distinct experts
whatever its numbers are, and nothing outside the outputs is written."""
import pytest
import torch

import quantized_matmul_affine_gb300 as aq

from . import _moe

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
SPOTS = [0, 256, 8, 264]  # a lane's own four values in the second summation, two of either sign


def _inputs(T, K, E, dtype=BF16, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g)
    w = torch.randn(E, K, generator=g) * K ** -0.5
    x[:, SPOTS] = 0
    w[:, SPOTS] = 0
    return x.to(dtype).cuda(), w.to(dtype).cuda()


def _guarded(x, router):
    """aq_moe_route with canaries before and after both outputs."""
    T, top = x.shape[0], router.top_k
    ids = torch.full((T + 8, top), -7, dtype=torch.int32, device="cuda")
    weights = torch.full((T + 8, top), -7.0, device="cuda")
    aq.aq_moe_route(x, router, out=(ids[4:T + 4], weights[4:T + 4]))
    for t in (ids, weights):
        assert (t[:4] == -7).all() and (t[T + 4:] == -7).all()
    ids, weights = ids[4:T + 4], weights[4:T + 4]
    assert (ids[:, 1:] > ids[:, :-1]).all() and (ids >= 0).all() and (ids < router.weight.shape[0]).all()
    return ids, weights


@pytest.mark.parametrize("mode", ["softmax", "plain", "sigmoid", "bias"])
@pytest.mark.parametrize("T,K,E,top", [(1, 512, 64, 1), (5, 512, 64, 2), (9, 576, 33, 8), (70, 512, 200, 3),
                                       (4, 2048, 512, 16), (3, 320, 5, 5)])
def test_products_that_cancel(T, K, E, top, mode):
    """Products of 2e38, twice with either sign: the logit is 0, the sums on the
    way to it are not finite in 32 bits."""
    x, w = _inputs(T, K, E, seed=T + E)
    kw = dict(score="softmax" if mode in ("softmax", "plain") else "sigmoid", normalize=mode != "plain",
              bias=torch.linspace(-0.2, 0.2, E).cuda() if mode == "bias" else None)
    rows = sorted({T // 2, T - 1})
    spots = [s for s in SPOTS if s < K]
    big = sorted({0, E // 2, E - 1})
    calm = _guarded(x, aq.AqRouter(w, top, **kw))
    w2, x2 = w.clone(), x.clone()
    w2[big] = 0
    w2[torch.tensor(big)[:, None], torch.tensor(spots)] = torch.tensor([1e19, 1e19, -1e19, -1e19][:len(spots)],
                                                                      dtype=BF16).cuda()
    x2[torch.tensor(rows)[:, None], torch.tensor(spots)] = torch.tensor(2e19, dtype=BF16).cuda()
    if len(spots) == 3:  # 0, 256 and 8: the pair that cancels, and one that does not take part
        w2[:, 256] = 0
    router = aq.AqRouter(w2, top, **kw)
    ids, p = _guarded(x2, router)
    want, exact, _ = _moe.route(x2, w2, top, **kw)
    assert torch.equal(ids.long(), want)
    # sums in 64 bits become logits of 32: half a step each, twice over as in the
    # models' bound, beside the roundings of exp and of the sum over experts
    logits = x2.double() @ w2.double().T
    assert (logits[rows][:, big] == 0).all()
    off = 2.0 ** -24 * logits.abs().amax(1, keepdim=True)
    mag = (x2.double().abs() @ w2.double().abs().T).amax(1, keepdim=True)
    off = torch.where(mag < 1e30, (K / 32 + 24) * 2.0 ** -22 * mag, off)
    rel = torch.expm1(2 * off) + (E + 32) * 2.0 ** -23
    assert ((p.double() - exact).abs() <= rel * exact).all()
    # the other tokens are those of a call without the large ones
    others = [t for t in range(T) if t not in rows]
    if others:
        again = _guarded(x, router)
        assert torch.equal(ids[others], again[0][others]) and torch.equal(p[others], again[1][others])
    # and the call itself repeats
    assert all(torch.equal(a, b) for a, b in zip(_guarded(x2, router), (ids, p)))
    assert calm[0].shape == ids.shape


@pytest.mark.parametrize("top", [1, 4])
def test_all_sums_past_the_range(top):
    """Every expert's magnitudes pass the largest float; the logits differ."""
    T, K, E = 3, 512, 40
    x, w = _inputs(T, K, E)
    w[:] = 0
    w[:, [0, 256]], w[:, [8, 264]] = 1e19, -1e19
    # (times 2^40, so that 64 bits tell 2e38 + v from 2e38)
    w[:, 5] = (torch.randperm(E, generator=torch.Generator().manual_seed(3)) * 2.0 ** 40).to(BF16).cuda()
    x[:] = 0
    x[:, SPOTS] = 2e19
    x[:, 5] = 2e19
    ids, _ = _guarded(x, aq.AqRouter(w, top))
    want = w[:, 5].float().sort(descending=True, stable=True).indices[:top].sort().values
    assert (ids.long() == want).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("mode", ["softmax", "bias"])
def test_tokens_that_are_not_finite(bad, mode):
    for dtype, T, E, top in ((BF16, 4, 64, 3), (F16, 70, 100, 16), (BF16, 2, 512, 16), (F16, 1, 3, 1)):
        x, w = _inputs(T, 320, E, dtype, seed=E)
        router = aq.AqRouter(w, top, score="softmax" if mode == "softmax" else "sigmoid",
                             bias=torch.zeros(E).cuda() if mode == "bias" else None)
        good = _guarded(x, router)
        x2 = x.clone()
        x2[T - 1, 7] = bad
        got = _guarded(x2, router)
        assert torch.equal(got[0][:-1], good[0][:-1]) and torch.equal(got[1][:-1], good[1][:-1])
        x2[T - 1] = bad
        _guarded(x2, router)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_experts_that_are_not_finite(bad):
    """An expert whose row is not finite: every token still has its experts, and
    one that is not a number is not among them."""
    x, w = _inputs(6, 320, 48)
    w[11, 3] = bad
    ids, _ = _guarded(x, aq.AqRouter(w, 4))
    if bad != bad:
        rest = w.clone()
        rest[11] = 0
        logits = x.double() @ rest.double().T
        logits[:, 11] = -torch.inf
        assert torch.equal(ids.long(), logits.sort(dim=1, descending=True, stable=True).indices[:, :4].sort(1).values)


def test_biases_that_are_not_finite():
    """Infinite biases beside sums past the range, and more forbidden experts
    than leave top_k."""
    x, w = _inputs(3, 512, 40)
    w[7] = 0
    w[7, SPOTS] = torch.tensor([1e19, 1e19, -1e19, -1e19], dtype=BF16).cuda()
    x[1, SPOTS] = 2e19
    bias = torch.zeros(40)
    bias[[0, 5]], bias[9] = -torch.inf, torch.inf
    ids, _ = _guarded(x, aq.AqRouter(w, 4, score="sigmoid", bias=bias.cuda()))
    want, _, _ = _moe.route(x, w, 4, score="sigmoid", bias=bias.cuda())
    assert torch.equal(ids.long(), want)
    bias[:] = -torch.inf
    bias[[2, 7]] = 0.0
    ids, _ = _guarded(x, aq.AqRouter(w, 4, score="sigmoid", bias=bias.cuda()))
    assert (ids == torch.tensor([0, 1, 2, 7], dtype=torch.int32, device="cuda")).all()
    bias[3] = torch.nan
    _guarded(x, aq.AqRouter(w, 4, score="sigmoid", bias=bias.cuda()))

"""The experts' layer (router, products, both) and the embedding lookup on the
GPU against the 64-bit models of tests/_moe.py."""
import pytest
import torch

import quantized_matmul_affine_gb300 as aq

from . import _moe

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _layer(E, K, inner, bits, group, seed):
    g = _gen(seed)
    return [_moe.stack(E, r, c, bits, group, g, "cuda")
            for r, c in ((inner, K), (inner, K), (K, inner))]


def _tokens(T, K, dtype, seed):
    g = _gen(seed)
    gain = 0.5 + torch.rand(K, generator=g)
    gain[torch.randint(0, K, (max(1, K // 100),), generator=g)] *= 8
    return (torch.randn(T, K, generator=g) * gain).to(dtype).cuda()


def _ids(T, E, top, seed, absent=0.0):
    g = _gen(seed)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :top].int()
    ids[torch.rand(T, top, generator=g) < absent] = -1
    return ids.contiguous().cuda()


def _weights(T, top, seed):
    return torch.randn(T, top, generator=_gen(seed)).cuda()


def _run(T, K, inner, E, top, bits, group, dtype, absent=0.0, ids=None, seed=3):
    mats = _layer(E, K, inner, bits, group, seed)
    x = _tokens(T, K, dtype, seed + 1)
    ids = _ids(T, E, top, seed + 2, absent) if ids is None else ids
    w = _weights(*ids.shape, seed + 3)
    y = aq.aq_moe_experts(x, aq.AqExperts(*mats, bits, group), ids, w)
    want, bound = _moe.experts(x, ids, w, *mats, bits, group)
    _moe.check(y, want, bound, dtype)
    return x, mats, ids, w, y


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("bits", [2, 3, 4, 5, 6, 8])
def test_experts_formats(bits, group, dtype):
    _run(3, 256, 128, 5, 2, bits, group, dtype)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("bits", [2, 3, 4, 5, 6, 8])
@pytest.mark.parametrize("T,K,inner,E,top", [
    (3, 8192, 128, 2, 2),   # 8 columns, packed rows
    (14, 640, 128, 3, 2),   # 16 columns
    (50, 384, 256, 2, 1),   # 32 columns
])
def test_experts_packed(T, K, inner, E, top, bits, group):
    _run(T, K, inner, E, top, bits, group, F16 if bits & 1 else BF16)


@pytest.mark.parametrize("K", [64, 128, 192, 256, 320, 512, 576])
@pytest.mark.parametrize("bits,group", [(3, 64), (5, 32), (4, 32), (8, 64)])
@pytest.mark.parametrize("T", [2, 20])
def test_experts_widths(T, K, bits, group):
    """Rows of codes and scales that are and are not whole 16-byte pieces."""
    _run(T, K, 64 * (K // 128 + 1), 3, 2, bits, group, F16)


@pytest.mark.parametrize("T", [2, 20])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_experts_offsets(T, group):
    """Scales and biases that are aligned to their elements only."""
    mats = _layer(3, 256, 128, 4, group, 5)

    def shifted(t):
        buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
        buf[1:] = t.flatten()
        return buf[1:].view(t.shape)

    moved = [(w, shifted(a), shifted(b)) for w, a, b in mats]
    assert all(a.data_ptr() % 4 == 2 for _, a, _ in moved)
    x, ids, w = _tokens(T, 256, BF16, 6), _ids(T, 3, 2, 7), _weights(T, 2, 8)
    y = aq.aq_moe_experts(x, aq.AqExperts(*moved, 4, group), ids, w)
    assert torch.equal(y, aq.aq_moe_experts(x, aq.AqExperts(*mats, 4, group), ids, w))


def test_experts_uneven():
    """One expert with most of the tokens, others with few or none."""
    ids = torch.full((200, 2), -1, dtype=torch.int32)
    ids[:, 0] = 5
    ids[3:9, 1] = 0
    ids[100, 1] = 39
    ids[::7, 1] = 20
    _run(200, 512, 256, 40, 2, 4, 64, BF16, ids=ids.cuda())


def test_written_just_before():
    """Weights, ids and tokens written by the launches right before the call,
    over and over: nothing is read before they are complete."""
    E, K, inner = 6, 512, 256
    w = [torch.randn(E * r, c, generator=_gen(i)).half().cuda() for i, (r, c) in
         enumerate(((inner, K), (inner, K), (K, inner)))]
    made = [tuple(t.view(E, -1, t.shape[1]) for t in aq.aq_quantize(m, 4)) for m in w]
    live = [tuple(t.clone() for t in m) for m in made]
    ex = aq.AqExperts(*live, 4, 64)
    x0, ids0, wt = _tokens(4, K, F16, 1), _ids(4, E, 2, 2), _weights(4, 2, 3)
    want = aq.aq_moe_experts(x0, aq.AqExperts(*made, 4, 64), ids0, wt)
    x, ids = torch.zeros_like(x0), torch.zeros_like(ids0)
    for _ in range(20):
        for m in live:
            for t in m:
                t.zero_()
        x.zero_()
        ids.fill_(-1)
        for a, b in zip(live, made):
            for t, s in zip(a, b):
                t.copy_(s)
        ids.copy_(ids0)
        x.copy_(x0)
        assert torch.equal(aq.aq_moe_experts(x, ex, ids, wt), want)


@pytest.mark.parametrize("T,K,inner,E,top,bits,group", [
    (1, 64, 64, 1, 1, 4, 64),          # the smallest
    (1, 64, 64, 1, 1, 3, 32),
    (1, 2048, 768, 128, 8, 4, 64),     # fewer tiles than CTAs and more
    (2, 64, 64, 512, 16, 4, 64),       # the most experts and experts a token
    (5, 1408, 192, 60, 4, 3, 64),      # units that do not divide by the warps
    (7, 5120, 64, 3, 2, 4, 64),        # a long K
    (1, 128, 13824, 2, 1, 4, 128),     # a long inner size: chunks of the second product
    (9, 64, 8192, 2, 2, 8, 32),
    (256, 320, 192, 2, 2, 4, 64),      # every token on both experts: 8 column blocks
    (256, 128, 64, 7, 3, 5, 32),
    (40, 8192, 64, 1, 1, 6, 32),       # chunks with 32 and with 8 columns
    (33, 4096, 128, 2, 1, 2, 128),
    (64, 1024, 512, 16, 4, 8, 128),
])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_experts_shapes(T, K, inner, E, top, bits, group, dtype):
    _run(T, K, inner, E, top, bits, group, dtype, absent=0.2 if T > 4 else 0.0)


@pytest.mark.parametrize("count", [1, 7, 8, 9, 16, 17, 31, 32, 33, 65])
def test_experts_columns(count):
    """Every number of an expert's tokens around the column blocks' ends."""
    ids = torch.full((70, 2), -1, dtype=torch.int32)
    ids[:count, 1] = 2
    ids[5:9, 0] = 0
    _run(70, 256, 64, 4, 2, 4, 64, BF16, ids=ids.cuda())


def test_experts_absent():
    """Rows without an expert are zeros; ids outside the range add nothing."""
    ids = torch.tensor([[-1, -1], [3, -2 ** 31], [2 ** 31 - 1, 4], [0, 1]], dtype=torch.int32).cuda()
    y = _run(4, 128, 64, 4, 2, 4, 32, F16, ids=ids)[-1]
    assert not y[0].any() and not y[2].any() and y[1].any()
    none = torch.full((4, 2), -1, dtype=torch.int32).cuda()
    assert not _run(4, 128, 64, 4, 2, 4, 32, F16, ids=none)[-1].any()


def test_experts_twice():
    """The same expert twice in a row counts twice."""
    ids = torch.tensor([[1, 1, 0], [2, 2, 2]], dtype=torch.int32).cuda()
    _run(2, 128, 64, 3, 3, 4, 64, BF16, ids=ids)


@pytest.mark.parametrize("dtype,size", [(F16, 6e4), (F16, 1e-6), (BF16, 1e30), (BF16, 1e-30)])
def test_experts_ranges(dtype, size):
    """Activations near the ends of their type, in one token of three: each
    token has its own power of two."""
    mats = _layer(2, 128, 64, 4, 64, 1)
    x = _tokens(3, 128, dtype, 2)
    x[1] = (x[1].float() / x[1].abs().max().float() * size).to(dtype)
    if size > 1e20:  # keep h within fp32: gate products of 1e30 saturate silu
        mats[1] = (mats[1][0], mats[1][1] * 0, mats[1][2] * 0)
    ids, w = torch.zeros(3, 1, dtype=torch.int32).cuda(), torch.ones(3, 1).cuda()
    y = aq.aq_moe_experts(x, aq.AqExperts(*mats, 4, 64), ids, w)
    want, bound = _moe.experts(x, ids, w, *mats, 4, 64)
    big = want.abs() + bound >= 6.5e4 if dtype == F16 else torch.zeros_like(want, dtype=torch.bool)
    _moe.check(torch.where(big, torch.zeros_like(y), y), torch.where(big, torch.zeros_like(want), want),
               torch.where(big, torch.zeros_like(want), bound), dtype)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_experts_not_finite(bad):
    """A token that is not finite leaves the others alone."""
    mats = _layer(3, 128, 64, 4, 64, 1)
    x, ids, w = _tokens(4, 128, BF16, 2), _ids(4, 3, 2, 3), _weights(4, 2, 4)
    ex = aq.AqExperts(*mats, 4, 64)
    good = aq.aq_moe_experts(x, ex, ids, w)
    x2 = x.clone()
    x2[2, 7] = bad
    y = aq.aq_moe_experts(x2, ex, ids, w)
    assert torch.equal(y[[0, 1, 3]], good[[0, 1, 3]]) and not torch.isfinite(y[2]).all()


def test_experts_neighbours():
    """Nothing outside y is written; the workspace needs no initial value."""
    mats = _layer(4, 256, 128, 4, 64, 1)
    ex = aq.AqExperts(*mats, 4, 64)
    x, ids, w = _tokens(6, 256, F16, 2), _ids(6, 4, 2, 3), _weights(6, 2, 4)
    want = aq.aq_moe_experts(x, ex, ids, w)
    buf = torch.full((8, 256), 7.0, dtype=F16, device="cuda")
    n = aq.aq_moe_workspace_bytes(ex, 6, 2)
    ws = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    aq.aq_moe_experts(x, ex, ids, w, out=buf[1:7], workspace=ws[256:256 + n])
    assert torch.equal(buf[1:7], want) and (buf[[0, 7]] == 7).all()
    assert (ws[:256] == 255).all() and (ws[256 + n:] == 255).all()


ROUTES = [(1, 64, 1, 1), (1, 2048, 128, 8), (3, 64, 5, 5), (8, 96 * 64, 60, 4), (9, 512, 16, 2),
          (17, 320, 17, 3), (64, 256, 512, 16), (65, 5120, 256, 8), (256, 1024, 100, 6), (2, 64, 33, 16)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("mode", ["softmax", "plain", "sigmoid", "bias"])
@pytest.mark.parametrize("T,K,E,top", ROUTES)
def test_route(T, K, E, top, mode, dtype):
    g = _gen(T + E)
    x = _tokens(T, K, dtype, T)
    w = (torch.randn(E, K, generator=g) * 2 * K ** -0.5).to(dtype).cuda()
    kw = dict(score="softmax" if mode in ("softmax", "plain") else "sigmoid",
              normalize=mode != "plain", scale=2.5 if mode != "softmax" else 1.0,
              bias=(0.3 * torch.randn(E, generator=g)).cuda() if mode == "bias" else None)
    ids, p = aq.aq_moe_route(x, aq.AqRouter(w, top, **kw))
    want, exact, rel = _moe.route(x, w, top, **kw)
    assert torch.equal(ids.long(), want)
    assert ((p.double() - exact).abs() <= rel * exact.abs()).all()


@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("bias", [False, True])
def test_route_border(T, bias):
    """Experts that differ by less than fp32 sums tell, and equal ones."""
    K, E, top = 2048, 64, 8
    g = _gen(5)
    x = _tokens(T, K, BF16, 6)
    base = torch.randn(K, generator=g) * K ** -0.5
    w = base.repeat(E, 1).bfloat16()
    for e in range(0, E, 2):  # one value a row moved by a step, where x is small: logits 1e-6 apart
        k = int(x[0].abs().cpu().argsort()[e + 1])
        w[e, k] = torch.nextafter(w[e, k].float(), torch.tensor(9.0)).bfloat16() * (1 + 2 ** -7)
    w = w.cuda()
    kw = dict(score="sigmoid", bias=torch.zeros(E).cuda()) if bias else {}
    ids, _ = aq.aq_moe_route(x, aq.AqRouter(w, top, **kw))
    want, _, _ = _moe.route(x, w, top, **kw)
    logits = x.double() @ w.double().T
    assert torch.equal(ids[:1].long(), want[:1])
    # beyond token 0 the model's own sums may tie differently: compare the chosen values
    a, b = (logits.gather(1, i.long()).sort(1).values for i in (ids, want))
    assert (a - b).abs().max() <= 2.0 ** -44 * (x.double().abs() @ w.double().abs().T).max()
    assert (ids[:, 1:] > ids[:, :-1]).all()
    same = torch.zeros(E, K, dtype=BF16).cuda() + base.bfloat16().cuda()
    ids, p = aq.aq_moe_route(x, aq.AqRouter(same, top, **kw))
    assert (ids == torch.arange(top, device="cuda")).all() and ((p - 1 / top).abs() < 1e-6).all()


def test_route_ends():
    """Biases that forbid and force experts; sigmoids that vanish; logits that
    are not finite."""
    x = _tokens(3, 128, F16, 1)
    w = torch.randn(9, 128, generator=_gen(2)).half().cuda()
    bias = torch.zeros(9)
    bias[[1, 4]], bias[7] = float("-inf"), float("inf")
    ids, p = aq.aq_moe_route(x, aq.AqRouter(w, 4, bias=bias.cuda(), score="sigmoid"))
    want, exact, rel = _moe.route(x, w, 4, bias=bias.cuda(), score="sigmoid")
    assert torch.equal(ids.long(), want) and (ids == 7).any(1).all()
    assert ((p.double() - exact).abs() <= rel * exact).all()
    low = -w.abs() * 3
    one = torch.full_like(x, 1.0)
    ids, p = aq.aq_moe_route(one, aq.AqRouter(low, 2, score="sigmoid"))
    want, exact, rel = _moe.route(one, low, 2, score="sigmoid")
    assert torch.equal(ids.long(), want) and ((p.double() - exact).abs() <= rel * exact).all()
    good = aq.aq_moe_route(x, aq.AqRouter(w, 4))
    for bad in (float("nan"), float("inf")):
        x2 = x.clone()
        x2[1, 5] = bad
        ids, p = aq.aq_moe_route(x2, aq.AqRouter(w, 4))
        for a, b in zip((ids, p), good):
            assert torch.equal(a[[0, 2]], b[[0, 2]])
        assert (ids[1, 1:] > ids[1, :-1]).all() and 0 <= int(ids[1, 0]) and int(ids[1, -1]) < 9


@pytest.mark.parametrize("T", [1, 6, 90])
def test_layer(T):
    """aq_moe is aq_moe_route and aq_moe_experts, bit for bit, call after call."""
    mats = _layer(24, 512, 192, 4, 64, 1)
    x = _tokens(T, 512, BF16, 2)
    router = aq.AqRouter((torch.randn(24, 512, generator=_gen(3)) / 16).bfloat16().cuda(), 3)
    ex = aq.AqExperts(*mats, 4, 64)
    y, ids, w = aq.aq_moe(x, router, ex)
    ids2, w2 = aq.aq_moe_route(x, router)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    assert torch.equal(y, aq.aq_moe_experts(x, ex, ids, w))
    want, bound = _moe.experts(x, ids, w, *mats, 4, 64)
    _moe.check(y, want, bound, BF16)
    for _ in range(5):
        again = aq.aq_moe(x, router, ex)
        assert all(torch.equal(a, b) for a, b in zip(again, (y, ids, w)))


def test_captured():
    """A captured layer follows its inputs' changes; two graphs share no memory
    that the calls need between replays."""
    mats = _layer(8, 256, 128, 3, 64, 1)
    router = aq.AqRouter((torch.randn(8, 256, generator=_gen(3)) / 16).half().cuda(), 2)
    ex = aq.AqExperts(*mats, 3, 64)
    xs = [_tokens(T, 256, F16, 10 + T) for T in (1, 5)]
    graphs = []
    for x in xs:
        aq.aq_moe(x, router, ex)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = aq.aq_moe(x, router, ex)
        graphs.append((g, x, got))
    for seed in (50, 60):
        for g, x, got in graphs:
            x.copy_(_tokens(*x.shape, F16, seed))
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, x, got in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, aq.aq_moe(x, router, ex)))


def test_streams():
    """Calls on two streams at once, each with memory of its own."""
    mats = _layer(8, 512, 256, 4, 64, 1)
    router = aq.AqRouter((torch.randn(8, 512, generator=_gen(3)) / 16).bfloat16().cuda(), 2)
    ex = aq.AqExperts(*mats, 4, 64)
    xs = [_tokens(7, 512, BF16, s) for s in (1, 2)]
    want = [aq.aq_moe(x, router, ex)[0] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for i in range(20):
        for x, s in zip(xs, streams):  # by argument, and as the current stream
            if i & 1:
                got.append(aq.aq_moe(x, router, ex, stream=s)[0])
            else:
                with torch.cuda.stream(s):
                    got.append(aq.aq_moe(x, router, ex)[0])
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])


@pytest.mark.parametrize("bits,group,K", [(2, 32, 64), (3, 64, 192), (3, 32, 32), (4, 64, 4096), (5, 128, 128),
                                          (5, 32, 96), (6, 64, 320), (6, 32, 32), (8, 128, 256), (8, 32, 32)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_embed(bits, group, K, dtype):
    N = 300
    words, s, b = (t[0] for t in _moe.stack(1, N, K, bits, group, _gen(bits), "cuda"))
    for T, index in ((1, torch.int32), (5, torch.int64), (1000, torch.int32)):
        ids = torch.randint(-1, N, (T,), generator=_gen(T)).to(index)
        ids[0] = N - 1  # the table's last row
        if T > 1:
            ids[1:5] = torch.tensor([0, N, -1, torch.iinfo(index).max]).to(index)
        buf = torch.full((T + 2, K), 7.0, dtype=dtype, device="cuda")
        got = aq.aq_embed(ids.cuda(), words, s, b, bits, group, dtype, scale=K ** 0.5, out=buf[1:T + 1])
        want, bound = _moe.embed(ids.cuda(), (words, s, b), bits, group, K ** 0.5)
        _moe.check(got, want, bound, dtype, f"T={T}")
        assert (buf[[0, -1]] == 7).all()


def test_embed_shapes():
    words, s, b = (t[0] for t in _moe.stack(1, 20, 64, 4, 64, _gen(1), "cuda"))
    ids = torch.arange(12, device="cuda").view(3, 4)
    out = aq.aq_embed(ids, words, s, b, 4, 64, F16)
    assert out.shape == (3, 4, 64)
    assert torch.equal(out[2, 1], aq.aq_embed(ids[2, 1:2], words, s, b, 4, 64, F16)[0])
    assert aq.aq_embed(ids[:0], words, s, b, 4, 64, F16).shape == (0, 4, 64)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_decoder_step(dtype):
    """Tokens to logits as a decoder has them: embedding rows, two experts'
    layers with their residuals, the same table as the vocabulary projection;
    each step against the model on the step's own input."""
    V, K, inner, E, top, T = 400, 512, 192, 12, 3, 5
    table = tuple(t[0] for t in _moe.stack(1, V, K, 4, 64, _gen(1), "cuda"))
    ids = torch.randint(0, V, (T,), generator=_gen(2)).cuda()
    x = aq.aq_embed(ids, *table, 4, 64, dtype, scale=K ** 0.5)
    want, bound = _moe.embed(ids, table, 4, 64, K ** 0.5)
    _moe.check(x, want, bound, dtype, "embed")
    for n in range(2):
        mats = _layer(E, K, inner, 4, 64, 7 + n)
        router = aq.AqRouter((torch.randn(E, K, generator=_gen(9 + n)) * K ** -0.5).to(dtype).cuda(), top)
        y, chosen, w = aq.aq_moe(x, router, aq.AqExperts(*mats, 4, 64))
        want_ids, want_w, rel = _moe.route(x, router.weight, top)
        assert torch.equal(chosen.long(), want_ids)
        assert ((w.double() - want_w).abs() <= rel * want_w).all()
        want, bound = _moe.experts(x, chosen, w, *mats, 4, 64)
        _moe.check(y, want, bound, dtype, f"layer {n}")
        x = x + y
    logits = (aq.aq_matmul if dtype == F16 else aq.aq_matmul_bf16)(x, *table, 4)
    v, mag = _moe.values(table, 4, 64)
    want = x.double() @ v.T
    assert ((logits.double() - want).abs() <= 2e-3 * (x.double().abs() @ v.abs().T) + 1e-5).all()
    assert aq.aq_device_error() == 0


def test_other_arguments():
    mats = _layer(4, 128, 64, 4, 64, 1)
    ex = aq.AqExperts(*mats, 4, 64)
    router = aq.AqRouter(torch.zeros(4, 128, dtype=F16, device="cuda"), 2)
    x = _tokens(3, 128, F16, 1)
    ids, w = aq.aq_moe_route(x, router)
    for call in (lambda: aq.aq_moe(x.bfloat16(), router, ex), lambda: aq.aq_moe_route(x.bfloat16(), router),
                 lambda: aq.aq_moe_experts(x[:, :64].contiguous(), ex, ids, w),
                 lambda: aq.aq_moe_experts(x, ex, ids[:2], w), lambda: aq.aq_moe_experts(x, ex, ids.long(), w),
                 lambda: aq.aq_moe_experts(x, ex, ids, w.half()), lambda: aq.aq_moe_experts(x.cpu(), ex, ids, w),
                 lambda: aq.aq_moe_experts(x.t().contiguous().t(), ex, ids, w),
                 lambda: aq.aq_moe_experts(x, ex, ids, w, out=x[:2]),
                 lambda: aq.aq_moe(x, aq.AqRouter(torch.zeros(5, 128, dtype=F16, device="cuda"), 2), ex),
                 lambda: aq.aq_moe_experts(x, ex, ids, w, workspace=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(aq.AqError):
        aq.aq_moe_experts(x, ex, ids, w, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(aq.AqError):
        aq.aq_moe_route(x[:0], router)
    with pytest.raises(aq.AqError):
        aq.aq_moe_route(x.expand(300, 3, 128)[:, 0].contiguous(), router)

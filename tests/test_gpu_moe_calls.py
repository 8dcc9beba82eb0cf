"""Ways to call the experts' layer and the embedding that its documentation
allows: a process's first call while a graph is captured, several host threads at
once, y over x, one workspace for calls of many sizes, the widest clusters in a
graph."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import quantized_matmul_affine_gb300 as aq

from . import _moe

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _layer(E, K, inner, bits, group, top, seed):
    g = torch.Generator().manual_seed(seed)
    mats = [_moe.stack(E, r, c, bits, group, g, "cuda") for r, c in ((inner, K), (inner, K), (K, inner))]
    w = (torch.randn(E, K, generator=g) * K ** -0.5).to(BF16).cuda()
    return aq.AqRouter(w, top), aq.AqExperts(*mats, bits, group)


def _x(T, K, seed):
    return torch.randn(T, K, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


FIRST = """
import torch, quantized_matmul_affine_gb300 as aq
from tests.test_gpu_moe_calls import _layer, _x
router, experts = _layer(256, 2048, 128, 4, 64, 8, 1)
table = [t[0] for t in experts.gate]
x, ids = _x(20, 2048, 2), torch.arange(20, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = aq.aq_moe(x, router, experts)
    e = aq.aq_embed(ids, *table, 4, 64, torch.float16)
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(y, aq.aq_moe(x, router, experts)))
assert torch.equal(e, aq.aq_embed(ids, *table, 4, 64, torch.float16))
print("same")
"""


def test_first_call_is_captured():
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and r.stdout == "same\n", r.stderr[-2000:]


def test_widest_clusters_in_a_graph():
    """A router over 16 CTAs a cluster, with the layer behind it, replayed after
    its tokens changed."""
    router, experts = _layer(256, 2048, 128, 4, 64, 8, 1)
    x = _x(20, 2048, 2)
    aq.aq_moe(x, router, experts)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = aq.aq_moe(x, router, experts)
    for seed in (3, 4):
        x.copy_(_x(20, 2048, seed))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, aq.aq_moe(x, router, experts)))


def test_threads():
    """Eight host threads, a stream each, layers of other sizes and widths."""
    sizes = [(1, 256, 128, 4, 64), (5, 512, 192, 3, 64), (20, 384, 128, 8, 32), (60, 256, 256, 5, 128),
             (200, 512, 64, 4, 64), (9, 2048, 128, 6, 64), (3, 8192, 64, 2, 64), (33, 1024, 128, 4, 32)]
    layers = [_layer(40, K, inner, bits, group, 3, i) for i, (T, K, inner, bits, group) in enumerate(sizes)]
    xs = [_x(s[0], s[1], 10 + i) for i, s in enumerate(sizes)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sizes]
    got, failed = [[] for _ in sizes], []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(15):
                    got[i].append(aq.aq_moe(xs[i], *layers[i]))
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for i, outs in enumerate(got):
        want = aq.aq_moe(xs[i], *layers[i])
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want)), i


@pytest.mark.parametrize("T", [1, 6, 20, 100])
def test_y_over_x(T):
    router, experts = _layer(12, 512, 128, 4, 64, 2, 1)
    x = _x(T, 512, 2)
    y, ids, w = aq.aq_moe(x, router, experts)
    z = x.clone()
    assert aq.aq_moe(z, router, experts, out=z)[0] is z and torch.equal(z, y)
    z = x.clone()
    aq.aq_moe_experts(z, experts, ids, w, out=z)
    assert torch.equal(z, y)


def test_one_workspace():
    """Calls of all sizes one after the other on one workspace, the largest's."""
    router, experts = _layer(12, 512, 128, 4, 64, 2, 1)
    n = max(aq.aq_moe_workspace_bytes(experts, T, 2) for T in range(1, 257))
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    sizes = [256, 1, 9, 130, 2, 33, 64, 17, 256, 3]
    xs = [_x(T, 512, T) for T in sizes]
    got = [aq.aq_moe(x, router, experts, workspace=ws)[0] for x in xs]
    for x, y in zip(xs, got):
        assert torch.equal(y, aq.aq_moe(x, router, experts)[0])


@pytest.mark.parametrize("top", [1, 16])
@pytest.mark.parametrize("T", [1, 2, 3, 256])
def test_one_expert_for_all(T, top):
    """The same expert in every slot of every token: the most entries of one."""
    K = inner = 128
    g = torch.Generator().manual_seed(1)
    mats = [_moe.stack(3, r, c, 4, 64, g, "cuda") for r, c in ((inner, K), (inner, K), (K, inner))]
    ids = torch.full((T, top), 2, dtype=torch.int32, device="cuda")
    w = torch.randn(T, top, generator=g).cuda()
    x = _x(T, K, 3)
    y = aq.aq_moe_experts(x, aq.AqExperts(*mats, 4, 64), ids, w)
    want, bound = _moe.experts(x, ids, w, *mats, 4, 64)
    _moe.check(y, want, bound, BF16)


def test_weights_of_the_sum():
    """Weights of entries that count are taken as they are, zeros and infinities
    too; those of empty slots are not read into y."""
    router, experts = _layer(6, 128, 64, 4, 64, 2, 1)
    x = _x(4, 128, 2)
    ids = torch.tensor([[0, 1], [-1, 3], [2, 99], [-1, -1]], dtype=torch.int32).cuda()
    w = torch.tensor([[0.0, 1.0], [float("nan"), 2.0], [1.0, float("inf")], [float("nan")] * 2]).cuda()
    y = aq.aq_moe_experts(x, experts, ids, w)
    w2 = torch.where(torch.isfinite(w), w, 0.0)
    assert torch.equal(y, aq.aq_moe_experts(x, experts, ids, w2)) and torch.isfinite(y).all() and not y[3].any()


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_embed_many(index):
    """Every row of a table, in an order that repeats, more tokens than a grid's
    usual size; ids whose low 32 bits alone would be rows."""
    g = torch.Generator().manual_seed(1)
    words, s, b = (t[0] for t in _moe.stack(1, 500, 96, 3, 32, g, "cuda"))
    ids = torch.randint(0, 500, (300001,), generator=g).to(index)
    ids[:500] = torch.arange(500)
    if index == torch.int64:
        ids[1000:1003] = torch.tensor([2 ** 32 + 5, -2 ** 32 + 5, 2 ** 62])
    ids = ids.cuda()
    out = aq.aq_embed(ids, words, s, b, 3, 32, BF16)
    rows = aq.aq_embed(torch.arange(500, device="cuda"), words, s, b, 3, 32, BF16)
    inside = (ids >= 0) & (ids < 500)
    want = torch.where(inside[:, None], rows[torch.where(inside, ids, 0).long()], torch.zeros((), dtype=BF16, device="cuda"))
    assert torch.equal(out, want)


def _random_stack(E, rows, cols, bits, group, gen):
    words = torch.randint(-2 ** 31, 2 ** 31, (E, rows, cols * bits // 32), dtype=torch.int32, device="cuda", generator=gen)
    s = (torch.rand((E, rows, cols // group), device="cuda", generator=gen) + 0.5) * (3.4 / 2 ** bits) * cols ** -0.5
    return words, s.half(), (-(2 ** bits - 1) / 2 * s).half()


@pytest.mark.parametrize("T", [1, 12])
def test_offsets_past_32_bits(T):
    """Stacks of 4.5 GB: the last experts' words lie past 2^32 bytes."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    E, K, inner = 80, 4096, 13824
    mats = [_random_stack(E, r, c, 8, 64, gen) for r, c in ((inner, K), (inner, K), (K, inner))]
    assert mats[0][0][E - 2].data_ptr() - mats[0][0].data_ptr() > 2 ** 32
    x, w = _x(T, K, 2), torch.ones(T, 2, device="cuda")
    ids = torch.tensor([[E - 2, E - 1], [0, E - 1]] * 6, dtype=torch.int32, device="cuda")[:T].contiguous()
    y = aq.aq_moe_experts(x, aq.AqExperts(*mats, 8, 64), ids, w)
    want, bound = _moe.experts(x, ids, w, *mats, 8, 64)
    _moe.check(y, want, bound, BF16)
    del mats
    torch.cuda.empty_cache()


def test_embed_past_32_bits():
    gen = torch.Generator(device="cuda").manual_seed(1)
    N, K = 1200000, 8192
    words, s, b = (t[0] for t in _random_stack(1, N, K, 4, 64, gen))
    assert words[N - 3].data_ptr() - words.data_ptr() > 2 ** 32
    ids = torch.tensor([N - 1, 0, N - 2, N, N // 2, 1048575, 1048576, 1048577], device="cuda")
    out = aq.aq_embed(ids, words, s, b, 4, 64, BF16, scale=2.0)
    want, bound = _moe.embed(ids, (words, s, b), 4, 64, 2.0)
    _moe.check(out, want, bound, BF16)
    del words, s, b
    torch.cuda.empty_cache()

"""The paged cache on the GPU: rows in and out bit for bit against an IEEE
fp32 model of the quantiser, page-table operations against plain loops, and
copies byte for byte."""
import numpy as np
import pytest
import torch

from . import _paged

pytestmark = pytest.mark.gpu

aq = pytest.importorskip("quantized_matmul_affine_gb300")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert aq.aq_device_error(clear=True) == 0


def _dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype))).cuda()


def _cache(pool, geo):
    return aq.AqCache(pool, geo.page, geo.D, geo.bits, geo.group)


def _rows(rng, T, heads, D, dtype):
    x = rng.standard_normal((T, heads, D)).astype(np.float32)
    x *= rng.random((1, heads, D)).astype(np.float32) * 4 + 0.05
    if T > 2:
        x[T // 2, 0, :] = 0.75           # a constant row: scale 0
    return torch.from_numpy(x).to(torch.bfloat16 if dtype == "bf16" else torch.float16)


def _quantised(x, geo):
    """codes uint8 [T, KV, D], pairs fp16 [T, KV, G, 2]: the rule in IEEE single precision."""
    w = x.float().numpy().reshape(*x.shape[:2], geo.groups, geo.group)
    lo, hi = w.min(-1, keepdims=True), w.max(-1, keepdims=True)
    top = np.float32(2 ** geo.bits - 1)
    s, b = ((hi - lo) / top).astype(np.float16), lo.astype(np.float16)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((w - b.astype(np.float32)) / s.astype(np.float32))
    q = np.where(s > 0, np.clip(np.nan_to_num(q), 0, top), 0)
    return q.reshape(x.shape).astype(np.uint8), np.concatenate((s, b), -1)


def _packed(codes, bits):
    b = (codes[..., None] >> np.arange(bits)) & 1
    return np.packbits(b.reshape(*codes.shape[:-1], -1).astype(np.uint8), axis=-1, bitorder="little")


CASES = [
    # KV, D, page, bits, group, lengths of the new tokens, dtype
    (2, 64, 16, 4, 32, [1], "bf16"),
    (1, 64, 16, 8, 64, [5, 0, 17], "fp16"),
    (8, 128, 64, 4, 64, [1] * 9, "bf16"),
    (8, 128, 32, 4, 128, [100, 3, 64, 31], "fp16"),
    (3, 256, 128, 8, 32, [7, 130], "bf16"),
    (1, 512, 16, 8, 128, [33], "fp16"),
    (2, 128, 16, 8, 32, [40, 1, 2, 3], "bf16"),
]


@pytest.mark.parametrize("KV,D,page,bits,group,new,dtype", CASES)
def test_append_and_read(KV, D, page, bits, group, new, dtype):
    geo = _paged.Geometry(KV, D, page, bits, group, layers=2)
    rng = np.random.default_rng(KV + D + page + bits + group)
    B, T = len(new), sum(new)
    start = rng.integers(0, 3 * page, size=B)
    have = [-(-int(s + n) // page) for s, n in zip(start, new)]
    n_pages = sum(have) + 2
    ids = rng.permutation(n_pages)
    table = np.full((B, max(have) + 1), -1)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = ids[at:at + n]
        at += n
    before = rng.integers(0, 256, size=(2, n_pages, KV, geo.rec), dtype=np.uint8)
    pool = torch.from_numpy(before.copy()).cuda()
    cache = _cache(pool, geo)
    # k and v are slices of one projection's output, with a padding token at its end
    fused = _rows(rng, T + 1, 2 * KV + 3, D, dtype)
    dev = fused.cuda()
    cu = np.concatenate(([0], np.cumsum(new)))
    k, v = dev[:, 3:3 + KV], dev[:, 3 + KV:]
    aq.aq_cache_append(cache, 1, k, v, _dev(cu), _dev(start), _dev(table))
    rk, rv = aq.aq_cache_read(cache, 1, _dev(cu), _dev(start), _dev(table), T + 1, dev.dtype)
    torch.cuda.synchronize()
    want = before.copy()
    for which, x in enumerate((fused[:T, 3:3 + KV], fused[:T, 3 + KV:])):
        codes, pairs = _quantised(x, geo)
        packed = _packed(codes, bits)
        sides = pairs.reshape(T, KV, -1).view(np.uint8)
        for b in range(B):
            for i in range(new[b]):
                pos, t = int(start[b]) + i, int(cu[b]) + i
                p, slot = table[b, pos // page], pos % page
                spans = geo.spans(slot)
                for data, (a, n) in ((packed, spans[which]), (sides, spans[2 + which])):
                    want[1, p, :, a:a + n] = data[t]
        val = pairs[..., :1].astype(np.float32) * codes.reshape(T, KV, geo.groups, group) + \
            pairs[..., 1:].astype(np.float32)
        val = torch.from_numpy(val.astype(np.float32).reshape(T, KV, D)).to(dev.dtype)
        got = (rk, rv)[which].cpu()
        assert torch.equal(got[:T], val)
        assert not got[T:].any()
    assert np.array_equal(pool.cpu().numpy(), want)


def test_append_places_outside_the_table():
    # a position past the table, a page number past the pool, an unset entry:
    # each is skipped and sets the error word, the others are written
    geo = _paged.Geometry(1, 64, 16, 4, 64)
    pool = torch.zeros(1, 3, 1, geo.rec, dtype=torch.uint8, device="cuda")
    cache = _cache(pool, geo)
    x = torch.ones(5, 1, 64, dtype=torch.float16, device="cuda")
    table = _dev([[0, -1], [3, 1], [2, 2], [2, 2], [-5, 2]])
    cu, start = _dev([0, 1, 2, 3, 4, 5]), _dev([16, 0, 32, -1, 3])
    assert aq.aq_device_error(clear=True) == 0
    aq.aq_cache_append(cache, 0, x, x, cu, start, table)
    torch.cuda.synchronize()
    assert aq.aq_device_error(clear=True) != 0
    assert not pool.any()
    k, v = aq.aq_cache_read(cache, 0, cu, start, table, 5, torch.float16)
    assert not k.any() and not v.any()
    assert aq.aq_device_error(clear=True) != 0


def test_copy():
    geo = _paged.Geometry(3, 128, 16, 4, 64, layers=3)
    rng = np.random.default_rng(5)
    host = rng.integers(0, 256, size=(3, 40, 3, geo.rec), dtype=np.uint8)
    pool = torch.from_numpy(host.copy()).cuda()
    order = rng.permutation(40)
    src, dst = order[:13], order[13:26]
    src[4] = dst[4]                          # onto itself
    aq.aq_cache_copy(_cache(pool, geo), _dev(src), _dev(dst))
    want = host.copy()
    want[:, dst] = host[:, src]
    assert np.array_equal(pool.cpu().numpy(), want)
    aq.aq_cache_copy(_cache(pool, geo), _dev([1, 40, -1]), _dev([40, 2, 3]))
    torch.cuda.synchronize()
    assert np.array_equal(pool.cpu().numpy(), want)
    assert aq.aq_device_error(clear=True) != 0


class Both:
    """The GPU's tables beside the plain model's."""

    def __init__(self, geo, n_pages, B, width, seed, in_place):
        self.geo, self.in_place = geo, in_place
        self.rng = np.random.default_rng(seed)
        self.host = self.rng.integers(0, 256, size=(geo.layers, n_pages, geo.KV, geo.rec), dtype=np.uint8)
        self.pool = torch.from_numpy(self.host.copy()).cuda()
        self.cache = _cache(self.pool, geo)
        self.refs, self.lens = _dev(np.zeros(n_pages)), _dev(np.zeros(B))
        self.table = _dev(np.full((B, width), -1))
        self.model = _paged.Tables(np.zeros(n_pages), np.full((B, width), -1), np.zeros(B), geo.page)

    def op(self, name, *args):
        f = getattr(aq, "aq_cache_" + name)
        before = [t.clone() for t in (self.refs, self.table, self.lens)]
        got = f(self.cache, self.refs, self.table, self.lens, *[_dev(a) for a in args],
                in_place=self.in_place)
        want = getattr(self.model, name)(*args)
        moves = []
        if isinstance(want, tuple):
            want, moves = want
        torch.cuda.synchronize()
        if not self.in_place:
            for t, b in zip((self.refs, self.table, self.lens), before):
                assert torch.equal(t, b), "an input changed"
        if name == "compact":
            self.refs, self.table, status = got
            for s, d in moves:
                self.host[:, d] = self.host[:, s]
        else:
            self.refs, self.table, self.lens, status = got
            for s, d, rows in moves:
                for slot in range(rows):
                    for a, n in self.geo.spans(slot):
                        self.host[:, d, :, a:a + n] = self.host[:, s, :, a:a + n]
        assert status.tolist() == want, (name, status.tolist(), want)
        assert self.refs.tolist() == self.model.refs, name
        assert self.lens.tolist() == self.model.lens, name
        assert self.table.tolist() == self.model.table, name
        if moves:
            assert np.array_equal(self.pool.cpu().numpy(), self.host), name
        return want


@pytest.mark.parametrize("B,width,n_pages,page,bits,D,layers,in_place", [
    (1, 4, 5, 16, 4, 64, 1, True),
    (7, 9, 40, 16, 4, 64, 2, True),
    (7, 9, 40, 32, 8, 64, 2, False),
    (40, 20, 300, 16, 4, 128, 1, False),
    (70, 33, 1000, 16, 4, 64, 1, True),
    (1500, 5, 9000, 16, 4, 64, 1, True),      # more rows than a CTA has threads
    (33, 300, 70001, 16, 4, 64, 1, False),    # more pages than the cluster has threads
])
def test_table_operations(B, width, n_pages, page, bits, D, layers, in_place):
    geo = _paged.Geometry(1, D, page, bits, 64, layers)
    both = Both(geo, n_pages, B, width, B + width, in_place)
    rng, model = both.rng, both.model
    room = n_pages * page // B
    seen = set()
    for step in range(12):
        kind = ("grow", "fork", "grow", "trim", "compact", "grow")[step % 6]
        if kind == "grow":
            top = max(2, min(width * page, room) // 2)
            add = [int(rng.integers(0, top)) if rng.random() < 0.6 else int(rng.integers(0, 2))
                   for _ in range(B)]
            if step % 4 != 2:  # mostly within the table's width
                add = [min(a, width * page - n) for a, n in zip(add, model.lens)]
            seen.add(both.op("grow", add)[0])
        elif kind == "fork":
            full = [b for b in range(B) if model.lens[b]]
            parent = [-1] * B
            for b in range(B):
                if not model.lens[b] and full and rng.random() < 0.8:
                    parent[b] = int(rng.choice(full))
            keep = [int(rng.integers(-1, model.lens[p] + 1)) if p >= 0 else 0 for p in parent]
            both.op("fork", parent, keep)
        elif kind == "trim":
            both.op("trim", [int(rng.integers(0, n + 2)) if rng.random() < 0.5 else (0 if rng.random() < 0.5 else -1)
                             for n in model.lens])
        else:
            both.op("compact")
    assert 0 in seen


def test_grow_refusals_change_nothing():
    geo = _paged.Geometry(1, 64, 16, 4, 64)
    for in_place in (True, False):
        both = Both(geo, 6, 3, 4, 1, in_place)
        assert both.op("grow", [20, 16, 0])[0] == 0
        assert both.op("grow", [20, 33, 30]) == [1, 3, 0, 0]
        assert both.op("grow", [0, -1, 0]) == [2, 1, 0, 0]
        assert both.op("grow", [45, 2 ** 31 - 1, 64])[:2] == [2, 2]
        assert both.op("grow", [0, 0, 0]) == [0, 0, 0, 0]
        assert both.op("fork", [-1, -1, 1], [0, 0, 17])[:2] == [2, 1]
        assert both.op("fork", [1, -1, 2], [0, 0, 0])[:2] == [2, 2]
        assert both.op("fork", [-1, -1, 3], [0, 0, 0])[:2] == [2, 1]
        assert both.op("fork", [-1, -1, 1], [0, 0, 16]) == [0, 0, 1, 0]


def test_copy_on_write_of_many_holders():
    # ten rows share a page of which five, then the others, grow
    geo = _paged.Geometry(2, 128, 32, 8, 64, layers=2)
    both = Both(geo, 64, 10, 3, 3, True)
    both.op("grow", [45] + [0] * 9)
    both.op("fork", [-1] + [0] * 9, [-1] * 10)
    assert both.op("grow", [1, 0] * 5) == [0, 0, 5, 5]
    assert both.op("grow", [0, 7] * 5) == [0, 0, 4, 4]      # the last of the five keeps the page
    assert both.op("trim", [-1] * 5 + [40] * 5)[2] == 0
    both.op("compact")


def test_entries_outside_the_pool():
    geo = _paged.Geometry(1, 64, 16, 4, 64)
    pool = torch.zeros(1, 4, 1, geo.rec, dtype=torch.uint8, device="cuda")
    cache = _cache(pool, geo)
    refs, lens = _dev([1, 0, 0, 1]), _dev([20, 20, 0])
    table = _dev([[0, 9], [3, -7], [-1, -1]])
    _, t, n, status = aq.aq_cache_trim(cache, refs, table, lens, _dev([0, 17, -1]), in_place=False)
    assert status.tolist()[0] == 3 and n.tolist() == [0, 17, 0] and t.tolist()[1] == [3, -7]
    r, t, n, status = aq.aq_cache_fork(cache, refs, table, lens, _dev([-1, -1, 0]), _dev([-1] * 3), in_place=False)
    assert status.tolist()[0] == 3 and r.tolist() == [2, 0, 0, 1] and t.tolist()[2] == [0, 9]
    r, t, n, status = aq.aq_cache_grow(cache, refs, table, lens, _dev([1, 1, 1]), in_place=False)
    assert status.tolist()[0] == 3 and r.tolist() == [1, 1, 0, 1] and n.tolist() == [21, 21, 1]
    r, t, status = aq.aq_cache_compact(cache, refs, table, lens, in_place=False)
    assert status.tolist() == [3, 0, 2, 1] and r.tolist() == [1, 1, 0, 0] and t.tolist()[:2] == [[0, 9], [1, -7]]


def test_streams_and_graphs():
    # a captured trim-fork-grow-append follows what the tensors hold at replay
    geo = _paged.Geometry(2, 64, 16, 4, 64)
    side = torch.cuda.Stream()
    n, B = 20, 3
    pool = torch.zeros(1, n, 2, geo.rec, dtype=torch.uint8, device="cuda")
    cache = _cache(pool, geo)
    refs, lens, table = _dev(np.zeros(n)), _dev(np.zeros(B)), _dev(np.full((B, 4), -1))
    add, cu = _dev([5, 20, 0]), _dev([0, 1, 2, 3])
    x = torch.randn(3, 2, 64, device="cuda").half()
    ws = torch.empty(aq.aq_cache_workspace_bytes(n, B), dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        aq.aq_cache_grow(cache, refs, table, lens, add, workspace=ws)
        start = lens.clone()
        add.fill_(1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        status = aq.aq_cache_grow(cache, refs, table, lens, add, workspace=ws)[3]
        aq.aq_cache_append(cache, 0, x, x, cu, start, table)
        start.add_(1)
    assert lens.tolist() == [5, 20, 0]
    for i in range(1, 14):
        g.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [5 + i, 20 + i, i] and status.tolist()[0] == 0
    assert refs.sum().item() == 2 + 3 + 1
    k, _ = aq.aq_cache_read(cache, 0, cu, lens - 1, table, 3, torch.float16)
    want, _ = aq.aq_cache_read(cache, 0, cu, lens - 4, table, 3, torch.float16)
    assert torch.equal(k, want) and k.any()

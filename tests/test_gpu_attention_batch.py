"""GPU parity of attention over the paged cache (aq_attention_batch) against a
plain model in 64 bits.

Tolerance per output element.  A score is off by at most tau: the loosest
kernel rounds K once to fp16 (2^-11 of sum_d |scale q k|; q itself is exact in
fp16 after its power-of-two scale, but for values 2^-28 below the row's
largest: 2^-20 more is allowed), sums in fp32 (covered by another 2^-15 of
it), plus 1e-5.  A weight then moves by a factor within exp(+-2 tau), so that
o moves by at most (exp(2 tau) - 1) sum_n p |v|.  The value product takes
fp16 operands: either p * scale against exact codes or p and v, each rounded:
at most 2^-10 (sum_n p |v| + max |bias|); fp32 sums add 2^-24 a key; o is
rounded once, 2^-8 (bf16) or 2^-11 (fp16) of its value.

Those bounds add absolute values over all keys.  Where scores are about unit
size the same roundings are independent and average out, so the error over a
whole output is also held in the 2-norm: p, k and v carry relative errors of
at most 2^-11 each, which moves o by less than 2^-9 of its norm, plus its own
rounding.
"""
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


def _ints(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


class Case:
    """groups: (members, shared tokens) in batch order; own: each sequence's own tokens."""

    def __init__(self, H, KV, D, page, bits, group, dtype, L, own, groups=(), seed=0, qscale=1.0,
                 layers=1, layer=0):
        self.geo = geo = _paged.Geometry(KV, D, page, bits, group, layers)
        self.rng = rng = np.random.default_rng(seed + H + D + page + bits + group + L + len(own))
        self.B, self.L, self.H, self.layer = len(own), L, H, layer
        share, starts, b = [], [0], 0
        for n, s in groups:
            share += [s] * n
            b += n
            starts.append(b)
        share += [0] * (self.B - b)
        self.lens = [s + o if s + o > 0 else 0 for s, o in zip(share, own)]
        width = -(-max(max(self.lens), 1) // page) + 1
        table, used, lead = np.full((self.B, width), -1), 0, {}
        copies = []
        for b, n in enumerate(self.lens):
            have = -(-n // page)
            g = next((g for g in range(len(groups)) if starts[g] <= b < starts[g + 1]), None)
            same = 0
            if g is not None and n >= share[b]:
                if g in lead:
                    same = share[b] // page
                    table[b, :same] = table[lead[g], :same]
                    if share[b] % page:
                        copies.append((b, lead[g], same, share[b] % page))
                else:
                    lead[g] = b
            table[b, same:have] = np.arange(used, used + have - same)
            used += have - same
        ids = rng.permutation(used + 3)
        self.table = np.where(table >= 0, ids[np.maximum(table, 0)], -1)
        self.pool = _paged.random_pool(rng, geo, used + 3)
        for b, a, spot, rows in copies:  # the partial page at the shared tokens' end
            for slot in range(rows):
                for at, n in geo.spans(slot):
                    self.pool[:, self.table[b, spot], :, at:at + n] = \
                        self.pool[:, self.table[a, spot], :, at:at + n]
        self.starts, self.shared = starts, [s for _, s in groups]
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float16
        self.q = torch.from_numpy(rng.standard_normal((self.B, L, H, D)).astype(np.float32) * qscale).to(self.dtype)
        self.scale = D ** -0.5

    def run(self, q=None, **kw):
        geo = self.geo
        cache = aq.AqCache(torch.from_numpy(self.pool).cuda(), geo.page, geo.D, geo.bits, geo.group)
        if self.shared:
            kw = dict(group_start=_ints(self.starts), shared=_ints(self.shared)) | kw
        o = aq.aq_attention_batch(self.q.cuda() if q is None else q, cache, self.layer, _ints(self.table),
                                  _ints(self.lens), scale=self.scale, **kw)
        torch.cuda.synchronize()
        return o

    def reference(self):
        return _paged.attention(self.geo, self.pool[self.layer], self.q.double().numpy(), self.table,
                                self.lens, self.scale)

    def check(self, o=None, norm=True, ref=None):
        o = self.run() if o is None else o
        want, smag, vmag, bmax = self.reference() if ref is None else ref
        got = o.double().cpu().numpy()
        rnd = 2.0 ** -8 if self.dtype == torch.bfloat16 else 2.0 ** -11
        tau = (2.0 ** -11 + 2.0 ** -20 + 2.0 ** -15) * smag + 1e-5
        tol = ((np.expm1(2 * tau) + 2.0 ** -24 * max(self.lens)) * vmag + 2.0 ** -10 * (vmag + bmax)
               + rnd * np.abs(want) + 1e-6)
        bad = np.argwhere(~(np.abs(got - want) <= tol))
        assert bad.size == 0, (len(bad), [(tuple(i), got[tuple(i)], want[tuple(i)], tol[tuple(i)]) for i in bad[:4]])
        if norm:
            off = np.linalg.norm(got - want)
            assert off <= (rnd + 2.0 ** -9) * np.linalg.norm(want) + 1e-6 * np.sqrt(want.size), off / np.linalg.norm(want)
        assert not got[np.array(self.lens) == 0].any()
        return o


GEOMETRIES = [
    # H, KV, D, page, bits, group, dtype
    (5, 1, 128, 16, 4, 64, "fp16"),
    (4, 4, 64, 16, 4, 32, "bf16"),
    (12, 2, 64, 32, 8, 64, "fp16"),
    (8, 1, 64, 64, 8, 32, "bf16"),
    (4, 2, 64, 128, 4, 64, "fp16"),
    (10, 2, 128, 64, 4, 128, "bf16"),
    (16, 2, 128, 32, 4, 32, "fp16"),
    (16, 1, 128, 128, 8, 64, "bf16"),
    (3, 3, 128, 16, 8, 32, "fp16"),
    (6, 2, 128, 64, 8, 128, "fp16"),
    (4, 2, 256, 64, 4, 64, "bf16"),
    (8, 2, 256, 16, 4, 32, "fp16"),
    (2, 1, 256, 32, 4, 128, "bf16"),
    (8, 1, 256, 32, 8, 128, "fp16"),
    (12, 1, 256, 128, 8, 64, "bf16"),
    (2, 2, 256, 16, 8, 32, "bf16"),
    (4, 2, 512, 16, 4, 64, "fp16"),
    (8, 1, 512, 64, 8, 128, "bf16"),
    (9, 1, 512, 32, 4, 32, "fp16"),
    (2, 2, 512, 16, 8, 32, "bf16"),
    (4, 1, 512, 128, 4, 128, "fp16"),
    (4, 2, 512, 16, 8, 64, "fp16"),
]


@pytest.mark.parametrize("H,KV,D,page,bits,group,dtype", GEOMETRIES)
def test_ragged_batch(H, KV, D, page, bits, group, dtype):
    # one token, one page, one past a page, an empty slot, longer ones
    own = [1, page, 0, page + 1, 300, 2 * page - 1, 777]
    Case(H, KV, D, page, bits, group, dtype, 1, own, layers=2, layer=1).check()


@pytest.mark.parametrize("H,KV,D,page,bits,group,dtype", GEOMETRIES)
def test_shared_prefix(H, KV, D, page, bits, group, dtype):
    # a group of one, a group of five with an empty slot and a member that is
    # shorter than what is shared, sequences in no group
    own = [40, 1, 3, -333, 50, -17, 9, 100]
    Case(H, KV, D, page, bits, group, dtype, 1, own, [(1, 100), (5, 333)]).check()


@pytest.mark.parametrize("L", [2, 3, 8])
@pytest.mark.parametrize("H,KV,D,page,bits,group,dtype", GEOMETRIES[::3])
def test_new_tokens(H, KV, D, page, bits, group, dtype, L):
    # the new tokens' triangle; sequences with fewer tokens than L: rows that
    # see nothing, and a member whose first tokens do not see all that is shared
    own = [L, 1, 200, L + 1, 1, 65]
    Case(H, KV, D, page, bits, group, dtype, L, own, [(3, 130)]).check()
    Case(H, KV, D, page, bits, group, dtype, L, own).check()


@pytest.mark.parametrize("H,KV,D,page,bits,group,dtype,L,members,shared", [
    (40, 8, 128, 64, 4, 64, "bf16", 1, 30, 1111),     # 150 rows a KV head
    (16, 8, 256, 64, 4, 64, "bf16", 1, 70, 500),      # 140 rows of 256
    (8, 1, 64, 16, 8, 32, "fp16", 3, 40, 2049),       # 960 rows of 64
    (16, 1, 128, 32, 8, 128, "fp16", 1, 16, 4096),    # 256 rows, whole tiles
    (16, 1, 128, 32, 8, 128, "bf16", 1, 17, 127),     # one row tile and a bit, less than a tile of keys
    (12, 2, 64, 128, 4, 32, "bf16", 2, 100, 640),
    (6, 1, 256, 16, 8, 64, "fp16", 5, 20, 1025),
    (8, 2, 512, 16, 4, 128, "fp16", 1, 24, 200),
])
def test_many_rows(H, KV, D, page, bits, group, dtype, L, members, shared):
    rng = np.random.default_rng(7)
    own = [int(x) for x in rng.integers(L, 40, size=members)]
    own[members // 2] = -shared                        # an empty slot
    Case(H, KV, D, page, bits, group, dtype, L, own, [(members, shared)]).check()


@pytest.mark.parametrize("H,KV,D,page,bits,group,dtype,L,members,shared", [
    (16, 8, 256, 64, 4, 64, "bf16", 1, 70, 500),      # two tiles of keys a piece, one row tile
    (6, 1, 256, 16, 8, 64, "fp16", 5, 20, 1025),
    (10, 2, 128, 16, 8, 32, "fp16", 1, 20, 3000),     # 100 rows: one row tile
    (8, 1, 128, 32, 4, 64, "bf16", 1, 40, 5000),      # 320 rows: two
    (8, 4, 64, 64, 4, 64, "bf16", 2, 30, 900),
])
def test_same_bits_every_time(H, KV, D, page, bits, group, dtype, L, members, shared):
    # many calls, with a cold and a warm L2, back to back: a wait that is one
    # phase short shows as a difference between calls
    rng = np.random.default_rng(9)
    c = Case(H, KV, D, page, bits, group, dtype, L, [int(x) for x in rng.integers(L, 40, size=members)],
             [(members, shared)])
    geo = c.geo
    cache = aq.AqCache(torch.from_numpy(c.pool).cuda(), geo.page, geo.D, geo.bits, geo.group)
    args = (c.q.cuda(), cache, 0, _ints(c.table), _ints(c.lens), c.scale, _ints(c.starts), _ints(c.shared))
    junk = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    outs = []
    for i in range(60):
        if i % 3 == 0:
            junk.fill_(i)
        outs.append(aq.aq_attention_batch(*args))
    torch.cuda.synchronize()
    c.check(o=outs[0])
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("H,KV,D,page,bits,group,dtype,groups", [
    (2, 2, 64, 16, 4, 32, "fp16", [(16, 333)]),        # 16 rows a KV head
    (2, 2, 64, 16, 4, 32, "fp16", [(17, 333)]),        # 17
    (10, 2, 128, 64, 8, 64, "bf16", [(3, 1000)]),      # 15
    (10, 2, 128, 64, 8, 64, "bf16", [(4, 1000)]),      # 20
    (2, 1, 256, 32, 4, 128, "bf16", [(9, 700)]),       # 18 of 256
    (4, 1, 128, 32, 4, 64, "fp16", [(1, 90), (2, 400), (12, 257), (0, 5)]),   # 15 on average, one group of 48
    (4, 1, 128, 32, 4, 64, "fp16", [(2, 400), (16, 257), (1, 70)]),           # 25 on average, one group of 8
])
def test_rows_around_the_choice_of_kernel(H, KV, D, page, bits, group, dtype, groups):
    rng = np.random.default_rng(10)
    own = [int(x) for x in rng.integers(1, 60, size=sum(n for n, _ in groups))]
    Case(H, KV, D, page, bits, group, dtype, 1, own, groups).check()


def test_several_large_groups():
    rng = np.random.default_rng(8)
    own = [int(x) for x in rng.integers(1, 100, size=75)]
    Case(8, 2, 128, 32, 4, 64, "bf16", 2, own, [(20, 513), (1, 64), (0, 33), (30, 100), (20, 1500)]).check()


def test_long_sequences():
    # enough keys for many pieces of one sequence and of the shared part
    Case(4, 1, 64, 64, 4, 64, "fp16", 1, [20011]).check()
    Case(4, 1, 64, 64, 8, 64, "bf16", 1, [5, 7000, 1], [(2, 15000)]).check()


def test_sharp_softmax():
    # scores of tens: one key decides a row, and the running maximum moves
    c = Case(8, 2, 128, 32, 8, 64, "bf16", 1, [500, 3, 90], [(2, 400)], qscale=40.0)
    c.check(norm=False)
    c = Case(16, 1, 128, 32, 4, 64, "fp16", 2, [60] * 12, [(12, 700)], qscale=40.0)
    c.check(norm=False)


def test_growing_scores_and_scales():
    # keys, and the values' scales, grow by orders of magnitude along the
    # sequence, so that every running maximum keeps moving
    c = Case(8, 1, 128, 16, 4, 64, "fp16", 1, [30] * 20, [(20, 800)])
    geo, lead = c.geo, c.table[0]
    for j in range(800):
        rec = c.pool[0, lead[j // 16], 0]
        for which, top in ((2, 6.0), (3, 9.0)):
            a, n = geo.spans(j % 16)[which]
            pair = rec[a:a + n].copy().view(np.float16).astype(np.float64) * 2.0 ** (top * j / 800 - top)
            rec[a:a + n] = pair.astype(np.float16).view(np.uint8)
    c.check(norm=False)


def test_masked_rows_may_hold_anything():
    # infinities and NaN past every sequence's end, before it in pages that
    # are not its own, and in the new tokens that earlier tokens do not see
    L = 4
    c = Case(8, 2, 128, 64, 4, 64, "bf16", L, [70, 5, 200, 33, 0, 90], [(3, 100)])
    geo, seen = c.geo, np.zeros((c.pool.shape[1], c.geo.page), bool)
    for b, n in enumerate(c.lens):
        for j in range(n):
            seen[c.table[b, j // geo.page], j % geo.page] = True
    ref = c.reference()
    odd = np.array([np.nan, np.inf, -np.inf, np.nan], np.float16)
    for p in range(c.pool.shape[1]):
        for slot in range(geo.page):
            if not seen[p, slot]:
                for a, n in geo.spans(slot)[2:]:
                    c.pool[0, p, :, a:a + n] = np.resize(odd, n // 2).view(np.uint8)
    c.check(ref=ref)
    # the last token of sequences 0 and 3 holds NaN and infinity: only their last rows see it
    for b in (0, 3):
        j = c.lens[b] - 1
        for a, n in geo.spans(j % geo.page)[2:]:
            c.pool[0, c.table[b, j // geo.page], :, a:a + n] = np.resize(odd, n // 2).view(np.uint8)
    o = c.run()
    want, smag, vmag, bmax = (x.copy() for x in ref)
    for b in (0, 3):
        assert torch.isnan(o[b, L - 1]).any()
        o[b, L - 1] = 0
        for x in (want, vmag, bmax, smag):
            x[b, L - 1] = 0
    c.check(o=o, ref=(want, smag, vmag, bmax))


def test_groups_that_do_not_ascend_share_nothing():
    c = Case(8, 2, 128, 32, 4, 64, "fp16", 1, [40, 9, 100], [(3, 64)])
    o = c.run(group_start=_ints([2, 1]), shared=_ints([64]))
    assert aq.aq_device_error(clear=True) != 0
    c.check(o=o)


def test_pages_outside_the_pool():
    # recorded, and the other sequences are right
    c = Case(8, 2, 128, 32, 4, 64, "fp16", 1, [40, 100, 9])
    ref = c.reference()
    c.table[1, 1] = c.pool.shape[1] + 1000
    c.table[1, 2] = -1
    o = c.run()
    assert aq.aq_device_error(clear=True) != 0
    o[1] = 0
    for x in ref:
        x[1] = 0
    c.check(o=o, ref=ref)


def test_lengths_past_the_table():
    # lens past the table's width read no further than the table
    c = Case(4, 1, 64, 16, 4, 64, "fp16", 1, [32, 5])
    c.table = c.table[:, :2]
    want = c.run()
    c.lens[0] = 10 ** 9
    assert torch.equal(c.run(), want)


def test_strided_queries_streams_and_repeats():
    c = Case(10, 2, 128, 32, 4, 64, "bf16", 2, [40, 300, 17, 64], [(3, 200)])
    want = c.check()
    fused = torch.randn(c.B, c.L, 10 + 4, 128, dtype=c.dtype, device="cuda")
    fused[:, :, 2:12] = c.q.cuda()
    assert torch.equal(c.run(q=fused[:, :, 2:12]), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        o = c.run(stream=side)
        assert torch.equal(o, want)


@pytest.mark.parametrize("D,members", [(128, 30), (128, 10), (256, 30)])   # two row tiles, one
def test_wait_runs_out_then_next_call_is_correct(D, members):
    # The test build of the library (1 ms waits) keeps the first k tile from
    # being announced: every wait on it gives up, the call returns and reports
    # it, and the next call is right.
    import ctypes
    from quantized_matmul_affine_gb300 import build
    if not build.up_to_date(build.TEST_LIB):
        build.build()
    prod, lib = aq.load(), ctypes.CDLL(build.TEST_LIB)
    for name in ("aq_attention_batch", "aq_attention_batch_workspace_bytes", "aq_device_error"):
        getattr(lib, name).argtypes = getattr(prod, name).argtypes
        getattr(lib, name).restype = getattr(prod, name).restype
    c = Case(10, 2, D, 32, 4, 64, "fp16", 1, [9] * members, [(members, 700)])
    geo = c.geo
    cache = aq.AqCache(torch.from_numpy(c.pool).cuda(), geo.page, geo.D, geo.bits, geo.group)
    q, table, lens = c.q.cuda(), _ints(c.table), _ints(c.lens)
    starts, shared = _ints(c.starts), _ints(c.shared)
    n = lib.aq_attention_batch_workspace_bytes(cache._ref, c.B, 1, 10, 1)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    code = ctypes.c_uint32(0)

    def call():
        st = lib.aq_attention_batch(cache._ref, 0, aq.AQ_F16, q.data_ptr(), 10 * D, table.data_ptr(),
                                    lens.data_ptr(), starts.data_ptr(), shared.data_ptr(), c.B, 1, 10, 1,
                                    table.shape[1], c.scale, out.data_ptr(), ws.data_ptr(), n,
                                    torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        assert lib.aq_device_error(ctypes.addressof(code), 1) == 0
        return code.value

    try:
        lib.aq_test_withhold(3)
        assert call() & 0xff == 0x06
    finally:
        lib.aq_test_withhold(0)
    for _ in range(3):
        assert call() == 0
        c.check(o=out)


def test_graph_follows_lengths():
    c = Case(8, 2, 64, 16, 4, 64, "fp16", 1, [300, 250, 200], [(2, 128)])
    geo = c.geo
    cache = aq.AqCache(torch.from_numpy(c.pool).cuda(), geo.page, geo.D, geo.bits, geo.group)
    table, lens, q = _ints(c.table), _ints(c.lens), c.q.cuda()
    gs, sh = _ints(c.starts), _ints(c.shared)
    ws = torch.empty(aq.aq_attention_batch_workspace_bytes(cache, 3, 1, 8, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def call():
        aq.aq_attention_batch(q, cache, 0, table, lens, c.scale, gs, sh, out=out, workspace=ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lengths, shared in (([300, 250, 200], 128), ([129, 250, 3], 128), ([5, 0, 1], 128), ([300, 200, 9], 64)):
        lens.copy_(_ints(lengths))
        sh.fill_(shared)
        out.fill_(float("nan"))
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        c.lens, c.shared = lengths, [shared]
        c.check(o=out)

"""Calls on another stream than torch's current one while both have work
waiting: results are those of calls made one at a time, and nothing is written
into memory that was given to something else."""
import numpy as np
import pytest
import torch

from . import _paged

pytestmark = pytest.mark.gpu

aq = pytest.importorskip("quantized_matmul_affine_gb300")

WAIT = 20_000_000  # cycles that a stream is kept busy: 10 ms


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert aq.aq_device_error(clear=True) == 0


def _ints(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def _batch(seed, members, shared):
    """(q, cache, table, lens, groups) of a group that shares its first tokens."""
    rng = np.random.default_rng(seed)
    geo = _paged.Geometry(2, 128, 32, 4, 64)
    own = rng.integers(1, 90, size=members)
    n = -(-int(shared + own.max()) // 32)
    head = shared // 32
    table = np.empty((members, n), np.int64)
    table[:, :head] = np.arange(head)
    table[:, head:] = head + np.arange(members * (n - head)).reshape(members, -1)
    pool = torch.from_numpy(_paged.random_pool(rng, geo, int(table.max()) + 1)).cuda()
    cache = aq.AqCache(pool, geo.page, geo.D, geo.bits, geo.group)
    q = torch.from_numpy(rng.standard_normal((members, 1, 10, 128)).astype(np.float32)).half().cuda()
    return q, cache, 0, _ints(table), _ints(shared + own), 128 ** -0.5, _ints([0, members]), _ints([shared // 32 * 32])


def test_attention_on_two_streams_at_once():
    a, b = _batch(1, 30, 1000), _batch(2, 25, 2000)
    alone = [aq.aq_attention_batch(*a), aq.aq_attention_batch(*b)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for first, second in ((None, stream), (stream, None)):
            outs = []
            for s in (first, second):  # both wait, so that both calls are in flight
                with torch.cuda.stream(None if s is None else side):
                    torch.cuda._sleep(WAIT)
            for _ in range(4):
                outs.append(aq.aq_attention_batch(*a, stream=first))
                outs.append(aq.aq_attention_batch(*b, stream=second))
            torch.cuda.synchronize()
            for i, o in enumerate(outs):
                assert torch.equal(o, alone[i & 1]), (i, stream is side)


def test_a_dropped_status_is_written_nowhere_else():
    geo = _paged.Geometry(1, 64, 16, 4, 64)
    cache = aq.AqCache.empty(1, 8, 1, geo.D, geo.page, geo.bits, geo.group)
    refs, table, lens, add = _ints([0] * 8), _ints([[-1] * 4] * 2), _ints([0, 0]), _ints([3, 20])
    keep = _ints([1, -1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    aq.aq_cache_grow(cache, refs, table, lens, add, stream=side)
    aq.aq_cache_trim(cache, refs, table, lens, keep, stream=side)
    aq.aq_cache_compact(cache, refs, table, lens, stream=side)
    aq.aq_cache_fork(cache, refs, table, lens, add, keep, in_place=False, stream=side)
    mine = [torch.full((n,), 7, dtype=torch.int32, device="cuda") for n in (2, 4, 8, 64, 512) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in mine)
    assert lens.tolist() == [1, 20] and refs.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]


def test_results_outlive_their_use_on_the_current_stream():
    # a result of a call on a side stream, read by a kernel that waits on the
    # current one and dropped before it runs: the next call on the side stream
    # must not be given its memory
    a = _batch(3, 9, 500)
    want = aq.aq_attention_batch(*a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o = aq.aq_attention_batch(*a, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(WAIT)
    copy = o + 0
    del o
    other = [aq.aq_attention_batch(-a[0], *a[1:], stream=side) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(other) == 3


def test_the_default_stream_by_its_handle():
    # 0 names the default stream, also while another one is current
    a = _batch(4, 9, 500)
    want = aq.aq_attention_batch(*a)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = aq.aq_attention_batch(*a, stream=0)
        status = aq.aq_cache_fork(a[1], _ints([0] * a[1].n_pages), a[3], torch.zeros_like(a[4]), a[4] * 0 - 1,
                                  a[4], in_place=False, stream=torch.cuda.default_stream())[3]
        torch.cuda.synchronize()
    assert torch.equal(got, want) and status.tolist() == [0, 0, 0, 0]


def test_workspace_of_decode_is_zero_on_the_calls_stream():
    # a call that allocates its workspace zeroes it where it runs: while the
    # current stream waits, the side stream's call is done and right
    rng = np.random.default_rng(5)
    KV, N, D = 2, 33000, 256
    n = aq.aq_attention_workspace_bytes(8, KV, N, D, 4, 64)
    assert n > 0
    w = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, size=(KV, N, D // 8), dtype=np.int64).astype(np.int32)).cuda()
    s = torch.full((KV, N, D // 64), 0.01, dtype=torch.float16, device="cuda")
    b = torch.full((KV, N, D // 64), -0.07, dtype=torch.float16, device="cuda")
    q = torch.from_numpy(rng.standard_normal((8, D)).astype(np.float32)).half().cuda()
    want = aq.aq_attention_decode_ws(q, (w, s, b), (w, s, b), 4, 64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    got = aq.aq_attention_decode_ws(q, (w, s, b), (w, s, b), 4, 64, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_the_current_stream_stays():
    a = _batch(6, 9, 500)
    side, mine = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (torch.cuda.default_stream(), mine):
        with torch.cuda.stream(s):
            aq.aq_attention_batch(*a, stream=side)
            assert torch.cuda.current_stream() == s
            with pytest.raises(aq.AqError):
                aq.aq_attention_batch(*a[:2], 5, *a[3:], stream=side)   # no such layer
            with pytest.raises((RuntimeError, MemoryError)):
                aq.aq_cache_read(a[1], 0, _ints([0] * 10), a[4], a[3], 2 ** 55, torch.float16, stream=side)
            assert torch.cuda.current_stream() == s
    torch.cuda.synchronize()

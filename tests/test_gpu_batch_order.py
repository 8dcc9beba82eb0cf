"""Batch attention right behind calls that rewrite what it reads: pages copied
over the ones a table names, tables and lengths changed in place, with nothing
waited for in between."""
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


@pytest.mark.parametrize("members", [3, 30])     # 15 and 150 rows a KV head
@pytest.mark.parametrize("bits", [4, 8])
def test_pages_copied_over(bits, members):
    rng = np.random.default_rng(bits + members)
    geo = _paged.Geometry(2, 128, 32, bits, 64)
    live, sets = 40 + 2 * members, 4
    pool = torch.from_numpy(_paged.random_pool(rng, geo, live * (1 + sets))).cuda()
    cache = aq.AqCache(pool, 32, 128, bits, 64)
    table = np.empty((members, 42), np.int64)
    table[:, :40] = np.arange(40)
    table[:, 40:] = 40 + np.arange(2 * members).reshape(members, 2)
    lens = _ints(1280 + rng.integers(1, 65, size=members))
    q = torch.from_numpy(rng.standard_normal((members, 1, 10, 128)).astype(np.float32)).half().cuda()
    groups = _ints([0, members]), _ints([1280])
    table = _ints(table)
    want = [aq.aq_attention_batch(q, cache, 0, table + live * (1 + i), lens, 0.09, *groups) for i in range(sets)]
    src = [_ints(live * (1 + i) + np.arange(live)) for i in range(sets)]
    dst = _ints(np.arange(live))
    torch.cuda.synchronize()
    got = []
    for i in range(10 * sets):
        aq.aq_cache_copy(cache, src[i % sets], dst)
        got.append(aq.aq_attention_batch(q, cache, 0, table, lens, 0.09, *groups))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % sets]) for i, o in enumerate(got))


@pytest.mark.parametrize("members", [3, 30])
def test_tables_changed_in_place(members):
    # trim and grow between the calls: the pages stay, the lengths move
    rng = np.random.default_rng(members)
    geo = _paged.Geometry(2, 128, 32, 4, 64)
    n_pages = 42 * members
    pool = torch.from_numpy(_paged.random_pool(rng, geo, n_pages)).cuda()
    cache = aq.AqCache(pool, 32, 128, 4, 64)
    refs, lens, table = _ints([0] * n_pages), _ints([0] * members), _ints([[-1] * 42] * members)
    aq.aq_cache_grow(cache, refs, table, lens, _ints([1280] + [0] * (members - 1)))
    aq.aq_cache_fork(cache, refs, table, lens, _ints([-1] + [0] * (members - 1)), _ints([-1] * members))
    aq.aq_cache_grow(cache, refs, table, lens, _ints([64] * members))
    q = torch.from_numpy(rng.standard_normal((members, 1, 10, 128)).astype(np.float32)).half().cuda()
    groups = _ints([0, members]), _ints([1280])
    cuts = [_ints(1280 + rng.integers(1, 65, size=members)) for _ in range(5)]
    want = [aq.aq_attention_batch(q, cache, 0, table.clone(), c, 0.09, *groups) for c in cuts]
    full = table.clone()
    torch.cuda.synchronize()
    got = []
    for i in range(30):
        c = cuts[i % 5]
        aq.aq_cache_trim(cache, refs, table, lens, c)
        got.append(aq.aq_attention_batch(q, cache, 0, table, lens, 0.09, *groups))
        # room for all again: lowest pages first, in row order, so each row's own
        aq.aq_cache_grow(cache, refs, table, lens, 1344 - lens)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 5]) for i, o in enumerate(got))
    assert torch.equal(table, full) and bool((lens == 1344).all())

"""Page-table operations whose totals over all rows pass 32 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

aq = pytest.importorskip("quantized_matmul_affine_gb300")

ROWS = 4096


def _world(width, n_pages):
    """Tables of as many entries as the totals (8 or 17 GB, which the calls
    leave alone: every row is empty)."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 5 * ROWS * width:
        pytest.skip("not enough device memory")
    cache = aq.AqCache.empty(1, n_pages, 1, 64, 16, 4, 64)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    lens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
    table = torch.empty((ROWS, width), dtype=torch.int32, device="cuda")
    table[:2] = -1
    table[-2:] = -1
    return cache, refs, table, lens


@pytest.mark.parametrize("each,one_more,missing", [
    (2 ** 19, 0, 2 ** 31 - 8),           # all rows together: 2^31 pages
    (2 ** 20, 0, 2 ** 31 - 1),           # 2^32, and more missing than status can say
    (2 ** 20, 5, 2 ** 31 - 1),           # 2^32 + 5, whose low 32 bits would fit the pool
])
def test_grow_refuses_more_pages_than_32_bits_count(each, one_more, missing):
    cache, refs, table, lens = _world(each + 1, 8)
    add = torch.full_like(lens, 16 * each)
    add[7:7 + one_more] += 16
    status = aq.aq_cache_grow(cache, refs, table, lens, add)[3]
    assert status.tolist() == [1, missing, 0, 0]
    assert not lens.any() and not refs.any() and bool((table[:2] == -1).all() and (table[-2:] == -1).all())
    # and a call that fits goes on as ever
    add.zero_()
    add[0], add[ROWS - 1] = 16 * 3, 1
    status = aq.aq_cache_grow(cache, refs, table, lens, add)[3]
    assert status.tolist() == [0, 0, 4, 0] and refs.tolist() == [1, 1, 1, 1, 0, 0, 0, 0]
    assert lens.tolist() == [48] + [0] * (ROWS - 2) + [1]
    assert table[0, :4].tolist() == [0, 1, 2, -1] and table[-1, :2].tolist() == [3, -1]
    assert aq.aq_device_error(clear=True) == 0


def test_fork_reports_more_entries_than_32_bits_count():
    # 4095 children of 2^19 + 200 pages are 2^31 + 294,712 entries
    width = 2 ** 19 + 200
    cache, refs, table, lens = _world(width, width)
    pages = torch.arange(width, dtype=torch.int32, device="cuda")
    refs.fill_(1)
    table[0] = pages
    lens[0] = 16 * width
    parent = torch.zeros_like(lens)
    parent[0] = -1
    status = aq.aq_cache_fork(cache, refs, table, lens, parent, torch.full_like(lens, -1))[3]
    assert status.tolist() == [0, 0, 2 ** 31 - 1, 0]
    assert bool((refs == ROWS).all() and (lens == 16 * width).all())
    assert torch.equal(table[1], pages) and torch.equal(table[-1], pages)
    assert aq.aq_device_error(clear=True) == 0

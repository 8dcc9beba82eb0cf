"""The plain models of tests/_paged.py against hand-computed values, and what
the paged cache's entry points refuse before anything is queued (no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import quantized_matmul_affine_gb300 as aq

from . import _paged

A = 0x100000  # a 256-byte-aligned placeholder address; validation never dereferences


def _cache(**kw):
    f = dict(pool_dev=A, layers=2, n_pages=8, KV=2, D=64, page=16, bits=4, group_size=32) | kw
    return aq._CacheStruct(f["pool_dev"], f["layers"], f["n_pages"], f["KV"], f["D"], f["page"],
                           f["bits"], f["group_size"])


def _ref(c):
    return ctypes.addressof(c)


def test_record_bytes():
    # 64 rows of 128 values at 4 bits: 64 bytes of codes a row and side, two
    # groups of one fp16 pair a row and side
    assert aq.aq_cache_record_bytes(128, 64, 4, 64) == 64 * (2 * 64 + 2 * 2 * 4)
    for D in (64, 128, 256, 512):
        for page in (16, 32, 64, 128):
            for bits in (4, 8):
                for group in (32, 64, 128):
                    want = _paged.record_bytes(D, page, bits, group) if D % group == 0 else 0
                    assert aq.aq_cache_record_bytes(D, page, bits, group) == want
    for bad in ((96, 64, 4, 32), (128, 48, 4, 64), (128, 64, 3, 64), (128, 64, 4, 16), (64, 16, 4, 128)):
        assert aq.aq_cache_record_bytes(*bad) == 0


def test_model_rows():
    geo = _paged.Geometry(1, 64, 16, 4, 32)
    rec = np.zeros(geo.rec, np.uint8)
    # row 3 of K: codes 0, 1, .. 15 repeating; scale 0.5, bias -1 in group 0, scale 2, bias 0 in group 1
    c0, n = geo.spans(3)[0]
    rec[c0:c0 + n] = np.tile(np.array([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE], np.uint8), 4)
    p0, m = geo.spans(3)[2]
    rec[p0:p0 + m] = np.array([0.5, -1.0, 2.0, 0.0], np.float16).view(np.uint8)
    codes, val, bias = _paged.row_values(geo, rec, 0, 3)
    assert codes.tolist() == list(range(16)) * 4
    assert val[:3].tolist() == [-1.0, -0.5, 0.0] and val[32:35].tolist() == [0.0, 2.0, 4.0]
    assert bias[0] == -1.0 and bias[63] == 0.0
    pool = rec[None, None]
    v, b = _paged.sequence_rows(geo, pool, [0], 4, 0)
    assert np.array_equal(v[3, 0], val) and np.array_equal(b[3, 0], bias)


def test_model_tables():
    # pages of 16; row 0 holds 20 tokens in pages 5 and 2
    t = _paged.Tables([0, 0, 1, 0, 0, 1], [[5, 2, -1], [-1] * 3, [-1] * 3], [20, 0, 0], 16)
    assert t.fork([-1, 0, 0], [0, -1, 16]) == [0, 0, 3, 0]
    assert t.lens == [20, 20, 16] and t.refs == [0, 0, 2, 0, 0, 3]
    assert t.table == [[5, 2, -1], [5, 2, -1], [5, -1, -1]]
    # both holders of page 2 grow: the first copies, the last keeps it; row 2 starts a page
    status, copies = t.grow([1, 1, 1])
    assert status == [0, 0, 2, 1] and copies == [(2, 0, 4)]
    assert t.table == [[5, 0, -1], [5, 2, -1], [5, 1, -1]] and t.refs == [1, 1, 1, 0, 0, 3]
    assert t.trim([-1, 0, 3]) == [0, 0, 2, 0]
    assert t.refs == [1, 0, 0, 0, 0, 2] and t.lens == [21, 0, 3]
    status, moves = t.compact()
    assert status == [0, 0, 2, 1] and moves == [(5, 1)]
    assert t.table[0][:2] == [1, 0] and t.table[2][0] == 1
    assert t.grow([200, 0, 0]) == ([2, 1, 0, 0], [])
    t.lens = [21, 0, 3]
    t.refs = [1, 1, 1, 1, 1, 1]
    assert t.grow([27, 0, 0]) == ([1, 1, 0, 0], [])


@pytest.mark.parametrize("bad", [
    dict(layers=0), dict(n_pages=0), dict(KV=0), dict(D=96), dict(page=48), dict(bits=3),
    dict(group_size=16), dict(pool_dev=None)])
def test_bad_caches(bad):
    lib, c = aq.load(), _cache(**bad)
    assert lib.aq_cache_append(_ref(c), 0, 0, A, 128, A, 128, 1, A, A, A, 1, 1, None) == 1
    assert lib.aq_cache_read(_ref(c), 0, 0, A, A, 1, A, A, A, 1, 1, None) == 1
    assert lib.aq_cache_copy(_ref(c), A, A, 1, None) == 1
    assert lib.aq_attention_batch(_ref(c), 0, 0, A, 128, A, A, None, None, 1, 1, 2, 0, 1, 1.0, A, A,
                                  1 << 40, None) == 1
    assert lib.aq_cache_grow(_ref(c), A, A, A, A, 1, 1, A, A, A, A, A, 1 << 30, None) == 1


def test_rows_refusals():
    lib, c = aq.load(), _cache()
    ok = [_ref(c), 0, 0, A, 128, A, 128, 1, A, A, A, 1, 1, None]

    def call(**change):
        a = list(ok)
        for i, v in change.items():
            a[int(i[1:])] = v
        return lib.aq_cache_append(*a)

    assert call(_0=None) == 1 and call(_1=2) == 1 and call(_1=-1) == 1 and call(_2=2) == 1
    assert call(_3=None) == 1 and call(_5=None) == 1 and call(_8=None) == 1 and call(_10=None) == 1
    assert call(_7=-1) == 1 and call(_11=0) == 1 and call(_12=0) == 1 and call(_12=1 << 40) == 1
    assert call(_7=2, _4=64) == 1            # tokens would overlap
    assert call(_3=A + 8) == 3 and call(_4=132) == 3 and call(_8=A + 2) == 3
    assert call(_7=0) == 0                   # nothing to do, nothing queued
    assert lib.aq_cache_read(_ref(c), 0, 0, A, A + 4, 1, A, A, A, 1, 1, None) == 3
    assert lib.aq_cache_read(_ref(c), 0, 7, A, A, 1, A, A, A, 1, 1, None) == 1
    assert lib.aq_cache_copy(_ref(c), A, A, 0, None) == 0
    assert lib.aq_cache_copy(_ref(c), None, A, 1, None) == 1
    assert lib.aq_cache_copy(_ref(c), A + 2, A, 1, None) == 3
    assert lib.aq_cache_copy(_ref(c), A, A, -1, None) == 1


def test_table_refusals():
    lib, c = aq.load(), _cache(pool_dev=None)  # fork and trim touch no page
    n = aq.aq_cache_workspace_bytes(8, 3)
    assert n > 0 and aq.aq_cache_workspace_bytes(0, 3) == 0
    assert lib.aq_cache_fork(_ref(c), A, A, A, A, None, 3, 4, A, A, A, A, None) == 1
    assert lib.aq_cache_fork(_ref(c), A, A, A, A, A, 0, 4, A, A, A, A, None) == 1
    assert lib.aq_cache_fork(_ref(c), A, A, A, A, A, 4097, 4, A, A, A, A, None) == 1
    assert lib.aq_cache_fork(_ref(c), A, A, A, A, A, 3, 0, A, A, A, A, None) == 1
    assert lib.aq_cache_fork(_ref(c), A, A + 2, A, A, A, 3, 4, A, A, A, A, None) == 3
    assert lib.aq_cache_trim(_ref(c), A, A, A, A, 3, 4, A, A, None, A, None) == 1
    assert lib.aq_cache_trim(_ref(c), A, A, A, A, 3, 4, A, A, A, A + 1, None) == 3
    assert lib.aq_cache_grow(_ref(c), A, A, A, A, 3, 4, A, A, A, A, A, n, None) == 1  # needs the pool
    c = _cache()
    assert lib.aq_cache_grow(_ref(c), A, A, A, A, 3, 4, A, A, A, A, A, n - 1, None) == 1
    assert lib.aq_cache_grow(_ref(c), A, A, A, A, 3, 4, A, A, A, A, None, n, None) == 1
    assert lib.aq_cache_compact(_ref(c), A, A, A, 3, 4, A, A, A, A, n - 1, None) == 1
    assert lib.aq_cache_compact(_ref(c), A, A, A, 3, 4, A, A, A, A + 2, n, None) == 3


def test_attention_refusals():
    lib, c = aq.load(), _cache()
    n = lib.aq_attention_batch_workspace_bytes(_ref(c), 2, 1, 4, 1)
    assert n > 0
    ok = [_ref(c), 0, 0, A, 256, A, A, A, A, 2, 1, 4, 1, 3, 0.125, A, A, n, None]

    def call(**change):
        a = list(ok)
        for i, v in change.items():
            a[int(i[1:])] = v
        return lib.aq_attention_batch(*a)

    assert call(_1=2) == 1 and call(_2=3) == 1 and call(_3=None) == 1 and call(_5=None) == 1
    assert call(_6=None) == 1 and call(_7=None) == 1 and call(_8=None) == 1 and call(_15=None) == 1
    assert call(_9=0) == 1 and call(_10=0) == 1 and call(_11=0) == 1 and call(_11=3) == 1
    assert call(_12=-1) == 1 and call(_13=0) == 1 and call(_13=1 << 30) == 1
    assert call(_14=math.inf) == 1 and call(_14=math.nan) == 1
    assert call(_16=None) == 1 and call(_17=n - 1) == 1
    assert call(_4=128) == 1                 # tokens would overlap
    assert call(_3=A + 2) == 3 and call(_4=260) == 3 and call(_15=A + 8) == 3
    assert call(_16=A + 128) == 3 and call(_5=A + 1) == 3
    assert call(_9=1025) == 2 and call(_10=65) == 2 and call(_12=257) == 2
    assert lib.aq_attention_batch_workspace_bytes(_ref(c), 1025, 1, 4, 0) == 0
    assert lib.aq_attention_batch_workspace_bytes(_ref(c), 1, 1, 3, 0) == 0


def test_binding_checks():
    rec = aq.aq_cache_record_bytes(64, 16, 4, 32)
    pool = torch.zeros(1, 4, 2, rec, dtype=torch.uint8)
    with pytest.raises(ValueError, match="uint8"):
        aq.AqCache(pool.int(), 16, 64, 4, 32)
    with pytest.raises(ValueError, match="bytes"):
        aq.AqCache(pool[..., :-4], 16, 64, 4, 32)
    with pytest.raises(ValueError, match="served"):
        aq.AqCache(pool, 16, 64, 5, 32)
    with pytest.raises(ValueError, match="CUDA"):
        aq.AqCache(pool, 16, 64, 4, 32)

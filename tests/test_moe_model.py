"""The plain models of tests/_moe.py against hand-computed values, and what the
entry points of the experts' layer and of the embedding lookup refuse before
anything is queued (no GPU)."""
import ctypes
import math

import pytest
import torch

import quantized_matmul_affine_gb300 as aq

from . import _moe

A = 0x100000  # a 256-byte-aligned placeholder address; validation never dereferences


def _router(**kw):
    f = dict(weight_dev=A, bias_dev=None, E=8, K=64, dtype=0, top_k=2, score=0, normalize=1,
             scale=1.0) | kw
    return aq._RouterStruct(*[f[n] for n, _ in aq._RouterStruct._fields_])


def _experts(**kw):
    f = {n: A for n, t in aq._ExpertsStruct._fields_ if t is ctypes.c_void_p}
    f |= dict(E=8, K=64, I=64, bits=4, group_size=64) | kw
    return aq._ExpertsStruct(*[f[n] for n, _ in aq._ExpertsStruct._fields_])


def _ref(s):
    return None if s is None else ctypes.addressof(s)


def test_model_codes():
    words = torch.tensor([[0x76543210, -0x01234568]], dtype=torch.int32)  # 0xFEDCBA98
    assert _moe.codes(words, 4).tolist() == [list(range(16))]
    # 3 bits, LSB first: 0b10_001_000 ... code 10 straddles the words
    w = torch.tensor([[sum(((i % 8) << (3 * i)) for i in range(11)) & 0xFFFFFFFF]], dtype=torch.int64)
    full = sum((i % 8) << (3 * i) for i in range(32))
    three = torch.tensor([[(full >> s) & 0xFFFFFFFF for s in (0, 32, 64)]]).to(torch.int32)
    assert int(three[0, 0]) & 0xFFFFFFFF == int(w)
    assert _moe.codes(three, 3).tolist() == [[i % 8 for i in range(32)]]


def test_model_experts():
    # one expert: gate weight 1 at (0, 0), up weight 2 at (0, 0), down weight 3 at (0, 0)
    def one(rows, cols, v):
        words = torch.zeros(2, rows, cols // 8, dtype=torch.int32)
        words[1, 0, 0] = 1
        s = torch.zeros(2, rows, cols // 64, dtype=torch.float16)
        s[1] = v
        return words, s, torch.zeros_like(s)

    x = torch.zeros(2, 64, dtype=torch.float16)
    x[0, 0] = 1.5
    y, bound = _moe.experts(x, torch.tensor([[1], [-1]]), torch.tensor([[0.5], [7.0]]),
                            one(64, 64, 1), one(64, 64, 2), one(64, 64, 3), 4, 64)
    want = 0.5 * 3 * (1.5 / (1 + math.exp(-1.5))) * 3.0
    assert float(y[0, 0]) == pytest.approx(want, rel=1e-12)
    assert not y[0, 1:].any() and not y[1].any() and (bound >= 0).all()
    assert float(bound[0, 0]) < 2.0 ** -9 * want  # two roundings of h to 11 bits, little else


def test_model_route():
    x = torch.zeros(1, 64, dtype=torch.bfloat16)
    x[0, 0] = 1.0
    w = torch.zeros(5, 64, dtype=torch.bfloat16)
    w[:, 0] = torch.tensor([0.0, 2.0, 1.0, 2.0, 2.0])
    ids, p, _ = _moe.route(x, w, 2)
    assert ids.tolist() == [[1, 3]] and p.tolist()[0] == pytest.approx([0.5, 0.5])
    ids, p, _ = _moe.route(x, w, 4, normalize=False, scale=2.0)
    z = 1 + math.e + 3 * math.e ** 2
    assert ids.tolist() == [[1, 2, 3, 4]]
    assert p.tolist()[0] == pytest.approx([2 * v / z for v in (math.e ** 2, math.e, math.e ** 2, math.e ** 2)])
    ids, p, _ = _moe.route(x, w, 1, bias=torch.tensor([0.5, 0.0, 0.0, 0.0, 0.0]), score="sigmoid",
                           normalize=False)
    assert ids.tolist() == [[0]] and p.item() == pytest.approx(0.5)


def test_model_embed():
    words = torch.tensor([[0x76543210] * 4, [-0x01234568] * 4], dtype=torch.int32)
    s, b = torch.tensor([[0.5], [2.0]]).half(), torch.tensor([[1.0], [-1.0]]).half()
    v, _ = _moe.embed(torch.tensor([1, -1, 0, 2]), (words, s, b), 4, 32, 3.0)
    assert v[0, :3].tolist() == [3 * (2 * 8 - 1), 3 * (2 * 9 - 1), 3 * (2 * 10 - 1)]
    assert not v[1].any() and not v[3].any() and v[2, :2].tolist() == [3.0, 4.5]


BAD_ROUTER = [dict(weight_dev=None), dict(E=0), dict(E=513), dict(K=0), dict(K=32), dict(K=96),
              dict(K=1 << 21), dict(dtype=2), dict(top_k=0), dict(top_k=9), dict(E=64, top_k=17),
              dict(score=2), dict(scale=math.inf), dict(scale=math.nan)]
BAD_EXPERTS = [dict(E=0), dict(E=513), dict(K=0), dict(K=96), dict(I=32), dict(I=0), dict(K=1 << 21),
               dict(bits=1), dict(bits=7), dict(group_size=16), dict(group_size=128),
               dict(I=192, K=128, group_size=128), dict(gate_words_dev=None), dict(up_scales_dev=None),
               dict(down_biases_dev=None)]


@pytest.mark.parametrize("bad", BAD_ROUTER + [None])
def test_route_refuses(bad):
    r = None if bad is None else _router(**bad)
    assert aq.load().aq_moe_route(_ref(r), A, 1, A, A, None) == 1
    if bad is not None and "E" not in bad and "K" not in bad:
        assert aq.load().aq_moe(_ref(r), _ref(_experts()), A, 1, A, A, A, A, 1 << 30, None) == 1


@pytest.mark.parametrize("bad", BAD_EXPERTS + [None])
def test_experts_refuses(bad):
    x = None if bad is None else _experts(**bad)
    lib = aq.load()
    assert lib.aq_moe_experts(_ref(x), 0, A, 1, 2, A, A, A, A, 1 << 30, None) == 1
    assert lib.aq_moe(_ref(_router()), _ref(x), A, 1, A, A, A, A, 1 << 30, None) == 1
    if bad is None or not any(k.endswith("_dev") for k in bad):
        assert lib.aq_moe_workspace_bytes(_ref(x), 1, 2) == 0


def test_calls_refuse():
    lib, r, x = aq.load(), _router(), _experts()
    need = lib.aq_moe_workspace_bytes(_ref(x), 4, 2)
    assert need == 2 * 4 * 2 * 64 * 4
    for T in (0, -1, 257):
        assert lib.aq_moe_route(_ref(r), A, T, A, A, None) == 1
        assert lib.aq_moe_experts(_ref(x), 0, A, T, 2, A, A, A, A, 1 << 40, None) == 1
        assert lib.aq_moe(_ref(r), _ref(x), A, T, A, A, A, A, 1 << 40, None) == 1
        assert lib.aq_moe_workspace_bytes(_ref(x), T, 2) == 0
    for top in (0, 17):
        assert lib.aq_moe_experts(_ref(x), 0, A, 1, top, A, A, A, A, 1 << 40, None) == 1
    assert lib.aq_moe_experts(_ref(x), 2, A, 1, 2, A, A, A, A, 1 << 40, None) == 1
    assert lib.aq_moe_experts(_ref(x), 0, A, 4, 2, A, A, A, A, need - 1, None) == 1
    for i, arg in enumerate((A, A, A, A, A)):  # x, ids, weights, out, workspace
        args = [A] * 5
        args[i] = None
        assert lib.aq_moe_experts(_ref(x), 0, args[0], 4, 2, args[1], args[2], args[3], args[4],
                                  need, None) == 1
        args[i] = A + 1
        assert lib.aq_moe_experts(_ref(x), 0, args[0], 4, 2, args[1], args[2], args[3], args[4],
                                  need, None) == 3
    assert lib.aq_moe_route(_ref(r), None, 1, A, A, None) == 1
    assert lib.aq_moe_route(_ref(r), A, 1, None, A, None) == 1
    assert lib.aq_moe_route(_ref(r), A + 8, 1, A, A, None) == 3
    assert lib.aq_moe_route(_ref(_router(weight_dev=A + 8)), A, 1, A, A, None) == 3
    assert lib.aq_moe_route(_ref(_router(bias_dev=A)), A, 1, A, A, None) == 2  # softmax with a bias
    for name, t in aq._ExpertsStruct._fields_:
        if t is ctypes.c_void_p:
            at = A + (8 if "words" in name else 1)
            assert lib.aq_moe_experts(_ref(_experts(**{name: at})), 0, A, 4, 2, A, A, A, A, need,
                                      None) == 3
    # router and experts of different sizes
    assert lib.aq_moe(_ref(_router(E=9)), _ref(x), A, 4, A, A, A, A, need, None) == 1
    assert lib.aq_moe(_ref(_router(K=128)), _ref(x), A, 4, A, A, A, A, need, None) == 1


def test_embed_refuses():
    lib = aq.load()

    def call(dtype=0, ids=A, index=4, T=1, Wq=A, s=A, b=A, N=10, K=64, bits=4, group=64, scale=1.0,
             out=A):
        return lib.aq_embed(dtype, ids, index, T, Wq, s, b, N, K, bits, group, scale, out, None)

    for bad in (dict(dtype=2), dict(index=2), dict(T=-1), dict(N=0), dict(K=0), dict(K=96), dict(bits=7),
                dict(group=16), dict(scale=math.nan), dict(scale=math.inf), dict(ids=None),
                dict(Wq=None), dict(s=None), dict(b=None), dict(out=None)):
        assert call(**bad) == 1, bad
    for bad in (dict(ids=A + 2), dict(ids=A + 4, index=8), dict(Wq=A + 2), dict(s=A + 1), dict(b=A + 1),
                dict(out=A + 8)):
        assert call(**bad) == 3, bad
    for bad in (dict(N=(1 << 31) + 1), dict(K=1 << 25), dict(T=(1 << 31) + 1)):
        assert call(**bad) == 2, bad
    assert call(T=0, ids=None, out=None) == 0


def test_binding_refuses():
    w = torch.zeros(8, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        aq.AqRouter(w, 2)
    with pytest.raises(ValueError, match="score"):
        aq.AqRouter(w, 2, score="max")
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        aq.AqRouter(w.float(), 2)
    with pytest.raises(ValueError, match="bias"):
        aq.AqRouter(w, 2, bias=torch.zeros(7))

    def m(rows, cols, E=4):
        return (torch.zeros(E, rows, cols // 8, dtype=torch.int32),
                *(torch.zeros(E, rows, cols // 64, dtype=torch.float16) for _ in range(2)))

    with pytest.raises(ValueError, match="CUDA"):
        aq.AqExperts(m(64, 128), m(64, 128), m(128, 64), 4, 64)
    with pytest.raises(ValueError, match="bits"):
        aq.AqExperts(m(64, 128), m(64, 128), m(128, 64), 7, 64)
    with pytest.raises(ValueError, match="multiples"):
        aq.AqExperts(m(96, 128), m(96, 128), m(128, 96), 4, 32)
    with pytest.raises(ValueError, match="up words must be"):
        aq.AqExperts(m(64, 128), m(64, 192), m(128, 64), 4, 64)
    with pytest.raises(ValueError, match="down scales must be"):
        aq.AqExperts(m(64, 128), m(64, 128), m(128, 64)[:1] + m(128, 128)[1:], 4, 64)
    with pytest.raises(ValueError, match="ids must be"):
        aq.aq_embed(torch.zeros(2), *(t[0] for t in m(64, 64)), 4, 64, torch.float16)
    with pytest.raises(ValueError, match="dtype"):
        aq.aq_embed(torch.zeros(2, dtype=torch.int32), *(t[0] for t in m(64, 64)), 4, 64, torch.float32)
    with pytest.raises(ValueError, match="Wq holds"):
        aq.aq_embed(torch.zeros(2, dtype=torch.int32), *(t[0] for t in m(64, 64)), 8, 64, torch.float16)


"""AqRouter and AqExperts are what the library reads: an attribute that changed
would have the binding make outputs of one size and the kernels write another
(no GPU: tensors that say they are the device's)."""
import copy
import ctypes

import pytest
import torch

import quantized_matmul_affine_gb300 as aq

from .test_binding_streams import _t

HALF = dict(dtype=torch.float16)


def _router():
    return aq.AqRouter(_t(4, 128, **HALF), 2, bias=_t(4, dtype=torch.float32), score="sigmoid")


def _experts():
    def stack(rows, cols):
        return (_t(4, rows, cols // 8), _t(4, rows, cols // 64, **HALF), _t(4, rows, cols // 64, **HALF))

    return aq.AqExperts(stack(64, 128), stack(64, 128), stack(128, 64), 4, 64)


@pytest.mark.parametrize("make,names", [
    (_router, ["top_k", "weight", "bias", "_struct", "_ref", "_shape", "_dtype", "_index"]),
    (_experts, ["gate", "up", "down", "bits", "group_size", "count", "hidden", "inner", "_struct", "_ref", "_index"])])
def test_attributes_are_fixed(make, names):
    o = make()
    for name in names:
        held = getattr(o, name)
        with pytest.raises(AttributeError, match="fixed"):
            setattr(o, name, 1)
        with pytest.raises(AttributeError, match="fixed"):
            delattr(o, name)
        assert getattr(o, name) is held or getattr(o, name) == held
    with pytest.raises(AttributeError):
        o.other = 1
    assert copy.copy(o) is o


def test_structs_say_the_same():
    r, x = _router(), _experts()
    s = ctypes.cast(r._ref, ctypes.POINTER(aq._RouterStruct)).contents
    assert (s.E, s.K, s.top_k, s.score, s.dtype) == (4, 128, r.top_k, aq.AQ_SCORE_SIGMOID, aq.AQ_F16)
    assert s.weight_dev == r.weight.data_ptr() and s.bias_dev == r.bias.data_ptr()
    s = ctypes.cast(x._ref, ctypes.POINTER(aq._ExpertsStruct)).contents
    assert (s.E, s.K, s.I, s.bits, s.group_size) == (x.count, x.hidden, x.inner, x.bits, x.group_size)
    assert [s.gate_words_dev, s.up_scales_dev, s.down_biases_dev] == \
        [t.data_ptr() for t in (x.gate[0], x.up[1], x.down[2])]


def test_subclasses_add_their_own():
    class Named(aq.AqRouter):
        def __init__(self, name, *args, **kw):
            super().__init__(*args, **kw)
            self.name = name

    r = Named("first", _t(4, 128, **HALF), 2)
    r.name = "second"
    assert r.name == "second" and r.top_k == 2
    del r.name
    with pytest.raises(AttributeError, match="fixed"):
        r.top_k = 3

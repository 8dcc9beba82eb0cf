"""Where the binding's memory comes from when a call names a stream other than
torch's current one (no GPU: torch's allocator and the library are stood in
for).  A block of the current stream's memory may still be in use by kernels
queued there, and one that is dropped returns to that stream at once: what a
call writes on another stream has to come from that stream's memory, and what
it hands back has to be known to the stream the caller is on."""
import types

import pytest
import torch

import quantized_matmul_affine_gb300 as aq


class _Stream:
    device_index, device_type = 0, 1

    def __init__(self, handle):
        self.cuda_stream = self.stream_id = handle


class _Tensor(torch.Tensor):
    """A host tensor that says it is the device's."""

    @staticmethod
    def of(t):
        t = t.as_subclass(_Tensor)
        t.known_to = []
        return t

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))
    __torch_function__ = torch._C._disabled_torch_function_impl

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.known_to.append(stream.cuda_stream)


def _t(*shape, dtype=torch.int32):
    return _Tensor.of(_real_zeros(*shape, dtype=dtype))


_real_zeros, _real_empty = torch.zeros, torch.empty
HERE, SIDE = 7, 11


@pytest.fixture
def world(monkeypatch):
    """Allocations as (stream that was current, tensor), in order."""
    w = types.SimpleNamespace(now=_Stream(HERE), made=[], called=[])

    def set_stream(stream_id, device_index, device_type):
        assert (device_index, device_type) == (0, 1)
        w.now = _Stream(stream_id)

    def made(t):
        t = _Tensor.of(t)
        w.made.append((w.now.cuda_stream, t))
        return t

    def empty(*shape, dtype=None, device=None, **kw):
        return made(_real_empty(*shape, dtype=dtype))

    def zeros(*shape, dtype=None, device=None, **kw):
        return made(_real_zeros(*shape, dtype=dtype))

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "zeros", zeros)
    monkeypatch.setattr(torch, "empty_like", lambda t, **kw: empty(tuple(t.shape), dtype=t.dtype))
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: _Stream(h))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentStream", lambda d: (w.now.cuda_stream, 0, 1), raising=False)
    monkeypatch.setattr(torch._C, "_cuda_setStream", set_stream, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.now)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: w.now.cuda_stream, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    class Lib:
        def __getattr__(self, name):
            def f(*args):
                if name.endswith("_bytes"):
                    return 4096
                w.called.append((name, args[-1]))
                return 0
            f.__name__ = name
            return f

    rec = aq.aq_cache_record_bytes(64, 16, 4, 32)
    w.cache = aq.AqCache(_t(1, 8, 2, rec, dtype=torch.uint8), 16, 64, 4, 32)
    aq._batch_workspace.cache_clear()
    aq.aq_cache_workspace_bytes.cache_clear()
    monkeypatch.setattr(aq, "load", lambda *a: Lib())
    yield w
    aq._batch_workspace.cache_clear()
    aq.aq_cache_workspace_bytes.cache_clear()


def _calls(cache):
    refs, table, lens, one = _t(8), _t(3, 4), _t(3), _t(3)
    half = dict(dtype=torch.float16)
    w4 = (_t(64, 16), _t(64, 2, **half), _t(64, 2, **half))
    x = _t(5, 128, **half)
    kv = (_t(2, 9, 8), _t(2, 9, 2, **half), _t(2, 9, 2, **half))
    out = []
    for in_place in (True, False):
        kw = dict(in_place=in_place)
        out += [
            ("aq_cache_fork", lambda s, kw=kw: aq.aq_cache_fork(cache, refs, table, lens, one, one, stream=s, **kw)),
            ("aq_cache_trim", lambda s, kw=kw: aq.aq_cache_trim(cache, refs, table, lens, one, stream=s, **kw)),
            ("aq_cache_grow", lambda s, kw=kw: aq.aq_cache_grow(cache, refs, table, lens, one, stream=s, **kw)),
            ("aq_cache_compact", lambda s, kw=kw: aq.aq_cache_compact(cache, refs, table, lens, stream=s, **kw)),
        ]
    out += [
        ("aq_cache_read", lambda s: aq.aq_cache_read(cache, 0, _t(4), lens, table, 6, torch.float16, stream=s)),
        ("aq_attention_batch", lambda s: aq.aq_attention_batch(_t(3, 1, 4, 64, **half), cache, 0, table, lens, 0.1,
                                                                stream=s)),
        ("aq_pack", lambda s: aq.aq_pack(_t(4, 32, dtype=torch.uint8), 4, stream=s)),
        ("aq_quantize", lambda s: aq.aq_quantize(x, 4, stream=s)),
        ("aq_quantize_ex", lambda s: aq.aq_quantize_ex(x, 4, 32, stream=s)),
        ("aq_matmul", lambda s: aq.aq_matmul(x, *w4, 4, stream=s)),
        ("aq_matmul_ex", lambda s: aq.aq_matmul_ex(x, *w4, 4, 64, stream=s)),
        ("aq_matmul_multi", lambda s: aq.aq_matmul_multi(x, [w4, w4], 4, stream=s)),
        ("aq_matmul_gate_up", lambda s: aq.aq_matmul_gate_up(x, w4, w4, 4, stream=s)),
        ("aq_attention_decode", lambda s: aq.aq_attention_decode(_t(4, 64, **half), kv, kv, 4, 32, stream=s)),
        ("aq_attention_decode_ws", lambda s: aq.aq_attention_decode_ws(_t(4, 64, **half), kv, kv, 4, 32, stream=s)),
    ]
    return out


def _flat(x):
    return [x] if isinstance(x, torch.Tensor) else [t for y in x for t in _flat(y)]


NAMES = range(19)


@pytest.mark.parametrize("i", NAMES)
@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_a_call_on_another_stream(world, i, handle):
    name, call = _calls(world.cache)[i]
    res = call(SIDE if handle else _Stream(SIDE))
    assert world.called[-1] == (name if name != "aq_matmul" else "aq_matmul_variant", SIDE)
    assert world.made and all(s == SIDE for s, _ in world.made), (name, [s for s, _ in world.made])
    given = {id(t) for t in _flat(res)}
    for _, t in world.made:  # what is handed back is freed under the caller's hands
        assert id(t) not in given or HERE in t.known_to, name
    assert world.now.cuda_stream == HERE


@pytest.mark.parametrize("i", NAMES)
@pytest.mark.parametrize("stream", [None, HERE, "current"])
def test_memory_of_a_call_on_the_current_stream(world, i, stream):
    name, call = _calls(world.cache)[i]
    call(world.now if stream == "current" else stream)
    assert world.called[-1][1] == HERE
    assert world.made and all(s == HERE and not t.known_to for s, t in world.made), name


def test_every_call_is_covered():
    import inspect
    made = {f for f in aq.__all__ if f.startswith("aq_") and "stream=None" in str(inspect.signature(getattr(aq, f)))}
    names = {n for n, _ in _calls(None)}
    # the others return nothing of their own, or share the code of one above
    assert made - names == {"aq_cache_append", "aq_cache_copy", "aq_quantize_bf16", "aq_matmul_bf16",
                            "aq_matmul_variant", "aq_matmul_host", "aq_attention_decode_static"}
    assert len(_calls(None)) == len(NAMES)

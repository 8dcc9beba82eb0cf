"""Every public call that takes a stream is in a list of calls whose memory is
looked at: by its parameter's name, however the signature writes its default."""
import inspect
import typing

import torch

import quantized_matmul_affine_gb300 as aq

from . import test_binding_streams, test_moe_streams

# these return nothing of their own, or share the code of a call that is listed
SHARED = {"aq_cache_append", "aq_cache_copy", "aq_quantize_bf16", "aq_matmul_bf16", "aq_matmul_variant",
          "aq_matmul_host", "aq_attention_decode_static"}


def _with_stream(names, of):
    return {n for n in names if inspect.isfunction(of(n)) and "stream" in inspect.signature(of(n)).parameters}


def test_found_by_name():
    def plain(x, stream=None): ...
    def typed(x, stream: typing.Optional[torch.cuda.Stream] = None): ...
    def needed(x, stream): ...
    def none(x, streams=None): ...
    made = {f.__name__: f for f in (plain, typed, needed, none)}
    assert _with_stream(made, made.get) == {"plain", "typed", "needed"}


def test_every_call_is_listed():
    calls = _with_stream(aq.__all__, lambda n: getattr(aq, n))
    listed = {n for n, _ in test_binding_streams._calls(None)} | set(test_moe_streams._calls())
    assert {"aq_moe_route", "aq_moe_experts", "aq_moe", "aq_embed"} <= calls
    assert calls - listed == SHARED
    assert listed <= calls


def test_annotations_admit_handles():
    """A stream may be torch's or a handle: what a signature says is what it takes."""
    for name in _with_stream(aq.__all__, lambda n: getattr(aq, n)):
        hint = typing.get_type_hints(getattr(aq, name)).get("stream")
        if hint is not None:
            assert {torch.cuda.Stream, int, type(None)} == set(typing.get_args(hint)), name

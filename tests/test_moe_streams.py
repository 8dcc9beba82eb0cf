"""Where the memory of the experts' layer and of the embedding lookup comes from
when a call names a stream other than torch's current one (no GPU: torch's
allocator and the library are stood in for, as for the other calls)."""
import pytest
import torch

import quantized_matmul_affine_gb300 as aq

from .test_binding_streams import HERE, SIDE, _flat, _Stream, _t, world  # noqa: F401

HALF = dict(dtype=torch.float16)


def _calls():
    def stack(rows, cols):
        return (_t(4, rows, cols // 8), _t(4, rows, cols // 64, **HALF), _t(4, rows, cols // 64, **HALF))

    x, ids, w = _t(3, 128, **HALF), _t(3, 2), _t(3, 2, dtype=torch.float32)
    router = aq.AqRouter(_t(4, 128, **HALF), 2)
    experts = aq.AqExperts(stack(64, 128), stack(64, 128), stack(128, 64), 4, 64)
    table = tuple(t[0].as_subclass(type(x)) for t in stack(64, 128))
    return {
        "aq_moe_route": lambda s: aq.aq_moe_route(x, router, stream=s),
        "aq_moe_experts": lambda s: aq.aq_moe_experts(x, experts, ids, w, stream=s),
        "aq_moe": lambda s: aq.aq_moe(x, router, experts, stream=s),
        "aq_embed": lambda s: aq.aq_embed(_t(5), *table, 4, 64, torch.float16, stream=s),
    }


@pytest.mark.parametrize("name", ["aq_moe_route", "aq_moe_experts", "aq_moe", "aq_embed"])
@pytest.mark.parametrize("handle", [False, True])
def test_on_another_stream(world, name, handle):  # noqa: F811
    res = _calls()[name](SIDE if handle else _Stream(SIDE))
    assert world.called[-1] == (name, SIDE)
    assert world.made and all(s == SIDE for s, _ in world.made)
    given = {id(t) for t in _flat(res)}
    for _, t in world.made:
        assert id(t) not in given or HERE in t.known_to
    assert world.now.cuda_stream == HERE


@pytest.mark.parametrize("name", ["aq_moe_route", "aq_moe_experts", "aq_moe", "aq_embed"])
@pytest.mark.parametrize("stream", [None, HERE, "current"])
def test_on_the_current_stream(world, name, stream):  # noqa: F811
    _calls()[name](world.now if stream == "current" else stream)
    assert world.called[-1] == (name, HERE)
    assert world.made and all(s == HERE and not t.known_to for s, t in world.made)

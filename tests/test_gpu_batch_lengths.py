"""Lengths below zero are empty rows, down to the lowest int32."""
import pytest
import torch

from .test_gpu_attention_batch import Case

pytestmark = pytest.mark.gpu

aq = pytest.importorskip("quantized_matmul_affine_gb300")


@pytest.mark.parametrize("members", [3, 12])     # 15 and 60 rows a KV head and token
@pytest.mark.parametrize("L", [1, 3])
def test_negative_lengths(L, members):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    c = Case(10, 2, 128, 32, 4, 64, "fp16", L, [40] * members + [50], [(members, 200)])
    for b, n in ((0, -2 ** 31), (members // 2, -2 ** 31 + 1), (members, -1)):
        c.lens[b] = n
    o = c.check()
    assert not o[0].any() and not o[members // 2].any() and not o[members].any()
    assert aq.aq_device_error(clear=True) == 0

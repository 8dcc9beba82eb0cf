"""Batch attention at scales other than D ** -0.5, on both sides of the choice
of kernel: zero (the plain mean of the values), negative, and so small that
the factor of a row's products underflows.  Shared lengths end inside a tile
of keys.  The tolerances are those of test_gpu_attention_batch."""
import pytest
import torch

from .test_gpu_attention_batch import Case

pytestmark = pytest.mark.gpu

aq = pytest.importorskip("quantized_matmul_affine_gb300")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert aq.aq_device_error(clear=True) == 0


@pytest.mark.parametrize("scale", [0.0, -0.0, -0.09, 1e-30, -2.0 ** -140])
@pytest.mark.parametrize("H,KV,D,bits,dtype,L,members", [
    (10, 2, 128, 4, "fp16", 1, 3),      # 15 rows a KV head
    (10, 2, 128, 4, "fp16", 1, 10),     # 50: one row tile
    (10, 2, 128, 8, "bf16", 1, 40),     # 200: two
    (6, 2, 256, 4, "bf16", 2, 12),
    (8, 2, 64, 8, "fp16", 1, 33),
])
def test_scales(H, KV, D, bits, dtype, L, members, scale):
    c = Case(H, KV, D, 32, bits, 64, dtype, L, [L + 5 * b % 70 for b in range(members)], [(members, 333)])
    c.scale = scale
    c.check()

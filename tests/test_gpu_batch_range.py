"""Batch attention where 16-bit floats run out of range: weights far below a
row's largest, and cached values next to the largest fp16 number.  Sizes are
those of the kernel for many rows."""
import numpy as np
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


def _set(c, page, slot, which, scale, bias):
    a, n = c.geo.spans(slot)[which]
    c.pool[:, page, :, a:a + n] = np.resize(np.array([scale, bias], np.float16), n // 2).view(np.uint8)


@pytest.mark.parametrize("D,bits", [(64, 4), (128, 8)])
def test_one_key_outweighs_the_others(D, bits):
    # The first key's weight is 2^17 to 2^21 times any other's, its value is
    # zero, and the others weigh alike: the output is theirs alone.  With 152
    # KV heads a piece of work is all the shared keys, so they meet the same
    # maximum.  Scores are exact here; a weight 2^-21 of the largest, rounded
    # once to fp16, is off by 2^-11 of itself, which the 2-norm bound of
    # test_gpu_attention_batch (2^-9 and the output's rounding) allows.
    c = Case(152, 152, D, 128, bits, 64, "fp16", 1, [1] * 17, [(17, 512)])
    for b in range(c.B):
        for j in range(c.lens[b]):
            page, slot = c.table[b, j // 128], j % 128
            _set(c, page, slot, 2, 0.0, 1.0 if j == 0 else 0.0)
            _set(c, page, slot, 3, *((0.0, 0.0) if j == 0 or j >= 512 else (0.5, 100.0)))
    power = np.random.default_rng(1).uniform(17, 21, size=(c.B, 1, c.H, 1))   # of two, by row
    c.q = torch.from_numpy(np.broadcast_to(power / 32, (c.B, 1, c.H, D)).copy()).to(torch.float16)
    c.scale = 32 * float(np.log(2)) / D
    c.check()


@pytest.mark.parametrize("D,bits,scale", [
    (128, 4, 8736.0),     # 15 * 8736 - 65504 = 65536
    (256, 4, 8736.0),
    (64, 8, 514.0),       # 255 * 514 - 65504 = 65566
    (128, 8, 514.0),
])
@pytest.mark.parametrize("which", [2, 3])
def test_values_next_to_the_largest_fp16(D, bits, scale, which):
    # What the quantiser makes of a group that holds both -65504 and 65504: its
    # rounded scale puts the top code past the largest fp16 number.  Taken as
    # 65504 it is off by 2^-10 of itself: twice the rounding that the score's
    # tolerance counts (so smag is doubled), and the value's counts 2^-10.
    assert np.float16(131008 / (2 ** bits - 1)) == scale
    c = Case(12, 2, D, 32, bits, 64, "bf16", 1, [20] * 9, [(9, 333)], qscale=2.0 ** -17 if which == 2 else 1.0)
    for j in range(0, 320, 3):
        _set(c, c.table[0, j // 32], j % 32, which, scale, -65504.0)
    want, smag, vmag, bmax = c.reference()
    c.check(ref=(want, 2 * smag, vmag, bmax))

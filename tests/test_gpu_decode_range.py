"""The few-token form near the ends of fp32: x scaled by a power of two, so h (its square) and the
outputs reach 2^124 and 2^-100, all finite and normal. Tolerance as in the test of the definition
(its terms scale with the values)."""
import pytest
import torch

from tests.gpu_helpers import lib
from tests.test_gpu_decode import DEV, _check, _deq, _inputs, _reference, _weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("power", [-50, -30, 40, 55, 58, 60])
def test_large_and_small_values(power, dtype):
    moe = lib()
    T, E, k, H, I = 3, 4, 2, 256, 320
    Wg, Wu, Wd = _weights(E, H, I)
    layer = moe.MoELayer(Wg, Wu, Wd, k, dtype=dtype)
    x, logits, _ = _inputs(T, H, E)
    x = (x.float() * 2.0 ** power).bfloat16()
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    out = layer.decode(x, logits, ids=ids, w=w)
    ref, mag = _reference(x, ids, w, [_deq(W, dtype) for W in (Wg, Wu, Wd)], None)
    assert float(ref.abs().max()) < 2.0 ** 127 and layer.check() == 0
    _check(out, ref, mag)

"""Sizes on both sides of the rules that choose a kernel of moe.linear, against float64: pairs or
128-wide tiles for rows that are not aligned (K 2048 | 2056, gated 1024 | 1032), two pairs to a
tile or 128-wide tiles (74 | 75 of them, K 2048 and 4096)."""
import pytest
import torch

from tests.gpu_helpers import lib
from tests.test_gpu_linear import BF, F32, _check, _make, _run

pytestmark = pytest.mark.gpu

SIZES = [  # M, N, K, gated
    (2500, 2041, 2048, False), (2500, 2041, 2056, False),
    (2500, 1021, 1024, True), (2500, 1021, 1032, True),
    (300, 2880, 4096, False), (300, 3200, 4096, False), (300, 3201, 4096, False),
    (600, 960, 4096, True), (600, 961, 4096, True), (257, 2300, 4104, False),
    (512, 2304, 2048, False), (512, 2432, 2048, False), (512, 1216, 2040, True),
]


@pytest.mark.parametrize("M,N,K,gated", SIZES)
def test_both_sides_of_a_choice(M, N, K, gated):
    moe = lib()
    for act, bias, residual, out in (("gelu", BF, True, BF), ("silu", None, False, F32)):
        c = _make(M, N, K, gated, bias, residual, out)
        y = _run(moe, c, act, gated, out)
        _check(y, c, act, gated)
        assert torch.equal(_run(moe, c, act, gated, out), y)
    assert moe.linear_status() == 0

"""The activations of moe.linear over their whole range, tails included: x W^T with one nonzero
term is an exact z, so the result's relative error is the activation's own.

Bound of the relative error, f32 out: a few ulp of the result (the polynomial of erfc 5, __expf 2,
the division 2, the products 1/2 each: 16 * 2^-24 covers them), and what the argument's own rounding does to the
factor.  GELU: erfc(a), a = -z / sqrt 2 off by 2^-23 relative (the constant's and the product's
rounding), changes by at most 2 a^2 + 1 = z^2 + 1 times that.  SiLU, and GELU's tanh form with
y = 2 sqrt(2 / pi) (z + 0.044715 z^3): the factor 1 / (1 + e^-y) changes by |y| times y's relative
error, 2^-21 for the few roundings of y; __expf adds |y| 1.44 2^-23 or less (its argument
times log2 e is rounded to 2^-24 of it)."""
import math

import pytest
import torch

from tests.gpu_helpers import lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _exact(z, act):
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z / (1 + torch.exp(-_inner(z)))


def _inner(z):
    return 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)


def _bound(z, act):
    ulp = 2.0 ** -24
    if act == "gelu":
        return 16 * ulp + 2 * ulp * (z.square() + 1)
    y = (z if act == "silu" else _inner(z)).abs()
    return 16 * ulp + 2.0 ** -21 * y + 2.0 ** -22 * y


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M", [16, 2000, 16000])
def test_relative_error_in_the_tails(M, act):
    moe = lib()
    K, N = 64, 128
    # bf16 values of [-8, 8], each in a row of x and a column of w: z = x[m, 0] w[n, 0]
    x = torch.zeros((M, K), dtype=BF, device=DEV)
    w = torch.zeros((N, K), dtype=BF, device=DEV)
    x[:, 0] = torch.linspace(-8, 8, M, device=DEV).to(BF)
    w[:, 0] = torch.linspace(1 / N, 1, N, device=DEV).to(BF)
    z = x[:, :1].double() * w[:, :1].double().t()
    want = _exact(z, act)
    for out_dtype in (F32, BF):
        out = moe.linear(x, w, act=getattr(moe, "ACT_" + act.upper()), out_dtype=out_dtype)
        half = torch.finfo(out_dtype).eps / 2
        err = (out.double() - want).abs()
        tol = (half + 2 * _bound(z, act)) * want.abs()
        assert bool((err <= tol).all()), float((err / want.abs().clamp(min=1e-300)).max())


@pytest.mark.parametrize("M", [4, 100])
def test_gelu_at_the_ends(M):
    """Zeros, infinities, NaN and values whose factor is 0 or 1 in fp32."""
    moe = lib()
    vals = [0.0, -0.0, 20.0, 1e30, float("inf"), -20.0, -1e30, float("nan")]
    x = torch.zeros((M, 8), dtype=BF, device=DEV)
    w = torch.zeros((8, 8), dtype=BF, device=DEV)
    out = moe.linear(x, w, bias=torch.tensor(vals, device=DEV), act=moe.ACT_GELU, out_dtype=F32)
    assert bool((out[:, :2] == 0).all())
    for c in (2, 3, 4):
        assert bool((out[:, c] == torch.tensor(vals[c], device=DEV, dtype=F32)).all())
    assert bool((out[:, 5:7].abs() < 1e-30).all()) and bool(torch.isnan(out[:, 7]).all())

"""moe_linear: act(x W^T + bias) [* (x W_up^T + bias_up)] + residual against float64.

Tolerance per element: the rounding of out, eps/2 of its type relative to the value, and the
fp32 sums.  Products of two bf16 values are exact in fp32; K additions in any order, truncating
ones of 2^-23 included, are off by at most K 2^-23 of the sum of magnitudes S.  The activations
have slopes below 1.13, gating multiplies by the other factor's size, and each of the few fp32
operations after the sums is off by some ulp (2^-20 of the magnitudes covers them, CUDA's erff,
tanhf and expf included).
"""
import math

import pytest
import torch

from tests.gpu_helpers import lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _make(M, N, K, gated, bias, residual, out, seed=0, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    rows = 2 * N if gated else N
    return dict(x=r(M, K + pad).to(BF)[:, :K], w=(r(rows, K + pad) / K ** 0.5).to(BF)[:, :K],
                bias=(0.5 * r(rows)).to(bias) if bias else None,
                residual=r(M, N + pad).to(out)[:, :N] if residual else None)


def _reference(c, act, gated):
    x, w = c["x"].double(), c["w"].double()
    z, S = x @ w.t(), x.abs() @ w.abs().t()
    if c["bias"] is not None:
        z, S = z + c["bias"].double(), S + c["bias"].double().abs()
    if gated:
        N = z.shape[1] // 2
        a, u = _act(z[:, :N], act), z[:, N:]
        y, E = a * u, 1.13 * S[:, :N] * u.abs() + a.abs() * S[:, N:]
    else:
        y, E = _act(z, act), 1.13 * S
    mag = y.abs()
    if c["residual"] is not None:
        y, mag = y + c["residual"].double(), mag + c["residual"].double().abs()
    return y, E, mag


def _check(out, c, act, gated):
    y, E, mag = _reference(c, act, gated)
    K = c["x"].shape[1]
    half = torch.finfo(out.dtype).eps / 2
    tol = half * y.abs() + (K + 64) * 2.0 ** -23 * E + 2.0 ** -20 * mag + 1e-30
    assert torch.isfinite(out).all()
    err = (out.double() - y).abs()
    assert not (err > tol).any(), f"worst {float((err / tol).max()):.2f} of the bound"
    rms = float(err.square().mean().sqrt() / y.square().mean().sqrt())
    # no element is off by more than half a step of its own value plus its sums' share, so the
    # root mean square is at most half a step (a few elements may all be near it) plus theirs
    assert rms < (half + 1e-4 if out.dtype == BF else 2e-5), rms


def _run(moe, c, act, gated, out_dtype, **kw):
    return moe.linear(c["x"], c["w"], bias=c["bias"], act=getattr(moe, "ACT_" + act.upper()),
                      gated=gated, residual=c["residual"], out_dtype=out_dtype, **kw)


# every kernel's edges: 16 | 17 tokens, 128- and 256-row tiles, ragged N and K, one k-block
SIZES = [(1, 8, 4096), (1, 1, 8), (3, 5, 72), (8, 256, 512), (9, 100, 200), (16, 257, 1024),
         (16, 4100, 64), (17, 64, 64), (17, 1, 8), (33, 100, 200), (100, 333, 520),
         (128, 64, 2048), (129, 130, 136), (300, 8, 4096), (513, 1000, 72),
         (520, 1001, 200), (260, 1003, 1024), (140, 301, 2048)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(M, N, K, gated):
    moe = lib()
    for act, bias, residual, out in (("none", None, False, F32), ("silu", BF, True, BF),
                                     ("gelu", F32, False, BF), ("relu", F32, True, F32)):
        c = _make(M, N, K, gated, bias, residual, out)
        _check(_run(moe, c, act, gated, out), c, act, gated)


# enough 256-row tiles for the CTA pairs (74 of them on 148 SMs), ragged in every direction
PAIR_SIZES = [(5000, 1000, 192), (2500, 2040, 520), (20000, 250, 72), (4864, 1024, 64),
              (1024, 5000, 136), (2500, 2041, 136), (4700, 1100, 64)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", PAIR_SIZES)
def test_pair_sizes(M, N, K, gated):
    moe = lib()
    for act, bias, residual, out in (("none", None, True, BF), ("gelu_tanh", F32, False, F32)):
        c = _make(M, N, K, gated, bias, residual, out)
        _check(_run(moe, c, act, gated, out), c, act, gated)


# 17 to 33 such tiles and a long K: two CTA pairs to a tile
SPLIT_SIZES = [(257, 2300, 4096, False), (257, 1200, 4104, True), (700, 1500, 4136, False),
               (129, 6001, 5000, False), (600, 799, 4096, True), (512, 2048, 4160, True)]


@pytest.mark.parametrize("M,N,K,gated", SPLIT_SIZES)
def test_split_sizes(M, N, K, gated):
    moe = lib()
    for act, bias, residual, out, pad in (("none", None, True, BF, 0), ("silu", BF, False, BF, 8),
                                          ("gelu_tanh", F32, True, F32, 0)):
        c = _make(M, N, K, gated, bias, residual, out, pad=pad)
        y = _run(moe, c, act, gated, out)
        _check(y, c, act, gated)
        for _ in range(3):
            assert torch.equal(_run(moe, c, act, gated, out), y)
    z = c["residual"].clone()                         # in place, and into wider rows
    assert torch.equal(moe.linear(c["x"], c["w"], bias=c["bias"], act=moe.ACT_GELU_TANH,
                                  gated=gated, residual=z, out=z), y)
    wide = torch.full((M, N + 24), 7.0, dtype=F32, device=DEV)
    _run(moe, c, "gelu_tanh", gated, F32, out=wide[:, 8:N + 8])
    assert torch.equal(wide[:, 8:N + 8], y)
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, N + 8:] == 7).all())
    # a non-finite value stays in its row (x) or its column (w)
    c["x"][M - 1, 0], c["w"][0, K - 1] = float("inf"), float("nan")
    bad = ~torch.isfinite(_run(moe, c, "gelu_tanh", gated, F32))
    assert bool(bad[:, 0].all()) and not bool(bad[:M - 1, 1:].any())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 40, 5000])
def test_activations(M, act):
    moe = lib()
    for gated in (False, True):
        c = _make(M, 1016, 128, gated, BF, True, BF, seed=3)
        _check(_run(moe, c, act, gated, BF), c, act, gated)


@pytest.mark.parametrize("M", [4, 60, 5000])
def test_strides_and_alignment(M):
    """Rows apart in every operand, and an output whose rows start at odd elements."""
    moe = lib()
    for N, pad in ((1001, 8), (1000, 24), (77, 64)):
        for out in (BF, F32):
            c = _make(M, N, 256, False, BF, True, out, pad=pad)
            buf = torch.full((M + 2, N + 5), 7.0, dtype=out, device=DEV)
            dst = buf[1:M + 1, 3:3 + N]
            _run(moe, c, "none", False, out, out=dst)
            _check(dst, c, "none", False)
            assert (buf[0] == 7).all() and (buf[M + 1] == 7).all()
            assert (buf[:, :3] == 7).all() and (buf[:, 3 + N:] == 7).all()


@pytest.mark.parametrize("M", [1, 7, 90, 5000])
def test_residual_in_place(M):
    moe = lib()
    c = _make(M, 1024, 128, True, None, True, BF)
    want = _run(moe, c, "silu", True, BF)
    buf = c["residual"].clone()
    c["residual"] = buf
    _run(moe, c, "silu", True, BF, out=buf)
    assert torch.equal(buf, want)


@pytest.mark.parametrize("M", [3, 50, 5000])
def test_non_finite_values(M):
    """NaN and infinity reach exactly the rows and columns that read them."""
    moe = lib()
    N, K = 1016, 200
    for act in ACTS:
        c = _make(M, N, K, False, F32, False, BF)
        clean = _run(moe, c, act, False, BF)
        c["x"][1, K - 1] = float("nan")
        c["w"][5, 0] = float("nan")
        c["bias"][9] = float("nan")
        c["bias"][11] = float("inf")
        out = _run(moe, c, act, False, BF)
        nan = torch.isnan(out)
        expect = torch.zeros_like(nan)
        expect[1, :] = True
        expect[:, 5] = True
        expect[:, 9] = True
        assert torch.equal(nan, expect)
        rows = [r for r in range(M) if r != 1]
        assert torch.isinf(out[rows, 11]).all()
        keep = ~expect
        keep[:, 11] = False
        assert torch.equal(out[keep], clean[keep])


def test_repeats_bit_for_bit():
    moe = lib()
    for M, N, K, gated in ((1, 256, 7168, False), (13, 64, 2048, True), (77, 320, 2880, False),
                           (5000, 1000, 192, True)):
        c = _make(M, N, K, gated, BF, True, BF)
        first = _run(moe, c, "silu", gated, BF)
        for _ in range(5):
            assert torch.equal(_run(moe, c, "silu", gated, BF), first)


def test_compiled_call_and_python_form_agree(monkeypatch):
    """Both forms of the call give the same bits and types, and return a given output itself."""
    moe = lib()
    from mixture_experts_expert_route_b200 import _binding, _lib
    cases = [(_make(M, N, 264, gated, bias, res, out, pad=pad), gated, out)
             for M, N, gated, bias, res, out, pad in (
                 (1, 40, False, None, False, BF, 0), (5, 33, True, BF, True, F32, 8),
                 (70, 64, False, F32, True, BF, 64), (300, 511, True, F32, False, F32, 0))]
    first = [_run(moe, c, "silu", gated, out) for c, gated, out in cases]
    given = torch.empty((5, 80), dtype=F32, device=DEV)[:, 8:41]
    assert _run(moe, cases[1][0], "silu", True, None, out=given) is given
    assert torch.equal(given, first[1])
    assert _lib._calls.linear is _binding.linear
    w = torch.nn.Parameter(cases[0][0]["w"].clone())        # a subclass that wants a gradient
    y = moe.linear(cases[0][0]["x"], w, act=moe.ACT_SILU)
    assert torch.equal(y, first[0]) and not y.requires_grad
    monkeypatch.setattr(_lib._calls, "linear", lambda *a: NotImplemented)
    for (c, gated, out), y in zip(cases, first):
        z = _run(moe, c, "silu", gated, out)
        assert z.dtype == y.dtype and z.stride() == y.stride() and torch.equal(z, y)
    assert _run(moe, cases[1][0], "silu", True, None, out=given) is given


def test_empty_batch():
    moe = lib()
    out = moe.linear(torch.empty((0, 64), dtype=BF, device=DEV),
                     torch.empty((8, 64), dtype=BF, device=DEV))
    assert out.shape == (0, 8)


def test_refusals():
    moe = lib()
    x = torch.zeros((4, 64), dtype=BF, device=DEV)
    w = torch.zeros((16, 64), dtype=BF, device=DEV)
    bad = [dict(w=w.float()), dict(w=w[:, :56]), dict(bias=torch.zeros(8, device=DEV)),
           dict(bias=torch.zeros(16, device=DEV, dtype=torch.float16)),
           dict(residual=torch.zeros((4, 16), device=DEV)), dict(out_dtype=torch.float16),
           dict(out=torch.zeros((4, 8), device=DEV, dtype=BF)), dict(x=x.t()[:4, :4]),
           dict(bias=torch.zeros(16))]
    for kw in bad:
        with pytest.raises(ValueError):
            moe.linear(**{**dict(x=x, w=w), **kw})
    with pytest.raises(moe.MoEError):                       # K % 8
        moe.linear(x[:, :60], w[:, :60])
    with pytest.raises(moe.MoEError):                       # rows off a 16-byte boundary
        moe.linear(torch.zeros((4, 72), dtype=BF, device=DEV)[:, 4:68], w)
    with pytest.raises(moe.MoEError):                       # a broadcast residual
        moe.linear(x, w, residual=torch.zeros((1, 16), device=DEV, dtype=BF).expand(4, 16))
    with pytest.raises(ValueError):
        moe.linear(x, w[:15], gated=True)


def test_streams_graphs_and_chains():
    """A chain of dependent products (early launches wait for their input), the same on two
    streams at once, and captured."""
    moe = lib()
    for M in (2, 40, 4000):
        H, I = 512, 768
        c = _make(M, I, H, True, None, False, BF)
        wd = (torch.randn((H, I), device=DEV) / I ** 0.5).to(BF)

        def chain(x, stream=None):
            for _ in range(3):
                h = moe.linear(x, c["w"], act=moe.ACT_SILU, gated=True, stream=stream)
                x = moe.linear(h, wd, residual=x, stream=stream)
            return x

        want = chain(c["x"])
        ref = c["x"].double()
        for _ in range(3):
            z = ref @ c["w"].double().t()
            h = (z[:, :I] / (1 + torch.exp(-z[:, :I])) * z[:, I:]).to(BF).double()
            ref = (h @ wd.double().t() + ref).to(BF).double()
        # a few flips of bf16 roundings on the way through
        assert float((want.double() - ref).norm() / ref.norm()) < 2.0 ** -8
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        got = [chain(c["x"], s) for _ in range(5) for s in (s1, s2)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in got)
        xs = c["x"].clone()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = chain(xs)
        for seed in (5, 6):
            xs.copy_(torch.randn((M, H), device=DEV).to(BF))
            gr.replay()
            assert torch.equal(o, chain(xs))


def test_offsets_past_32_bits():
    """x, then out and the residual, of more than 2^31 elements: the first and last rows."""
    moe = lib()
    M, K, N = 270000, 8192, 16
    x = torch.empty((M, K), dtype=BF, device=DEV).normal_()
    w = (torch.randn((N, K), device=DEV) / K ** 0.5).to(BF)
    out = moe.linear(x, w, act=moe.ACT_RELU)
    for rows in (slice(0, 300), slice(M - 300, M)):
        c = dict(x=x[rows], w=w, bias=None, residual=None)
        _check(out[rows], c, "relu", False)
    del x, out
    M, K, N = 70000, 64, 32768
    x = torch.randn((M, K), device=DEV).to(BF)
    w = (torch.randn((N, K), device=DEV) / K ** 0.5).to(BF)
    res = torch.empty((M, N), dtype=BF, device=DEV).normal_()
    rows = slice(M - 200, M)
    keep = res[rows].clone()
    out = moe.linear(x, w, residual=res, out=res)
    assert out is res
    _check(out[rows], dict(x=x[rows], w=w, bias=None, residual=keep), "none", False)

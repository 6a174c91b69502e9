"""The whole layer for a few tokens in one kernel (moe_decode_forward) against the layer's
definition in float64: out = residual + sum_j w_j (SiLU(x Wg) * (x Wu)) Wd.

Tolerance of out, per element:
    |out - ref| <= 2^-8 |ref| + 2^-10 * mag
2^-8 (half of bf16's eps) is the one rounding of out.  mag is the sum of magnitudes that an
error in the sums is relative to, sum_j w_j sum_i (|h_i| + how g's and u's sums of magnitudes
move h_i) |Wd_i|; its factor covers h's representation (hi + lo of two bf16 values, 2^-17; with
e4m3 weights f16, 2^-12) and the fp32 sums: the products are exact, and n additions in any order, truncating ones of
2^-23 included, are off by at most n 2^-23 of the sum of magnitudes: 2^-11 for the n <= 2^12
terms here at the very worst, into h and down.
"""
import pytest
import torch

from tests.gpu_helpers import check_routing, lib

pytestmark = pytest.mark.gpu

BF16, FP8 = 0, 1
DEV = "cuda:0"
C = 2.0 ** -10


def _weights(E, H, I, seed=0, dev=DEV):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    return ((r(E, H, I) / H ** 0.5).bfloat16(), (r(E, H, I) / H ** 0.5).bfloat16(),
            (r(E, I, H) / I ** 0.5).bfloat16())


def _inputs(T, H, E, seed=1, dev=DEV):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn((T, H), generator=g, device=dev).bfloat16(),
            torch.randn((T, E), generator=g, device=dev),
            torch.randn((T, H), generator=g, device=dev).bfloat16())


def _deq(W, dtype):
    """The expert matrices as the kernel's weights stand for them, float64."""
    if dtype == BF16:
        return W.double()
    # a quotient of two tensors: torch divides by a Python number through its reciprocal
    s = W.float().abs().amax(dim=(1, 2), keepdim=True)
    s = s / torch.full_like(s, 448.0)
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (W.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.double() * s.double()


def _reference(x, ids, w, Ws, residual):
    """(out, magnitude) in float64; magnitude = sum_j w_j sum_i |h_i Wd_i|."""
    Wg, Wu, Wd = Ws
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    xd = x.double()
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            g, u = xd[t] @ Wg[e], xd[t] @ Wu[e]
            h = g / (1 + torch.exp(-g)) * u
            out[t] += w[t, j].double() * (h @ Wd[e])
            # |dh| <= |u| |dg| |silu'| + |silu(g)| |du|, |silu'| < 1.1: through the sums of
            # magnitudes of g and u
            ga, ua = xd[t].abs() @ Wg[e].abs(), xd[t].abs() @ Wu[e].abs()
            bound = h.abs() + 1.1 * u.abs() * ga + g.abs() * ua
            mag[t] += w[t, j].double() * (bound @ Wd[e].abs())
    if residual is not None:
        out += residual.double()
    return out, mag


def _check(out, ref, mag):
    err = (out.double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + C * mag + 1e-30
    assert torch.isfinite(out).all()
    bad = err > tol
    assert not bad.any(), f"{int(bad.sum())} off, worst {float((err / tol).max()):.2f} of the bound"
    # and in the mean: the rounding of out alone is eps / 2 / sqrt(3) at most
    rms = float((err.square().mean() / ref.square().mean()).sqrt())
    assert rms < 2.0 ** -8


SHAPES = [  # T, E, k, H, I
    (1, 8, 2, 256, 512), (2, 8, 2, 256, 512), (7, 8, 2, 256, 512), (8, 8, 2, 256, 512),
    (9, 8, 2, 256, 512), (16, 8, 2, 256, 512), (16, 8, 8, 256, 512),
    (1, 1, 1, 64, 64), (16, 1, 1, 64, 64),              # one expert, one tile
    (1, 128, 8, 2048, 768), (5, 128, 8, 2048, 768), (16, 128, 8, 512, 768),
    (3, 32, 4, 2880, 2880), (13, 32, 4, 576, 320),      # H, I not multiples of 128
    (4, 256, 8, 192, 192), (1, 256, 128, 64, 128), (2, 60, 6, 320, 1344),
    (16, 4, 1, 64, 2048), (1, 2, 2, 64, 4096),          # one row tile, many k-blocks
    (2, 4, 2, 4096, 64),                                  # many row tiles, one k-block
]


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("T,E,k,H,I", SHAPES)
def test_matches_definition(T, E, k, H, I, dtype):
    moe = lib()
    Wg, Wu, Wd = _weights(E, H, I)
    layer = moe.MoELayer(Wg, Wu, Wd, k, dtype=dtype)
    Ws = [_deq(W, dtype) for W in (Wg, Wu, Wd)]
    for seed, with_res in ((1, True), (2, False)):
        x, logits, res = _inputs(T, H, E, seed)
        ids = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
        w = torch.full((T, k), -7.0, device=DEV)
        out = layer.decode(x, logits, residual=res if with_res else None, ids=ids, w=w)
        assert layer.check() == 0
        check_routing(ids, w, logits)
        _check(out, *_reference(x, ids, w, Ws, res if with_res else None))


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_routing_equals_route_topk_and_ties(dtype):
    """Ties, signed zeros, infinities and NaN logits: ids and w bit for bit as moe_route_topk."""
    moe = lib()
    T, E, k, H, I = 6, 40, 5, 128, 64
    layer = moe.MoELayer(*_weights(E, H, I), k, dtype=dtype)
    x, logits, _ = _inputs(T, H, E)
    logits[0] = 0.0
    logits[0, ::2] = -0.0
    logits[1] = logits[1].round()
    logits[2, 7] = float("nan")
    logits[3, :] = float("-inf")
    logits[3, 5:] = -3.0e38
    logits[4, :36] = float("nan")
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    layer.decode(x, logits, ids=ids, w=w)
    ids_r, w_r = moe.route_topk(logits, k)
    assert layer.check() == 0
    assert torch.equal(ids, ids_r)
    assert torch.equal(w.view(torch.int32), w_r.view(torch.int32))


def test_all_tokens_on_the_same_experts():
    """One expert takes every token (16 columns), and token order does not matter."""
    moe = lib()
    T, E, k, H, I = 16, 16, 3, 384, 640
    Wg, Wu, Wd = _weights(E, H, I)
    layer = moe.MoELayer(Wg, Wu, Wd, k)
    x, logits, res = _inputs(T, H, E)
    logits[:, 3] += 50.0
    logits[:, 9] += 40.0
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    out = layer.decode(x, logits, residual=res, ids=ids, w=w)
    assert (ids[:, 0] == 3).all() and (ids[:, 1] == 9).all()
    _check(out, *_reference(x, ids, w, [W.double() for W in (Wg, Wu, Wd)], res))
    p = torch.randperm(T, generator=torch.Generator().manual_seed(3)).to(DEV)
    out_p = layer.decode(x[p].contiguous(), logits[p].contiguous(),
                         residual=res[p].contiguous())
    assert torch.equal(out_p, out[p])
    # each token alone: its sums are cut at other places, so equal up to the bound only
    one = torch.cat([layer.decode(x[t:t + 1], logits[t:t + 1], residual=res[t:t + 1])
                     for t in range(T)])
    _check(one, *_reference(x, ids, w, [W.double() for W in (Wg, Wu, Wd)], res))


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_repeats_bit_for_bit_and_shares_a_workspace(dtype):
    """The same call gives the same bits; one workspace serves calls of other T and layers."""
    moe = lib()
    E, k, H, I = 32, 4, 512, 448
    layer = moe.MoELayer(*_weights(E, H, I), k, dtype=dtype)
    other = moe.MoELayer(*_weights(8, 256, 128, seed=5), 2, dtype=dtype)
    x, logits, res = _inputs(16, H, E)
    xo, lo, _ = _inputs(3, 256, 8)
    ws = layer.decode_workspace(16)
    first = {}
    for rep in range(10):
        for T in (1, 16, 5):
            out = layer.decode(x[:T].contiguous(), logits[:T].contiguous(),
                               residual=res[:T].contiguous())
            assert T not in first or torch.equal(first[T], out)
            first.setdefault(T, out)
        moe.decode_forward(dtype, xo, lo, other.packed, other.scales, 8, 128, 2, ws=ws)
    assert layer.decode_workspace(5) is ws
    assert other.decode_workspace(3) is ws            # one per stream, whichever layer asks
    assert layer.check() == 0


@pytest.mark.parametrize("T,E,k,H,I,dtype", [(1, 8, 2, 2048, 3584, BF16), (1, 64, 8, 1024, 512, BF16),
                                             (16, 32, 4, 1024, 768, BF16), (1, 32, 4, 1472, 1472, FP8),
                                             (13, 32, 4, 1472, 1472, FP8), (3, 2, 1, 64, 64, BF16)])
def test_no_partial_sum_is_read_before_it_is_written(T, E, k, H, I, dtype):
    """With NaN in all of the workspace but its header every output is the same: each CTA waits
    for the others' sums, and reads only sums of this call."""
    moe = lib()
    layer = moe.MoELayer(*_weights(E, H, I), k, dtype=dtype)
    ws = moe.decode_workspace(dtype, T, k, E, H, I, torch.device(DEV))
    for seed in range(8):
        x, logits, res = _inputs(T, H, E, seed=seed)
        args = (dtype, x, logits, layer.packed, layer.scales, E, I, k, res)
        out = moe.decode_forward(*args, ws=ws)
        for _ in range(4):
            poisoned = torch.full_like(ws, 0xFF)
            code = moe._lib.lib().moe_decode_workspace_init(
                poisoned.data_ptr(), poisoned.numel(), torch.cuda.current_stream().cuda_stream)
            assert code == 0
            assert torch.equal(moe.decode_forward(*args, ws=poisoned), out)


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_compiled_call_and_python_form_agree(dtype, monkeypatch):
    """Both forms of the call give the same bits and optional outputs."""
    moe = lib()
    from mixture_experts_expert_route_b200 import _binding, _lib
    T, E, k, H, I = 5, 16, 3, 256, 192
    layer = moe.MoELayer(*_weights(E, H, I), k, dtype=dtype)
    x, logits, res = _inputs(T, H, E)
    def call(**kw):
        ids = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
        w = torch.zeros((T, k), device=DEV)
        return layer.decode(x, logits, ids=ids, w=w, **kw), ids, w
    first = [call(), call(residual=res)]
    given = torch.empty_like(x)
    assert layer.decode(x, logits, residual=res, out=given) is given
    assert torch.equal(given, first[1][0]) and _lib._calls.decode is _binding.decode
    monkeypatch.setattr(_lib._calls, "decode", lambda *a: NotImplemented)
    for got, want in zip([call(), call(residual=res)], first):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert layer.check() == 0


def test_a_timeout_makes_the_workspaces_anew():
    """After MOE_ERR_TIMEOUT (here written by the host) decode calls do not use the old one."""
    moe = lib()
    layer = moe.MoELayer(*_weights(8, 256, 128), 2)
    x, logits, _ = _inputs(3, 256, 8)
    out, ws = layer.decode(x, logits), layer.decode_workspace(3)
    assert layer.check() == 0 and layer.decode_workspace(3) is ws
    layer.status.fill_(5)
    assert layer.check() == 5 and layer.decode_workspace(3) is not ws
    layer.status.zero_()
    assert torch.equal(layer.decode(x, logits), out) and layer.check() == 0


def test_residual_may_be_the_output():
    moe = lib()
    T, E, k, H, I = 5, 8, 2, 256, 192
    layer = moe.MoELayer(*_weights(E, H, I), k)
    x, logits, res = _inputs(T, H, E)
    want = layer.decode(x, logits, residual=res)
    got = res.clone()
    layer.decode(x, logits, residual=got, out=got)
    assert torch.equal(got, want)
    # the input itself as residual and output: a layer updating the stream in place
    want = layer.decode(x, logits, residual=x)
    layer.decode(x, logits, residual=x, out=x)
    assert torch.equal(x, want)


def test_rows_behind_the_batch_stay():
    moe = lib()
    T, E, k, H, I = 3, 8, 2, 192, 128
    layer = moe.MoELayer(*_weights(E, H, I), k)
    x, logits, _ = _inputs(T, H, E)
    buf = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device=DEV)
    layer.decode(x, logits, out=buf[1:T + 1])
    assert (buf[0] == 7).all() and (buf[T + 1] == 7).all()
    assert torch.equal(buf[1:T + 1], layer.decode(x, logits))


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_non_finite_values_stay_in_their_token(dtype):
    """NaN or infinity in one token's x reaches that token's output only, also where tokens
    share an expert; a huge finite x is not squashed."""
    moe = lib()
    T, E, k, H, I = 4, 4, 4, 128, 192
    Wg, Wu, Wd = _weights(E, H, I)
    layer = moe.MoELayer(Wg, Wu, Wd, k, dtype=dtype)
    x, logits, _ = _inputs(T, H, E)
    clean = layer.decode(x, logits)
    x2 = x.clone()
    x2[1, 5] = float("nan")
    x2[2, 17] = float("inf")
    out = layer.decode(x2, logits)
    assert torch.equal(out[0], clean[0]) and torch.equal(out[3], clean[3])
    assert torch.isnan(out[1]).all()
    assert not torch.isfinite(out[2]).any()
    x3 = x.clone()
    x3[0] *= 2.0 ** 40
    ids, w = moe.route_topk(logits, k)
    ref, mag = _reference(x3[:1], ids[:1], w[:1], [_deq(W, dtype) for W in (Wg, Wu, Wd)], None)
    out = layer.decode(x3, logits)
    _check(out[:1], ref, mag)


def test_nan_weight_stays_nan():
    """A NaN among the e4m3 codes is a NaN in the outputs that read it, not a number."""
    moe = lib()
    E, k, H, I = 2, 1, 128, 128
    Wg, Wu, Wd = _weights(E, H, I)
    Wd[0, 3, 10] = float("nan")
    layer = moe.MoELayer(Wg, Wu, Wd, k, dtype=FP8)
    x, logits, _ = _inputs(2, H, E)
    logits[:] = 0
    logits[0, 0] = 5.0
    logits[1, 1] = 5.0
    out = layer.decode(x, logits)
    assert torch.isnan(out[0, 10]) and torch.isfinite(out[1]).all()
    assert int(torch.isnan(out[0]).sum()) == 1


def test_near_moe_forward():
    """The same layer through moe_forward (h in bf16): within that path's tolerance."""
    moe = lib()
    T, E, k, H, I = 16, 32, 4, 1024, 512
    layer = moe.MoELayer(*_weights(E, H, I), k)
    x, logits, _ = _inputs(T, H, E)
    a, b = layer(x, logits).double(), layer.decode(x, logits).double()
    assert float((a - b).abs().max() / b.abs().max()) < 2e-2


def test_zero_tokens():
    moe = lib()
    layer = moe.MoELayer(*_weights(8, 64, 64), 2)
    out = layer.decode(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV),
                       torch.empty((0, 8), device=DEV))
    assert out.shape == (0, 64) and layer.check() == 0


def test_uninitialised_workspace_is_reported():
    """A workspace that moe_decode_workspace_init never saw: an error status, no wait."""
    moe = lib()
    E, k, H, I = 8, 2, 64, 64
    layer = moe.MoELayer(*_weights(E, H, I), k)
    x, logits, _ = _inputs(2, H, E)
    n = moe.lib().moe_decode_workspace_size(BF16, 2, k, E, H, I)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((2, H), 3.0, dtype=torch.bfloat16, device=DEV)
    moe.decode_forward(BF16, x, logits, layer.packed, None, E, I, k, out=out, ws=ws,
                       status=status)
    assert moe.check_status(status) == 6          # MOE_ERR_DEVICE
    assert (out == 3).all()


def test_streams_and_graphs():
    """Calls on two streams at once, on a stream given by hand, and two captured graphs of
    one layer replayed in turn and beside eager calls."""
    moe = lib()
    E, k, H, I = 16, 2, 512, 768
    layer = moe.MoELayer(*_weights(E, H, I), k)
    ins = [_inputs(T, H, E, seed=T) for T in (1, 4, 16)]
    want = [layer.decode(x, lg, residual=r) for x, lg, r in ins]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for rep in range(20):
        for s in (s1, s2):
            for n, (x, lg, r) in enumerate(ins):
                got.append((n, layer.decode(x, lg, residual=r, stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[n]) for n, o in got)

    graphs, outs = [], []
    statics = [[t.clone() for t in i] for i in ins[:2]]
    side = torch.cuda.Stream()
    for st in statics:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            o1 = layer.decode(st[0], st[1], residual=st[2])
            o2 = layer.decode(o1, st[1], residual=st[2])
        graphs.append(gr)
        outs.append((o1, o2))
    for rep in range(3):
        for n in (1, 0):
            x, lg, r = _inputs(ins[n][0].shape[0], H, E, seed=50 + rep)
            for dst, src in zip(statics[n], (x, lg, r)):
                dst.copy_(src)
            graphs[n].replay()
            o1 = layer.decode(x, lg, residual=r)
            o2 = layer.decode(o1, lg, residual=r)
            assert torch.equal(outs[n][0], o1) and torch.equal(outs[n][1], o2)
    assert layer.check() == 0


@pytest.mark.parametrize("H,I,E,k,T,dtype", [(4096, 14336, 8, 2, 1, BF16),
                                             (7168, 2048, 16, 8, 6, BF16),
                                             (2880, 2880, 32, 4, 13, FP8)])
def test_full_size(H, I, E, k, T, dtype):
    """Full layer sizes: relative 2-norm error within what out's rounding alone gives."""
    moe = lib()
    Wg, Wu, Wd = _weights(E, H, I)
    layer = moe.MoELayer(Wg, Wu, Wd, k, dtype=dtype)
    x, logits, res = _inputs(T, H, E)
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    out = layer.decode(x, logits, residual=res, ids=ids, w=w)
    assert layer.check() == 0
    ref = res.double()
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        D = [_deq(W[e:e + 1], dtype)[0] for W in (Wg, Wu, Wd)]
        g, u = x[t].double() @ D[0], x[t].double() @ D[1]
        ref[t] += w[t, j].double()[:, None] * ((g / (1 + torch.exp(-g)) * u) @ D[2])
    err = (out.double() - ref).norm() / ref.norm()
    # half a step of bf16, uniform in it: at most 2^-8 / sqrt(3) = 0.00226
    assert float(err) < 2.0 ** -8 / 3 ** 0.5


def test_binding_refuses():
    moe = lib()
    E, k, H, I = 8, 2, 64, 64
    layer = moe.MoELayer(*_weights(E, H, I), k)
    x, logits, res = _inputs(3, H, E)
    for bad in (dict(x=x.float()), dict(logits=logits.double()), dict(logits=logits[:2]),
                dict(residual=res[:2]), dict(residual=res.float()),
                dict(x=torch.zeros((3, 2 * H), dtype=torch.bfloat16, device=DEV)[:, :H]),
                dict(out=torch.zeros((3, H), device=DEV)),
                dict(ids=torch.zeros((3, k), dtype=torch.int64, device=DEV)),
                dict(w=torch.zeros((3, k + 1), device=DEV)), dict(logits=logits.cpu())):
        with pytest.raises(ValueError):
            layer.decode(**{**dict(x=x, logits=logits), **bad})
    big = _inputs(17, H, E)
    with pytest.raises(moe.MoEError):                     # more than 16 tokens
        layer.decode(big[0], big[1])
    with pytest.raises(moe.MoEError):                     # a workspace for fewer tokens
        moe.decode_forward(BF16, *big[:2], layer.packed, None, E, I, k,
                           ws=moe.decode_workspace(BF16, 1, k, E, H, I, DEV))
    with pytest.raises(ValueError):                       # weights of a smaller layer
        moe.decode_forward(BF16, x, logits, layer.packed[:-16384], None, E, I, k)

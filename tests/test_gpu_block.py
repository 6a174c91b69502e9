"""The feed-forward part of a decoder block, as a user runs it: router product, top-k, routed
experts (the few-token form or the layer's call), a shared expert, the residual."""
import pytest
import torch

import oracle
from tests.gpu_helpers import lib, to_host

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def _block(moe, E, k, H, I, S, dtype=0, bias=True, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    W = dict(Wg=(r(E, H, I) / H ** 0.5).to(BF), Wu=(r(E, H, I) / H ** 0.5).to(BF),
             Wd=(r(E, I, H) / I ** 0.5).to(BF), Wr=(r(E, H) / H ** 0.5).to(BF),
             br=0.3 * r(E) if bias else None,
             gu=(r(2 * S, H) / H ** 0.5).to(BF) if S else None,
             dn=(r(H, S) / S ** 0.5).to(BF) if S else None)
    layer = moe.MoELayer(W["Wg"], W["Wu"], W["Wd"], k, dtype=dtype)
    return moe.MoEBlock(layer, W["Wr"], W["br"], W["gu"], W["dn"]), W


def _ffn(x, g, u, d):
    a = x @ g
    return (a / (1 + torch.exp(-a)) * (x @ u)) @ d


def _reference(W, k, x, logits, residual):
    """The block in float64 from the logits that its router gives (top-k near a tie is the
    router's rounding, not the experts')."""
    xd = x.double()
    ids, w = oracle.route_topk(to_host(logits), k)
    out = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
    for t in range(x.shape[0]):
        for j in range(k):
            e = int(ids[t, j])
            out[t] += float(w[t, j]) * _ffn(xd[t], *(W[n][e].double() for n in ("Wg", "Wu", "Wd")))
    if W["gu"] is not None:
        S = W["dn"].shape[1]
        gu = W["gu"].double()
        out += _ffn(xd, gu[:S].t(), gu[S:].t(), W["dn"].double().t())
    return out if residual is None else out + residual.double()


@pytest.mark.parametrize("S", [0, 320])
@pytest.mark.parametrize("T", [1, 6, 16, 17, 40])
def test_block_matches_definition(T, S):
    moe = lib()
    E, k, H, I = 40, 4, 512, 256
    block, W = _block(moe, E, k, H, I, S)
    assert block.layer.decodes(T) == (T <= 16)
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn((T, H), generator=g, device=DEV).to(BF)
    res = torch.randn((T, H), generator=g, device=DEV).to(BF)
    for residual in (res, None):
        before = None if residual is None else residual.clone()
        out = block(x, residual)
        logits = moe.linear(x, W["Wr"], bias=W["br"], out_dtype=torch.float32)
        want = x.double() @ W["Wr"].double().t() + W["br"].double()
        assert float((logits.double() - want).abs().max()) < 1e-4
        ref = _reference(W, k, x, logits, residual)
        # at most four roundings to bf16 on an element's way (the shared expert's h and sum, the
        # routed sum, out; the layer's own h and rows in its call), 2^-8 of the terms each
        err = (out.double() - ref).norm() / ref.norm()
        assert float(err) < 4 * 2.0 ** -8
        assert block.layer.check() == 0
        assert residual is None or torch.equal(residual, before)      # left as it was


def test_decode_steps_in_a_graph():
    """Three blocks of a decode step captured once and replayed on new inputs."""
    moe = lib()
    T, E, k, H, I, S = 3, 16, 2, 256, 192, 128
    blocks = [_block(moe, E, k, H, I, S, seed=s)[0] for s in range(3)]

    def step(x):
        for b in blocks:
            x = b(x, residual=x)
        return x

    x = torch.randn((T, H), device=DEV).to(BF)
    step(x)
    torch.cuda.synchronize()
    xs = x.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = step(xs)
    for seed in range(4):
        xs.copy_(torch.randn((T, H), generator=torch.Generator(device=DEV).manual_seed(seed),
                             device=DEV).to(BF))
        gr.replay()
        assert torch.equal(out, step(xs))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = blocks[0](xs, residual=xs, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, blocks[0](xs, residual=xs))


def test_block_e4m3():
    moe = lib()
    T, E, k, H, I, S = 5, 8, 2, 256, 192, 128
    block, W = _block(moe, E, k, H, I, S, dtype=1, bias=False)
    x = torch.randn((T, H), device=DEV).to(BF)
    out = block(x, residual=x)
    logits = moe.linear(x, W["Wr"], out_dtype=torch.float32)
    ref = _reference(W, k, x, logits, x)
    # e4m3 weights: off by at most 2^-4 of each, half that in the mean over the products
    assert float((out.double() - ref).norm() / ref.norm()) < 2.0 ** -4


def test_block_refuses_half_a_shared_expert():
    moe = lib()
    block, W = _block(moe, 8, 2, 128, 64, 64)
    with pytest.raises(ValueError):
        moe.MoEBlock(block.layer, W["Wr"], shared_gu=W["gu"])

"""Calls that the layer, the block and the few-token form refuse: arguments whose memory the
kernels would read as something else."""
import pytest
import torch

from tests.gpu_helpers import lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def _layer(moe, E=8, k=2, H=256, I=128, dtype=0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    return moe.MoELayer((r(E, H, I) / H ** 0.5).to(BF), (r(E, H, I) / H ** 0.5).to(BF),
                        (r(E, I, H) / I ** 0.5).to(BF), k, dtype=dtype)


def _inputs(T, H, E, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn((T, H), generator=g, device=DEV).to(BF),
            torch.randn((T, E), generator=g, device=DEV))


@pytest.mark.parametrize("T", [2, 16, 17, 40])
def test_rows_that_are_apart(T):
    """A slice of a fused projection as x: moe.linear takes it, the experts' kernels have no row
    stride, so the layer and the block refuse it (contiguous, it is the same as any other)."""
    moe = lib()
    layer = _layer(moe)
    w_router = (torch.randn((8, 256), device=DEV) / 16).to(BF)
    block = moe.MoEBlock(layer, w_router)
    wide = torch.randn((T, 3 * 256), device=DEV).to(BF)
    x = wide[:, 256:512]
    logits = moe.linear(x, w_router, out_dtype=torch.float32)
    for call in (lambda: block(x), lambda: layer(x, logits),
                 lambda: moe.forward(0, x, logits, layer.packed, None, 8, 128, 2)):
        with pytest.raises(ValueError, match="x: must be contiguous"):
            call()
    own = x.contiguous()
    assert torch.equal(moe.linear(own, w_router, out_dtype=torch.float32), logits)
    assert torch.equal(block(own), layer.decode(own, logits) if T <= 16 else layer(own, logits))


def test_arguments_of_the_layers_call():
    moe = lib()
    T, E, k, H = 20, 8, 2, 256
    layer = _layer(moe)
    x, logits = _inputs(T, H, E)
    want = layer(x, logits)
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    args = dict(dtype=0, x=x, logits=logits, packed=layer.packed, scales=None, E=E, I=128, k=k)
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(x=x[0]), dict(logits=logits.to(BF)),
                dict(logits=logits.t().contiguous().t()), dict(logits=logits[:T - 1]),
                dict(logits=logits[:, :4].contiguous()), dict(logits=logits.cpu()),
                dict(out=torch.empty((T, H), device=DEV)), dict(out=torch.empty_like(x)[:T - 1]),
                dict(out=torch.empty((T, 2 * H), dtype=BF, device=DEV)[:, :H]),
                dict(ids=ids.long()), dict(ids=ids[:T - 1]), dict(w=w.double()),
                dict(w=torch.empty((T, k + 1), device=DEV))):
        with pytest.raises(ValueError):
            moe.forward(**{**args, **bad})
    out = torch.empty_like(x)
    assert moe.forward(**args, out=out, ids=ids, w=w) is out and torch.equal(out, want)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T", [4, 20])
def test_x_of_another_width(T, dtype):
    """x narrower or wider than the layer's H (H = 192 and 256 have e4m3 tiles of one size)."""
    moe = lib()
    layer = _layer(moe, H=256, dtype=dtype)
    for H in (64, 128, 192, 320, 512):
        x, logits = _inputs(T, H, 8)
        with pytest.raises(ValueError, match="H = 256"):
            layer(x, logits)
        with pytest.raises(ValueError, match="H = 256"):
            layer.decode(x, logits)
    for x in (x[0], x[:, :, None]):
        with pytest.raises(ValueError):
            layer(x, logits)
        with pytest.raises(ValueError):
            layer.decode(x, logits)


@pytest.mark.parametrize("T", [4, 40])
def test_residuals_that_a_block_refuses(T):
    """The same ones for every T: nothing is broadcast or converted."""
    moe = lib()
    layer = _layer(moe)
    block = moe.MoEBlock(layer, (torch.randn((8, 256), device=DEV) / 16).to(BF))
    x, _ = _inputs(T, 256, 8)
    for residual in (x[0].contiguous(), x[:1].contiguous(), x.float(), x[:T - 1], x.cpu(),
                     torch.zeros((T, 512), dtype=BF, device=DEV)[:, :256], x[:1].expand(T, 256)):
        with pytest.raises(ValueError, match="residual"):
            block(x, residual)
    before = x.clone()
    assert torch.equal(block(x, x), block(x, residual=before)) and torch.equal(x, before)


@pytest.mark.parametrize("T", [3, 20])
def test_buffers_of_another_type_or_layout(T):
    """Packed weights, workspace and status word: a broadcast buffer has fewer bytes than its
    numel says, a status word of another type fewer than the kernel writes."""
    moe = lib()
    layer = _layer(moe)
    x, logits = _inputs(T, 256, 8)
    if T <= 16:
        ws = moe.decode_workspace(0, T, 2, 8, 256, 128, DEV)

        def call(packed=layer.packed, ws=ws, status=layer.status):
            return moe.decode_forward(0, x, logits, packed, None, 8, 128, 2, ws=ws, status=status)
    else:
        ws = layer.workspace(T)

        def call(packed=layer.packed, ws=ws, status=layer.status):
            return moe.forward(0, x, logits, packed, None, 8, 128, 2, ws=ws, status=status)
    want = call()
    one = torch.zeros(1, dtype=torch.uint8, device=DEV)
    for name, t in (("packed", layer.packed), ("ws", ws)):
        for bad in (one.expand(t.numel()), torch.zeros(2 * t.numel(), dtype=torch.uint8,
                                                       device=DEV)[::2],
                    torch.zeros(t.numel(), dtype=torch.float16, device=DEV), t.cpu()):
            with pytest.raises(ValueError, match=name):
                call(**{name: bad})
    for bad in (one, torch.zeros(1, dtype=torch.int64, device=DEV), layer.status.cpu(),
                torch.zeros(0, dtype=torch.int32, device=DEV)):
        with pytest.raises(ValueError, match="status"):
            call(status=bad)
    assert torch.equal(call(), want) and layer.check() == 0

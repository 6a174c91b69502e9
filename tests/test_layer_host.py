"""The layer's and the block's Python side without a GPU: which device, stream, workspace and
status word their calls use.  Tensors and streams are stand-ins; nothing is launched."""
import contextlib

import pytest
import torch


class OnDevice:
    """A CUDA tensor as far as the calls' device handling looks at it."""
    is_cuda = True

    def __init__(self, shape, index, dtype=torch.bfloat16):
        self.shape, self.index, self.dtype = shape, index, dtype
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 0x1000

    def is_contiguous(self):
        return True

    def numel(self):
        return 1 << 40


@pytest.fixture
def L(monkeypatch):
    from mixture_experts_expert_route_b200 import _lib, build
    build.build()
    _lib.lib()
    current = [0]

    @contextlib.contextmanager
    def on_device(dev, stream=None):
        before = current[0]
        current[0] = dev.index
        yield
        current[0] = before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0])
    monkeypatch.setattr(_lib, "_on_device", on_device)
    _lib.test_current = current
    yield _lib
    del _lib.test_current


def _layer(L, E=8, k=2, H=256, I=128, index=1):
    layer = object.__new__(L.MoELayer)
    layer.E, layer.H, layer.I, layer.k, layer.dtype = E, H, I, k, 0
    layer.block_m = layer.max_ctas = layer.combine = 0
    layer.packed, layer.scales = OnDevice((1,), index, torch.uint8), None
    layer.status, layer.device = OnDevice((1,), index, torch.int32), torch.device("cuda", index)
    layer._ws, layer._decode_need, layer._decode_ws = {}, {}, {}
    return layer


@pytest.mark.parametrize("T", [4, 40])
def test_every_step_of_a_block_runs_on_the_tensors_device(L, monkeypatch, T):
    """The current device is 0, the tensors are on 1: so are products, experts and the sum."""
    layer = _layer(L)
    seen = []
    result = OnDevice((T, 256), 1)
    result.add_ = lambda r: seen.append(("add", L.test_current[0])) or result

    def record(name):
        def call(*a, **kw):
            seen.append((name, L.test_current[0]))
            return result
        return call

    monkeypatch.setattr(L, "linear", record("linear"))
    monkeypatch.setattr(L, "forward", record("forward"))
    monkeypatch.setattr(L, "decode_forward", record("decode"))
    monkeypatch.setattr(L.MoELayer, "workspace", record("workspace"))
    monkeypatch.setattr(L.MoELayer, "decode_workspace", record("workspace"))
    monkeypatch.setattr(L.MoELayer, "decodes", lambda self, T: T <= 16)
    block = L.MoEBlock(layer, OnDevice((8, 256), 1), None, OnDevice((64, 256), 1),
                       OnDevice((256, 32), 1))
    block(OnDevice((T, 256), 1), OnDevice((T, 256), 1))
    assert {n for n, _ in seen} >= {"linear", "workspace", "decode" if T <= 16 else "forward"}
    assert all(dev == 1 for _, dev in seen), seen
    assert L.test_current[0] == 0


def test_forward_runs_on_the_tensors_device(L, monkeypatch):
    seen = []

    class Lib:
        def __getattr__(self, name):
            def call(*a):
                seen.append((name, L.test_current[0]))
                return 0 if name == "moe_forward" else 64
            return call

    monkeypatch.setattr(L, "lib", lambda: Lib())
    monkeypatch.setattr(L, "_stream", lambda stream=None: 0)
    x, logits = OnDevice((20, 256), 1), OnDevice((20, 8), 1, torch.float32)
    packed, ws, out = (OnDevice((1,), 1, torch.uint8), OnDevice((1,), 1, torch.uint8),
                       OnDevice((20, 256), 1))
    assert L.forward(0, x, logits, packed, None, 8, 128, 2, out=out, ws=ws) is out
    assert ("moe_forward", 1) in seen and all(dev == 1 for _, dev in seen)
    # weights, scales, status and workspace of another device are refused
    for bad in (dict(packed=OnDevice((1,), 0, torch.uint8)), dict(scales=OnDevice((8, 3), 0, torch.float32)),
                dict(status=OnDevice((1,), 0, torch.int32)), dict(ws=OnDevice((1,), 0, torch.uint8)),
                dict(logits=OnDevice((20, 8), 0, torch.float32)), dict(out=OnDevice((20, 256), 0))):
        with pytest.raises(ValueError, match="cuda:1"):
            L.forward(**{**dict(dtype=0, x=x, logits=logits, packed=packed, scales=None, E=8,
                                I=128, k=2, out=out, ws=ws), **bad})


def test_check_waits_on_the_layers_device(L, monkeypatch):
    seen = []
    monkeypatch.setattr(L, "check_status", lambda t: seen.append(L.test_current[0]) or 0)
    assert _layer(L).check() == 0 and seen == [1]


def test_workspaces_of_streams_and_captures(L, monkeypatch):
    """Calls that may run at the same time do not share a workspace: another stream has its own,
    and a captured call has one that nothing else is given."""
    layer, state = _layer(L), dict(stream=7, capturing=False)
    monkeypatch.setattr(L, "forward_workspace_size", lambda *a: 100)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: bytearray(n))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda idx: state["stream"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    first = layer.workspace(40)
    assert layer.workspace(40) is first and layer.workspace(41) is not first
    state["stream"] = 8
    second = layer.workspace(40)
    assert second is not first and layer.workspace(40) is second
    state["capturing"] = True
    captured = [layer.workspace(40), layer.workspace(40)]
    assert captured[0] is not captured[1] and all(c is not second for c in captured)
    state.update(stream=7, capturing=False)
    assert layer.workspace(40) is first


@pytest.mark.parametrize("T", [4, 40])
def test_a_blocks_products_report_to_the_layer(L, monkeypatch, T):
    """A wait that runs out in any of the block's products is seen by layer.check()."""
    layer, seen = _layer(L), []
    result = OnDevice((T, 256), 1)

    def linear(*a, status=None, **kw):
        seen.append(status)
        return result

    monkeypatch.setattr(L, "linear", linear)
    monkeypatch.setattr(L.MoELayer, "__call__", lambda *a, **kw: result)
    monkeypatch.setattr(L.MoELayer, "decode", lambda *a, **kw: result)
    monkeypatch.setattr(L.MoELayer, "decodes", lambda self, T: T <= 16)
    L.MoEBlock(layer, OnDevice((8, 256), 1), None, OnDevice((64, 256), 1),
               OnDevice((256, 32), 1))(OnDevice((T, 256), 1))
    assert len(seen) == 3 and all(s is layer.status for s in seen)


def test_linear_passes_its_status_word_on(L, monkeypatch):
    """The compiled call gets it (a call with a status word is not a slower one)."""
    seen = []
    monkeypatch.setattr(L._calls, "linear", lambda *a: seen.append(a) or "out")
    status = OnDevice((1,), 0, torch.int32)
    assert L.linear(OnDevice((4, 64), 0), OnDevice((8, 64), 0), status=status) == "out"
    assert seen[0][-1] is status


@pytest.mark.parametrize("form", ["__call__", "decode"])
def test_x_of_another_width_is_refused(L, monkeypatch, form):
    """Before anything is launched, for every T and type (e4m3 tiles of H = 192 and 256 have the
    same size, so the size of the packed weights does not tell them apart)."""
    for name in ("forward", "decode_forward", "decode_workspace"):
        monkeypatch.setattr(L, name, lambda *a, **kw: pytest.fail("launched"))
    layer = _layer(L, H=256, index=0)
    for dtype in (0, 1):
        layer.dtype = dtype
        for shape in ((4, 192), (20, 128), (4, 320), (256,), (4, 256, 1)):
            with pytest.raises(ValueError):
                getattr(layer, form)(OnDevice(shape, 0), OnDevice((shape[0], 8), 0))


@pytest.mark.parametrize("T", [4, 40])
def test_a_blocks_residual_is_checked_before_anything_runs(L, monkeypatch, T):
    monkeypatch.setattr(L, "linear", lambda *a, **kw: pytest.fail("launched"))
    block = L.MoEBlock(_layer(L, index=0), OnDevice((8, 256), 0))
    x = OnDevice((T, 256), 0)
    for bad in (OnDevice((256,), 0), OnDevice((1, 256), 0), OnDevice((T, 256), 0, torch.float32),
                OnDevice((T, 256), 1)):
        with pytest.raises(ValueError, match="residual"):
            block(x, bad)


def test_buffers_are_checked_as_bytes(L):
    """(on host tensors, whose device index is -1)"""
    flat = torch.zeros(64, dtype=torch.uint8)
    assert L._bytes(flat, "ws", -1) == flat.data_ptr()
    for bad in (flat[:1].expand(64), flat[::2], flat.view(torch.float16)):
        with pytest.raises(ValueError, match="ws: expected contiguous uint8"):
            L._bytes(bad, "ws", -1)
    with pytest.raises(ValueError, match="ws: on cpu"):
        L._bytes(flat, "ws", 0)
    word = torch.zeros(1, dtype=torch.int32)
    assert L._word(word, -1) == word.data_ptr() and L._word(None, -1) is None
    for bad in (flat, word.long(), word[:0]):
        with pytest.raises(ValueError, match="status"):
            L._word(bad, -1)
    with pytest.raises(ValueError, match="status"):
        L._word(word, 0)


def test_a_device_without_an_index_is_the_current_one(monkeypatch):
    """device="cuda" and a stream of the current device; a stream of another one is refused."""
    from types import SimpleNamespace

    from mixture_experts_expert_route_b200 import _lib
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: ("stream", s))
    monkeypatch.setattr(torch.cuda, "device", lambda d: ("device", d))
    here, there = (SimpleNamespace(device=torch.device("cuda", i)) for i in (1, 0))
    assert _lib._on_device(torch.device("cuda"), here) == ("stream", here)
    assert isinstance(_lib._on_device(torch.device("cuda")), contextlib.nullcontext)
    assert _lib._on_device(torch.device("cuda", 0)) == ("device", torch.device("cuda", 0))
    with pytest.raises(ValueError, match="another device"):
        _lib._on_device(torch.device("cuda"), there)


def test_decode_workspaces_are_shared_and_released(L, monkeypatch):
    """One per stream for all layers, grown for the largest call; gone with the last layer."""
    class Workspace:
        def __init__(self, n):
            self.n = n

        def numel(self):
            return self.n

    class Lib:
        moe_decode_workspace_size = staticmethod(lambda dtype, T, k, E, H, I: 1000 * T)

    monkeypatch.setattr(L, "lib", lambda: Lib)
    monkeypatch.setattr(L, "decode_workspace",
                        lambda dtype, T, k, E, H, I, dev, stream=None: Workspace(1000 * T))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda idx: 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    a, b, key = _layer(L, index=93), _layer(L, index=93), (93, 7)
    small = a.decode_workspace(2)
    assert b.decode_workspace(1) is small and L._DECODE_WS[key] is small
    large = b.decode_workspace(5)
    assert large is not small and a.decode_workspace(2) is large
    del small, large, a
    assert key in L._DECODE_WS
    del b
    assert key not in L._DECODE_WS


def test_a_block_refuses_host_tensors(monkeypatch):
    """(and does not look for their device for ever)"""
    from mixture_experts_expert_route_b200 import _lib
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    block = _lib.MoEBlock(None, None)
    with pytest.raises(ValueError, match="CUDA tensor"):
        block(torch.zeros((4, 64), dtype=torch.bfloat16))


def test_linear_status_reads_the_word_of_the_streams_device(L, monkeypatch):
    from types import SimpleNamespace
    seen = []

    @contextlib.contextmanager
    def stream_context(s):
        before = L.test_current[0]
        if s is not None:
            L.test_current[0] = s.device.index
        yield
        L.test_current[0] = before

    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(L, "_stream", lambda s: 0 if s is None else s.cuda_stream)
    monkeypatch.setattr(L, "lib", lambda: SimpleNamespace(
        moe_linear_status=lambda s: seen.append((s, L.test_current[0])) or 0))
    assert L.linear_status() == 0
    assert L.linear_status(SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=7)) == 0
    assert seen == [(0, 0), (7, 1)]

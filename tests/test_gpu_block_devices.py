"""The block and the layer on a device that is not the current one.  Skipped where fewer than
two GPUs are visible."""
import pytest
import torch

from tests.gpu_helpers import lib

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.skipif(not torch.cuda.is_available() or torch.cuda.device_count() < 2,
                    reason="needs two visible GPUs")
@pytest.mark.parametrize("T", [3, 40])
def test_block_on_the_second_device(T):
    moe = lib()
    E, k, H, I, S = 8, 2, 256, 128, 64
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    host = [(r(E, H, I) / 16).to(BF), (r(E, H, I) / 16).to(BF), (r(E, I, H) / 11).to(BF),
            (r(E, H) / 16).to(BF), (r(2 * S, H) / 16).to(BF), (r(H, S) / 8).to(BF),
            r(T, H).to(BF)]
    outs = []
    for dev in ("cuda:0", "cuda:1"):
        with torch.cuda.device(dev):
            t = [a.to(dev) for a in host]
            layer = moe.MoELayer(*t[:3], k)
        block = moe.MoEBlock(layer, t[3], None, t[4], t[5])
        out = block(t[6], residual=t[6])          # the current device is 0
        torch.cuda.synchronize(dev)
        assert out.device == torch.device(dev) and layer.check() == 0
        outs.append(out.cpu())
    assert torch.equal(outs[0], outs[1])

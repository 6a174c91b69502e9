"""MoELayer's call and MoEBlock beyond a few tokens: at the same time on several streams, and
captured into graphs that are replayed beside one another and beside eager calls."""
import pytest
import torch

from tests.gpu_helpers import lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def _block(moe, E=16, k=2, H=512, I=384, S=128, dtype=0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    layer = moe.MoELayer((r(E, H, I) / H ** 0.5).to(BF), (r(E, H, I) / H ** 0.5).to(BF),
                         (r(E, I, H) / I ** 0.5).to(BF), k, dtype=dtype)
    return moe.MoEBlock(layer, (r(E, H) / H ** 0.5).to(BF), None,
                        (r(2 * S, H) / H ** 0.5).to(BF), (r(H, S) / S ** 0.5).to(BF))


def _x(T, seed, H=512):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((T, H), generator=g, device=DEV).to(BF)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T", [40, 600])
def test_block_on_two_streams_at_once(T, dtype):
    moe = lib()
    block = _block(moe, dtype=dtype)
    xs = [_x(T, s) for s in range(4)]
    want = [block(x, residual=x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for rep in range(20):
        for n, x in enumerate(xs):
            got.append((n, block(x, residual=x, stream=streams[n % 2])))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[n]) for n, y in got)
    assert block.layer.check() == 0


@pytest.mark.parametrize("T", [40, 600])
def test_graphs_beside_one_another_and_beside_eager_calls(T):
    moe = lib()
    block = _block(moe)
    statics = [_x(T, s) for s in range(2)]
    block(statics[0], residual=statics[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in statics:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(block(x, residual=x))
        graphs.append(gr)
    eager_x = _x(T, 9)
    eager_want = block(eager_x, residual=eager_x)
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(10):
        for n, x in enumerate(statics):
            x.copy_(_x(T, 100 + 2 * rep + n))
        want = [block(x, residual=x) for x in statics]
        torch.cuda.synchronize()
        for n in range(2):
            with torch.cuda.stream(streams[n]):
                graphs[n].replay()
        eager = [block(eager_x, residual=eager_x, stream=streams[2]) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(outs[n], want[n]) for n in range(2))
        assert all(torch.equal(e, eager_want) for e in eager)
    assert block.layer.check() == 0


def test_a_decode_workspace_made_on_a_stream():
    """With the device named without its index too."""
    moe = lib()
    block = _block(moe)
    layer, x = block.layer, _x(4, 0)
    logits = moe.linear(x, block.w_router, out_dtype=torch.float32)
    want = layer.decode(x, logits)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for device in ("cuda", "cuda:0", torch.device("cuda", 0)):
        ws = moe.decode_workspace(0, 4, 2, 16, 512, 384, device, stream=side)
        got = moe.decode_forward(0, x, logits, layer.packed, None, 16, 384, 2, ws=ws, stream=side)
        side.synchronize()
        assert torch.equal(got, want)


def test_few_tokens_beside_a_busy_stream():
    """The few-token form, whose blocks wait on one another, on one stream while another is full
    of products and layer calls that start early (and each other's): no wait runs out."""
    moe = lib()
    few, many = _block(moe, seed=1), _block(moe, seed=2)
    xs, xl = [_x(T, T) for T in (1, 5, 16)], _x(900, 3)
    want = [few(x, residual=x) for x in xs]
    want_l = many(xl, residual=xl)
    torch.cuda.synchronize()
    s1, s2, s3 = (torch.cuda.Stream() for _ in range(3))
    got, got_l = [], []
    for rep in range(30):
        got_l += [many(xl, residual=xl, stream=s2) for _ in range(3)]
        got += [(n, few(x, residual=x, stream=s)) for n, x in enumerate(xs) for s in (s1, s3)]
    torch.cuda.synchronize()
    assert few.layer.check() == 0 and many.layer.check() == 0
    assert all(torch.equal(y, want[n]) for n, y in got)
    assert all(torch.equal(y, want_l) for y in got_l)

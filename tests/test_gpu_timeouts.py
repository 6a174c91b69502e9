"""Waits that run out in the few-token layer and in the dense products: the copies that they wait for are withheld
(moe_selftest_withhold, in a child process with the debug build) and the limit is 2 ms.  The call
ends, MOE_ERR_TIMEOUT is in the status word, and the next call is right.  Nothing faults or hangs:
every wait is bounded, and no copy or product is under way when a block leaves."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PRELUDE = r'''
import sys, torch
sys.path.insert(0, ROOT)
from tests.gpu_helpers import lib
moe = lib()
assert moe._lib.DEBUG_CHECKS and moe.LIB_PATH.endswith("libmoe_b200_debug.so")
DEV, BF = "cuda:0", torch.bfloat16
gen = torch.Generator(device=DEV).manual_seed(0)
def r(*s): return torch.randn(s, generator=gen, device=DEV)
'''

DECODE = PRELUDE + r'''
for dtype in (0, 1):
    # about 20 (e4m3: 10) gate/up and 10 (5) down tiles a block, in rings of 8 or 12
    E, k, H, I = 8, 2, 1024, 2048
    layer = moe.MoELayer((r(E, H, I) / 32).to(BF), (r(E, H, I) / 32).to(BF),
                         (r(E, I, H) / 45).to(BF), k, dtype=dtype)
    for T in (4, 16):
        x, logits = r(T, H).to(BF), r(T, E)
        if T == 16:
            logits[:, 3] += 50.0          # an expert with more than 8 tokens
        args = (dtype, x, logits, layer.packed, layer.scales, E, I, k)
        def ws(): return moe.decode_workspace(dtype, T, k, E, H, I, DEV)
        want = moe.decode_forward(*args, ws=ws(), status=layer.status)
        assert layer.check() == 0
        for copies in (0, 1, 7, 13, 17, 22, 26):
            for block in (0, 77):
                moe.selftest_withhold(copies, block)
                out = moe.decode_forward(*args, ws=ws(), status=layer.status)
                code = layer.check()
                moe.selftest_withhold(-1)
                # (a block with fewer tiles has none withheld)
                assert code == 5 or (code == 0 and copies > 10 and torch.equal(out, want)), \
                    (dtype, T, copies, block, code)
                seen = code == 5 if copies == 0 else seen
                layer.status.zero_()
                assert torch.equal(moe.decode_forward(*args, ws=ws(), status=layer.status), want)
                assert layer.check() == 0
        assert seen
print("timeouts ok")
'''

LINEAR = PRELUDE + r'''
SHAPES = [  # M, K, N, gated, ranks of a cluster
    (512, 512, 4096, False, 1),       # 128-wide tiles, one block each
    (77, 2880, 2880, False, 4),       # 64-wide tiles, four blocks
    (4864, 1024, 1024, False, 2),     # CTA pairs, several tiles each
    (2500, 2112, 2041, False, 2),     # ... with rows that are not aligned
    (5000, 512, 1000, True, 2),
    (512, 4160, 2048, True, 4),       # two pairs to a tile
]
for M, K, N, gated, ranks in SHAPES:
    x, w = r(M, K).to(BF), (r(2 * N if gated else N, K) / K ** 0.5).to(BF)
    def call(**kw):
        return moe.linear(x, w, act=moe.ACT_SILU, gated=gated, **kw)
    want = call()
    assert moe.linear_status() == 0
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for copies in (0, 1, 5, 6, 9, 20, 33):
        for rank in range(ranks):
            moe.selftest_withhold(copies, rank)
            own = copies % 2 == 0         # a status word, or the device's
            out = call(status=status if own else None)
            code = moe.check_status(status) if own else moe.linear_status()
            moe.selftest_withhold(-1)
            assert code == 5 or (code == 0 and copies > 4 and torch.equal(out, want)), \
                (M, K, N, copies, rank, code)
            assert code == 5 or copies > 0
            status.zero_()
            assert torch.equal(call(status=status), want) and moe.check_status(status) == 0
            assert moe.linear_status() == 0
# a block tells of its products
E, k, H, I = 8, 2, 256, 128
layer = moe.MoELayer((r(E, H, I) / 16).to(BF), (r(E, H, I) / 16).to(BF), (r(E, I, H) / 11).to(BF), k)
block = moe.MoEBlock(layer, (r(E, H) / 16).to(BF))
x = r(40, H).to(BF)
want = block(x)
assert layer.check() == 0
moe.selftest_withhold(0)
block(x)
assert layer.check() == 5
moe.selftest_withhold(-1)
layer.status.zero_()
assert torch.equal(block(x), want) and layer.check() == 0
print("timeouts ok")
'''


def _child(code):
    env = dict(os.environ, MOE_B200_DEBUG_CHECKS="1")
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n" + code], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "timeouts ok" in r.stdout


def test_decode_waits_run_out():
    _child(DECODE)


def test_linear_waits_run_out():
    _child(LINEAR)


def test_the_release_build_withholds_nothing():
    from tests.gpu_helpers import lib
    moe = lib()
    if moe._lib.DEBUG_CHECKS:
        pytest.skip("the debug build")
    with pytest.raises(moe.MoEError, match="MOE_ERR_UNSUPPORTED"):
        moe.selftest_withhold(0)

"""Host-side checks of the C ABI that need no GPU: the library loads, exports
every entry point include/*.h declares, and rejects bad arguments
synchronously (nothing is launched, so no device is touched)."""
import ctypes
import os
import re

import pytest
import torch

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    from mixture_experts_expert_route_b200 import _lib, build
    build.build(debug=_lib.DEBUG_CHECKS)
    import mixture_experts_expert_route_b200 as moe
    return moe


def declared_functions():
    src = ""
    inc = os.path.join(ROOT, "include")
    for name in sorted(os.listdir(inc)):
        if name.endswith(".h"):
            with open(os.path.join(inc, name)) as f:
                src += f.read()
    return sorted(set(re.findall(r"MOE_API [^;(]*?\b(moe_\w+)\s*\(", src)))


def test_exports_every_declared_symbol(L):
    names = declared_functions()
    assert len(names) >= 24
    lib = ctypes.CDLL(L.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    # the binding wires the same names
    from mixture_experts_expert_route_b200._lib import _SIGS
    assert sorted(_SIGS) == names


def test_status_strings(L):
    for code, name in L._lib.STATUS.items():
        assert L.status_string(code) == name
    assert L.status_string(99) == "MOE_ERR_UNKNOWN"
    assert "sm_100a" in L.version()


@pytest.mark.parametrize("T,k,E,bm", [(0, 2, 8, 16), (1, 2, 8, 16), (64, 2, 8, 16), (17, 8, 128, 64),
                                      (8192, 8, 256, 16), (4096, 8, 128, 128), (3, 3, 3, 1)])
def test_capacity_matches_oracle(L, T, k, E, bm):
    assert L.permute_capacity(T, k, E, bm) == oracle.permute_capacity(T, k, E, bm)


def test_workspace_sizes(L):
    lib = L.lib()
    assert lib.moe_align_permute_workspace_size(64, 2, 8) == 0       # single chunk
    assert lib.moe_align_permute_workspace_size(4096, 8, 128) == 64 * 128 * 4   # 512 per chunk
    assert lib.moe_align_permute_workspace_size(256, 8, 128) == 0                # one CTA up to 2048
    # 16 KB tiles of 128 rows x 128 bytes, padded per expert matrix
    assert lib.moe_packed_weights_size(0, 8, 4096, 14336) == 3 * 8 * 4096 * 14336 * 2
    tiles = 32 * ((2 * 2880 // 128) * 23 + 23 * 23)
    assert lib.moe_packed_weights_size(1, 32, 2880, 2880) == tiles * 16384
    a = lib.moe_forward_workspace_size(0, 64, 2, 8, 4096, 14336, 0)
    b = lib.moe_forward_workspace_size(0, 64, 2, 8, 4096, 14336, 16)
    assert a == b > 0
    assert lib.moe_forward_workspace_size(1, 64, 2, 8, 4096, 14336, 16) > 0
    # unsupported shapes report size 0
    assert lib.moe_forward_workspace_size(0, 64, 2, 8, 4000, 14336, 16) == 0
    assert lib.moe_grouped_ffn_workspace_size(0, 64, 2, 8, 4096, 14336, 8) == 0


def test_argument_errors_return_synchronously(L):
    lib = L.lib()
    INVALID, UNSUP, WS = 1, 2, 3
    fake = ctypes.c_void_p(0x1000)
    assert lib.moe_route_topk(fake, 4, 8, 9, fake, fake, None) == INVALID      # k > E
    assert lib.moe_route_topk(fake, 4, 8, 0, fake, fake, None) == INVALID      # k < 1
    assert lib.moe_route_topk(fake, -1, 8, 2, fake, fake, None) == INVALID
    assert lib.moe_route_topk(fake, 4, 300, 2, fake, fake, None) == UNSUP      # E > 256
    assert lib.moe_route_topk(None, 4, 8, 2, fake, fake, None) == INVALID
    assert lib.moe_route_topk(None, 0, 8, 2, None, None, None) == 0            # T = 0 no-op
    cap = lib.moe_permute_capacity(64, 2, 8, 16)
    assert lib.moe_align_permute(fake, 64, 2, 8, 16, fake, fake, fake, fake, fake, fake,
                                 cap - 1, None, 0, None) == WS
    assert lib.moe_align_permute(fake, 8192, 8, 256, 16, fake, fake, fake, fake, fake, fake,
                                 lib.moe_permute_capacity(8192, 8, 256, 16), None, 0, None) == WS
    assert lib.moe_pack_weights(0, 8, 4000, 512, fake, fake, fake, fake, None, None) == UNSUP
    assert lib.moe_pack_weights(1, 8, 256, 512, fake, fake, fake, fake, None, None) == INVALID
    assert lib.moe_pack_weights(0, 8, 256, 512, ctypes.c_void_p(0x1001), fake, fake, fake,
                                None, None) == INVALID                            # misaligned
    assert lib.moe_combine(fake, fake, 4, 2, 100, fake, None) == INVALID          # H % 8
    assert lib.moe_check_status(None, None) == INVALID
    assert lib.moe_selftest_wait_timeout(fake, 0, None) == INVALID
    assert lib.moe_selftest_wait_timeout(fake, 2000000, None) == INVALID


def _fwd(L, **kw):
    base = dict(dtype=0, T=4, k=2, E=8, H=256, I=512, block_m=16, x=0x1000, logits=0x1000,
                packed=0x1000, scales=None, out=0x1000, ids=None, w=None, status=None,
                max_ctas=0, events=None, n_events=0, combine=0, lora=None)
    base.update(kw)
    a = L._lib.ForwardArgs(*[base[f] for f, _ in L._lib.ForwardArgs._fields_])
    return a


def test_forward_argument_errors(L):
    lib = L.lib()
    INVALID, UNSUP, WS = 1, 2, 3
    ws = ctypes.c_void_p(0x1000)
    big = 1 << 40
    call = lambda a, n=big: lib.moe_forward(ctypes.byref(a), ws, n, None)
    assert call(_fwd(L, k=9)) == INVALID
    assert call(_fwd(L, H=200)) == INVALID or call(_fwd(L, H=200)) == UNSUP
    assert call(_fwd(L, H=320 - 32)) == UNSUP                 # not a multiple of 64
    assert call(_fwd(L, block_m=8)) == INVALID
    assert call(_fwd(L, block_m=24)) == UNSUP
    assert call(_fwd(L, dtype=7)) == INVALID
    assert call(_fwd(L, dtype=1)) == INVALID                  # FP8 needs scales
    assert call(_fwd(L, x=0x1004)) == INVALID                 # misaligned
    assert call(_fwd(L, logits=None)) == INVALID
    assert call(_fwd(L, max_ctas=-1)) == INVALID
    assert call(_fwd(L, events=0x1000, n_events=3)) == INVALID
    assert call(_fwd(L, combine=3)) == INVALID                # unknown combine mode
    assert call(_fwd(L, combine=-1)) == INVALID
    # adapters: bf16 only, n * r <= 64, pointers required
    la = L._lib.LoraArgs(4, 16, 0x1000, 0x1000, 0x1000)
    assert call(_fwd(L, lora=ctypes.pointer(la), dtype=1, scales=0x1000)) == UNSUP
    assert call(_fwd(L, lora=ctypes.pointer(L._lib.LoraArgs(5, 16, 0x1000, 0x1000, 0x1000)))) == UNSUP
    assert call(_fwd(L, lora=ctypes.pointer(L._lib.LoraArgs(0, 16, 0x1000, 0x1000, 0x1000)))) == INVALID
    assert call(_fwd(L, lora=ctypes.pointer(L._lib.LoraArgs(4, 16, None, 0x1000, 0x1000)))) == INVALID
    assert lib.moe_packed_lora_size(8, 256, 512, 4, 16) > 0
    assert lib.moe_packed_lora_size(8, 256, 512, 4, 17) == 0
    assert call(_fwd(L), 64) == WS                            # workspace too small
    assert call(_fwd(L, T=0, x=None, logits=None)) == 0       # T = 0 no-op
    assert lib.moe_forward(None, ws, big, None) == INVALID


def test_missing_library_fails_loudly(monkeypatch, tmp_path):
    """No silent fallback: without the built library the binding raises."""
    import mixture_experts_expert_route_b200._lib as binding
    monkeypatch.setattr(binding, "LIB_PATH", str(tmp_path / "absent.so"))
    monkeypatch.setattr(binding, "_lib", None)
    with pytest.raises(ImportError):
        binding.lib()
    # and a CUDA tensor argument is required: host tensors are refused, not copied
    with pytest.raises(ValueError):
        binding._ptr(torch.zeros(1))


def _decode_args(L, **kw):
    base = dict(dtype=0, T=4, k=2, E=8, H=256, I=512, x=0x1000, logits=0x1000, packed=0x1000,
                scales=None, residual=None, out=0x1000, ids=None, w=None, status=None)
    base.update(kw)
    return L._lib.DecodeArgs(*[base[f] for f, _ in L._lib.DecodeArgs._fields_])


def test_decode_argument_errors(L):
    lib = L.lib()
    INVALID, UNSUP, WS = 1, 2, 3
    ws, big = ctypes.c_void_p(0x1000), 1 << 40

    def call(ws=ws, n=big, **kw):
        return lib.moe_decode_forward(ctypes.byref(_decode_args(L, **kw)), ws, n, None)

    assert lib.moe_decode_forward(None, ws, big, None) == INVALID
    assert call(T=-1) == INVALID
    assert call(T=0, x=None, out=None, ws=None, n=0) == 0            # no-op
    assert call(T=17) == UNSUP
    assert call(T=16, k=9, E=16) == UNSUP                            # T * k > 128
    assert call(k=9) == INVALID
    assert call(E=300) == UNSUP
    assert call(H=100) == UNSUP
    assert call(I=32) == INVALID
    assert call(dtype=5) == INVALID
    assert call(dtype=1) == INVALID                                  # e4m3 without scales
    for name in ("x", "logits", "packed", "out"):
        assert call(**{name: None}) == INVALID
    for name in ("x", "packed", "out", "residual"):
        assert call(**{name: 0x1008}) == INVALID
    need = lib.moe_decode_workspace_size(0, 4, 2, 8, 256, 512)
    assert need > 0
    assert call(n=need - 1) == WS
    assert call(ws=None) == WS
    assert call(ws=ctypes.c_void_p(0x1008)) == WS
    assert lib.moe_decode_workspace_size(0, 17, 2, 8, 256, 512) == 0
    assert lib.moe_decode_workspace_size(0, 4, 2, 8, 200, 512) == 0
    assert lib.moe_decode_workspace_size(0, 16, 2, 8, 256, 512) > need
    assert lib.moe_decode_workspace_init(None, big, None) == WS
    assert lib.moe_decode_workspace_init(ws, 16, None) == WS


def test_decode_binding_refuses_host_tensors(L):
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        L.decode_forward(0, x, torch.zeros((2, 8)), x, None, 8, 64, 2)
    with pytest.raises(ValueError):
        L.decode_forward(0, x[0], torch.zeros((2, 8)), x, None, 8, 64, 2)


def _linear_args(L, **kw):
    base = dict(M=4, N=64, K=128, act=0, gated=0, x=0x1000, w=0x1000, ldx=128, ldw=128, bias=None,
                bias_type=0, residual=None, ldr=0, out=0x1000, ldo=64, out_type=0, status=None)
    base.update(kw)
    return L._lib.LinearArgs(*[base[f] for f, _ in L._lib.LinearArgs._fields_])


def test_linear_argument_errors(L):
    lib = L.lib()
    INVALID, UNSUP = 1, 2

    def call(**kw):
        return lib.moe_linear(ctypes.byref(_linear_args(L, **kw)), None)

    assert lib.moe_linear(None, None) == INVALID
    assert call(M=-1) == INVALID and call(N=0) == INVALID and call(K=0) == INVALID
    assert call(M=0, x=None, out=None) == 0                    # no-op
    assert call(act=-1) == INVALID and call(act=5) == INVALID
    assert call(bias_type=2) == INVALID and call(out_type=-1) == INVALID
    assert call(K=100) == UNSUP                                # K % 8
    assert call(M=(1 << 30) + 1) == UNSUP and call(N=(1 << 29) + 1) == UNSUP
    assert call(ldx=132) == UNSUP and call(ldw=130) == UNSUP
    assert call(ldx=120) == INVALID and call(ldw=64) == INVALID and call(ldo=63) == INVALID
    assert call(residual=0x1000, ldr=32) == INVALID
    for name in ("x", "w", "out"):
        assert call(**{name: None}) == INVALID
    assert call(x=0x1008) == INVALID and call(w=0x1002) == INVALID
    assert call(out=0x1001) == INVALID and call(out=0x1002, out_type=1) == INVALID
    assert call(residual=0x1001, ldr=64) == INVALID
    assert call(bias=0x1002, bias_type=1) == INVALID


def test_linear_binding_refuses(L):
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        L.linear(x, x)                                         # host tensors
    with pytest.raises(ValueError):
        L.linear(x[0], x)


def test_linear_packing_matches_the_structure(L):
    """The binding packs moe_linear_args as bytes: every field where the C struct has it."""
    vals = dict(M=1, N=2, K=3, act=4, gated=1, x=0x1000, w=0x2000, ldx=5, ldw=6, bias=0x3000,
                bias_type=7, residual=0x4000, ldr=8, out=0x5000, ldo=9, out_type=10, status=0x6000)
    s = L._lib.LinearArgs(*[vals[f] for f, _ in L._lib.LinearArgs._fields_])
    packed = L._lib._LINEAR_ARGS.pack(*[vals[f] for f, _ in L._lib.LinearArgs._fields_])
    assert len(packed) == ctypes.sizeof(s)
    back = L._lib.LinearArgs.from_buffer_copy(packed)
    for f, _ in L._lib.LinearArgs._fields_:
        assert getattr(back, f) == getattr(s, f), f

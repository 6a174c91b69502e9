"""ctypes binding of libmoe_b200.so (the C ABI of include/moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch provides device memory and the current stream.  There is no
CPU fallback: if the library is missing, importing this module's functions
raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
import warnings
import weakref

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# MOE_B200_DEBUG_CHECKS=1 selects the build whose kernels validate the
# permutation they are handed (see build.py --debug-checks)
DEBUG_CHECKS = os.environ.get("MOE_B200_DEBUG_CHECKS", "0") == "1"
LIB_PATH = os.path.join(_HERE, "libmoe_b200_debug.so" if DEBUG_CHECKS else "libmoe_b200.so")

BF16, FP8_E4M3 = 0, 1
COMBINE_AUTO, COMBINE_DETERMINISTIC, COMBINE_FUSED = 0, 1, 2
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3, 4
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
          3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT",
          6: "MOE_ERR_DEVICE"}

P = ctypes.c_void_p
I32 = ctypes.c_int
SZ = ctypes.c_size_t


class MoEError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}")


class FfnArgs(ctypes.Structure):
    _fields_ = [("dtype", I32), ("T", I32), ("k", I32), ("E", I32), ("H", I32), ("I", I32),
                ("block_m", I32), ("capacity", I32), ("x", P), ("w", P), ("counts", P),
                ("offsets", P), ("sorted_ids", P), ("packed", P), ("scales", P),
                ("y_perm", P), ("status", P), ("max_ctas", I32)]


class LoraArgs(ctypes.Structure):
    _fields_ = [("n_adapters", I32), ("rank", I32), ("adapter", P), ("packed", P),
                ("scale", P)]


class ForwardArgs(ctypes.Structure):
    _fields_ = [("dtype", I32), ("T", I32), ("k", I32), ("E", I32), ("H", I32), ("I", I32),
                ("block_m", I32), ("x", P), ("logits", P), ("packed", P), ("scales", P),
                ("out", P), ("ids", P), ("w", P), ("status", P), ("max_ctas", I32),
                ("events", P), ("n_events", I32), ("combine", I32),
                ("lora", ctypes.POINTER(LoraArgs))]


class DecodeArgs(ctypes.Structure):
    _fields_ = [("dtype", I32), ("T", I32), ("k", I32), ("E", I32), ("H", I32), ("I", I32),
                ("x", P), ("logits", P), ("packed", P), ("scales", P), ("residual", P),
                ("out", P), ("ids", P), ("w", P), ("status", P)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("M", I32), ("N", I32), ("K", I32), ("act", I32), ("gated", I32), ("x", P),
                ("w", P), ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64), ("bias", P),
                ("bias_type", I32), ("residual", P), ("ldr", ctypes.c_int64), ("out", P),
                ("ldo", ctypes.c_int64), ("out_type", I32), ("status", P)]


class SplitCosts(ctypes.Structure):
    _fields_ = [("cpu_us", ctypes.c_double), ("cpu_us_per_token", ctypes.c_double),
                ("xfer_us", ctypes.c_double), ("gpu_us", ctypes.c_double),
                ("gpu_us_per_token", ctypes.c_double)]


class HostFfnArgs(ctypes.Structure):
    _fields_ = [("H", I32), ("I", I32), ("n", I32), ("weights", P), ("x", P), ("w", P),
                ("h", P), ("y", P), ("threads", I32), ("flags", I32)]


class SplitArgs(ctypes.Structure):
    _fields_ = [("T", I32), ("k", I32), ("E", I32), ("H", I32), ("I", I32), ("block_m", I32),
                ("x", P), ("logits", P), ("out", P), ("resident", P), ("resident_packed", P),
                ("stage_packed", P), ("n_stage", I32), ("host_packed", P), ("host_weights", P),
                ("costs", ctypes.POINTER(SplitCosts)), ("policy", I32), ("where", P),
                ("status", P), ("copy_stream", P), ("copy_event", P), ("host_threads", I32)]


_SIGS = {
    "moe_status_string": ([I32], ctypes.c_char_p),
    "moe_version": ([], ctypes.c_char_p),
    "moe_route_topk": ([P, I32, I32, I32, P, P, P], I32),
    "moe_permute_capacity": ([I32, I32, I32, I32], I32),
    "moe_align_permute_workspace_size": ([I32, I32, I32], SZ),
    "moe_align_permute": ([P, I32, I32, I32, I32, P, P, P, P, P, P, I32, P, SZ, P], I32),
    "moe_align_permute_noalloc": ([P, I32, I32, I32, I32, P, P, P, P, P, P, I32, P], I32),
    "moe_packed_weights_size": ([I32, I32, I32, I32], SZ),
    "moe_pack_weights": ([I32, I32, I32, I32, P, P, P, P, P, P], I32),
    "moe_packed_lora_size": ([I32, I32, I32, I32, I32], SZ),
    "moe_pack_lora": ([I32, I32, I32, I32, I32, P, P, P, P, P, P, P, P], I32),
    "moe_grouped_ffn_workspace_size": ([I32, I32, I32, I32, I32, I32, I32], SZ),
    "moe_grouped_ffn": ([ctypes.POINTER(FfnArgs), P, SZ, P], I32),
    "moe_combine": ([P, P, I32, I32, I32, P, P], I32),
    "moe_forward_workspace_size": ([I32, I32, I32, I32, I32, I32, I32], SZ),
    "moe_forward": ([ctypes.POINTER(ForwardArgs), P, SZ, P], I32),
    "moe_decode_workspace_size": ([I32, I32, I32, I32, I32, I32], SZ),
    "moe_decode_workspace_init": ([P, SZ, P], I32),
    "moe_decode_forward": ([ctypes.POINTER(DecodeArgs), P, SZ, P], I32),
    "moe_linear": ([P, P], I32),
    "moe_linear_status": ([P], I32),
    "moe_check_status": ([P, P], I32),
    "moe_selftest_wait_timeout": ([P, I32, P], I32),
    "moe_selftest_withhold": ([I32, I32, I32], I32),
    # CPU/GPU split (include/moe_split.h)
    "moe_split_place": ([P, I32, I32, P], I32),
    "moe_split_plan": ([P, P, I32, ctypes.POINTER(SplitCosts), I32, P], I32),
    "moe_split_plan_balanced": ([P, P, I32, ctypes.POINTER(SplitCosts), I32, P], I32),
    "moe_host_packed_size": ([I32, I32], SZ),
    "moe_host_pack_weights": ([I32, I32, I32, P, P, P, P], I32),
    "moe_host_isa": ([], I32),
    "moe_host_expert_ffn": ([ctypes.POINTER(HostFfnArgs)], I32),
    "moe_split_calibrate": ([I32, I32, I32, P, P, P, P, SZ, I32, P, ctypes.POINTER(SplitCosts)],
                            I32),
    "moe_split_workspace_size": ([I32, I32, I32, I32, I32, I32, I32, I32], SZ),
    "moe_split_host_workspace_size": ([I32, I32, I32, I32], SZ),
    "moe_split_forward": ([ctypes.POINTER(SplitArgs), P, SZ, P, SZ, P], I32),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m mixture_experts_expert_route_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(code: int, where: str) -> None:
    if code != 0:
        raise MoEError(code, where)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def status_string(code: int) -> str:
    return lib().moe_status_string(code).decode()


def version() -> str:
    return lib().moe_version().decode()


def permute_capacity(T: int, k: int, E: int, block_m: int) -> int:
    return lib().moe_permute_capacity(T, k, E, block_m)


def route_topk(logits: torch.Tensor, k: int, ids=None, w=None, stream=None):
    T, E = logits.shape
    dev = logits.device
    ids = torch.empty((T, k), dtype=torch.int32, device=dev) if ids is None else ids
    w = torch.empty((T, k), dtype=torch.float32, device=dev) if w is None else w
    _check(lib().moe_route_topk(_ptr(logits), T, E, k, _ptr(ids), _ptr(w), _stream(stream)),
           "moe_route_topk")
    return ids, w


def align_permute(ids: torch.Tensor, E: int, block_m: int, capacity: int | None = None,
                  stream=None):
    T, k = ids.shape
    dev = ids.device
    cap = permute_capacity(T, k, E, block_m) if capacity is None else capacity
    out = dict(counts=torch.empty(E, dtype=torch.int32, device=dev),
               offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
               sorted_ids=torch.empty(max(cap, 1), dtype=torch.int32, device=dev),
               inv_perm=torch.empty(max(T * k, 1), dtype=torch.int32, device=dev),
               tiles=torch.empty(max(cap // block_m, 1), dtype=torch.int32, device=dev),
               num_tiles=torch.empty(1, dtype=torch.int32, device=dev))
    nws = lib().moe_align_permute_workspace_size(T, k, E)
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev)
    _check(lib().moe_align_permute(_ptr(ids), T, k, E, block_m, _ptr(out["counts"]),
                                   _ptr(out["offsets"]), _ptr(out["sorted_ids"]),
                                   _ptr(out["inv_perm"]), _ptr(out["tiles"]),
                                   _ptr(out["num_tiles"]), cap, _ptr(ws), nws, _stream(stream)),
           "moe_align_permute")
    out["capacity"] = cap
    out["block_m"] = block_m
    return out


def align_permute_noalloc(ids: torch.Tensor, E: int, block_m: int, capacity: int | None = None,
                          stream=None):
    """align_permute without a workspace (the library's built-in scratch)."""
    T, k = ids.shape
    dev = ids.device
    cap = permute_capacity(T, k, E, block_m) if capacity is None else capacity
    out = dict(counts=torch.empty(E, dtype=torch.int32, device=dev),
               offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
               sorted_ids=torch.empty(max(cap, 1), dtype=torch.int32, device=dev),
               inv_perm=torch.empty(max(T * k, 1), dtype=torch.int32, device=dev),
               tiles=torch.empty(max(cap // block_m, 1), dtype=torch.int32, device=dev),
               num_tiles=torch.empty(1, dtype=torch.int32, device=dev))
    _check(lib().moe_align_permute_noalloc(_ptr(ids), T, k, E, block_m, _ptr(out["counts"]),
                                           _ptr(out["offsets"]), _ptr(out["sorted_ids"]),
                                           _ptr(out["inv_perm"]), _ptr(out["tiles"]),
                                           _ptr(out["num_tiles"]), cap, _stream(stream)),
           "moe_align_permute_noalloc")
    out["capacity"] = cap
    out["block_m"] = block_m
    return out


def pack_weights(dtype: int, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, stream=None):
    """Packs bf16 master weights once.  Returns (packed uint8 tensor, scales or None)."""
    E, H, I = Wg.shape
    for W in (Wg, Wu, Wd):
        if W.dtype != torch.bfloat16 or not W.is_contiguous():
            raise ValueError("master weights must be contiguous bf16")
    n = lib().moe_packed_weights_size(dtype, E, H, I)
    packed = torch.empty(n, dtype=torch.uint8, device=Wg.device)
    scales = torch.empty((E, 3), dtype=torch.float32, device=Wg.device) \
        if dtype == FP8_E4M3 else None
    _check(lib().moe_pack_weights(dtype, E, H, I, _ptr(Wg), _ptr(Wu), _ptr(Wd), _ptr(packed),
                                  _ptr(scales), _stream(stream)), "moe_pack_weights")
    return packed, scales


class Lora:
    """Packed multi-LoRA adapters on the device (see moe_pack_lora)."""

    def __init__(self, Ag, Bg, Au, Bu, Ad, Bd, scale, stream=None):
        n, E, H, r = Ag.shape
        I = Bg.shape[3]
        for M in (Ag, Bg, Au, Bu, Ad, Bd):
            if M.dtype != torch.bfloat16 or not M.is_contiguous() or not M.is_cuda:
                raise ValueError("adapter matrices must be contiguous bf16 CUDA tensors")
        self.n_adapters, self.rank, self.E, self.H, self.I = n, r, E, H, I
        size = lib().moe_packed_lora_size(E, H, I, n, r)
        if size == 0:
            raise MoEError(2, "moe_packed_lora_size")
        self.packed = torch.empty(size, dtype=torch.uint8, device=Ag.device)
        _check(lib().moe_pack_lora(E, H, I, n, r, _ptr(Ag), _ptr(Bg), _ptr(Au), _ptr(Bu),
                                   _ptr(Ad), _ptr(Bd), _ptr(self.packed), _stream(stream)),
               "moe_pack_lora")
        self.scale = scale.to(device=Ag.device, dtype=torch.float32).contiguous()

    def args(self, adapter):
        """The C struct for tokens whose adapters are `adapter` (device int32 [T])."""
        if adapter.dtype != torch.int32 or not adapter.is_cuda:
            raise ValueError("adapter must be a CUDA int32 tensor")
        return LoraArgs(self.n_adapters, self.rank, _ptr(adapter), _ptr(self.packed),
                        _ptr(self.scale))


def grouped_ffn_workspace_size(dtype, T, k, E, H, I, block_m) -> int:
    return lib().moe_grouped_ffn_workspace_size(dtype, T, k, E, H, I, block_m)


def grouped_ffn(dtype: int, x: torch.Tensor, w: torch.Tensor, perm: dict, packed, scales,
                E: int, I: int, k: int, y_perm=None, status=None, ws=None, max_ctas: int = 0,
                stream=None):
    T, H = x.shape
    bm, cap = perm["block_m"], perm["capacity"]
    y_perm = torch.empty((max(cap, 1), H), dtype=torch.bfloat16, device=x.device) \
        if y_perm is None else y_perm
    n = grouped_ffn_workspace_size(dtype, T, k, E, H, I, bm)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=x.device) if ws is None else ws
    a = FfnArgs(dtype, T, k, E, H, I, bm, cap, _ptr(x), _ptr(w), _ptr(perm["counts"]),
                _ptr(perm["offsets"]), _ptr(perm["sorted_ids"]), _ptr(packed), _ptr(scales),
                _ptr(y_perm), _ptr(status), max_ctas)
    _check(lib().moe_grouped_ffn(ctypes.byref(a), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_grouped_ffn")
    return y_perm, ws


def combine(y_perm, inv_perm, T: int, k: int, H: int, out=None, stream=None):
    out = torch.empty((T, H), dtype=torch.bfloat16, device=y_perm.device) if out is None else out
    _check(lib().moe_combine(_ptr(y_perm), _ptr(inv_perm), T, k, H, _ptr(out), _stream(stream)),
           "moe_combine")
    return out


def _on_device(dev: torch.device, stream=None):
    """Makes the tensors' device the current one, and the given stream (if any) torch's
    current stream, so that buffers made inside belong to it."""
    if dev.type != "cuda":
        raise ValueError("expected a CUDA tensor")
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if stream is not None:
        if stream.device != dev:
            raise ValueError("the stream belongs to another device than the tensors")
        return torch.cuda.stream(stream)
    if dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _take(t, name, shape, dtype, idx):
    """Address of an optional contiguous argument tensor of a layer entry point, checked."""
    if t is None:
        return None
    if t.get_device() != idx:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{idx}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _bytes(t, name, idx):
    """Address of a buffer of bytes (packed weights, a workspace), whose numel is its size."""
    if t.get_device() != idx:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{idx}")
    if t.dtype is not torch.uint8 or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous uint8")
    return t.data_ptr()


def _word(t, idx):
    """Address of an optional status word."""
    if t is None:
        return None
    if t.get_device() != idx or t.dtype is not torch.int32 or t.numel() < 1:
        raise ValueError(f"status: expected int32 on cuda:{idx}")
    return t.data_ptr()


def forward_workspace_size(dtype, T, k, E, H, I, block_m=0) -> int:
    return lib().moe_forward_workspace_size(dtype, T, k, E, H, I, block_m)


def forward(dtype: int, x, logits, packed, scales, E: int, I: int, k: int, out=None, ids=None,
            w=None, status=None, ws=None, block_m: int = 0, max_ctas: int = 0, events=None,
            combine: int = COMBINE_AUTO, lora=None, adapter=None, stream=None):
    """The whole layer.  ``events`` (7 torch.cuda.Event, optional) are recorded after
    each stage: entry, route+permute, FP8 x quantisation, gate/up, h quant, down,
    combine.  ``combine``: COMBINE_AUTO, COMBINE_DETERMINISTIC or COMBINE_FUSED.
    ``lora`` (a Lora) with ``adapter`` (CUDA int32 [T], -1 = none) applies
    multi-LoRA adapters (bf16 layers).  x, logits, out, ids and w are contiguous.
    Runs on x's device, on ``stream`` or the device's current one."""
    idx = x.get_device()
    if idx < 0:
        raise ValueError("expected a CUDA tensor")
    if x.dim() != 2:
        raise ValueError("x: expected [T, H]")
    if stream is not None or idx != torch._C._cuda_getDevice():
        with _on_device(x.device, stream):
            return forward(dtype, x, logits, packed, scales, E, I, k, out, ids, w, status, ws,
                           block_m, max_ctas, events, combine, lora, adapter)
    if scales is not None and scales.get_device() != idx:
        raise ValueError(f"scales: on {scales.device}, expected cuda:{idx}")
    T, H = x.shape
    bf16, f32 = torch.bfloat16, torch.float32
    if out is None:
        out = x.new_empty((T, H), dtype=bf16)
        out_p = out.data_ptr()
    else:
        out_p = _take(out, "out", (T, H), bf16, idx)
    if ws is None:
        n = forward_workspace_size(dtype, T, k, E, H, I, block_m)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=x.device)
    ev_arr = None
    if events is not None:
        if len(events) != 7:
            raise ValueError("events must hold 7 torch.cuda.Event")
        for e in events:
            if e.cuda_event == 0:  # create lazily-initialised events
                e.record()
        ev_arr = (ctypes.c_void_p * 7)(*[e.cuda_event for e in events])
    largs = lora.args(adapter) if lora is not None else None
    a = ForwardArgs(dtype, T, k, E, H, I, block_m, _take(x, "x", (T, H), bf16, idx),
                    _take(logits, "logits", (T, E), f32, idx), _bytes(packed, "packed", idx),
                    _ptr(scales),
                    out_p, _take(ids, "ids", (T, k), torch.int32, idx),
                    _take(w, "w", (T, k), f32, idx), _word(status, idx), max_ctas,
                    ctypes.cast(ev_arr, ctypes.c_void_p) if ev_arr is not None else None,
                    7 if ev_arr is not None else 0, combine,
                    ctypes.pointer(largs) if largs is not None else None)
    _check(lib().moe_forward(ctypes.byref(a), _bytes(ws, "ws", idx), ws.numel(), _stream(stream)),
           "moe_forward")
    return out


DECODE_MAX_T, DECODE_MAX_ASSIGN = 16, 128     # tokens, T * k
# (device index, stream) -> the workspace of MoELayer.decode calls there, kept by the layers
# that use it
_DECODE_WS = weakref.WeakValueDictionary()


def decode_workspace(dtype: int, T: int, k: int, E: int, H: int, I: int, device,
                     stream=None) -> torch.Tensor:
    """A workspace of decode_forward, initialised on the stream."""
    n = lib().moe_decode_workspace_size(dtype, T, k, E, H, I)
    if n == 0:
        raise MoEError(2, "moe_decode_workspace_size")
    with _on_device(torch.device(device), stream):
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        _check(lib().moe_decode_workspace_init(ws.data_ptr(), n, _stream(stream)),
               "moe_decode_workspace_init")
    return ws


class _Calls:
    """The compiled calls of moe_linear and moe_decode_forward (csrc/binding.cpp), bound to the
    library by the first of them; without the extension every call goes through ctypes, and
    costs the host twice as much."""

    def __init__(self):
        self.linear = lambda *args: self._bind().linear(*args)
        self.decode = lambda *args: self._bind().decode(*args)

    def _bind(self):
        addresses = [ctypes.cast(getattr(lib(), name), ctypes.c_void_p).value for name in
                     ("moe_linear", "moe_decode_forward", "moe_packed_weights_size")]
        why = None
        try:
            from . import _binding as b
            if b.torch_version != torch.__version__.split("+")[0]:
                why = f"built for torch {b.torch_version}"
        except ModuleNotFoundError:         # (not built: build.py has said why)
            b = None
        except ImportError as e:            # of another torch or Python, say
            b, why = None, e
        if why is not None:
            warnings.warn(f"_binding.so is not used, calls go through ctypes: {why}")
        if b is not None and why is None:
            b.init(*addresses)
            self.linear, self.decode = b.linear, b.decode
        else:
            self.linear = self.decode = lambda *args: NotImplemented
        return self


_calls = _Calls()


def decode_forward(dtype: int, x, logits, packed, scales, E: int, I: int, k: int,
                   residual=None, out=None, ids=None, w=None, status=None, ws=None,
                   stream=None):
    """The whole layer for T <= 16 tokens (T * k <= 128) in one kernel:
    out = residual + sum_j w_j * FFN_{id_j}(x).  ``ws`` comes from decode_workspace
    and is reused from call to call (None: a new one for this call)."""
    if stream is None and ws is not None:
        y = _calls.decode(dtype, x, logits, packed, scales, E, I, k, residual, out, ids, w, status,
                          ws)
        if y is not NotImplemented:
            return y
    # another device or stream, no workspace, or an argument to refuse
    idx = x.get_device()
    if idx < 0:
        raise ValueError("expected a CUDA tensor")
    if x.dim() != 2:
        raise ValueError("x: expected [T, H]")
    if stream is not None or idx != torch._C._cuda_getDevice():
        with _on_device(x.device, stream):
            return decode_forward(dtype, x, logits, packed, scales, E, I, k, residual, out, ids,
                                  w, status, ws)
    T, H = x.shape
    bf16, f32 = torch.bfloat16, torch.float32
    packed_p = _bytes(packed, "packed", idx)
    if packed.numel() < lib().moe_packed_weights_size(dtype, E, H, I):
        raise ValueError("packed: smaller than these sizes need")
    if out is None:
        out = x.new_empty((T, H))
    if ws is None and T > 0:
        ws = decode_workspace(dtype, T, k, E, H, I, x.device)
    a = DecodeArgs(dtype, T, k, E, H, I, _take(x, "x", (T, H), bf16, idx),
                   _take(logits, "logits", (T, E), f32, idx), packed_p,
                   _take(scales, "scales", (E, 3), f32, idx),
                   _take(residual, "residual", (T, H), bf16, idx),
                   _take(out, "out", (T, H), bf16, idx), _take(ids, "ids", (T, k), torch.int32, idx),
                   _take(w, "w", (T, k), f32, idx), _word(status, idx))
    code = lib().moe_decode_forward(ctypes.byref(a),
                                    None if ws is None else _bytes(ws, "ws", idx),
                                    0 if ws is None else ws.numel(),
                                    torch._C._cuda_getCurrentRawStream(idx))
    if code:
        raise MoEError(code, "moe_decode_forward")
    return out


_FLOAT_TYPE = {torch.bfloat16: 0, torch.float32: 1}


# moe_linear_args as bytes: packing costs a third of filling a ctypes structure,
# and a product of a few tokens takes the GPU no longer than its call
_LINEAR_ARGS = struct.Struct("@iiiiiPPqqPiPqPqiP")


def _rows(t, name, rows, cols, dtype, idx):
    """Checks a matrix argument of linear (rows may be apart) and returns its row stride."""
    if t.get_device() != idx:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{idx}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(rows, cols)}")
    rs, cs = t.stride()
    if cs != 1 and cols > 1:
        raise ValueError(f"{name}: columns must be contiguous")
    # the stride of a single row is of no account
    return rs if rows > 1 else (cols + 7) // 8 * 8


def linear(x, w, bias=None, act: int = ACT_NONE, gated: bool = False, residual=None, out=None,
           out_dtype=None, status=None, stream=None):
    """act(x w^T + bias) + residual, or with ``gated`` act(z[:, :N]) * z[:, N:] + residual.

    x bf16 [M, K] and w bf16 [N, K] (gated: [2N, K], gate rows then up rows), rows any multiple
    of 8 elements apart; bias bf16 or f32 [rows of w]; residual and out of ``out_dtype`` (bf16,
    the default, or f32).  ``out`` may be the residual.  ``status`` (int32, on x's device) gets
    the code of a wait that runs out; without one linear_status tells."""
    if stream is None:
        y = _calls.linear(x, w, bias, act, gated, residual, out, out_dtype, status)
        if y is not NotImplemented:
            return y
    # another device or stream, or an argument to refuse
    idx = x.get_device()
    if idx < 0:
        raise ValueError("expected a CUDA tensor")
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w: expected [M, K] and [N, K]")
    if stream is not None or idx != torch._C._cuda_getDevice():
        with _on_device(x.device, stream):
            return linear(x, w, bias, act, gated, residual, out, out_dtype, status)
    bf16 = torch.bfloat16
    M, K = x.shape
    N = rows = w.shape[0]
    if gated:
        if rows % 2:
            raise ValueError("w: a gated product has an even number of rows")
        N = rows // 2
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else bf16
    out_type = _FLOAT_TYPE.get(out_dtype)
    if out_type is None:
        raise ValueError(f"out_dtype: {out_dtype}, expected bfloat16 or float32")
    ldx = _rows(x, "x", M, K, bf16, idx)
    ldw = _rows(w, "w", rows, K, bf16, idx)
    bias_type = bias_p = ldr = res_p = 0
    if bias is not None:
        bias_type = _FLOAT_TYPE.get(bias.dtype)
        if bias_type is None:
            raise ValueError(f"bias: {bias.dtype}, expected bfloat16 or float32")
        if bias.get_device() != idx or bias.shape != (rows,) or not bias.is_contiguous():
            raise ValueError(f"bias: expected [{rows}], contiguous, on cuda:{idx}")
        bias_p = bias.data_ptr()
    if residual is not None:
        ldr = _rows(residual, "residual", M, N, out_dtype, idx)
        res_p = residual.data_ptr()
    status_p = _word(status, idx) or 0
    if out is None:
        out, ldo = x.new_empty((M, N)) if out_type == 0 else x.new_empty((M, N), dtype=out_dtype), N
    else:
        ldo = _rows(out, "out", M, N, out_dtype, idx)
    a = _LINEAR_ARGS.pack(M, N, K, act, gated, x.data_ptr(), w.data_ptr(), ldx, ldw, bias_p,
                          bias_type, res_p, ldr, out.data_ptr(), ldo, out_type, status_p)
    code = lib().moe_linear(a, torch._C._cuda_getCurrentRawStream(idx))
    if code:
        raise MoEError(code, "moe_linear")
    return out


def linear_status(stream=None) -> int:
    """Synchronises the stream (None: the current one) and returns the code that linear calls
    without a status word recorded on the current device since this was last called: 0, or 5
    where a wait ran out.  With a stream of another device, that device's."""
    with torch.cuda.stream(stream):      # (None: nothing changes)
        return lib().moe_linear_status(_stream(stream))


def check_status(status: torch.Tensor, stream=None) -> int:
    return lib().moe_check_status(_ptr(status), _stream(stream))


def selftest_wait_timeout(status: torch.Tensor, timeout_us: int, stream=None) -> None:
    _check(lib().moe_selftest_wait_timeout(_ptr(status), timeout_us, _stream(stream)),
           "moe_selftest_wait_timeout")


def selftest_withhold(copies: int, rank: int = 0, limit_us: int = 2000) -> None:
    """Debug builds: decode and linear launches leave out copies, so that their waits run out
    (see moe.h); copies < 0 ends it."""
    _check(lib().moe_selftest_withhold(copies, rank, limit_us), "moe_selftest_withhold")


class MoELayer:
    """A fused MoE layer with packed weights and a reusable workspace.

    >>> layer = MoELayer(Wg, Wu, Wd, k=2, dtype=BF16)   # bf16 [E,H,I], [E,I,H] on cuda
    >>> out = layer(x, logits)                            # x bf16 [T,H], logits f32 [T,E]
    """

    def __init__(self, Wg, Wu, Wd, k: int, dtype: int = BF16, block_m: int = 0,
                 max_ctas: int = 0, combine: int = COMBINE_AUTO):
        self.E, self.H, self.I = Wg.shape
        self.k, self.dtype, self.block_m, self.max_ctas = k, dtype, block_m, max_ctas
        self.combine = combine
        self.packed, self.scales = pack_weights(dtype, Wg, Wu, Wd)
        self.device = Wg.device
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._ws = {}
        self._decode_need, self._decode_ws = {}, {}

    def workspace(self, T: int) -> torch.Tensor:
        """The workspace of a call with T tokens on the device's current stream: one per T and
        stream (calls on one stream follow one another, on different streams they may overlap).
        A call captured into a graph gets one of its own: the graph may be replayed on any
        stream, beside other calls."""
        capturing = torch.cuda.is_current_stream_capturing()
        key = (T, torch._C._cuda_getCurrentRawStream(self.device.index))
        ws = None if capturing else self._ws.get(key)
        if ws is None:
            n = forward_workspace_size(self.dtype, T, self.k, self.E, self.H, self.I,
                                       self.block_m)
            ws = torch.empty(max(n, 16), dtype=torch.uint8, device=self.device)
            if not capturing:
                self._ws[key] = ws
        return ws

    def _tokens(self, x) -> int:
        """The rows of x, whose width must be the layer's: the packed tiles of another H would be
        read as this one's."""
        T, H = x.shape
        if H != self.H:
            raise ValueError(f"x: {H} columns, the layer has H = {self.H}")
        return T

    def __call__(self, x, logits, out=None, events=None, stream=None):
        if stream is not None or self.device.index != torch._C._cuda_getDevice():
            with _on_device(self.device, stream):
                return self(x, logits, out, events)
        T = self._tokens(x)
        return forward(self.dtype, x, logits, self.packed, self.scales, self.E, self.I,
                       self.k, out=out, status=self.status, ws=self.workspace(T),
                       block_m=self.block_m, max_ctas=self.max_ctas, events=events,
                       combine=self.combine)

    def decode_workspace(self, T: int, stream=None) -> torch.Tensor:
        """The workspace of decode calls on a stream: one per device and stream, shared by all
        layers (calls on one stream follow one another, on different streams they may overlap)
        and released with the last of them.  A call captured into a graph gets one of its own,
        whose initialisation is captured with it: the graph may be replayed on any stream, and
        outlive the cache."""
        if torch.cuda.is_current_stream_capturing():
            return decode_workspace(self.dtype, T, self.k, self.E, self.H, self.I,
                                    self.device, stream)
        need = self._decode_need.get(T)
        if need is None:
            need = lib().moe_decode_workspace_size(self.dtype, T, self.k, self.E, self.H, self.I)
            self._decode_need[T] = need
        key = (self.device.index, _stream(stream) if stream is not None else
               torch._C._cuda_getCurrentRawStream(self.device.index))
        ws = _DECODE_WS.get(key)
        if ws is None or need == 0 or ws.numel() < need:
            ws = decode_workspace(self.dtype, T, self.k, self.E, self.H, self.I, self.device,
                                  stream)
            _DECODE_WS[key] = ws
        self._decode_ws[key] = ws
        return ws

    def decodes(self, T: int) -> bool:
        """Whether decode is the faster form for T tokens: within its limits, and at most 1 GiB
        of experts that the tokens may activate.  Measured on B200, us, decode / call on the same
        inputs: E = 128 H = 2048 I = 768 top-8, T = 1 27 / 40, T = 8 86 / 98, T = 16 130 / 142;
        e4m3 E = 32 H = I = 2880 top-4, T = 1 31 / 46, T = 8 102 / 111, T = 16 141 / 141; E = 64
        H = 7168 I = 2048 top-8, T = 1 119 / 125, T = 2 204 / 205, T = 4 367 / 348; E = 8 H = 4096
        I = 14336 top-2, T = 1 116 / 124, T = 4 286 / 275."""
        n = self.packed.numel() // self.E * min(T * self.k, self.E)
        return T <= DECODE_MAX_T and T * self.k <= DECODE_MAX_ASSIGN and n <= 1 << 30

    def decode(self, x, logits, residual=None, out=None, ids=None, w=None, stream=None):
        """The layer for a few tokens in one kernel (see decode_forward)."""
        if stream is not None or self.device.index != torch._C._cuda_getDevice():
            with _on_device(self.device, stream):
                return self.decode(x, logits, residual, out, ids, w)
        T = self._tokens(x)
        return decode_forward(self.dtype, x, logits, self.packed, self.scales, self.E, self.I,
                              self.k, residual, out, ids, w, self.status,
                              self.decode_workspace(T) if T > 0 else None)

    def check(self, stream=None) -> int:
        """The status word after the work on the stream (None: the device's current one)."""
        with _on_device(self.device, stream):
            code = check_status(self.status)
        if code == 5:       # a wait ran out: later decode calls get workspaces made anew
            for key in [key for key in list(_DECODE_WS) if key[0] == self.device.index]:
                _DECODE_WS.pop(key, None)
        return code


class MoEBlock:
    """The feed-forward part of a decoder block around a MoELayer:

        logits = x w_router^T (+ b_router)                       f32
        out = residual + layer(x, logits) + shared(x)            bf16
        shared(x) = (SiLU(x G^T) * (x U^T)) D^T

    w_router bf16 [E, H] with an optional bias [E]; shared_gu bf16 [2S, H] (G's rows, then
    U's) and shared_down bf16 [H, S], or neither.  A few tokens run through the layer's decode
    form (see MoELayer.decodes), more through its call; both take contiguous rows of x only.
    A fault in any part is in the layer's status word (layer.check()).  The two forms differ in
    precision (decode keeps h in 16 bits, the call in bf16's 8), most for e4m3 experts, whose
    activations only the call quantises; shared(x) and the routed sum are bf16 on their way."""

    def __init__(self, layer: MoELayer, w_router, b_router=None, shared_gu=None,
                 shared_down=None):
        if (shared_gu is None) != (shared_down is None):
            raise ValueError("a shared expert has both shared_gu and shared_down")
        self.layer, self.w_router, self.b_router = layer, w_router, b_router
        self.shared_gu, self.shared_down = shared_gu, shared_down

    def __call__(self, x, residual=None, stream=None):
        if stream is not None or x.get_device() != torch._C._cuda_getDevice():
            with _on_device(x.device, stream):
                return self(x, residual)
        _take(residual, "residual", x.shape, torch.bfloat16, x.get_device())
        st = self.layer.status       # of the products too: layer.check() tells of the whole block
        logits = linear(x, self.w_router, bias=self.b_router, out_dtype=torch.float32, status=st)
        few = self.layer.decodes(x.shape[0])
        out = residual if few else self.layer(x, logits)
        if self.shared_gu is not None:
            h = linear(x, self.shared_gu, act=ACT_SILU, gated=True, status=st)
            # (in place where the routed experts' sum is this call's own)
            out = linear(h, self.shared_down, residual=out, out=None if few else out,
                         status=st)
        if few:
            return self.layer.decode(x, logits, residual=out)
        return out if residual is None else out.add_(residual)


# ---- CPU/GPU expert split (include/moe_split.h) ----------------------------

SPLIT_IDLE, SPLIT_RESIDENT, SPLIT_STAGED, SPLIT_CPU = 0, 1, 2, 3
POLICY_DYNAMIC, POLICY_ALL_CPU, POLICY_ALL_STAGED, POLICY_BALANCED = 0, 1, 2, 3
HOST_ISA_PORTABLE, HOST_ISA_AVX512_BF16, HOST_ISA_AMX_BF16 = 0, 1, 2
HOST_PATHS = {"auto": 0, "portable": 1, "avx512_bf16": 2}   # moe_host_ffn_args.flags


def _hptr(t):
    """Address of a host (CPU) tensor or numpy array."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if t.is_cuda:
            raise ValueError("expected a host tensor")
        return t.data_ptr()
    return t.ctypes.data


def _i32(a):
    import numpy as np
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def split_place(hits, budget: int):
    """resident int32 [E]: 1 for the `budget` experts with the most hits."""
    import numpy as np
    h = np.ascontiguousarray(np.asarray(hits, dtype=np.int64))
    resident = np.zeros(len(h), np.int32)
    _check(lib().moe_split_place(_hptr(h), len(h), budget, _hptr(resident)), "moe_split_place")
    return resident


def split_costs(cpu_us=0.0, cpu_us_per_token=0.0, xfer_us=0.0, gpu_us=0.0,
                gpu_us_per_token=0.0) -> SplitCosts:
    return SplitCosts(cpu_us, cpu_us_per_token, xfer_us, gpu_us, gpu_us_per_token)


def split_plan(counts, resident, costs: SplitCosts, n_stage: int, balanced: bool = False):
    """where int32 [E] (SPLIT_IDLE / RESIDENT / STAGED / CPU) for one batch:
    the per-expert rule, or with ``balanced`` the host/link balanced plan."""
    import numpy as np
    c, r = _i32(counts), _i32(resident)
    where = np.zeros(len(c), np.int32)
    fn = lib().moe_split_plan_balanced if balanced else lib().moe_split_plan
    _check(fn(_hptr(c), _hptr(r), len(c), ctypes.byref(costs), n_stage, _hptr(where)),
           "moe_split_plan")
    return where


def host_isa() -> int:
    return lib().moe_host_isa()


def host_packed_size(H: int, I: int) -> int:
    return lib().moe_host_packed_size(H, I)


def host_pack_weights(Wg, Wu, Wd):
    """Host layout of bf16 master weights (CPU tensors) -> uint8 CPU tensor [E, bytes]."""
    E, H, I = Wg.shape
    for W in (Wg, Wu, Wd):
        if W.dtype != torch.bfloat16 or W.is_cuda or not W.is_contiguous():
            raise ValueError("host master weights must be contiguous bf16 CPU tensors")
    out = torch.empty((E, host_packed_size(H, I)), dtype=torch.uint8)
    _check(lib().moe_host_pack_weights(E, H, I, _hptr(Wg), _hptr(Wu), _hptr(Wd), _hptr(out)),
           "moe_host_pack_weights")
    return out


def host_expert_ffn(weights, x, w, threads: int = 0, path: str = "auto"):
    """One expert on the host: (h bf16 [n,I], y bf16 [n,H]).  weights: one row of
    host_pack_weights' output; x bf16 [n,H]; w f32 [n] (CPU tensors).  path:
    "auto" (the fastest this CPU has), "avx512_bf16" (no AMX) or "portable"."""
    n, H = x.shape
    I = weights.numel() // (3 * H * 2)
    x = x.contiguous()
    w = w.to(torch.float32).contiguous()
    h = torch.empty((n, I), dtype=torch.bfloat16)
    y = torch.empty((n, H), dtype=torch.bfloat16)
    a = HostFfnArgs(H, I, n, _hptr(weights), _hptr(x), _hptr(w), _hptr(h), _hptr(y), threads,
                    HOST_PATHS[path])
    _check(lib().moe_host_expert_ffn(ctypes.byref(a)), "moe_host_expert_ffn")
    return h, y


class SplitLayer:
    """The CPU/GPU split layer (moe_split_forward): `resident` experts' weights
    live on the GPU, the rest in host memory; each batch runs every other
    expert it routes to either on the host or after copying its weights to
    one of `n_stage` staging slots, as `policy` and `costs` decide.

    Wg, Wu [E,H,I], Wd [E,I,H]: bf16 master weights on the host."""

    def __init__(self, Wg, Wu, Wd, k: int, resident, n_stage: int = 2,
                 policy: int = POLICY_DYNAMIC, costs: SplitCosts | None = None,
                 host_threads: int = 0, block_m: int = 0, device="cuda"):
        self.E, self.H, self.I = Wg.shape
        self.k, self.n_stage, self.policy = k, n_stage, policy
        self.host_threads, self.block_m = host_threads, block_m
        self.device = torch.device(device)
        self.resident = _i32(resident)
        self.S = int(self.resident.sum())
        E, H, I = self.E, self.H, self.I
        self.host_weights = host_pack_weights(Wg, Wu, Wd)
        # the GPU layout of each expert, made on the device one expert at a
        # time and kept in page-locked host memory as the source of the
        # staging copies (the GPU never holds more than one expert's copy)
        per = lib().moe_packed_weights_size(BF16, 1, H, I)
        self.host_packed = torch.empty((E, per), dtype=torch.uint8, pin_memory=True)
        for e in range(E):
            pk, _ = pack_weights(BF16, Wg[e:e + 1].to(self.device), Wu[e:e + 1].to(self.device),
                                 Wd[e:e + 1].to(self.device))
            self.host_packed[e].copy_(pk)
        del pk
        idx = [e for e in range(E) if self.resident[e]]
        self.resident_packed = None
        if idx:
            self.resident_packed, _ = pack_weights(BF16, Wg[idx].to(self.device),
                                                   Wu[idx].to(self.device),
                                                   Wd[idx].to(self.device))
        self.stage_packed = torch.empty(
            max(lib().moe_packed_weights_size(BF16, max(n_stage, 1), H, I), 16),
            dtype=torch.uint8, device=self.device)
        self.copy_stream = torch.cuda.Stream(device=self.device)
        self.copy_event = torch.cuda.Event()
        self.copy_event.record(self.copy_stream)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.where = _i32([0] * E)
        self._ws, self._hws = {}, {}
        self.costs = costs if costs is not None else self.calibrate()

    def calibrate(self, n_max: int = 128) -> SplitCosts:
        """The latency model measured here: the host kernel on 1 and n_max
        tokens (a line through both: flat while the host streams weights,
        steeper once its tile products bound it, so n_max sits where a copy
        starts to compete) and one expert's copy to the GPU."""
        c = SplitCosts()
        hws = torch.empty(lib().moe_split_host_workspace_size(n_max, 1, self.H, self.I),
                          dtype=torch.uint8, pin_memory=True)
        dst = self.stage_packed if self.n_stage > 0 else torch.empty(
            3 * self.H * self.I * 2, dtype=torch.uint8, device=self.device)
        _check(lib().moe_split_calibrate(self.H, self.I, n_max, _hptr(self.host_weights[0]),
                                         _hptr(self.host_packed), _ptr(dst), _hptr(hws),
                                         hws.numel(), self.host_threads, _stream(None),
                                         ctypes.byref(c)), "moe_split_calibrate")
        return c

    def workspaces(self, T: int):
        if T not in self._ws:
            n = lib().moe_split_workspace_size(T, self.k, self.E, self.S, self.n_stage, self.H,
                                               self.I, self.block_m)
            if n == 0:
                raise MoEError(1, "moe_split_workspace_size")
            self._ws[T] = torch.empty(n, dtype=torch.uint8, device=self.device)
            m = lib().moe_split_host_workspace_size(T, self.k, self.H, self.I)
            self._hws[T] = torch.empty(max(m, 16), dtype=torch.uint8, pin_memory=True)
        return self._ws[T], self._hws[T]

    def __call__(self, x, logits, out=None, stream=None, policy: int | None = None):
        T = x.shape[0]
        out = torch.empty((T, self.H), dtype=torch.bfloat16, device=x.device) \
            if out is None else out
        ws, hws = self.workspaces(T)
        a = SplitArgs(T, self.k, self.E, self.H, self.I, self.block_m, _ptr(x), _ptr(logits),
                      _ptr(out), _hptr(self.resident), _ptr(self.resident_packed),
                      _ptr(self.stage_packed) if self.n_stage > 0 else None, self.n_stage,
                      _hptr(self.host_packed), _hptr(self.host_weights),
                      ctypes.pointer(self.costs), self.policy if policy is None else policy,
                      _hptr(self.where), _ptr(self.status), self.copy_stream.cuda_stream,
                      self.copy_event.cuda_event, self.host_threads)
        _check(lib().moe_split_forward(ctypes.byref(a), _ptr(ws), ws.numel(), _hptr(hws),
                                       hws.numel(), _stream(stream)), "moe_split_forward")
        return out

    def check(self) -> int:
        return check_status(self.status)

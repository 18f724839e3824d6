"""Thin Python binding of the C ABI in ``include/moe_b200.h`` (ctypes).

Argument marshalling only: every step of the layer runs in the CUDA library.
PyTorch provides device memory and streams. There is no fallback: if the
shared library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import numpy as np

from . import _build

FMT_CODE = {"bf16": 16, "int8": 8, "int4": 4, "nvfp4": 41, "fp16": 17}
ACT_CODE = {"silu": 0, "gelu": 1}
PATH_CODE = {"auto": 0, "gemv": 1, "tc": 2, "fused": 3}
N_MARKS = 6

STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported", -3: "CUDA error",
          -4: "device timeout", -5: "workspace", -6: "device check failed",
          -7: "too large for the built-in scratch"}


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status})")
        self.status = status


class MoeBank(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("group", ctypes.c_int32), ("n_exp", ctypes.c_int32),
                ("reserved", ctypes.c_int32),
                ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p),
                ("g_gate", ctypes.c_void_p), ("g_up", ctypes.c_void_p), ("g_down", ctypes.c_void_p)]


class MoeLayer(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("f", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("path", ctypes.c_int32),
                ("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("routed", MoeBank), ("shared", MoeBank)]


class MoeMatrix(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("group", ctypes.c_int32), ("x_type", ctypes.c_int32), ("y_type", ctypes.c_int32),
                ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64),
                ("w", ctypes.c_void_p), ("s", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class MoeFfn(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("f", ctypes.c_int32),
                ("act", ctypes.c_int32), ("bank", MoeBank)]


_LIB = None
EXPORTS = ["moe_abi_version", "moe_status_str", "moe_validate", "moe_workspace_size",
           "moe_route", "moe_permute", "moe_grouped_ffn", "moe_combine", "moe_layer_forward",
           "moe_layer_forward_marked", "moe_device_status", "moe_launches_per_call",
           "moe_layer_forward_static", "moe_static_device_status", "moe_test_inject_hold",
           "moe_nvfp4_pack_scales", "moe_nvfp4_quantize_rows", "moe_device_wait_site",
           "moe_matvec_validate", "moe_matvec_workspace_size", "moe_matvec",
           "moe_matvec_device_status", "moe_ffn_validate", "moe_ffn_workspace_size",
           "moe_ffn_forward", "moe_ffn_backward", "moe_ffn_device_status",
           "moe_test_inject_dense_hold"]


def load_library(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load ``libmoe_b200.so`` (in-tree). Raises if it is absent."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = _build.LIB_PATH
    if not os.path.exists(path):
        if build_if_missing:
            _build.build()
        else:
            raise RuntimeError(f"CUDA library not built: {path} (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    LP = ctypes.POINTER(MoeLayer)
    MP = ctypes.POINTER(MoeMatrix)
    FP = ctypes.POINTER(MoeFfn)
    sig = {
        "moe_abi_version": (I32, []),
        "moe_status_str": (ctypes.c_char_p, [I32]),
        "moe_validate": (I32, [LP]),
        "moe_workspace_size": (SZ, [LP]),
        "moe_route": (I32, [LP, P, P, P, P, SZ, P]),
        "moe_permute": (I32, [LP, P, P, P, P, P, SZ, P]),
        "moe_grouped_ffn": (I32, [LP, P, P, P, P, P, P, SZ, P]),
        "moe_combine": (I32, [LP, P, P, P, P, P, P]),
        "moe_layer_forward": (I32, [LP, P, P, P, P, P, P, P, SZ, P]),
        "moe_layer_forward_marked": (I32, [LP, P, P, P, P, P, P, P, SZ, P,
                                           ctypes.POINTER(P), I32]),
        "moe_device_status": (I32, [LP, P, SZ, ctypes.POINTER(I32), P]),
        "moe_device_wait_site": (I32, [LP, P, SZ, ctypes.POINTER(I32), P]),
        "moe_launches_per_call": (I32, [LP]),
        "moe_layer_forward_static": (I32, [LP, P, P, P]),
        "moe_static_device_status": (I32, [ctypes.POINTER(I32), P]),
        "moe_test_inject_hold": (I32, [LP, P, SZ, I32, I32, P]),
        "moe_nvfp4_pack_scales": (I32, [P, P, I32, I32, I32, P]),
        "moe_nvfp4_quantize_rows": (I32, [P, I32, I32, P, P, P, P]),
        "moe_matvec_validate": (I32, [MP]),
        "moe_matvec_workspace_size": (SZ, [MP]),
        "moe_matvec": (I32, [MP, P, P, P, SZ, P]),
        "moe_matvec_device_status": (I32, [MP, P, SZ, ctypes.POINTER(I32), ctypes.POINTER(I32),
                                           P]),
        "moe_ffn_validate": (I32, [FP]),
        "moe_ffn_workspace_size": (SZ, [FP, I32]),
        "moe_ffn_forward": (I32, [FP, P, P, P, P, SZ, P]),
        "moe_ffn_backward": (I32, [FP, P, P, P, P, P, P, P, P, SZ, P]),
        "moe_ffn_device_status": (I32, [FP, P, SZ, ctypes.POINTER(I32), ctypes.POINTER(I32), P]),
        "moe_test_inject_dense_hold": (I32, [I32, I32]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        raise MoeError(status, what)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def bank_struct(b) -> MoeBank:
    """A bank dict (fmt, group, n_exp and device tensors w_*, s_*, g_*) -> moe_bank."""
    if b is None:
        return MoeBank(16, 128, 0, 0, None, None, None, None, None, None, None, None, None)
    return MoeBank(FMT_CODE[b["fmt"]], b["group"], b["n_exp"], 0,
                   _ptr(b["w_gate"]), _ptr(b["w_up"]), _ptr(b["w_down"]),
                   _ptr(b.get("s_gate")), _ptr(b.get("s_up")), _ptr(b.get("s_down")),
                   _ptr(b.get("g_gate")), _ptr(b.get("g_up")), _ptr(b.get("g_down")))


class DeviceLayer:
    """Device-resident inputs of one layer that do not depend on the tokens:
    router weights, optional router bias, routed and shared expert banks."""

    def __init__(self, inputs, device="cuda", path: str = "auto"):
        import torch
        cfg = inputs.cfg
        self.cfg = cfg
        self.d, self.f, self.E, self.k = cfg.d, cfg.f, cfg.E, cfg.k
        self.path = PATH_CODE[path]
        dev = torch.device(device)

        def up(a, dtype=None):
            if a is None:
                return None
            if a.dtype == np.uint16:
                return torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)
            if a.dtype == np.uint32:
                return torch.from_numpy(a.view(np.int32)).to(dev)
            return torch.from_numpy(a).to(dev)

        self.router_w = up(inputs.router_w)
        self.router_bias = None if inputs.router_bias is None else \
            torch.from_numpy(inputs.router_bias.astype(np.float32)).to(dev)
        self.banks = {}
        for name, bank in (("routed", inputs.routed), ("shared", inputs.shared)):
            if bank is None:
                self.banks[name] = None
                continue
            self.banks[name] = dict(fmt=bank.fmt, group=bank.group, n_exp=bank.n_exp,
                                    **{k: up(v) for k, v in bank.arrays().items()})
            if bank.fmt == "nvfp4":  # block scales into the layout the kernels read
                b = self.banks[name]
                for m, (N, K) in (("gate", (cfg.f, cfg.d)), ("up", (cfg.f, cfg.d)),
                                  ("down", (cfg.d, cfg.f))):
                    b["s_" + m] = nvfp4_pack_scales(b["s_" + m], bank.n_exp, N, K)

    @classmethod
    def from_tensors(cls, cfg, router_w, router_bias, routed: dict, shared: dict | None,
                     path="auto"):
        self = cls.__new__(cls)
        self.cfg = cfg
        self.d, self.f, self.E, self.k = cfg.d, cfg.f, cfg.E, cfg.k
        self.path = PATH_CODE[path]
        self.router_w, self.router_bias = router_w, router_bias
        self.banks = {"routed": routed, "shared": shared}
        return self

    def _bank(self, b) -> MoeBank:
        return bank_struct(b)

    def descriptor(self, T: int, path: str | None = None) -> MoeLayer:
        return MoeLayer(T, self.d, self.f, self.E, self.k,
                        self.path if path is None else PATH_CODE[path],
                        _ptr(self.router_w), _ptr(self.router_bias),
                        self._bank(self.banks["routed"]), self._bank(self.banks["shared"]))

    @property
    def has_shared(self) -> bool:
        return self.banks["shared"] is not None


def _stream(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def workspace_size(L: MoeLayer) -> int:
    n = load_library().moe_workspace_size(ctypes.byref(L))
    if n == 0:
        raise MoeError(load_library().moe_validate(ctypes.byref(L)), "moe_workspace_size")
    return n


def alloc_workspace(L: MoeLayer, device="cuda"):
    """A zeroed workspace (the status word at its start must begin at zero). The fill is
    waited for here, so the workspace may be used on any stream: a fill still queued behind
    other work while a call runs on another stream would reset the call's barrier words."""
    import torch
    ws = torch.zeros(workspace_size(L), dtype=torch.uint8, device=device)
    torch.cuda.current_stream(ws.device).synchronize()
    return ws


def _on_stream(stream):
    """The context in which a call's results are allocated: with a given stream current, so that
    their memory is that stream's (a block of another stream's pool may still be in use by what is
    queued there). Tensors that the caller brings are the caller's to keep and to order."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


def _used_here(stream, *results):
    """Marks results allocated for a given stream as used by the caller's current stream too: dropped
    while work queued here still reads them, they are not handed out again before it has run."""
    import torch
    if stream is None:
        return
    for t in results:
        if t is not None and t.is_cuda:
            t.record_stream(torch.cuda.current_stream(t.device))


def route(L: MoeLayer, x, ws, stream=None):
    import torch
    with _on_stream(stream):
        idx = torch.empty((L.T, L.k), dtype=torch.int32, device=x.device)
        w = torch.empty((L.T, L.k), dtype=torch.float32, device=x.device)
    _used_here(stream, idx, w)
    _check(load_library().moe_route(ctypes.byref(L), x.data_ptr(), idx.data_ptr(), w.data_ptr(),
                                    ws.data_ptr(), ws.numel(), _stream(stream)), "moe_route")
    return idx, w


def permute(L: MoeLayer, topk_idx, ws, stream=None):
    import torch
    dev = topk_idx.device
    with _on_stream(stream):
        offsets = torch.empty(L.E + 1, dtype=torch.int32, device=dev)
        perm = torch.empty(L.T * L.k, dtype=torch.int32, device=dev)
        inv = torch.empty(L.T * L.k, dtype=torch.int32, device=dev)
    _used_here(stream, offsets, perm, inv)
    _check(load_library().moe_permute(ctypes.byref(L), topk_idx.data_ptr(), offsets.data_ptr(),
                                      perm.data_ptr(), inv.data_ptr(), ws.data_ptr(), ws.numel(),
                                      _stream(stream)), "moe_permute")
    return offsets, perm, inv


def grouped_ffn(L: MoeLayer, x, offsets, perm, ws, has_shared=True, stream=None):
    import torch
    dev = x.device
    with _on_stream(stream):
        y_assign = torch.empty((L.T * L.k, L.d), dtype=torch.float32, device=dev)
        y_shared = torch.empty((L.T, L.d), dtype=torch.float32, device=dev) if has_shared else None
    _used_here(stream, y_assign, y_shared)
    _check(load_library().moe_grouped_ffn(ctypes.byref(L), x.data_ptr(), offsets.data_ptr(),
                                          perm.data_ptr(), y_assign.data_ptr(), _ptr(y_shared),
                                          ws.data_ptr(), ws.numel(), _stream(stream)),
           "moe_grouped_ffn")
    return y_assign, y_shared


def combine(L: MoeLayer, y_assign, y_shared, inv, topk_w, out=None, stream=None):
    import torch
    if out is None:
        with _on_stream(stream):
            out = torch.empty((L.T, L.d), dtype=torch.bfloat16, device=y_assign.device)
        _used_here(stream, out)
    _check(load_library().moe_combine(ctypes.byref(L), y_assign.data_ptr(), _ptr(y_shared),
                                      inv.data_ptr(), topk_w.data_ptr(), out.data_ptr(),
                                      _stream(stream)), "moe_combine")
    return out


def layer_forward(L: MoeLayer, x, ws, out=None, topk_idx=None, topk_w=None, offsets=None,
                  perm=None, marks=None, stream=None):
    """The fused layer call. Optional outputs are written when tensors are given."""
    import torch
    if out is None:
        with _on_stream(stream):
            out = torch.empty((L.T, L.d), dtype=torch.bfloat16, device=x.device)
        _used_here(stream, out)
    lib = load_library()
    if marks is None:
        st = lib.moe_layer_forward(ctypes.byref(L), x.data_ptr(), out.data_ptr(), _ptr(topk_idx),
                                   _ptr(topk_w), _ptr(offsets), _ptr(perm), ws.data_ptr(),
                                   ws.numel(), _stream(stream))
    else:
        arr = (ctypes.c_void_p * len(marks))(*[None if m is None else m.cuda_event for m in marks])
        st = lib.moe_layer_forward_marked(ctypes.byref(L), x.data_ptr(), out.data_ptr(),
                                          _ptr(topk_idx), _ptr(topk_w), _ptr(offsets),
                                          _ptr(perm), ws.data_ptr(), ws.numel(),
                                          _stream(stream), arr, len(marks))
    _check(st, "moe_layer_forward")
    return out


def nvfp4_pack_scales(src, n_mats: int, rows: int, K: int, stream=None):
    """Block scales of an NVFP4 bank, uint8 [n_mats][rows][K/16] on the device, rearranged
    into the layout the FP4 tensor-core kernels read (a new tensor of the same size)."""
    import torch
    with _on_stream(stream):
        src = src.contiguous()
        dst = torch.empty_like(src)
    _used_here(stream, dst)
    _check(load_library().moe_nvfp4_pack_scales(src.data_ptr(), dst.data_ptr(), n_mats, rows, K,
                                                _stream(stream)), "moe_nvfp4_pack_scales")
    return dst


def nvfp4_quantize_rows(v, stream=None):
    """fp32 rows [R, K] on the device -> (E2M1 codes uint8 [R, K/2], E4M3 block-scale codes
    uint8 [R, K/16], fp32 row scales [R]) by the layer's activation quantiser."""
    import torch
    R, K = v.shape
    with _on_stream(stream):
        v = v.contiguous()
        codes = torch.empty((R, K // 2), dtype=torch.uint8, device=v.device)
        scales = torch.empty((R, K // 16), dtype=torch.uint8, device=v.device)
        g = torch.empty(R, dtype=torch.float32, device=v.device)
    _used_here(stream, codes, scales, g)
    _check(load_library().moe_nvfp4_quantize_rows(v.data_ptr(), R, K, codes.data_ptr(),
                                                  scales.data_ptr(), g.data_ptr(),
                                                  _stream(stream)), "moe_nvfp4_quantize_rows")
    return codes, scales, g


def launches_per_call(L: MoeLayer) -> int:
    return load_library().moe_launches_per_call(ctypes.byref(L))


def device_status(L: MoeLayer, ws, stream=None) -> int:
    code = ctypes.c_int32(0)
    _check(load_library().moe_device_status(ctypes.byref(L), ws.data_ptr(), ws.numel(),
                                            ctypes.byref(code), _stream(stream)),
           "moe_device_status")
    return code.value


def device_wait_site(L: MoeLayer, ws, stream=None) -> int:
    """Site of the first device-side wait that gave up since the last read (0: none)."""
    site = ctypes.c_int32(0)
    _check(load_library().moe_device_wait_site(ctypes.byref(L), ws.data_ptr(), ws.numel(),
                                               ctypes.byref(site), _stream(stream)),
           "moe_device_wait_site")
    return site.value


def layer_forward_static(L: MoeLayer, x, out=None, stream=None):
    """The layer with the library's built-in scratch (no workspace argument): for callers
    that cannot allocate device memory. Limits and sharing rules: include/moe_b200.h."""
    import torch
    if out is None:
        with _on_stream(stream):
            out = torch.empty((L.T, L.d), dtype=torch.bfloat16, device=x.device)
        _used_here(stream, out)
    _check(load_library().moe_layer_forward_static(ctypes.byref(L), x.data_ptr(),
                                                   out.data_ptr(), _stream(stream)),
           "moe_layer_forward_static")
    return out


def static_device_status(stream=None) -> int:
    """Reads and clears the status word of the built-in scratch (moe_layer_forward_static)."""
    code = ctypes.c_int32(0)
    _check(load_library().moe_static_device_status(ctypes.byref(code), _stream(stream)),
           "moe_static_device_status")
    return code.value


def test_inject_hold(L: MoeLayer, ws, hold: bool, budget_cycles: int = 0, stream=None):
    """Sets or clears the workspace's failure-injection hold word (see the header)."""
    _check(load_library().moe_test_inject_hold(ctypes.byref(L), ws.data_ptr(), ws.numel(),
                                               int(bool(hold)), int(budget_cycles),
                                               _stream(stream)), "moe_test_inject_hold")


# ---------------------------------------------------------------------- dense operators
#
# Unlike the layer's calls above, these check their tensors (type, shape, layout, device)
# before handing over pointers, and raise ValueError. The work runs on the tensors' device,
# on its current stream unless one is given. A given stream is the current one during the call:
# its work comes after what that stream holds, and a caller who goes on on another stream orders
# the two, as with torch.cuda.stream; the memory of what the call uses and returns is safe to drop.


def _dtype_code(t) -> int:
    import torch
    try:
        return {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}[t]
    except KeyError:
        raise ValueError(f"element type {t} is not supported") from None


def _check_rows(t, name, shape, dtype, index, stride=None):
    """A 2-D tensor of `shape` on CUDA device `index` with contiguous rows, `stride` elements
    apart where there is more than one (dense without a stride)."""
    if t.dtype != dtype or t.get_device() != index or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {list(shape)} on cuda:{index}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    rows, cols = shape
    want = cols if stride is None else stride
    if (rows > 1 and t.stride(0) != want) or (cols > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected rows of contiguous elements, {want} apart, got strides "
                         f"{list(t.stride())}")


def _check_ws(ws, index):
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"the workspace must be contiguous and on cuda:{index}")


_CURRENT = None  # (current device, its raw stream), bound at the first call


def _call(index, fn, *args):
    """fn(*args, stream) with CUDA device `index` current, on its current stream; returns its status.
    The stream is asked for as a raw handle: building a torch stream object takes as long as a
    kernel launch."""
    global _CURRENT
    if _CURRENT is None:
        import torch
        _CURRENT = (torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
    current_device, raw_stream = _CURRENT
    if index == current_device():
        return fn(*args, raw_stream(index))
    import torch
    with torch.cuda.device(index):
        return fn(*args, raw_stream(index))


def _on(stream, fn, *args):
    """fn(*args) with the given `stream` current, so that its results are allocated for that stream
    (a block of another stream's pool may still be in use by what is queued there). What the call
    reads and writes is marked as used by the stream, and its results as used by the caller's
    current one: freed early, they are not handed out again before both are done with them."""
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    for a in args:
        owner = getattr(a, "owner", None)  # a descriptor: its weights
        held = (a,) if owner is None else (*vars(owner).values(), *getattr(owner, "bank", {}).values())
        for t in held:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                if t.get_device() != stream.device_index:
                    raise ValueError(f"the stream is on cuda:{stream.device_index}, a tensor of the "
                                     f"call on {t.device}")
                t.record_stream(stream)
    with torch.cuda.stream(stream):
        result = fn(*args)
    _used_here(stream, *(t for t in (result if isinstance(result, tuple) else (result,))
                         if isinstance(t, torch.Tensor)))
    return result


def _alloc_zeroed(nbytes: int, device):
    """A zeroed workspace whose fill is waited for (see alloc_workspace)."""
    import torch
    ws = torch.zeros(nbytes, dtype=torch.uint8, device=device)
    torch.cuda.current_stream(ws.device).synchronize()
    return ws


class QuantMatrix:
    """A weight matrix [N, K] of 4-bit integers with group scales, on the device: ``codes``
    int32 [N, K/8] (8 two's-complement nibbles a word along K), ``scales`` bf16
    [N, K/group], ``bias`` fp32 [N] or None (the int4 encoding of the expert banks)."""

    def __init__(self, codes, scales, K: int, group: int = 128, bias=None):
        import torch
        if group not in (32, 64, 128) or K < 1 or K % group:
            raise ValueError(f"K must be a multiple of the group (32, 64 or 128): {K}, {group}")
        if codes.dim() != 2 or not codes.is_cuda:
            raise ValueError("codes must be a CUDA tensor [N, K/8]")
        N, dev = codes.shape[0], codes.device
        if codes.dtype not in (torch.int32, torch.uint32):
            raise ValueError("codes must hold 32-bit words")
        _check_rows(codes, "codes", (N, K // 8), codes.dtype, dev.index)
        _check_rows(scales, "scales", (N, K // group), torch.bfloat16, dev.index)
        if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (N,) or
                                 bias.device != dev or not bias.is_contiguous()):
            raise ValueError(f"bias: expected contiguous fp32 [{N}] on {dev}")
        self.codes, self.scales, self.bias = codes, scales, bias
        self.N, self.K, self.group, self.device = N, K, group, dev

    def descriptor(self, T: int, x_dtype=None, y_dtype=None, ldx: int | None = None,
                   ldy: int | None = None) -> MoeMatrix:
        """The call's descriptor: T rows of x_dtype (bf16 by default) giving rows of y_dtype
        (x_dtype by default, or fp32); ldx, ldy: elements between rows (dense by default).
        It holds pointers into this object's tensors, which must outlive it."""
        import torch
        x_dtype = torch.bfloat16 if x_dtype is None else x_dtype
        y_dtype = x_dtype if y_dtype is None else y_dtype
        M = MoeMatrix(T, self.N, self.K, self.group, _dtype_code(x_dtype), _dtype_code(y_dtype),
                      self.K if ldx is None else ldx, self.N if ldy is None else ldy,
                      self.codes.data_ptr(), self.scales.data_ptr(), _ptr(self.bias))
        M.owner = self
        lib = load_library()
        _check(lib.moe_matvec_validate(ctypes.byref(M)), "moe_matvec_validate")
        # what each call needs, at hand: a call costs the host little more than its launch. (No
        # reference to M itself: the cycle would keep the weights until a garbage collection.)
        M.call = ((T, self.K), (T, self.N), M.ldx, M.ldy, x_dtype, y_dtype, self.device.index,
                  lib.moe_matvec)
        return M


def matvec_workspace_size(M: MoeMatrix) -> int:
    return load_library().moe_matvec_workspace_size(ctypes.byref(M))


def alloc_matvec_workspace(M: MoeMatrix):
    return _alloc_zeroed(matvec_workspace_size(M), M.owner.device)


def matvec(M: MoeMatrix, x, ws, out=None, stream=None):
    """y = x W^T (+ bias) for the T <= 32 rows of x: [T, K] -> [T, N] (include/moe_b200.h)."""
    if stream is not None:
        return _on(stream, matvec, M, x, ws, out)
    x_shape, y_shape, ldx, ldy, xt, yt, index, fn = M.call
    _check_rows(x, "x", x_shape, xt, index, ldx)
    if out is None:
        # (sizes as numbers: a tuple costs the call half a microsecond more)
        rows, cols = y_shape
        out = x.new_empty(rows, ldy) if yt == xt else x.new_empty((rows, ldy), dtype=yt)
        if ldy != cols:
            out = out[:, :cols]
    else:
        _check_rows(out, "out", y_shape, yt, index, ldy)
    _check_ws(ws, index)
    status = _call(index, fn, M, x.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel())
    if status:
        _check(status, "moe_matvec")
    return out


class DeviceFfn:
    """A dense gated feed-forward block y = Wd (act(Wg x) * (Wu x)) on the device. ``bank``: a
    bank dict as for the layer, of one expert: fmt "bf16", "fp16" or "int4" (group 128, s_*
    scales), device tensors w_gate, w_up [f, d] and w_down [d, f] (a leading dimension of 1 is
    accepted; int4: int32 words, K/8 a row). act: "silu" or "gelu" (tanh form)."""

    def __init__(self, bank: dict, d: int, f: int, act: str = "silu"):
        import torch
        if act not in ACT_CODE:
            raise ValueError(f"act must be one of {sorted(ACT_CODE)}")
        if bank.get("n_exp", 1) != 1 or bank["fmt"] not in ("bf16", "fp16", "int4"):
            raise ValueError("the block takes a bank of one expert in bf16, fp16 or int4")
        fmt = bank["fmt"]
        if fmt == "int4" and bank.get("group", 128) != 128:
            raise ValueError("int4 blocks have groups of 128")
        step = 128 if fmt == "int4" else 8
        if d < step or f < step or d % step or f % step:
            raise ValueError(f"d and f must be multiples of {step}: {d}, {f}")
        self.dtype = torch.float16 if fmt == "fp16" else torch.bfloat16
        self.device = bank["w_gate"].device
        if self.device.type != "cuda":
            raise ValueError("the weights must be on a CUDA device")
        self.d, self.f, self.act, self.fmt = d, f, act, fmt
        self.bank = dict(fmt=fmt, group=128, n_exp=1)
        for m, N, K in (("gate", f, d), ("up", f, d), ("down", d, f)):
            w = bank["w_" + m]
            w = w[0] if w.dim() == 3 and w.shape[0] == 1 else w
            int4 = fmt == "int4"
            want = w.dtype if int4 and w.dtype in (torch.int32, torch.uint32) else \
                torch.int32 if int4 else self.dtype
            _check_rows(w, "w_" + m, (N, K // 8 if int4 else K), want, self.device.index)
            self.bank["w_" + m] = w
            if int4:
                s = bank["s_" + m]
                s = s[0] if s.dim() == 3 and s.shape[0] == 1 else s
                _check_rows(s, "s_" + m, (N, K // 128), torch.bfloat16, self.device.index)
                self.bank["s_" + m] = s

    def descriptor(self, T: int) -> MoeFfn:
        """The descriptor of calls on T rows. It holds pointers into this object's tensors,
        which must outlive it."""
        F = MoeFfn(T, self.d, self.f, ACT_CODE[self.act], bank_struct(self.bank))
        F.owner = self
        lib = load_library()
        _check(lib.moe_ffn_validate(ctypes.byref(F)), "moe_ffn_validate")
        F.call = ((T, self.d), (2, T, self.f), self.dtype, self.device.index,
                  lib.moe_ffn_forward, lib.moe_ffn_backward)
        return F


def ffn_workspace_size(F: MoeFfn, backward: bool = False) -> int:
    n = load_library().moe_ffn_workspace_size(ctypes.byref(F), int(backward))
    if n == 0:
        raise MoeError(-2, "moe_ffn_workspace_size")  # an int4 block has no backward pass
    return n


def alloc_ffn_workspace(F: MoeFfn, backward: bool = False):
    """A zeroed workspace for ffn_forward, with ``backward`` for training calls (ffn_forward with
    pre, and ffn_backward)."""
    return _alloc_zeroed(ffn_workspace_size(F, backward), F.owner.device)


def ffn_pre(F: MoeFfn, device=None):
    """The fp32 tensor [2, T, f] in which ffn_forward keeps Wg x and Wu x for ffn_backward."""
    import torch
    return torch.empty((2, F.T, F.f), dtype=torch.float32, device=device or F.owner.device)


def _check_pre(pre, shape, index):
    import torch
    if pre.dtype != torch.float32 or pre.shape != shape or pre.get_device() != index or \
            not pre.is_contiguous():
        raise ValueError(f"pre: expected contiguous fp32 {list(shape)} on cuda:{index}")


def ffn_forward(F: MoeFfn, x, ws, out=None, pre=None, stream=None):
    """y = Wd (act(Wg x) * (Wu x)) for the rows of x [T, d]; ``pre`` (ffn_pre) keeps what
    ffn_backward needs (include/moe_b200.h)."""
    if stream is not None:
        return _on(stream, ffn_forward, F, x, ws, out, pre)
    shape, pre_shape, dtype, index, fn, _ = F.call
    _check_rows(x, "x", shape, dtype, index)
    if out is None:
        out = x.new_empty(*shape)
    else:
        _check_rows(out, "out", shape, dtype, index)
    if pre is not None:
        _check_pre(pre, pre_shape, index)
    _check_ws(ws, index)
    status = _call(index, fn, F, x.data_ptr(), out.data_ptr(), _ptr(pre), ws.data_ptr(),
                   ws.numel())
    if status:
        _check(status, "moe_ffn_forward")
    return out


def ffn_backward(F: MoeFfn, x, dy, pre, ws, need_dx: bool = True, need_dw: bool = True,
                 stream=None):
    """(dx, dw_gate, dw_up, dw_down) from dy [T, d], x and the ``pre`` of ffn_forward; what is
    not needed is None and not computed. ``ws``: alloc_ffn_workspace(F, backward=True)."""
    if stream is not None:
        return _on(stream, ffn_backward, F, x, dy, pre, ws, need_dx, need_dw)
    shape, pre_shape, dtype, index, _, fn = F.call
    _check_rows(x, "x", shape, dtype, index)
    _check_rows(dy, "dy", shape, dtype, index)
    _check_pre(pre, pre_shape, index)
    _check_ws(ws, index)
    dx = x.new_empty(*shape) if need_dx else None
    dwg = dwu = dwd = None
    if need_dw:
        dwg, dwu, dwd = x.new_empty(F.f, F.d), x.new_empty(F.f, F.d), x.new_empty(F.d, F.f)
    _check(_call(index, fn, F, x.data_ptr(), dy.data_ptr(), pre.data_ptr(), _ptr(dx),
                 _ptr(dwg), _ptr(dwu), _ptr(dwd), ws.data_ptr(), ws.numel()), "moe_ffn_backward")
    return dx, dwg, dwu, dwd


def _device_status(fn, D, ws, stream):
    if stream is not None:
        return _on(stream, _device_status, fn, D, ws, None)
    code, site = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(_call(D.owner.device.index, fn, ctypes.byref(D), ws.data_ptr(), ws.numel(),
                 ctypes.byref(code), ctypes.byref(site)), fn.__name__)
    return code.value, site.value


def ffn_device_status(F: MoeFfn, ws, stream=None):
    """(status code, wait site) kept in a block's workspace since the last read (0, 0: none)."""
    return _device_status(load_library().moe_ffn_device_status, F, ws, stream)


def matvec_device_status(M: MoeMatrix, ws, stream=None):
    """(status code, wait site) kept in a matvec workspace since the last read (0, 0: none)."""
    return _device_status(load_library().moe_matvec_device_status, M, ws, stream)


def test_inject_dense_hold(hold: bool, budget_cycles: int = 0):
    """Sets or clears the dense operators' failure injection for this thread's calls (see the
    header)."""
    _check(load_library().moe_test_inject_dense_hold(int(bool(hold)), int(budget_cycles)),
           "moe_test_inject_dense_hold")

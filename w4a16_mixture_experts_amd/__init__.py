"""Python binding of libexmoe, the fused grouped W4A16 MoE expert layer for MI355X.

Argument marshalling only: tensors are passed to the C ABI as device pointers with
torch's current HIP stream; every step of the layer runs in the library's HIP kernels
(host C++ for the offline packer and the slot-cache policy). PyTorch provides device
memory and streams. Importing this package fails loudly if libexmoe.so is not built.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import NamedTuple, Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libexmoe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libexmoe.so is not built ({LIB_PATH}); run python w4a16_mixture_experts_amd/build_lib.py")
# torch ships its own HIP runtime under the SONAME libamdhip64.so.7 but links it by the
# name libamdhip64.so. Loading torch first makes this library bind to that same runtime;
# loaded the other way round, the process would hold two HIP runtimes, and a kernel
# launched from one does not see the device the other initialised.
try:
    import torch  # noqa: F401
except ImportError:
    pass
_lib = ctypes.CDLL(LIB_PATH)

# status codes (exmoe.h)
OK = 0
ERR_INVALID_ARGUMENT = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE = -3
ERR_HIP = -4
ERR_OUT_OF_MEMORY = -5
ERR_CACHE = -6

PATH_AUTO, PATH_DECODE, PATH_PREFILL, PATH_SEQUENTIAL = 0, 1, 2, 3
WEIGHTS_BF16 = 0x100       # flag: the bank holds dense bf16 experts (bf16_pack)
DEBUG_COUNTERS = 0x200     # flag: expert kernels count the rows they ran per expert (workspace_rows)
CACHE_DRY_RUN = 1
DTYPE_BF16, DTYPE_FP16, DTYPE_FP32 = 0, 1, 2
GROUPED_MM, GROUPED_DGRAD, GROUPED_WGRAD = 0, 1, 2

_vp = ctypes.c_void_p
_cp = ctypes.c_char_p      # a struct of arguments, packed into bytes
_i = ctypes.c_int
_sz = ctypes.c_size_t


class ExpertBankC(ctypes.Structure):
    _fields_ = [("base", _vp), ("stride", _sz), ("expert_to_slot", _vp)]


class LoraBankC(ctypes.Structure):
    _fields_ = [("a", _vp), ("lda", _sz), ("a_stride", _sz), ("b", _vp), ("ldb", _sz), ("b_stride", _sz),
                ("ranks", _vp), ("scales", _vp), ("adapters", _i), ("rank_max", _i)]


class CacheStatsC(ctypes.Structure):
    _fields_ = [("lookups", ctypes.c_uint64), ("hits", ctypes.c_uint64), ("misses", ctypes.c_uint64),
                ("evictions", ctypes.c_uint64), ("h2d_bytes", ctypes.c_uint64), ("h2d_copies", ctypes.c_uint64),
                ("device_bytes", ctypes.c_uint64), ("pinned_host_bytes", ctypes.c_uint64), ("resident", _i)]


_SIGS = {
    "exmoe_status_string": (ctypes.c_char_p, [_i]),
    "exmoe_last_error": (ctypes.c_char_p, []),
    "exmoe_abi_version": (_i, []),
    "exmoe_packed_expert_bytes": (_sz, [_i, _i]),
    "exmoe_quantize_pack": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _sz]),
    "exmoe_unpack_expert": (_i, [_vp, _sz, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "exmoe_route_topk": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "exmoe_topk_from_logits": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp]),
    "exmoe_route_weights": (_i, [_vp, _vp, _i, _i, _i, _i, _vp, _vp]),
    "exmoe_group_workspace_bytes": (_sz, [_i, _i, _i]),
    "exmoe_group_tokens": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "exmoe_active_experts": (_i, [_vp, _i, _vp, _vp, _vp]),
    "exmoe_moe_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "exmoe_bf16_expert_bytes": (_sz, [_i, _i]),
    "exmoe_workspace_flags": (_i, [_vp, _sz, _i, ctypes.POINTER(ctypes.c_uint32), _vp]),
    "exmoe_workspace_rows": (_i, [_vp, _sz, _i, _i, _vp, _vp]),
    "exmoe_bf16_pack": (_i, [_vp, _vp, _vp, _i, _i, _vp, _sz]),
    "exmoe_moe_forward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(ExpertBankC), _i, _i, _i, _i, _i, _i,
                               _vp, _vp, _sz, _vp]),
    "exmoe_moe_forward_cached": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i, _i,
                                      _vp, _vp, _sz, _vp]),
    "exmoe_moe_layer_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "exmoe_moe_layer": (_i, [_vp, _vp, _vp, ctypes.POINTER(ExpertBankC), _i, _i, _i, _i, _i, _i, _i,
                             _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "exmoe_moe_layer_noalloc": (_i, [_vp, _vp, _vp, ctypes.POINTER(ExpertBankC), _i, _i, _i, _i, _i, _i, _i,
                                     _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "exmoe_slot_cache_create": (_i, [_i, _i, _i, _sz, _i, ctypes.POINTER(_vp)]),
    "exmoe_slot_cache_host_slot": (_i, [_vp, _i, _i, ctypes.POINTER(_vp)]),
    "exmoe_slot_cache_preload": (_i, [_vp, _vp]),
    "exmoe_slot_cache_acquire": (_i, [_vp, _i, _vp, _i, _vp, ctypes.POINTER(ExpertBankC)]),
    "exmoe_slot_cache_table": (_i, [_vp, _i, _vp]),
    "exmoe_slot_cache_waves": (_i, [_vp, _i, _vp, _i, _i, _vp, ctypes.POINTER(_i), ctypes.POINTER(_i)]),
    "exmoe_slot_cache_stats": (_i, [_vp, ctypes.POINTER(CacheStatsC)]),
    "exmoe_slot_cache_reset_stats": (_i, [_vp]),
    "exmoe_slot_cache_destroy": (_i, [_vp]),
    "exmoe_profile_enable": (_i, [_i]),
    "exmoe_profile_reset": (_i, []),
    "exmoe_profile_read": (_i, [ctypes.c_char_p, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_uint64)]),
    "exmoe_span_enable": (_i, [_i]),
    "exmoe_span_clear": (_i, []),
    "exmoe_span_read": (_i, [ctypes.c_char_p, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_uint64)]),
    "exmoe_device_copy": (_i, [_vp, _vp, _sz, _vp]),
    "exmoe_grouped_mm_workspace_bytes": (_sz, [_i] * 6),
    "exmoe_grouped_mm": (_i, [_vp, _sz, _i, _vp, _i, _vp, _vp, _sz, _sz, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp, _sz,
                              _vp]),
    "exmoe_grouped_mm_dgrad": (_i, [_vp, _sz, _vp, _vp, _sz, _sz, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp, _sz,
                                    _vp]),
    "exmoe_grouped_mm_wgrad": (_i, [_vp, _sz, _vp, _sz, _i, _vp, _i, _vp, _i, _i, _i, _i, _i, _i, _vp, _sz, _sz, _vp,
                                    _sz, _vp]),
    "exmoe_rms_norm": (_i, [_cp, _vp]),
    "exmoe_quantize_fp8": (_i, [_cp, _vp]),
    "exmoe_swiglu_fp8": (_i, [_cp, _vp]),
    "exmoe_quantize_fp8_weights": (_i, [_cp, _vp]),
    "exmoe_grouped_mm_fp8": (_i, [_cp, _vp]),
    "exmoe_moe_layer_fp8_workspace_bytes": (_sz, [_i] * 5),
    "exmoe_moe_layer_fp8": (_i, [_cp, _vp, _sz, _vp]),
    "exmoe_balance_loss_workspace_bytes": (_sz, [_i, _i]),
    "exmoe_balance_loss": (_i, [_cp, _vp, _sz, _vp]),
    "exmoe_balance_loss_backward": (_i, [_cp, _vp]),
    "exmoe_lora_workspace_bytes": (_sz, [_i] * 5),
    "exmoe_lora_linear": (_i, [_vp, _sz, _vp, _sz, ctypes.POINTER(LoraBankC), _vp, _i, _i, _i, _i, _vp, _sz, _vp, _sz,
                               _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGS)


class ExmoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_lib.exmoe_status_string(status).decode()} ({status}): {msg}")
        self.status = status


def _check(status: int):
    if status != OK:
        raise ExmoeError(status, _lib.exmoe_last_error().decode())


def last_error() -> str:
    return _lib.exmoe_last_error().decode()


def abi_version() -> int:
    return _lib.exmoe_abi_version()


def packed_expert_bytes(H: int, I: int) -> int:
    return _lib.exmoe_packed_expert_bytes(H, I)


# ----------------------------------------------------------------------------- host packer
def bf16_expert_bytes(H: int, I: int) -> int:
    return _lib.exmoe_bf16_expert_bytes(H, I)


def bf16_pack(g_bits: np.ndarray, u_bits: np.ndarray, d_bits: np.ndarray) -> np.ndarray:
    """bf16 bits gate [I,H], up [I,H], down [H,I] (uint16) -> dense bf16 blob (uint8 numpy)."""
    g = np.ascontiguousarray(g_bits, dtype=np.uint16)
    u = np.ascontiguousarray(u_bits, dtype=np.uint16)
    d = np.ascontiguousarray(d_bits, dtype=np.uint16)
    I, H = g.shape
    if u.shape != (I, H) or d.shape != (H, I):
        raise ValueError("shape mismatch: gate/up [I,H], down [H,I]")
    nb = bf16_expert_bytes(H, I)
    out = np.empty(nb, dtype=np.uint8)
    _check(_lib.exmoe_bf16_pack(g.ctypes.data, u.ctypes.data, d.ctypes.data, H, I, out.ctypes.data, nb))
    return out


def quantize_pack(w_gate: np.ndarray, w_up: np.ndarray, w_down: np.ndarray, out: Optional[np.ndarray] = None,
                  out_ptr: Optional[int] = None) -> np.ndarray:
    """fp32 gate [I,H], up [I,H], down [H,I] -> packed blob (uint8 numpy, or written to out_ptr)."""
    g = np.ascontiguousarray(w_gate, dtype=np.float32)
    u = np.ascontiguousarray(w_up, dtype=np.float32)
    d = np.ascontiguousarray(w_down, dtype=np.float32)
    I, H = g.shape
    if u.shape != (I, H) or d.shape != (H, I):
        raise ValueError("shape mismatch: gate/up [I,H], down [H,I]")
    nb = packed_expert_bytes(H, I)
    if out_ptr is None:
        if out is None:
            out = np.empty(nb, dtype=np.uint8)
        ptr = out.ctypes.data
        size = out.nbytes
    else:
        ptr, size = out_ptr, nb
    _check(_lib.exmoe_quantize_pack(g.ctypes.data, u.ctypes.data, d.ctypes.data, H, I, 128, ptr, size))
    return out


def unpack_expert(blob: np.ndarray, H: int, I: int):
    blob = np.ascontiguousarray(blob, dtype=np.uint8)
    qg = np.empty((I, H), np.int8); qu = np.empty((I, H), np.int8); qd = np.empty((H, I), np.int8)
    sg = np.empty((I, H // 128), np.uint16); su = np.empty_like(sg); sd = np.empty((H, I // 128), np.uint16)
    _check(_lib.exmoe_unpack_expert(blob.ctypes.data, blob.nbytes, H, I, qg.ctypes.data, qu.ctypes.data,
                                    qd.ctypes.data, sg.ctypes.data, su.ctypes.data, sd.ctypes.data))
    return qg, sg, qu, su, qd, sd


# ----------------------------------------------------------------------------- device calls
_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    return _torch().cuda.current_stream().cuda_stream


def route_topk(x, w_router, k: int, bias=None, renormalize: bool = True, logits=None, ids=None, weights=None):
    """x bf16 [T,H], w_router bf16 [E,H], bias fp32 [E] -> (logits bf16 [T,E], ids int32 [T,k], weights fp32 [T,k])."""
    torch = _torch()
    T, H = x.shape
    E = w_router.shape[0]
    dev = x.device
    logits = torch.empty((T, E), dtype=torch.bfloat16, device=dev) if logits is None else logits
    ids = torch.empty((T, k), dtype=torch.int32, device=dev) if ids is None else ids
    weights = torch.empty((T, k), dtype=torch.float32, device=dev) if weights is None else weights
    _check(_lib.exmoe_route_topk(_ptr(x), _ptr(w_router), _ptr(bias), T, H, E, k, int(renormalize), _ptr(logits),
                                 _ptr(ids), _ptr(weights), _stream()))
    return logits, ids, weights


def topk_from_logits(logits, k: int, renormalize: bool = True):
    torch = _torch()
    T, E = logits.shape
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(_lib.exmoe_topk_from_logits(_ptr(logits), T, E, k, int(renormalize), _ptr(ids), _ptr(weights), _stream()))
    return ids, weights


def route_weights(logits, ids, renormalize: bool = True, weights=None):
    torch = _torch()
    T, E = logits.shape
    k = ids.shape[1]
    weights = torch.empty((T, k), dtype=torch.float32, device=logits.device) if weights is None else weights
    _check(_lib.exmoe_route_weights(_ptr(logits), _ptr(ids), T, E, k, int(renormalize), _ptr(weights), _stream()))
    return weights


def group_tokens(ids, E: int, offsets=None, sorted_flat=None, flat_to_sorted=None):
    torch = _torch()
    T, k = ids.shape
    dev = ids.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if offsets is None else offsets
    sorted_flat = torch.empty(T * k, dtype=torch.int32, device=dev) if sorted_flat is None else sorted_flat
    flat_to_sorted = torch.empty(T * k, dtype=torch.int32, device=dev) if flat_to_sorted is None else flat_to_sorted
    nws = _lib.exmoe_group_workspace_bytes(T, k, E)
    ws = torch.empty(max(nws, 4), dtype=torch.uint8, device=dev) if nws else None
    _check(_lib.exmoe_group_tokens(_ptr(ids), T, k, E, _ptr(offsets), _ptr(sorted_flat), _ptr(flat_to_sorted),
                                   _ptr(ws) if ws is not None else None, nws, _stream()))
    return offsets, sorted_flat, flat_to_sorted


def active_experts(offsets) -> list[int]:
    E = offsets.numel() - 1
    buf = (ctypes.c_int32 * E)()
    n = ctypes.c_int(0)
    _check(_lib.exmoe_active_experts(_ptr(offsets), E, ctypes.cast(buf, _vp), ctypes.byref(n), _stream()))
    return [buf[i] for i in range(n.value)]


@dataclass
class ExpertBank:
    """Packed experts in device memory: expert e's blob at base + stride * slot(e)."""
    base: object                 # torch uint8 tensor (kept alive) or raw int pointer
    stride: int
    expert_to_slot: object = None   # torch int32 [E] or None
    base_ptr: Optional[int] = None

    def c(self) -> ExpertBankC:
        base = self.base_ptr if self.base_ptr is not None else self.base.data_ptr()
        e2s = None if self.expert_to_slot is None else (
            self.expert_to_slot if isinstance(self.expert_to_slot, int) else self.expert_to_slot.data_ptr())
        return ExpertBankC(base, self.stride, e2s)


def bank_from_blobs(blobs, device="cuda") -> ExpertBank:
    """Upload a list of packed blobs (numpy uint8) into one device bank, stride rounded to 256 B."""
    torch = _torch()
    nb = blobs[0].nbytes
    stride = (nb + 255) // 256 * 256
    host = np.zeros((len(blobs), stride), dtype=np.uint8)
    for i, b in enumerate(blobs):
        host[i, :nb] = b
    dev = torch.from_numpy(host.reshape(-1)).to(device)
    return ExpertBank(base=dev, stride=stride)


def moe_workspace_bytes(T, H, I, E, k, flags=PATH_AUTO) -> int:
    return _lib.exmoe_moe_workspace_bytes(T, H, I, E, k, flags)


def alloc_workspace(nbytes: int, device="cuda"):
    """Zero-filled workspace: the layer call keeps arrival counters, zero between calls,
    in its first 4096 bytes."""
    torch = _torch()
    return torch.zeros(max(nbytes, 4096), dtype=torch.uint8, device=device)


FLAG_EXPERT_WITHOUT_SLOT = 1
FLAG_ROWS_UNGROUPED = 2


def workspace_flags(workspace, clear: bool = True) -> int:
    """Conditions the expert kernels recorded in a workspace (bit 0: a routed expert had no
    slot); synchronizes the current stream."""
    v = ctypes.c_uint32(0)
    _check(_lib.exmoe_workspace_flags(_ptr(workspace), workspace.numel(), int(clear), ctypes.byref(v), _stream()))
    return v.value


def workspace_rows(workspace, E: int, clear: bool = True) -> np.ndarray:
    """Per-expert counters of routed rows run since the last clear (DEBUG_COUNTERS calls);
    synchronizes the current stream."""
    out = np.empty(E, dtype=np.int32)
    _check(_lib.exmoe_workspace_rows(_ptr(workspace), workspace.numel(), E, int(clear), out.ctypes.data, _stream()))
    return out


def moe_forward(x, ids, weights, offsets, sorted_flat, flat_to_sorted, bank: ExpertBank, I: int,
                flags: int = PATH_AUTO, y=None, workspace=None):
    torch = _torch()
    T, H = x.shape
    k = ids.shape[1]
    E = offsets.numel() - 1
    y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device) if y is None else y
    need = moe_workspace_bytes(T, H, I, E, k, flags)
    workspace = alloc_workspace(need, x.device) if workspace is None else workspace
    bc = bank.c()
    _check(_lib.exmoe_moe_forward(_ptr(x), _ptr(ids), _ptr(weights), _ptr(offsets), _ptr(sorted_flat),
                                  _ptr(flat_to_sorted), ctypes.byref(bc), T, H, I, E, k, flags, _ptr(y),
                                  _ptr(workspace), workspace.numel(), _stream()))
    return y


class LayerBuffers:
    """Preallocated outputs and workspace of one layer call (no allocation per call)."""

    def __init__(self, T, H, I, E, k, flags=PATH_AUTO, device="cuda"):
        torch = _torch()
        self.T, self.H, self.I, self.E, self.k, self.flags = T, H, I, E, k, flags
        self.logits = torch.empty((T, E), dtype=torch.bfloat16, device=device)
        self.ids = torch.empty((T, k), dtype=torch.int32, device=device)
        self.weights = torch.empty((T, k), dtype=torch.float32, device=device)
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=device)
        self.sorted_flat = torch.empty(max(T * k, 1), dtype=torch.int32, device=device)
        self.flat_to_sorted = torch.empty(max(T * k, 1), dtype=torch.int32, device=device)
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.workspace = alloc_workspace(_lib.exmoe_moe_layer_workspace_bytes(T, H, I, E, k, flags), device)


def moe_layer(x, w_router, bank: ExpertBank, I: int, k: int, bias=None, renormalize: bool = True,
              flags: int = PATH_AUTO, buffers: Optional[LayerBuffers] = None, stream: Optional[int] = None):
    """route + group + experts in one call; returns the LayerBuffers holding every output."""
    T, H = x.shape
    E = w_router.shape[0]
    b = buffers or LayerBuffers(T, H, I, E, k, flags, x.device)
    bc = bank.c()
    _check(_lib.exmoe_moe_layer(_ptr(x), _ptr(w_router), _ptr(bias), ctypes.byref(bc), T, H, I, E, k,
                                int(renormalize), flags, _ptr(b.logits), _ptr(b.ids), _ptr(b.weights), _ptr(b.offsets),
                                _ptr(b.sorted_flat), _ptr(b.flat_to_sorted), _ptr(b.y), _ptr(b.workspace),
                                b.workspace.numel(), _stream() if stream is None else stream))
    return b


def moe_layer_noalloc(x, w_router, bank: ExpertBank, I: int, k: int, buffers: LayerBuffers, bias=None,
                      renormalize: bool = True, flags: int = PATH_AUTO):
    """moe_layer without a workspace (the library's fixed per-GPU array serves as one):
    every output goes to the preallocated `buffers` (its workspace is not used)."""
    T, H = x.shape
    E = w_router.shape[0]
    b = buffers
    bc = bank.c()
    _check(_lib.exmoe_moe_layer_noalloc(_ptr(x), _ptr(w_router), _ptr(bias), ctypes.byref(bc), T, H, I, E, k,
                                        int(renormalize), flags, _ptr(b.logits), _ptr(b.ids), _ptr(b.weights),
                                        _ptr(b.offsets), _ptr(b.sorted_flat), _ptr(b.flat_to_sorted), _ptr(b.y),
                                        _stream()))
    return b


# ----------------------------------------------------------------------------- grouped products
def _dtype_code(dtype) -> int:
    global _DTYPE_CODES
    if _DTYPE_CODES is None:
        torch = _torch()
        _DTYPE_CODES = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16, torch.float32: DTYPE_FP32}
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}: bfloat16, float16 or float32")
    return code


_DTYPE_CODES = None


def _rows_ld(name: str, t, ndim: int = 2) -> int:
    """Elements between the rows of a GPU tensor whose last axis is contiguous."""
    stride, shape = t.stride(), t.shape
    if len(stride) != ndim:
        raise ValueError(f"{name} must have {ndim} axes (got shape {tuple(shape)})")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return stride[-2] if shape[-2] > 1 else shape[-1]   # (the stride of a single row means nothing)


def _int32(name: str, t, dev: int, numel: Optional[int] = None):
    if t is None:
        return None
    if t.dtype is not (_TORCH or _torch()).int32 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on GPU {dev}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} entries (got {t.numel()})")
    return t.data_ptr()


def _result(name: str, out, shape, dtype, dev: int, like):
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    if out.shape != shape or out.dtype is not dtype or out.get_device() != dev:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype} on GPU {dev}")
    return out


def _scratch(workspace, need, dev: int):
    """(pointer, bytes, tensor) of the caller's workspace, or of a new one of need() bytes."""
    if workspace is None:
        n = need()
        if not n:
            return None, 0, None
        workspace = _torch().empty(n, dtype=_torch().uint8, device=f"cuda:{dev}")
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on GPU {dev}")
    return workspace.data_ptr(), workspace.nbytes, workspace


def _run_on(dev: int, fn, *args):
    """Calls a C entry point on GPU dev, on that device's current stream."""
    torch = _TORCH or _torch()
    if dev == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st)


def _same(name: str, t, dtype, dev: int):
    if t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} on GPU {dev}")


def _no_gradient():
    if _torch().is_grad_enabled():
        raise ValueError("a tensor requires a gradient, and this call records none: pass it detached or call under "
                         "torch.no_grad() (an autograd function around grouped_mm calls grouped_mm_dgrad and grouped_mm_wgrad)")


def grouped_mm_workspace_bytes(op: int, rows: int, N: int, K: int, E: int, k: int = 0) -> int:
    return _lib.exmoe_grouped_mm_workspace_bytes(op, rows, N, K, E, k)


def grouped_mm(x, w, offsets, row_index=None, row_div: int = 1, out_dtype=None, y=None, workspace=None):
    """y[s, :] = w[e] @ x[src(s), :] for the rows s of every expert's segment.

    x [x_rows, K], w [E, N, K] (both bf16 or both fp16, last axis contiguous), offsets int32
    [E + 1]; row_index int32 [rows] with src(s) = row_index[s] // row_div (sorted_flat and k
    of a routed batch), or None for src(s) = s. Returns y [rows, N] in out_dtype (x's type
    or fp32); its rows outside every segment are left as they are. Records no gradient: tensors
    that require one are refused unless gradients are off."""
    if x.requires_grad or w.requires_grad or y is not None and y.requires_grad:
        _no_gradient()
    ldx, ldw = _rows_ld("x", x), _rows_ld("w", w, 3)
    dev, dtype = x.get_device(), x.dtype
    _same("w", w, dtype, dev)
    E, N, K = w.shape
    x_rows, x_cols = x.shape
    if x_cols != K:
        raise ValueError(f"x has {x_cols} columns, w takes {K}")
    rows = x_rows if row_index is None else row_index.numel()
    out_dtype = dtype if out_dtype is None else out_dtype
    y = _result("y", y, (rows, N), out_dtype, dev, x)
    ws, ws_bytes, _keep = _scratch(workspace, lambda: grouped_mm_workspace_bytes(GROUPED_MM, rows, N, K, E), dev)
    _run_on(dev, _lib.exmoe_grouped_mm, x.data_ptr(), ldx, x_rows, _int32("row_index", row_index, dev), row_div,
            _int32("offsets", offsets, dev, E + 1), w.data_ptr(), ldw, w.stride(0), rows, N, K, E,
            _dtype_code(dtype), _dtype_code(out_dtype), y.data_ptr(), _rows_ld("y", y), ws, ws_bytes)
    return y


def grouped_mm_dgrad(dy, w, offsets, flat_to_sorted=None, k: int = 1, out_dtype=None, dx=None, workspace=None):
    """Gradient of grouped_mm with respect to x: dx[s, :] = dy[s, :] @ w[e] per row, or, with
    flat_to_sorted int32 [T * k], summed over the k rows of each token (dx [T, K]). Records no
    gradient, as grouped_mm."""
    if dy.requires_grad or w.requires_grad or dx is not None and dx.requires_grad:
        _no_gradient()
    lddy, ldw = _rows_ld("dy", dy), _rows_ld("w", w, 3)
    dev, dtype = dy.get_device(), dy.dtype
    _same("w", w, dtype, dev)
    E, N, K = w.shape
    rows, dy_cols = dy.shape
    if dy_cols != N:
        raise ValueError(f"dy has {dy_cols} columns, w gives {N}")
    if flat_to_sorted is not None and (k < 1 or rows % k):
        raise ValueError(f"dy's {rows} rows are no multiple of k = {k}")
    out_dtype = dtype if out_dtype is None else out_dtype
    dx = _result("dx", dx, (rows if flat_to_sorted is None else rows // k, K), out_dtype, dev, dy)
    ws, ws_bytes, _keep = _scratch(
        workspace, lambda: grouped_mm_workspace_bytes(GROUPED_DGRAD, rows, N, K, E, 0 if flat_to_sorted is None else k), dev)
    _run_on(dev, _lib.exmoe_grouped_mm_dgrad, dy.data_ptr(), lddy, _int32("offsets", offsets, dev, E + 1), w.data_ptr(),
            ldw, w.stride(0), _int32("flat_to_sorted", flat_to_sorted, dev, rows), k, rows, N, K, E,
            _dtype_code(dtype), _dtype_code(out_dtype), dx.data_ptr(), _rows_ld("dx", dx), ws, ws_bytes)
    return dx


def grouped_mm_wgrad(dy, x, offsets, row_index=None, row_div: int = 1, out_dtype=None, dw=None, workspace=None):
    """Gradient of grouped_mm with respect to w: dw[e] = sum over its rows of dy[s]^T x[src(s)],
    zeros for an expert without rows. out_dtype defaults to fp32. Records no gradient, as
    grouped_mm."""
    if dy.requires_grad or x.requires_grad or dw is not None and dw.requires_grad:
        _no_gradient()
    lddy, ldx = _rows_ld("dy", dy), _rows_ld("x", x)
    dev, dtype = dy.get_device(), dy.dtype
    _same("x", x, dtype, dev)
    rows, N = dy.shape
    x_rows, K = x.shape
    E = offsets.numel() - 1
    if row_index is None and x_rows < rows:
        raise ValueError(f"x has {x_rows} rows, dy has {rows}")
    out_dtype = _torch().float32 if out_dtype is None else out_dtype
    dw = _result("dw", dw, (E, N, K), out_dtype, dev, x)
    lddw = _rows_ld("dw", dw, 3)
    ws, ws_bytes, _keep = _scratch(workspace, lambda: grouped_mm_workspace_bytes(GROUPED_WGRAD, rows, N, K, E), dev)
    _run_on(dev, _lib.exmoe_grouped_mm_wgrad, dy.data_ptr(), lddy, x.data_ptr(), ldx, x_rows,
            _int32("row_index", row_index, dev, rows), row_div, _int32("offsets", offsets, dev, E + 1), rows, N, K, E,
            _dtype_code(dtype), _dtype_code(out_dtype), dw.data_ptr(), lddw, dw.stride(0), ws, ws_bytes)
    return dw


# ----------------------------------------------------------------------------- low-rank adapters
class LoraBank:
    """Low-rank adapters in device memory: a [L, R, K], b [L, N, R] (16-bit, last axis
    contiguous), ranks int32 [L] (None: all R) and scales fp32 [L] (None: all 1)."""

    def __init__(self, a, b, ranks=None, scales=None):
        lda, ldb = _rows_ld("a", a, 3), _rows_ld("b", b, 3)
        dev = a.get_device()
        _same("b", b, a.dtype, dev)
        if a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise ValueError(f"a {tuple(a.shape)} and b {tuple(b.shape)} must be [L, R, K] and [L, N, R]")
        L, R, self.K = a.shape
        self.N = b.shape[1]
        if scales is not None and (scales.dtype is not _torch().float32 or scales.get_device() != dev
                                   or not scales.is_contiguous() or scales.numel() != L):
            raise ValueError(f"scales must be a contiguous float32 tensor of {L} on GPU {dev}")
        self.a, self.b, self.ranks, self.scales = a, b, ranks, scales      # kept alive
        self.c = LoraBankC(a.data_ptr(), lda, a.stride(0), b.data_ptr(), ldb, b.stride(0),
                           _int32("ranks", ranks, dev, L), _ptr(scales), L, R)
        self.ref = ctypes.byref(self.c)


def lora_workspace_bytes(T: int, N: int, K: int, adapters: int, rank_max: int) -> int:
    return _lib.exmoe_lora_workspace_bytes(T, N, K, adapters, rank_max)


def lora_linear(x, w, bank: LoraBank, ids, y=None, workspace=None):
    """y[t] = w @ x[t] + scale * b[id] @ (a[id] @ x[t]) with id = ids[t] (int32 [T]; outside
    [0, L): no adapter). w [N, K], or None: the adapters' part is added to y in place. Records no
    gradient: tensors that require one are refused unless gradients are off."""
    if (x.requires_grad or bank.a.requires_grad or bank.b.requires_grad or w is not None and w.requires_grad
            or y is not None and y.requires_grad):
        _no_gradient()
    ldx = _rows_ld("x", x)
    T, K = x.shape
    dev, dtype = x.get_device(), x.dtype
    _same("bank", bank.a, dtype, dev)
    N = bank.N
    if bank.K != K:
        raise ValueError(f"x has {K} columns, the adapters take {bank.K}")
    if w is None:
        if y is None:
            raise ValueError("without w, y must be given (it is added to)")
        wp, ldw = None, 0
    else:
        wp, ldw = w.data_ptr(), _rows_ld("w", w)
        _same("w", w, dtype, dev)
        if w.shape != (N, K):
            raise ValueError(f"w must be {(N, K)} (got {tuple(w.shape)})")
    y = _result("y", y, (T, N), dtype, dev, x)
    ws, ws_bytes, _keep = _scratch(workspace, lambda: lora_workspace_bytes(T, N, K, bank.c.adapters, bank.c.rank_max), dev)
    _run_on(dev, _lib.exmoe_lora_linear, x.data_ptr(), ldx, wp, ldw, bank.ref, _int32("ids", ids, dev, T), T, N, K,
            _dtype_code(dtype), y.data_ptr(), _rows_ld("y", y), ws, ws_bytes)
    return y


# ----------------------------------------------------------------------------- experts in 8 bits
# Argument structs of exmoe.h: pointers and sizes, then ints. (One bytes object per call: ctypes
# spends about 0.1 us on each argument of its own.)
_NORM = struct.Struct("13Qf5i")
_FP8_ROWS = struct.Struct("8Q4i")
_FP8_MATRICES = struct.Struct("9Q4i")
_GROUPED_FP8 = struct.Struct("14Q7i4x")
_BALANCE = struct.Struct("9Q5i4x")
_LAYER_FP8 = struct.Struct("16Qf6i4x")


def _wrong(name: str, t, shape, dtype, dev: int):
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape:
        raise ValueError(f"{name}: the last axis must be contiguous")
    raise ValueError(f"{name} must be {tuple(shape)} {dtype} on GPU {dev} (got {tuple(t.shape)} {t.dtype})")


def _mat(name: str, t, shape, dtype, dev: int):
    """(pointer, elements between rows) of a matrix of this shape and type on GPU dev, last axis contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _wrong(name, t, shape, dtype, dev)
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        _wrong(name, t, shape, dtype, dev)
    return t.data_ptr(), ld if shape[0] > 1 else shape[1]   # (the stride of a single row means nothing)


def _mats(name: str, t, shape, dtype, dev: int):
    """(pointer, elements between rows, between experts) of one matrix per expert."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _wrong(name, t, shape, dtype, dev)
    stride, ld, one = t.stride()
    if one != 1 and shape[2] > 1:
        _wrong(name, t, shape, dtype, dev)
    return t.data_ptr(), ld if shape[1] > 1 else shape[2], stride


def _axes(name: str, t, n: int):
    """The shape of a tensor of n axes."""
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{name} must have {n} axes (got shape {tuple(shape)})")
    return shape


def _on_gpu(name: str, t) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return dev


def _f8_outputs(q, scale, rows: int, K: int, dev: int, like):
    """The given outputs, or new ones (q with rows of a multiple of 16 bytes, as the product reads
    them), and their pointers and strides."""
    torch = _TORCH or _torch()
    if q is None:
        q = like.new_empty((rows, (K + 15) // 16 * 16), dtype=torch.float8_e4m3fn)[:, :K]
    elif q.requires_grad:
        _no_gradient()
    if scale is None:
        scale = like.new_empty((rows, (K + 127) // 128), dtype=torch.float32)
    elif scale.requires_grad:
        _no_gradient()
    return q, scale, (_mat("q", q, (rows, K), torch.float8_e4m3fn, dev)
                      + _mat("scale", scale, (rows, (K + 127) // 128), torch.float32, dev))


class NormOutputs(NamedTuple):
    """What rms_norm wrote (None: not asked for)."""
    y: object          # [T, H] of x's type
    q: object          # [T, H] float8_e4m3fn
    scale: object      # [T, ceil(H / 128)] float32
    residual: object   # [T, H]: x + residual


def rms_norm(x, w, eps: float = 1e-6, residual=None, out: str = "y", y=None, q=None, scale=None, residual_out=None) -> NormOutputs:
    """y = h / sqrt(mean(h^2) + eps) * w over the rows of h = x + residual (or x).

    x [T, H] (bf16, fp16 or fp32), w [H] and residual [T, H] of x's type or fp32. out: "y" (x's
    type), "fp8" (e4m3 q with a scale per 128 columns) or "both". h is rounded to the residual's type
    and written to residual_out (a new tensor, or the residual itself). Records no gradient."""
    if (x.requires_grad or w.requires_grad or residual is not None and (residual.requires_grad or residual_out is not None
                                                                        and residual_out.requires_grad)
            or y is not None and y.requires_grad):
        _no_gradient()
    dev, dtype = _on_gpu("x", x), x.dtype
    T, H = shape = _axes("x", x, 2)
    px, ldx = _mat("x", x, shape, dtype, dev)
    if w.shape != (H,) or w.get_device() != dev or not w.is_contiguous():
        raise ValueError(f"w must be a contiguous tensor of {H} on GPU {dev}")
    pr = ldr = po = ldo = py = ldy = res_code = 0
    f8 = (0, 0, 0, 0)
    if residual is not None:
        res_dtype = residual.dtype
        pr, ldr = _mat("residual", residual, shape, res_dtype, dev)
        res_code = _dtype_code(res_dtype)
        if residual_out is None:
            residual_out = residual.new_empty(shape)
        po, ldo = _mat("residual_out", residual_out, shape, res_dtype, dev)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if out == "y" or out == "both":
        if y is None:
            y = x.new_empty(shape)
        py, ldy = _mat("y", y, shape, dtype, dev)
    elif out != "fp8":
        raise ValueError(f'out must be "y", "fp8" or "both" (got {out!r})')
    elif y is not None:
        raise ValueError('y with out="fp8"')
    if out != "y":
        q, scale, f8 = _f8_outputs(q, scale, T, H, dev, x)
    elif q is not None or scale is not None:
        raise ValueError('q or scale with out="y"')
    _run_on(dev, _lib.exmoe_rms_norm, _NORM.pack(px, ldx, w.data_ptr(), pr, ldr, po, ldo, py, ldy, *f8, eps, T, H,
                                                 _dtype_code(dtype), _dtype_code(w.dtype), res_code))
    return NormOutputs(y, q, scale, residual_out)


def _row_weights(weights, dev: int):
    """(pointer, number) of the rows' weights."""
    if weights.dtype is not _torch().float32 or weights.get_device() != dev or not weights.is_contiguous():
        raise ValueError(f"weights must be a contiguous float32 tensor on GPU {dev}")
    return weights.data_ptr(), weights.numel()


def quantize_fp8(x, q=None, scale=None, weights=None, row_index=None):
    """(q, scale) of x [rows, K] (bf16, fp16 or fp32): e4m3 with a scale per 128 columns of a row; weights
    and row_index as in swiglu_fp8."""
    if x.requires_grad or weights is not None and weights.requires_grad:
        _no_gradient()
    dev, dtype = _on_gpu("x", x), x.dtype
    rows, K = shape = _axes("x", x, 2)
    px, ldx = _mat("x", x, shape, dtype, dev)
    pw, n = (0, 0) if weights is None else _row_weights(weights, dev)
    pi = 0 if row_index is None else _int32("row_index", row_index, dev, rows)
    q, scale, f8 = _f8_outputs(q, scale, rows, K, dev, x)
    _run_on(dev, _lib.exmoe_quantize_fp8, _FP8_ROWS.pack(px, ldx, pw, pi, *f8, n, rows, K, _dtype_code(dtype)))
    return q, scale


def swiglu_fp8(gate_up, weights=None, row_index=None, q=None, scale=None):
    """(q, scale) of silu(gate) * up [rows, I], gate_up [rows, 2 I] with the gate's columns first.
    weights fp32 (any shape, contiguous): row r's scales are multiplied by weights.view(-1)[row_index[r]]
    (row_index int32 [rows]: sorted_flat of a routed batch), or by its r-th without row_index."""
    if gate_up.requires_grad or weights is not None and weights.requires_grad:
        _no_gradient()
    dev, dtype = _on_gpu("gate_up", gate_up), gate_up.dtype
    rows, cols = shape = _axes("gate_up", gate_up, 2)
    px, ldx = _mat("gate_up", gate_up, shape, dtype, dev)
    if cols % 2:
        raise ValueError(f"gate_up has {cols} columns: gate and up side by side are an even number")
    pw, n = (0, 0) if weights is None else _row_weights(weights, dev)
    I = cols // 2
    q, scale, f8 = _f8_outputs(q, scale, rows, I, dev, gate_up)
    _run_on(dev, _lib.exmoe_swiglu_fp8, _FP8_ROWS.pack(px, ldx, pw, _int32("row_index", row_index, dev, rows) or 0, *f8, n, rows,
                                                       I, _dtype_code(dtype)))
    return q, scale


def quantize_fp8_weights(w, q=None, scale=None):
    """(q, scale) of w [E, N, K] (bf16, fp16 or fp32): e4m3 with a scale per 128 x 128 block, scale
    fp32 [E, ceil(N / 128), ceil(K / 128)]."""
    if w.requires_grad or q is not None and q.requires_grad or scale is not None and scale.requires_grad:
        _no_gradient()
    torch = _torch()
    dev, dtype = _on_gpu("w", w), w.dtype
    E, N, K = shape = _axes("w", w, 3)
    pw = _mats("w", w, shape, dtype, dev)
    blocks = (E, (N + 127) // 128, (K + 127) // 128)
    if q is None:
        q = w.new_empty((E, N, (K + 15) // 16 * 16), dtype=torch.float8_e4m3fn)[..., :K]
    if scale is None:
        scale = w.new_empty(blocks, dtype=torch.float32)
    _run_on(dev, _lib.exmoe_quantize_fp8_weights, _FP8_MATRICES.pack(*pw, *_mats("q", q, shape, torch.float8_e4m3fn, dev),
                                                                     *_mats("scale", scale, blocks, torch.float32, dev), E, N, K,
                                                                     _dtype_code(dtype)))
    return q, scale


def grouped_mm_fp8(x, x_scale, w, w_scale, offsets=None, row_index=None, row_div: int = 1, out_dtype=None, y=None):
    """grouped_mm on 8-bit operands: y[s, :] = (w[e] * w_scale[e]) @ (x * x_scale)[src(s), :].

    x [x_rows, K] and w [E, N, K] float8_e4m3fn with 16-byte aligned rows, K a multiple of 16;
    x_scale fp32 [x_rows, ceil(K / 128)], w_scale fp32 [E, ceil(N / 128), ceil(K / 128)]; offsets,
    row_index and row_div as in grouped_mm, offsets None for one expert with every row. Returns y
    [rows, N] in out_dtype (bf16, the default, fp16 or fp32); rows outside every segment are left
    as they are. 16-bit outputs may lose small products beside large ones of the same 8 positions
    (7 x 2^-13 of the largest one of them), 32-bit outputs lose none."""
    if (x.requires_grad or w.requires_grad or x_scale.requires_grad or w_scale.requires_grad
            or y is not None and y.requires_grad):
        _no_gradient()
    torch = _TORCH or _torch()
    dev, f8, f32 = _on_gpu("x", x), torch.float8_e4m3fn, torch.float32
    E, N, K = shape = _axes("w", w, 3)
    pw, ldw, sw = _mats("w", w, shape, f8, dev)
    rows, cols = shape = _axes("x", x, 2)
    if cols != K:
        raise ValueError(f"x has {cols} columns, w takes {K}")
    px, ldx = _mat("x", x, shape, f8, dev)
    kb, x_rows, pi, pf = (K + 127) // 128, rows, 0, 0
    pxs, ldxs = _mat("x_scale", x_scale, (rows, kb), f32, dev)
    pws, ldws, sws = _mats("w_scale", w_scale, (E, (N + 127) // 128, kb), f32, dev)
    if row_index is not None:
        rows, pi = row_index.numel(), _int32("row_index", row_index, dev)
    if offsets is not None:
        pf = _int32("offsets", offsets, dev, E + 1)
    if out_dtype is None:
        out_dtype = torch.bfloat16
    if y is None:
        y = x.new_empty((rows, N), dtype=out_dtype)
    py, ldy = _mat("y", y, (rows, N), out_dtype, dev)
    _run_on(dev, _lib.exmoe_grouped_mm_fp8, _GROUPED_FP8.pack(px, ldx, pxs, ldxs, pi, pf, pw, ldw, sw, pws, ldws, sws, py, ldy,
                                                              x_rows, row_div, rows, N, K, E, _dtype_code(out_dtype)))
    return y


class Fp8Experts:
    """Experts in 8 bits: gate_up [E, 2 I, H] (gate's rows first) and down [E, H, I] in bf16, fp16 or fp32,
    quantised here (quantize_fp8_weights)."""

    def __init__(self, gate_up, down):
        E, rows, H = _axes("gate_up", gate_up, 3)
        if rows % 2 or tuple(down.shape) != (E, H, rows // 2):
            raise ValueError(f"gate_up {tuple(gate_up.shape)} and down {tuple(down.shape)} must be [E, 2 I, H] and [E, H, I]")
        if gate_up.device != down.device:
            raise ValueError(f"gate_up and down must be on the same device (got {gate_up.device} and {down.device})")
        self.E, self.H, self.I = E, H, rows // 2
        if H % 128 or self.I % 128:
            raise ValueError(f"H and I must be multiples of 128 (got {H}, {self.I})")
        self.gate_up, self.gate_up_scale = quantize_fp8_weights(gate_up)
        self.down, self.down_scale = quantize_fp8_weights(down)


class Fp8LayerBuffers:
    """Preallocated outputs and workspace of a moe_layer_fp8 call (no allocation per call)."""

    def __init__(self, T, H, I, E, k, device="cuda"):
        torch = _torch()
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.logits = torch.empty((T, E), dtype=torch.bfloat16, device=device)
        self.ids = torch.empty((T, k), dtype=torch.int32, device=device)
        self.weights = torch.empty((T, k), dtype=torch.float32, device=device)
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=device)
        self.sorted_flat = torch.empty(max(T * k, 1), dtype=torch.int32, device=device)
        self.flat_to_sorted = torch.empty(max(T * k, 1), dtype=torch.int32, device=device)
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.workspace = torch.empty(max(_lib.exmoe_moe_layer_fp8_workspace_bytes(T, H, I, E, k), 16), dtype=torch.uint8, device=device)


def moe_layer_fp8(x, w_norm, w_router, experts: Fp8Experts, k: int, residual=None, bias=None, eps: float = 1e-6,
                  renormalize: bool = True, buffers: Optional[Fp8LayerBuffers] = None) -> Fp8LayerBuffers:
    """residual += x (in place, or without one), its norm, routing, grouping and the experts in 8 bits in
    one call; returns the Fp8LayerBuffers holding every output. x and residual bf16 [T, H], w_norm bf16 [H],
    w_router bf16 [E, H], bias fp32 [E], all contiguous. Records no gradient."""
    for t in (x, w_norm, w_router, residual, bias):
        if t is not None and t.requires_grad:
            _no_gradient()
    torch = _torch()
    dev, bf16 = _on_gpu("x", x), torch.bfloat16
    T, H = _axes("x", x, 2)
    E, I, f8, f32 = experts.E, experts.I, torch.float8_e4m3fn, torch.float32
    held = experts.gate_up, experts.gate_up_scale, experts.down, experts.down_scale   # (a program may have put others there)
    if any(t.requires_grad for t in held):
        _no_gradient()
    for name, t, shape, dtype in (("x", x, (T, experts.H), bf16), ("w_norm", w_norm, (H,), bf16), ("w_router", w_router, (E, H), bf16),
                                  ("residual", residual, (T, H), bf16), ("bias", bias, (E,), f32),
                                  ("experts.gate_up", held[0], (E, 2 * I, H), f8),
                                  ("experts.gate_up_scale", held[1], (E, 2 * I // 128, H // 128), f32),
                                  ("experts.down", held[2], (E, H, I), f8),
                                  ("experts.down_scale", held[3], (E, H // 128, I // 128), f32)):
        if t is not None and (t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on GPU {dev} (got {tuple(t.shape)} {t.dtype})")
    b = buffers or Fp8LayerBuffers(T, H, I, E, k, x.device)
    if (b.T, b.H, b.I, b.E, b.k) != (T, H, I, E, k) or b.y.get_device() != dev:
        raise ValueError(f"buffers are of another call: {(b.T, b.H, b.I, b.E, b.k)}, not {(T, H, I, E, k)} on GPU {dev}")
    _run_on(dev, _lib.exmoe_moe_layer_fp8,
            _LAYER_FP8.pack(x.data_ptr(), w_norm.data_ptr(), _ptr(residual) or 0, w_router.data_ptr(), _ptr(bias) or 0,
                            *(t.data_ptr() for t in held), b.logits.data_ptr(), b.ids.data_ptr(), b.weights.data_ptr(),
                            b.offsets.data_ptr(), b.sorted_flat.data_ptr(), b.flat_to_sorted.data_ptr(), b.y.data_ptr(), eps, T, H, I,
                            E, k, int(renormalize)), b.workspace.data_ptr(), b.workspace.numel())
    return b


# ----------------------------------------------------------------------------- router losses
def _mask(mask, T: int, dev: int) -> int:
    if mask is None:
        return 0
    if mask.dtype not in (_torch().bool, _torch().uint8) or mask.get_device() != dev or not mask.is_contiguous() or mask.numel() != T:
        raise ValueError(f"mask must be a contiguous bool tensor of {T} on GPU {dev}")
    return mask.data_ptr()


def balance_loss_workspace_bytes(T: int, E: int) -> int:
    return _lib.exmoe_balance_loss_workspace_bytes(T, E)


def balance_loss(logits, ids, mask=None, losses=None, counts=None, workspace=None):
    """(losses fp32 [2], counts int32 [E + 1]) of router logits [T, E] (bf16, fp16 or fp32) and their
    top-k ids int32 [T, k], over the tokens whose mask (bool [T]; None: all) is set: losses[0] = E
    sum_e f_e P_e (f: share of the routed pairs, P: mean probability), losses[1] = mean squared
    log-sum-exp, counts: pairs per expert, then the number of tokens. Records no gradient: an autograd
    function around it calls balance_loss_backward."""
    if logits.requires_grad or losses is not None and losses.requires_grad:
        _no_gradient()
    torch = _torch()
    dev, dtype = _on_gpu("logits", logits), logits.dtype
    T, E = shape = _axes("logits", logits, 2)
    pl, ldl = _mat("logits", logits, shape, dtype, dev)
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids must be [{T}, k] (got {tuple(ids.shape)})")
    losses = _result("losses", losses, (2,), torch.float32, dev, logits)
    counts = _result("counts", counts, (E + 1,), torch.int32, dev, logits)
    if not losses.is_contiguous() or not counts.is_contiguous():
        raise ValueError("losses and counts must be contiguous")
    ws, ws_bytes, _keep = _scratch(workspace, lambda: balance_loss_workspace_bytes(T, E), dev)
    _run_on(dev, _lib.exmoe_balance_loss, _BALANCE.pack(pl, ldl, _int32("ids", ids, dev), _mask(mask, T, dev), losses.data_ptr(),
                                                        counts.data_ptr(), 0, 0, 0, T, E, ids.shape[1], _dtype_code(dtype), 0),
            ws, ws_bytes)
    return losses, counts


def balance_loss_backward(logits, counts, k: int, grad_losses, mask=None, out_dtype=None, dlogits=None):
    """Gradient of grad_losses[0] * losses[0] + grad_losses[1] * losses[1] (fp32 [2], on the GPU) with
    respect to logits: [T, E] in out_dtype (logits' type, the default, or fp32). counts: what
    balance_loss returned. dlogits may be logits itself."""
    if logits.requires_grad or grad_losses.requires_grad or dlogits is not None and dlogits.requires_grad:
        _no_gradient()
    dev, dtype = _on_gpu("logits", logits), logits.dtype
    T, E = shape = _axes("logits", logits, 2)
    pl, ldl = _mat("logits", logits, shape, dtype, dev)
    if (grad_losses.dtype is not _torch().float32 or grad_losses.get_device() != dev or not grad_losses.is_contiguous()
            or grad_losses.numel() != 2):
        raise ValueError(f"grad_losses must be a contiguous float32 tensor of 2 on GPU {dev}")
    if out_dtype is None:
        out_dtype = dtype
    if dlogits is None:
        dlogits = logits.new_empty(shape, dtype=out_dtype)
    pd, ldd = _mat("dlogits", dlogits, shape, out_dtype, dev)
    _run_on(dev, _lib.exmoe_balance_loss_backward,
            _BALANCE.pack(pl, ldl, 0, _mask(mask, T, dev), 0, _int32("counts", counts, dev, E + 1), grad_losses.data_ptr(), pd, ldd, T,
                          E, k, _dtype_code(dtype), _dtype_code(out_dtype)))
    return dlogits


# ----------------------------------------------------------------------------- slot cache
def moe_forward_cached(x, ids, weights, offsets, sorted_flat, flat_to_sorted, cache: "SlotCache", layer: int,
                       active, I: int, flags: int = PATH_AUTO, y=None, workspace=None):
    """Expert layer through a slot cache in cache-sized waves (active: every routed expert id)."""
    torch = _torch()
    T, H = x.shape
    k = ids.shape[1]
    E = offsets.numel() - 1
    y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device) if y is None else y
    need = moe_workspace_bytes(T, H, I, E, k, flags)
    workspace = alloc_workspace(need, x.device) if workspace is None else workspace
    arr = (ctypes.c_int32 * max(len(active), 1))(*[int(e) for e in active])
    _check(_lib.exmoe_moe_forward_cached(_ptr(x), _ptr(ids), _ptr(weights), _ptr(offsets), _ptr(sorted_flat),
                                         _ptr(flat_to_sorted), cache._h, layer, ctypes.cast(arr, _vp), len(active),
                                         T, H, I, E, k, flags, _ptr(y), _ptr(workspace), workspace.numel(),
                                         _stream()))
    return y


class SlotCache:
    """GPU slot cache over a pinned host pool (policy in C++, copies on a side stream)."""

    def __init__(self, layers: int, E: int, slots: int, expert_bytes: int, dry_run: bool = False):
        h = _vp()
        _check(_lib.exmoe_slot_cache_create(layers, E, slots, expert_bytes, CACHE_DRY_RUN if dry_run else 0,
                                            ctypes.byref(h)))
        self._h = h
        self.dry_run = dry_run
        self.layers, self.E, self.slots, self.expert_bytes = layers, E, slots, expert_bytes

    def host_slot(self, layer: int, expert: int) -> int:
        p = _vp()
        _check(_lib.exmoe_slot_cache_host_slot(self._h, layer, expert, ctypes.byref(p)))
        return p.value

    def fill(self, layer: int, expert: int, blob: np.ndarray):
        ctypes.memmove(self.host_slot(layer, expert), blob.ctypes.data, blob.nbytes)

    def preload(self):
        _check(_lib.exmoe_slot_cache_preload(self._h, _stream()))

    def acquire(self, layer: int, active) -> ExpertBank:
        arr = (ctypes.c_int32 * max(len(active), 1))(*[int(e) for e in active])
        bc = ExpertBankC()
        _check(_lib.exmoe_slot_cache_acquire(self._h, layer, ctypes.cast(arr, _vp), len(active),
                                             None if self.dry_run else _stream(), ctypes.byref(bc)))
        return ExpertBank(base=None, stride=bc.stride, expert_to_slot=bc.expert_to_slot, base_ptr=bc.base)

    def waves(self, layer: int, active, run: bool = False):
        """The cache-sized waves a cached forward on `layer` would run: list of id lists.
        run=True (dry-run caches only) also looks the waves up, as that forward does."""
        arr = (ctypes.c_int32 * max(len(active), 1))(*[int(e) for e in active])
        order = np.empty(max(len(active), 1), dtype=np.int32)
        n, w = _i(0), _i(0)
        _check(_lib.exmoe_slot_cache_waves(self._h, layer, ctypes.cast(arr, _vp), len(active), int(run),
                                           order.ctypes.data, ctypes.byref(n), ctypes.byref(w)))
        ids = order[:n.value].tolist()
        return [ids[i:i + w.value] for i in range(0, len(ids), w.value)] if ids else []

    def table(self, layer: int) -> np.ndarray:
        out = np.empty(self.E, dtype=np.int32)
        _check(_lib.exmoe_slot_cache_table(self._h, layer, out.ctypes.data))
        return out

    def stats(self) -> dict:
        s = CacheStatsC()
        _check(_lib.exmoe_slot_cache_stats(self._h, ctypes.byref(s)))
        return {f: getattr(s, f) for f, _ in CacheStatsC._fields_}

    def reset_stats(self):
        _check(_lib.exmoe_slot_cache_reset_stats(self._h))

    def close(self):
        if self._h:
            _check(_lib.exmoe_slot_cache_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ----------------------------------------------------------------------------- kernel timing
def profile_enable(on: bool = True):
    _check(_lib.exmoe_profile_enable(int(on)))


def profile_reset():
    _check(_lib.exmoe_profile_reset())


def profile_read(kernel: str):
    """(total milliseconds, launches) of one library kernel since the last reset."""
    ms = ctypes.c_double(0.0)
    n = ctypes.c_uint64(0)
    _check(_lib.exmoe_profile_read(kernel.encode(), ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


def span_enable(max_launches: int):
    """Launch span stamps for the next `max_launches` expert-layer kernel launches (0: off)."""
    _check(_lib.exmoe_span_enable(int(max_launches)))


def span_clear():
    """Reset the span stamps, keeping the slots' assignment (replay a graph, then read)."""
    _check(_lib.exmoe_span_clear())


def span_read(kernel: str):
    """(total microseconds, launches) of one kernel's spans since the last clear."""
    us = ctypes.c_double(0.0)
    n = ctypes.c_uint64(0)
    _check(_lib.exmoe_span_read(kernel.encode(), ctypes.byref(us), ctypes.byref(n)))
    return us.value, n.value


def device_copy(dst, src):
    """Plain device copy of src into dst (same byte size, multiple of 16) on the current stream."""
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != n:
        raise ValueError("device_copy: size mismatch")
    _check(_lib.exmoe_device_copy(_vp(dst.data_ptr()), _vp(src.data_ptr()), n, _stream()))

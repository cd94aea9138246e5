"""GPTQ per-layer weight quantization on GB300 — Python binding of libgptq.

Thin ctypes marshalling over the C ABI declared in ``include/gptq.h``: every
function here has the C entry point's name, checks tensor shapes/dtypes/devices,
allocates outputs with PyTorch (device memory and streams only) and calls the
library on the current CUDA stream. All arithmetic runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback — if the library is missing or no
GPU is present, the calls raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, NamedTuple, Optional, Tuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgptq.so")

GPTQ_F32 = 0
GPTQ_BF16 = 1

STATUS = {
    0: "GPTQ_OK", 1: "GPTQ_ERR_INVALID_ARG", 2: "GPTQ_ERR_UNSUPPORTED", 3: "GPTQ_ERR_NOT_SPD",
    4: "GPTQ_ERR_CUDA", 5: "GPTQ_ERR_TIMEOUT", 6: "GPTQ_ERR_WORKSPACE", 7: "GPTQ_ERR_NONFINITE",
}

# every symbol include/gptq.h declares
EXPORTS = [
    "gptq_hessian_create", "gptq_hessian_reset", "gptq_hessian_accumulate", "gptq_hessian_finalize",
    "gptq_hessian_destroy", "gptq_prepare_workspace_bytes", "gptq_prepare", "gptq_prepare_noalloc",
    "gptq_quantize_workspace_bytes",
    "gptq_quantize", "gptq_prune_workspace_bytes", "gptq_prune", "rtn_quantize", "gptq_packed_words_per_row", "gptq_pack", "gptq_dequant_matmul",
    "gptq_fp4_code_pitch", "gptq_fp4_scale_bytes", "gptq_fp4_tensor_scale", "gptq_fp4_quantize", "gptq_fp4_dequantize",
    "gptq_fp4_tile_scales", "gptq_fp4_matmul", "gptq_expert_sort_workspace_bytes", "gptq_expert_sort",
    "gptq_expert_gather", "gptq_expert_combine", "gptq_expert_combine_grad",
    "gptq_int8_pitch", "gptq_int8_quantize", "gptq_int8_dequantize", "gptq_int8_rms_norm",
    "gptq_int8_rms_norm_grad_workspace_bytes", "gptq_int8_rms_norm_grad", "gptq_int8_matmul",
    "gptq_expert_balance_workspace_bytes", "gptq_expert_balance", "gptq_expert_balance_grad",
    "gptq_status_string", "gptq_set_status_mode", "gptq_status_mode", "gptq_status_sync",
    "gptq_launch_count", "gptq_profile_enable", "gptq_profile_read", "gptq_profile_kernel_count",
    "gptq_profile_kernel_name",
]


class GptqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({_str(status)})")


class QConfig(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("group", ctypes.c_int32), ("sym", ctypes.c_int32),
                ("zero_in_range", ctypes.c_int32)]


_lib: Optional[ctypes.CDLL] = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t


def _declare(lib: ctypes.CDLL) -> None:
    sig = {
        "gptq_hessian_create": (_I, [_I64, ctypes.POINTER(_P)]),
        "gptq_hessian_reset": (_I, [_P, _P]),
        "gptq_hessian_accumulate": (_I, [_P, _P, _I, _I64, _I64, _P]),
        "gptq_hessian_finalize": (_I, [_P, _P, _P, ctypes.POINTER(_I64), _P]),
        "gptq_hessian_destroy": (_I, [_P]),
        "gptq_prepare_workspace_bytes": (_SZ, [_I64, _I]),
        "gptq_prepare": (_I, [_P, _P, _I64, _F, _I, _P, _P, _P, _P, _SZ, _P]),
        "gptq_prepare_noalloc": (_I, [_P, _P, _I64, _F, _I, _P, _P, _P, _P]),
        "gptq_quantize_workspace_bytes": (_SZ, [_I64, _I64, QConfig]),
        "gptq_quantize": (_I, [_P, _I64, _I64, _P, _P, _P, QConfig, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
        "rtn_quantize": (_I, [_P, _I64, _I64, _P, QConfig, _P, _P, _P, _P, _P, _P]),
        "gptq_prune_workspace_bytes": (_SZ, [_I64, _I64]),
        "gptq_prune": (_I, [_P, _I64, _I64, _P, _P, _P, _F, _P, _P, _P, _P, _SZ, _P]),
        "gptq_packed_words_per_row": (_I64, [_I64, _I]),
        "gptq_pack": (_I, [_P, _I64, _I64, _I, _I, _P, _P]),
        "gptq_dequant_matmul": (_I, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _I64, _I64, _I, _I, _P, _I64, _P]),
        "gptq_fp4_code_pitch": (_I64, [_I64]),
        "gptq_fp4_scale_bytes": (_I64, [_I64, _I64, _I]),
        "gptq_fp4_tensor_scale": (_I, [_P, _I, _I64, _I64, _I64, _P, _P]),
        "gptq_fp4_quantize": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _I64, _I, _P, _P, _P, _P]),
        "gptq_fp4_dequantize": (_I, [_P, _P, _P, _I64, _I64, _I, _P, _I, _I64, _P]),
        "gptq_fp4_tile_scales": (_I, [_P, _I64, _I64, _I64, _I, _P, _P]),
        "gptq_fp4_matmul": (_I, [_P, _P, _P, _I64, _P, _P, _P, _I64, _I64, _I, _P, _I64, _I, _P, _I64, _P]),
        "gptq_expert_sort_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
        "gptq_expert_sort": (_I, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _SZ, _P]),
        "gptq_expert_gather": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _P]),
        "gptq_expert_combine": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _P, _P, _I64, _P]),
        "gptq_expert_combine_grad": (_I, [_P, _I64, _P, _I64, _I, _I64, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _P, _P]),
        "gptq_int8_pitch": (_I64, [_I64]),
        "gptq_int8_quantize": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _P]),
        "gptq_int8_dequantize": (_I, [_P, _P, _I64, _I64, _P, _I, _I64, _P]),
        "gptq_int8_rms_norm": (_I, [_P, _I64, _P, _I64, _I, _I64, _I64, _P, _F, _P, _P, _P, _I64, _P, _P]),
        "gptq_int8_rms_norm_grad_workspace_bytes": (_SZ, [_I64, _I64]),
        "gptq_int8_rms_norm_grad": (_I, [_P, _I64, _P, _I64, _P, _I64, _I, _I64, _I64, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
        "gptq_int8_matmul": (_I, [_P, _P, _I64, _P, _P, _I64, _I64, _P, _I64, _I, _P, _I64, _P]),
        "gptq_expert_balance_workspace_bytes": (_SZ, [_I64, _I64]),
        "gptq_expert_balance": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _P, _P, _P, _P, _SZ, _P]),
        "gptq_expert_balance_grad": (_I, [_P, _P, _I, _I64, _I64, _I64, _P, _I64, _P, _P, _I64, _P]),
        "gptq_status_string": (ctypes.c_char_p, [_I]),
        "gptq_set_status_mode": (_I, [_I]),
        "gptq_status_mode": (_I, []),
        "gptq_status_sync": (_I, [_P]),
        "gptq_launch_count": (ctypes.c_ulonglong, []),
        "gptq_profile_enable": (None, [_I]),
        "gptq_profile_read": (_I, [_P, _P, _I]),
        "gptq_profile_kernel_count": (_I, []),
        "gptq_profile_kernel_name": (ctypes.c_char_p, [_I]),
        # test hook (exported, deliberately not declared in gptq.h)
        "gptq_test_set_wait_limit_ns": (_I, [ctypes.c_ulonglong]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgptq.so (built in-tree by ``build.py``; the environment variable GPTQ_LIB names
    another build of the same library instead); raises if it is missing."""
    global _lib
    if _lib is None:
        path = os.environ.get("GPTQ_LIB", path)
        if not os.path.exists(path):
            raise RuntimeError(f"libgptq.so not built ({path}); run post_weight_quantization_04_gb300.build")
        lib = ctypes.CDLL(path)
        _declare(lib)
        _setup_call(lib)
        _lib = lib
    return _lib


def _setup_call(lib: ctypes.CDLL) -> None:
    """Hands the C module of the serving calls what it needs: torch's types and the library's entry points."""
    from . import _call
    names = ("gptq_fp4_quantize", "gptq_fp4_dequantize", "gptq_fp4_matmul", "gptq_expert_sort_workspace_bytes",
             "gptq_expert_sort", "gptq_expert_gather", "gptq_expert_combine", "gptq_expert_combine_grad", "gptq_int8_quantize",
             "gptq_int8_dequantize", "gptq_int8_matmul", "gptq_int8_rms_norm", "gptq_int8_rms_norm_grad_workspace_bytes",
             "gptq_int8_rms_norm_grad", "gptq_expert_balance_workspace_bytes", "gptq_expert_balance", "gptq_expert_balance_grad")
    _call.setup({"float32": torch.float32, "bfloat16": torch.bfloat16, "uint8": torch.uint8, "int8": torch.int8, "bool": torch.bool,
                 "int32": torch.int32, "empty": torch.empty, "raw_stream": _current_raw_stream, "current_device": _current_device,
                 "Fp4": Fp4, "Int8": Int8, "Route": Route, "Balance": Balance, "check": _check},
                {n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names})
    globals()["_fast"] = _call


def _str(status: int) -> str:
    try:
        return load().gptq_status_string(status).decode()
    except Exception:  # noqa: BLE001
        return "?"


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise GptqError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t: torch.Tensor, dtype, name: str, shape=None) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def qconfig(bits: int, group: int = 0, sym: bool = True, zero_in_range: bool = False) -> QConfig:
    return QConfig(int(bits), int(group), 1 if sym else 0, 1 if zero_in_range else 0)


def gptq_packed_words_per_row(cols: int, bits: int) -> int:
    return int(load().gptq_packed_words_per_row(cols, bits))


# ------------------------------------------------------------------------------ Hessian

class Hessian:
    """The library's accumulator: S += X^T X over token batches; H = 2 S / n."""

    def __init__(self, d: int, device=None):
        lib = load()
        self.d = int(d)
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check("gptq_hessian_create", lib.gptq_hessian_create(self.d, ctypes.byref(h)))
        self._h = h

    def reset(self, stream=None) -> None:
        _check("gptq_hessian_reset", load().gptq_hessian_reset(self._h, _stream(stream)))

    def accumulate(self, X: torch.Tensor, stream=None) -> None:
        if X.dim() != 2 or X.shape[1] != self.d:
            raise ValueError(f"X must be (n, {self.d})")
        if X.dtype not in (torch.bfloat16, torch.float32) or not X.is_cuda:
            raise ValueError("X must be a CUDA bf16 or fp32 tensor")
        if X.stride(1) != 1:
            raise ValueError("X rows must be contiguous")
        dt = GPTQ_BF16 if X.dtype == torch.bfloat16 else GPTQ_F32
        _check("gptq_hessian_accumulate",
               load().gptq_hessian_accumulate(self._h, _ptr(X), dt, X.shape[0], X.stride(0), _stream(stream)))

    def finalize(self, stream=None) -> Tuple[torch.Tensor, torch.Tensor, int]:
        H = torch.empty(self.d, self.d, dtype=torch.float32, device=self.device)
        diag = torch.empty(self.d, dtype=torch.float32, device=self.device)
        n = ctypes.c_int64(0)
        _check("gptq_hessian_finalize",
               load().gptq_hessian_finalize(self._h, _ptr(H), _ptr(diag), ctypes.byref(n), _stream(stream)))
        return H, diag, int(n.value)

    def close(self) -> None:
        if getattr(self, "_h", None):
            load().gptq_hessian_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001
            pass


def gptq_hessian_create(d: int, device=None) -> Hessian:
    return Hessian(d, device)


def gptq_hessian_accumulate(h: Hessian, X: torch.Tensor, stream=None) -> None:
    h.accumulate(X, stream)


def gptq_hessian_finalize(h: Hessian, stream=None):
    return h.finalize(stream)


# ------------------------------------------------------------------------------ prepare

def gptq_prepare_workspace_bytes(d: int, act_order: bool = False) -> int:
    return int(load().gptq_prepare_workspace_bytes(d, 1 if act_order else 0))


def gptq_prepare(H: torch.Tensor, diag_xtx: Optional[torch.Tensor] = None, damp: float = 0.01,
                 act_order: bool = False, ws: Optional[torch.Tensor] = None, stream=None):
    """(U, perm, dead) from H (the upper triangle is read)."""
    d = H.shape[0]
    _dev(H, torch.float32, "H", (d, d))
    if act_order:
        if diag_xtx is None:
            raise ValueError("act_order needs diag_xtx")
        _dev(diag_xtx, torch.float32, "diag_xtx", (d,))
    dev = H.device
    U = torch.empty(d, d, dtype=torch.float32, device=dev)
    perm = torch.empty(d, dtype=torch.int32, device=dev)
    dead = torch.empty(d, dtype=torch.uint8, device=dev)
    nb = gptq_prepare_workspace_bytes(d, act_order)
    if ws is None:
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    _check("gptq_prepare", load().gptq_prepare(_ptr(H), _ptr(diag_xtx), d, float(damp), 1 if act_order else 0,
                                               _ptr(U), _ptr(perm), _ptr(dead), _ptr(ws), ws.numel(), _stream(stream)))
    return U, perm, dead


# ----------------------------------------------------------------------------- quantize

def gptq_quantize_workspace_bytes(rows: int, cols: int, bits: int = 4, group: int = 0, sym: bool = True) -> int:
    return int(load().gptq_quantize_workspace_bytes(rows, cols, qconfig(bits, group, sym)))


def _outputs(rows, cols, bits, group, dev):
    G = -(-cols // group) if group else 1
    return {
        "codes": torch.empty(rows, cols, dtype=torch.int8, device=dev),
        "scales": torch.empty(rows, G, dtype=torch.float32, device=dev),
        "zeros": torch.empty(rows, G, dtype=torch.uint8, device=dev),
        "Wq": torch.empty(rows, cols, dtype=torch.float32, device=dev),
        "packed": torch.empty(rows, gptq_packed_words_per_row(cols, bits), dtype=torch.int32, device=dev),
    }


def gptq_quantize(W: torch.Tensor, U: torch.Tensor, perm: Optional[torch.Tensor] = None,
                  dead: Optional[torch.Tensor] = None, bits: int = 4, group: int = 0, sym: bool = True,
                  ws: Optional[torch.Tensor] = None, out: Optional[Dict[str, torch.Tensor]] = None,
                  stream=None, zero_in_range: bool = False) -> Dict[str, torch.Tensor]:
    """GPTQ's column loop on W (rows, cols) given U (loop order), perm and dead.
    zero_in_range: asymmetric grid over the min/max range widened to contain 0."""
    rows, cols = W.shape
    _dev(W, torch.float32, "W")
    _dev(U, torch.float32, "U", (cols, cols))
    if perm is not None:
        _dev(perm, torch.int32, "perm", (cols,))
    if dead is not None:
        _dev(dead, torch.uint8, "dead", (cols,))
    dev = W.device
    o = out if out is not None else _outputs(rows, cols, bits, group, dev)
    if "g_idx" not in o:
        o["g_idx"] = torch.empty(cols, dtype=torch.int32, device=dev)
    if "row_loss" not in o:
        o["row_loss"] = torch.empty(rows, dtype=torch.float32, device=dev)
    nb = gptq_quantize_workspace_bytes(rows, cols, bits, group, sym)
    if ws is None:
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    _check("gptq_quantize", load().gptq_quantize(
        _ptr(W), rows, cols, _ptr(U), _ptr(perm), _ptr(dead), qconfig(bits, group, sym, zero_in_range),
        _ptr(o["codes"]), _ptr(o["scales"]), _ptr(o["zeros"]), _ptr(o["g_idx"]), _ptr(o.get("Wq")),
        _ptr(o.get("packed")), _ptr(o["row_loss"]), _ptr(ws), ws.numel(), _stream(stream)))
    return o


def gptq_prune_workspace_bytes(rows: int, cols: int) -> int:
    return int(load().gptq_prune_workspace_bytes(rows, cols))


def gptq_prune(W: torch.Tensor, U: torch.Tensor, perm: Optional[torch.Tensor] = None,
               dead: Optional[torch.Tensor] = None, sparsity: float = 0.5, ws: Optional[torch.Tensor] = None,
               out: Optional[Dict[str, torch.Tensor]] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Pruning with GPTQ's update: Wp (pruned and compensated, 0 where pruned), mask (uint8,
    1 where pruned) and row_loss, all in the original column order."""
    rows, cols = W.shape
    _dev(W, torch.float32, "W")
    _dev(U, torch.float32, "U", (cols, cols))
    if perm is not None:
        _dev(perm, torch.int32, "perm", (cols,))
    if dead is not None:
        _dev(dead, torch.uint8, "dead", (cols,))
    dev = W.device
    nb = gptq_prune_workspace_bytes(rows, cols)
    if ws is None:
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    o = out if out is not None else {
        "Wp": torch.empty(rows, cols, dtype=torch.float32, device=dev),
        "mask": torch.empty(rows, cols, dtype=torch.uint8, device=dev),
        "row_loss": torch.empty(rows, dtype=torch.float32, device=dev),
    }
    _check("gptq_prune", load().gptq_prune(
        _ptr(W), rows, cols, _ptr(U), _ptr(perm), _ptr(dead), float(sparsity), _ptr(o["Wp"]), _ptr(o.get("mask")),
        _ptr(o.get("row_loss")), _ptr(ws), ws.numel(), _stream(stream)))
    return o


def rtn_quantize(W: torch.Tensor, bits: int = 4, group: int = 0, sym: bool = True,
                 dead: Optional[torch.Tensor] = None, out: Optional[Dict[str, torch.Tensor]] = None,
                 stream=None, zero_in_range: bool = False) -> Dict[str, torch.Tensor]:
    rows, cols = W.shape
    _dev(W, torch.float32, "W")
    if dead is not None:
        _dev(dead, torch.uint8, "dead", (cols,))
    o = out if out is not None else _outputs(rows, cols, bits, group, W.device)
    _check("rtn_quantize", load().rtn_quantize(
        _ptr(W), rows, cols, _ptr(dead), qconfig(bits, group, sym, zero_in_range), _ptr(o["codes"]), _ptr(o["scales"]),
        _ptr(o["zeros"]), _ptr(o.get("Wq")), _ptr(o.get("packed")), _stream(stream)))
    return o


def gptq_pack(codes: torch.Tensor, bits: int, sym: bool = True, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    rows, cols = codes.shape
    _dev(codes, torch.int8, "codes")
    p = out if out is not None else torch.empty(rows, gptq_packed_words_per_row(cols, bits), dtype=torch.int32,
                                                device=codes.device)
    _check("gptq_pack", load().gptq_pack(_ptr(codes), rows, cols, bits, 1 if sym else 0, _ptr(p), _stream(stream)))
    return p


STATUS_SYNC, STATUS_DEFERRED = 0, 1


def set_status_mode(deferred: bool) -> None:
    """Deferred: the calls that synchronise to report device-side errors return once their
    work is enqueued; `status_sync` reports the first such error since its last call."""
    _check("gptq_set_status_mode", load().gptq_set_status_mode(STATUS_DEFERRED if deferred else STATUS_SYNC))


def status_sync(stream=None) -> None:
    """Synchronise the stream and raise the first device-side error recorded in deferred
    mode since the last call (clearing it)."""
    _check("gptq_status_sync", load().gptq_status_sync(_stream(stream)))


class deferred_status:
    """Context manager: deferred status reporting inside, the previous mode restored after
    (pending errors are left for `status_sync`)."""

    def __enter__(self):
        self._prev = int(load().gptq_status_mode())
        _check("gptq_set_status_mode", load().gptq_set_status_mode(STATUS_DEFERRED))
        return self

    def __exit__(self, *exc):
        load().gptq_set_status_mode(self._prev)
        return False


DQ_RELU, DQ_BF16_OUT = 1, 2


def gptq_dequant_matmul(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                        g_idx: torch.Tensor, bits: int, out: Optional[torch.Tensor] = None, relu: bool = False,
                        out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """Y = X Wq^T (optionally max(., 0)) straight from the stored form (packed codes,
    scales, zeros, g_idx); Y fp32 or bf16."""
    T, K = X.shape
    N, G = scales.shape
    _dev(X, torch.bfloat16, "X")
    _dev(packed, torch.int32, "packed", (N, gptq_packed_words_per_row(K, bits)))
    _dev(scales, torch.float32, "scales")
    _dev(zeros, torch.uint8, "zeros", (N, G))
    _dev(g_idx, torch.int32, "g_idx", (K,))
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out_dtype must be float32 or bfloat16")
    Y = out if out is not None else torch.empty(T, N, dtype=out_dtype, device=X.device)
    _dev(Y, out_dtype, "Y", (T, N))
    flags = (DQ_RELU if relu else 0) | (DQ_BF16_OUT if out_dtype == torch.bfloat16 else 0)
    _check("gptq_dequant_matmul", load().gptq_dequant_matmul(
        _ptr(X), T, K, K, _ptr(packed), _ptr(scales), _ptr(zeros), _ptr(g_idx), N, G, bits, flags, _ptr(Y), N,
        _stream(stream)))
    return Y


def gptq_layerwise(X: torch.Tensor, Ws, bits: int = 4, group: int = 0, sym: bool = True, damp: float = 0.01,
                   act_order: bool = False, stream=None):
    """GPTQ guide page's `apply_layerwise` on the GPU: every layer is calibrated on the
    inputs it will actually see — the bf16 outputs of the layers before it, already
    quantised — and the forward pass runs on the stored form (gptq_dequant_matmul; relu on
    the hidden layers, bf16 activations, the last layer's output fp32). Returns one dict
    per layer (its calibration input, H, U, perm, dead and the gptq_quantize outputs) and
    the network's output. Host orchestration only: every step runs in the library."""
    h = X
    layers = []
    for i, W in enumerate(Ws):
        last = i == len(Ws) - 1
        acc = Hessian(h.shape[1], h.device)
        acc.accumulate(h, stream=stream)
        H, diag, _ = acc.finalize(stream=stream)
        acc.close()
        U, perm, dead = gptq_prepare(H, diag, damp, act_order=act_order, stream=stream)
        st = gptq_quantize(W, U, perm, dead, bits, group, sym, stream=stream)
        out = gptq_dequant_matmul(h, st["packed"], st["scales"], st["zeros"], st["g_idx"], bits, relu=not last,
                                  out_dtype=torch.float32 if last else torch.bfloat16, stream=stream)
        layers.append({"input": h, "H": H, "U": U, "perm": perm, "dead": dead, **st})
        h = out
    return layers, h


# -------------------------------------------------- the microscaled 4-bit form (e2m1 codes)

MXFP4, NVFP4 = 0, 1
_FP4 = {"mx": MXFP4, "nv": NVFP4}
FP4_EXPERT_G = 4


class Fp4(NamedTuple):
    """A matrix (rows, cols), or one per expert, in the microscaled 4-bit form: codes uint8
    ([experts,] rows, gptq_fp4_code_pitch(cols)), scales uint8 ([experts,] row tiles, column
    tiles, 512), the format ("mx" or "nv") and, for "nv", the fp32 tensor scale (one, or one
    per expert). Layouts: include/gptq.h."""
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int
    format: str
    tensor_scale: Optional[torch.Tensor] = None

    @property
    def rows(self) -> int:
        return self.codes.shape[-2]


def _fp4_format(format: str) -> int:
    f = _FP4.get(format)
    if f is None:
        raise ValueError(f"format must be 'mx' or 'nv', got {format!r}")
    return f


def gptq_fp4_code_pitch(cols: int) -> int:
    return (cols + 31) // 32 * 16


def _fp4_scale_shape(rows: int, cols: int, format: str) -> Tuple[int, int, int]:
    return ((rows + 127) // 128, -(-cols // (128 if format == "mx" else 64)), 512)


def gptq_fp4_scale_bytes(rows: int, cols: int, format: str) -> int:
    return int(load().gptq_fp4_scale_bytes(rows, cols, _fp4_format(format)))


# The calls of a serving step are short. Their common form (results allocated here, on the current
# stream) goes through the C module _call, which returns NotImplemented for what it does not
# recognise; the functions below then check in Python, and raise. With `stream`, results are still
# allocated on the current stream: a caller keeps them and the inputs until that stream is done.
# All tensors are on the current device. Results have no autograd graph, whether or not an input requires
# a gradient; gptq_expert_gather_grad and gptq_expert_combine_grad are the gradients there are, and the
# 4-bit product has none.
_fast = None


def _load_fast():
    load()
    return _fast


_DTYPES = {torch.float32: GPTQ_F32, torch.bfloat16: GPTQ_BF16}
_current_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _raw_stream(stream) -> int:
    return _current_raw_stream(_current_device()) if stream is None else stream.cuda_stream


def _addr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _here(t: torch.Tensor, name: str) -> None:
    """The library launches on the current device, and only reaches the tensors there."""
    if t.get_device() != _current_device():
        raise ValueError(f"{name} must be on the current CUDA device")


def _dev_here(t: torch.Tensor, dtype, name: str, shape=None) -> None:
    _dev(t, dtype, name, shape)
    _here(t, name)


def _matrix(t: torch.Tensor, name: str) -> Tuple[int, int, int, int]:
    """(dtype code, rows, columns, row stride) of a matrix whose rows are contiguous."""
    dt = _DTYPES.get(t.dtype)
    if dt is None or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA bf16 or fp32 tensor")
    _here(t, name)
    rows, cols = t.shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name} rows must be contiguous")
    if rows <= 1:
        ld = max(cols, 1)
    elif ld < cols:
        raise ValueError(f"{name} rows must not overlap")
    return dt, rows, cols, ld


def _matrix_like(t: torch.Tensor, name: str, dtype, rows: int, cols: int) -> int:
    """The row stride of a matrix that has to have this type and shape."""
    _, r, c, ld = _matrix(t, name)
    if r != rows or c != cols or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {(rows, cols)}, got {t.dtype} {tuple(t.shape)}")
    return ld


def _check_fp4(q: Fp4, name: str, experts: Optional[int] = None) -> int:
    """The format code of a stored matrix whose buffers fit its columns (experts: one per expert)."""
    codes, scales, cols, format, g = q
    f = _fp4_format(format)
    tiles = _fp4_scale_shape(codes.shape[-2], cols, format)
    lead = () if experts is None else (experts,)
    if codes.shape != (*lead, codes.shape[-2], (cols + 31) // 32 * 16) or scales.shape != (*lead, *tiles):
        raise ValueError(f"{name}: codes {tuple(codes.shape)} and scales {tuple(scales.shape)} are not those of "
                         f"{'one matrix' if experts is None else f'{experts} matrices'} of {cols} columns in format {format!r}")
    if not (codes.is_cuda and scales.is_cuda and codes.dtype is torch.uint8 and scales.dtype is torch.uint8
            and codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name}: codes and scales must be contiguous CUDA uint8 tensors")
    _here(codes, name + ".codes")
    _here(scales, name + ".scales")
    if f == NVFP4:
        if g is None:
            raise ValueError(f"{name}: format 'nv' needs a tensor scale")
        _dev_here(g, torch.float32, name + ".tensor_scale")
        if g.numel() not in (1, experts):
            raise ValueError(f"{name}.tensor_scale must hold one number, or one per expert")
    return f


def gptq_fp4_tensor_scale(X: torch.Tensor, stream=None) -> torch.Tensor:
    """The "nv" tensor scale of X: the least power of two for which no block scale saturates."""
    dt, rows, cols, ld = _matrix(X, "X")
    g = torch.empty(1, dtype=torch.float32, device=X.device)
    _check("gptq_fp4_tensor_scale", load().gptq_fp4_tensor_scale(X.data_ptr(), dt, rows, cols, ld, g.data_ptr(),
                                                                 _raw_stream(stream)))
    return g


def gptq_fp4_quantize(X: torch.Tensor, format: str = "mx", tensor_scale: Optional[torch.Tensor] = None,
                      index: Optional[torch.Tensor] = None, per: int = 1, out: Optional[Fp4] = None,
                      stream=None) -> Fp4:
    """X (bf16 or fp32, any stride between rows that do not overlap) in the microscaled 4-bit form. index (int32): row r is X row
    index[r] // per, zeros where index[r] < 0 (a Route's src with per = top gathers the experts' rows
    in the same pass). "nv" without a tensor scale takes gptq_fp4_tensor_scale(X)."""
    if out is None and stream is None:
        r = (_fast or _load_fast()).quantize(X, format, tensor_scale, index, per)
        if r is not NotImplemented:
            return r
    f = _fp4_format(format)
    dt, n, cols, ld = _matrix(X, "X")
    rows = n
    if index is not None:
        _dev_here(index, torch.int32, "index")
        rows = index.numel()
    if f == NVFP4:
        if tensor_scale is None:
            tensor_scale = gptq_fp4_tensor_scale(X, stream)
        _dev_here(tensor_scale, torch.float32, "tensor_scale")
        if tensor_scale.numel() != 1:
            raise ValueError("tensor_scale must hold one number")
    else:
        tensor_scale = None
    if out is None:
        dev = X.device
        out = Fp4(torch.empty((rows, (cols + 31) // 32 * 16), dtype=torch.uint8, device=dev),
                  torch.empty(_fp4_scale_shape(rows, cols, format), dtype=torch.uint8, device=dev), cols, format, tensor_scale)
    else:
        if out.cols != cols or out.format != format or out.rows != rows:
            raise ValueError("out has another shape or format")
        out = out._replace(tensor_scale=tensor_scale)
        _check_fp4(out, "out")
    _check("gptq_fp4_quantize", load().gptq_fp4_quantize(
        X.data_ptr(), dt, n, cols, ld, _addr(index), per, rows, f, _addr(tensor_scale), out.codes.data_ptr(),
        out.scales.data_ptr(), _raw_stream(stream)))
    return out


def gptq_fp4_dequantize(q: Fp4, dtype=torch.float32, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values that q's codes and scales stand for."""
    if out is None and stream is None:
        r = (_fast or _load_fast()).dequantize(q, dtype)
        if r is not NotImplemented:
            return r
    f = _check_fp4(q, "q")
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise ValueError("dtype must be float32 or bfloat16")
    rows, cols = q.rows, q.cols
    Y = out if out is not None else torch.empty((rows, cols), dtype=dtype, device=q.codes.device)
    ld = cols if out is None else _matrix_like(Y, "out", dtype, rows, cols)
    _check("gptq_fp4_dequantize", load().gptq_fp4_dequantize(
        q.codes.data_ptr(), q.scales.data_ptr(), _addr(q.tensor_scale), rows, cols, f, Y.data_ptr(), dt, ld,
        _raw_stream(stream)))
    return Y


def gptq_fp4_tile_scales(scales: torch.Tensor, cols: int, format: str, stream=None) -> torch.Tensor:
    """Row-major scale bytes (rows, blocks) of a checkpoint, in the tiled order of Fp4.scales."""
    f = _fp4_format(format)
    rows = scales.shape[0]
    _dev_here(scales, torch.uint8, "scales", (rows, -(-cols // (32 if f == MXFP4 else 16))))
    out = torch.empty(_fp4_scale_shape(rows, cols, format), dtype=torch.uint8, device=scales.device)
    _check("gptq_fp4_tile_scales", load().gptq_fp4_tile_scales(scales.data_ptr(), rows, cols, scales.shape[1], f,
                                                               out.data_ptr(), _raw_stream(stream)))
    return out


def gptq_fp4_matmul(X: Fp4, W: Fp4, offsets: Optional[torch.Tensor] = None, relu: bool = False,
                    out_dtype=torch.float32, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = X W^T (optionally max(., 0)) of two matrices in the microscaled 4-bit form. With offsets
    (int32, experts + 1, a Route's) W holds one weight per expert and rows offsets[e]..offsets[e+1]
    of X use weight e; rows in no expert's range give zeros."""
    if out is None and stream is None:
        r = (_fast or _load_fast()).matmul(X, W, offsets, relu, out_dtype)
        if r is not NotImplemented:
            return r
    f = _check_fp4(X, "X")
    experts = 1
    if offsets is None:
        _check_fp4(W, "W")
    else:
        experts = W.codes.shape[0]
        _check_fp4(W, "W", experts)
        _dev_here(offsets, torch.int32, "offsets", (experts + 1,))
    if X.format != W.format or X.cols != W.cols:
        raise ValueError("X and W must have the same format and columns")
    if out_dtype not in _DTYPES:
        raise ValueError("out_dtype must be float32 or bfloat16")
    T, N = X.codes.shape[0], W.codes.shape[-2]
    Y = out if out is not None else torch.empty((T, N), dtype=out_dtype, device=X.codes.device)
    ld = N if out is None else _matrix_like(Y, "out", out_dtype, T, N)
    if X.cols == 0:   # a sum of nothing; the library's products have a column or more
        with torch.cuda.stream(stream):
            return Y.zero_()
    flags = (DQ_RELU if relu else 0) | (DQ_BF16_OUT if out_dtype is torch.bfloat16 else 0)
    if f == NVFP4 and experts > 1 and W.tensor_scale.numel() == experts:
        flags |= FP4_EXPERT_G
    _check("gptq_fp4_matmul", load().gptq_fp4_matmul(
        X.codes.data_ptr(), X.scales.data_ptr(), _addr(X.tensor_scale), T, W.codes.data_ptr(), W.scales.data_ptr(),
        _addr(W.tensor_scale), N, X.cols, f, _addr(offsets), experts, flags, Y.data_ptr(), ld, _raw_stream(stream)))
    return Y


# ---------------------------------------------------------------------- the 8-bit integer form

class Int8(NamedTuple):
    """A matrix (rows, cols), or one per expert, as whole numbers with a scale per row: codes int8
    ([experts,] rows, gptq_int8_pitch(cols)), zeros past cols, and scales fp32 ([experts,] rows), not
    negative; value = code * scale."""
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int

    @property
    def rows(self) -> int:
        return self.codes.shape[-2]


def gptq_int8_pitch(cols: int) -> int:
    return (cols + 15) // 16 * 16


def _check_int8(q: Int8, name: str, experts: Optional[int] = None) -> None:
    """A stored matrix whose buffers fit its columns (experts: one per expert)."""
    codes, scales, cols = q
    rows = codes.shape[-2] if codes.dim() >= 2 else 0
    lead = () if experts is None else (experts,)
    if cols < 0 or codes.shape != (*lead, rows, gptq_int8_pitch(cols)) or scales.shape != (*lead, rows):
        raise ValueError(f"{name}: codes {tuple(codes.shape)} and scales {tuple(scales.shape)} are not those of "
                         f"{'one matrix' if experts is None else f'{experts} matrices'} of {cols} columns")
    _dev_here(codes, torch.int8, name + ".codes")
    _dev_here(scales, torch.float32, name + ".scales")


def _new_int8(rows: int, cols: int, dev) -> Int8:
    return Int8(torch.empty((rows, gptq_int8_pitch(cols)), dtype=torch.int8, device=dev),
                torch.empty((rows,), dtype=torch.float32, device=dev), cols)


def _int8_out(out: Optional[Int8], rows: int, cols: int, dev) -> Int8:
    if out is None:
        return _new_int8(rows, cols, dev)
    _check_int8(out, "out")
    if out.cols != cols or out.rows != rows:
        raise ValueError("out has another shape")
    return out


def gptq_int8_quantize(X: torch.Tensor, index: Optional[torch.Tensor] = None, per: int = 1, out: Optional[Int8] = None,
                       stream=None) -> Int8:
    """X (bf16 or fp32, any stride between rows that do not overlap) in 8-bit integers, scale = max|x| / 127 of each
    row. index (int32): row r is X row index[r] // per, zeros where index[r] < 0 (a Route's src with per = top
    gathers the experts' rows in the same pass)."""
    if out is None and stream is None:
        r = (_fast or _load_fast()).int8_quantize(X, index, per)
        if r is not NotImplemented:
            return r
    dt, n, cols, ld = _matrix(X, "X")
    rows = n
    if index is not None:
        _dev_here(index, torch.int32, "index")
        rows = index.numel()
    out = _int8_out(out, rows, cols, X.device)
    _check("gptq_int8_quantize", load().gptq_int8_quantize(
        X.data_ptr(), dt, n, cols, ld, _addr(index), per, rows, out.codes.data_ptr(), out.scales.data_ptr(), _raw_stream(stream)))
    return out


def gptq_int8_dequantize(q: Int8, dtype=torch.float32, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values that q's codes and scales stand for."""
    if out is None and stream is None:
        r = (_fast or _load_fast()).int8_dequantize(q, dtype)
        if r is not NotImplemented:
            return r
    _check_int8(q, "q")
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise ValueError("dtype must be float32 or bfloat16")
    rows, cols = q.rows, q.cols
    Y = out if out is not None else torch.empty((rows, cols), dtype=dtype, device=q.codes.device)
    ld = cols if out is None else _matrix_like(Y, "out", dtype, rows, cols)
    _check("gptq_int8_dequantize", load().gptq_int8_dequantize(
        q.codes.data_ptr(), q.scales.data_ptr(), rows, cols, Y.data_ptr(), dt, ld, _raw_stream(stream)))
    return Y


def gptq_int8_rms_norm(X: torch.Tensor, gain: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                       out: Optional[Tuple[Int8, Optional[torch.Tensor], torch.Tensor]] = None,
                       stream=None) -> Tuple[Int8, torch.Tensor, torch.Tensor]:
    """(q, h, rstd): h = X + residual in X's type (X itself without a residual), rstd = 1 / sqrt(mean h^2 + eps) per
    row, and q = (h rstd) gain in 8-bit integers. gain fp32 (cols). h and rstd are what gptq_int8_rms_norm_grad needs.
    out: (q, h, rstd) to write to; its h may be X or residual itself."""
    if out is None and stream is None:
        r = (_fast or _load_fast()).rms_norm(X, gain, eps, residual)
        if r is not NotImplemented:
            return r
    dt, rows, cols, ld = _matrix(X, "X")
    _dev_here(gain, torch.float32, "gain", (cols,))
    ldr = _matrix_like(residual, "residual", X.dtype, rows, cols) if residual is not None else 0
    q, h, rstd = out if out is not None else (None, None, None)
    q = _int8_out(q, rows, cols, X.device)
    if residual is None:
        if h is not None and h is not X:
            raise ValueError("out[1] must be X or None without a residual: h is X")
        h, ldh = X, ld
    elif h is None:
        h, ldh = torch.empty((rows, cols), dtype=X.dtype, device=X.device), cols
    else:
        ldh = _matrix_like(h, "out[1]", X.dtype, rows, cols)
    if rstd is None:
        rstd = torch.empty((rows,), dtype=torch.float32, device=X.device)
    else:
        _dev_here(rstd, torch.float32, "out[2]", (rows,))
    _check("gptq_int8_rms_norm", load().gptq_int8_rms_norm(
        X.data_ptr(), ld, _addr(residual), ldr, dt, rows, cols, gain.data_ptr(), float(eps), q.codes.data_ptr(),
        q.scales.data_ptr(), None if residual is None else h.data_ptr(), ldh, rstd.data_ptr(), _raw_stream(stream)))
    return q, h, rstd


def gptq_int8_rms_norm_grad_workspace_bytes(rows: int, cols: int) -> int:
    return int(load().gptq_int8_rms_norm_grad_workspace_bytes(rows, cols))


def _workspace(ws: Optional[torch.Tensor], need: int, dev, stream) -> Tuple[Optional[torch.Tensor], int]:
    """A workspace and its bytes: the caller's, or a new one."""
    if ws is not None:
        if not (ws.is_cuda and ws.is_contiguous()):
            raise ValueError("ws must be a contiguous CUDA tensor")
        _here(ws, "ws")
        return ws, ws.numel() * ws.element_size()
    if need:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        if stream is not None:
            ws.record_stream(stream)
    return ws, need


def gptq_int8_rms_norm_grad(dY: torch.Tensor, h: torch.Tensor, gain: torch.Tensor, rstd: torch.Tensor,
                            dh: Optional[torch.Tensor] = None, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                            ws: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dX, dgain) of gptq_int8_rms_norm, straight through the rounding: dY is the gradient of q's values, dh (None: 0)
    the one that reaches h past the norm. dX, of X's type, is residual's gradient too; it may be written to dY, h or dh
    (out). dgain is fp32."""
    if out is None and ws is None and stream is None:
        r = (_fast or _load_fast()).rms_norm_grad(dY, h, gain, rstd, dh)
        if r is not NotImplemented:
            return r
    dt, rows, cols, ldh = _matrix(h, "h")
    lddy = _matrix_like(dY, "dY", h.dtype, rows, cols)
    lddh = _matrix_like(dh, "dh", h.dtype, rows, cols) if dh is not None else 0
    _dev_here(gain, torch.float32, "gain", (cols,))
    _dev_here(rstd, torch.float32, "rstd", (rows,))
    if out is None:
        dX, dgain = torch.empty((rows, cols), dtype=h.dtype, device=h.device), torch.empty((cols,), dtype=torch.float32, device=h.device)
        lddx = cols
    else:
        dX, dgain = out
        lddx = _matrix_like(dX, "out[0]", h.dtype, rows, cols)
        _dev_here(dgain, torch.float32, "out[1]", (cols,))
    lib = load()
    ws, nb = _workspace(ws, int(lib.gptq_int8_rms_norm_grad_workspace_bytes(rows, cols)), h.device, stream)
    _check("gptq_int8_rms_norm_grad", lib.gptq_int8_rms_norm_grad(
        dY.data_ptr(), lddy, h.data_ptr(), ldh, _addr(dh), lddh, dt, rows, cols, gain.data_ptr(), rstd.data_ptr(), dX.data_ptr(),
        lddx, dgain.data_ptr(), _addr(ws), nb, _raw_stream(stream)))
    return dX, dgain


def gptq_int8_matmul(X: Int8, W: Int8, offsets: Optional[torch.Tensor] = None, relu: bool = False, out_dtype=torch.float32,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = X W^T (optionally max(., 0)) of two matrices in 8-bit integers, times the scales of X's row and of W's. With
    offsets (int32, experts + 1, a Route's) W holds one weight per expert and rows offsets[e]..offsets[e+1] of X use
    weight e; rows in no expert's range give zeros."""
    if out is None and stream is None:
        r = (_fast or _load_fast()).int8_matmul(X, W, offsets, relu, out_dtype)
        if r is not NotImplemented:
            return r
    _check_int8(X, "X")
    experts = 1
    if offsets is None:
        _check_int8(W, "W")
    else:
        experts = W.codes.shape[0]
        _check_int8(W, "W", experts)
        _dev_here(offsets, torch.int32, "offsets", (experts + 1,))
    if X.cols != W.cols:
        raise ValueError("X and W must have the same columns")
    if out_dtype not in _DTYPES:
        raise ValueError("out_dtype must be float32 or bfloat16")
    T, N = X.rows, W.rows
    Y = out if out is not None else torch.empty((T, N), dtype=out_dtype, device=X.codes.device)
    ld = N if out is None else _matrix_like(Y, "out", out_dtype, T, N)
    flags = (DQ_RELU if relu else 0) | (DQ_BF16_OUT if out_dtype is torch.bfloat16 else 0)
    _check("gptq_int8_matmul", load().gptq_int8_matmul(
        X.codes.data_ptr(), X.scales.data_ptr(), T, W.codes.data_ptr(), W.scales.data_ptr(), N, X.cols, _addr(offsets), experts,
        flags, Y.data_ptr(), ld, _raw_stream(stream)))
    return Y


# ------------------------------------------------------- tokens sorted by expert, and back

class Route(NamedTuple):
    """Where each token's slots go (gptq_expert_sort): offsets int32 (experts + 1), src int32
    (tokens * top), pos int32 (tokens, top)."""
    offsets: torch.Tensor
    src: torch.Tensor
    pos: torch.Tensor

    @property
    def experts(self) -> int:
        return self.offsets.numel() - 1


def gptq_expert_sort_workspace_bytes(tokens: int, top: int, experts: int) -> int:
    return int(load().gptq_expert_sort_workspace_bytes(tokens, top, experts))


def gptq_expert_sort(ids: torch.Tensor, experts: int, ws: Optional[torch.Tensor] = None, stream=None) -> Route:
    """ids (tokens, top) int32, each slot's expert (negative: dropped) -> the slots' places, stably
    sorted by expert."""
    if ws is None and stream is None:
        r = (_fast or _load_fast()).sort(ids, experts)
        if r is not NotImplemented:
            return r
    _dev_here(ids, torch.int32, "ids")
    if ids.dim() != 2:
        raise ValueError("ids must be (tokens, top)")
    tokens, top = ids.shape
    dev = ids.device
    route = Route(torch.empty(experts + 1, dtype=torch.int32, device=dev),
                  torch.empty(tokens * top, dtype=torch.int32, device=dev), torch.empty_like(ids))
    lib = load()
    if ws is not None and not (ws.is_cuda and ws.is_contiguous()):
        raise ValueError("ws must be a contiguous CUDA tensor")
    if ws is not None:
        _here(ws, "ws")
    nb = ws.numel() * ws.element_size() if ws is not None else int(lib.gptq_expert_sort_workspace_bytes(tokens, top, experts))
    if ws is None and nb:
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        if stream is not None:
            ws.record_stream(stream)
    _check("gptq_expert_sort", lib.gptq_expert_sort(
        ids.data_ptr(), tokens, top, experts, route.offsets.data_ptr(), route.src.data_ptr(), route.pos.data_ptr(),
        _addr(ws), nb, _raw_stream(stream)))
    return route


def _check_route(route: Route) -> Tuple[int, int]:
    offsets, src, pos = route
    tokens, top = pos.shape
    if (pos.dtype is not torch.int32 or src.dtype is not torch.int32 or offsets.dtype is not torch.int32 or not pos.is_cuda
            or not src.is_cuda or not offsets.is_cuda or not pos.is_contiguous() or not src.is_contiguous()
            or not offsets.is_contiguous() or src.shape != (tokens * top,) or offsets.dim() != 1):
        raise ValueError("route must hold contiguous CUDA int32 tensors: offsets (experts + 1), src (tokens * top), pos (tokens, top)")
    for t in route:
        _here(t, "route")
    return tokens, top


def gptq_expert_gather(X: torch.Tensor, route: Route, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The tokens' rows in the order of their experts (tokens * top rows, zeros past the live ones)."""
    if out is None and stream is None:
        r = (_fast or _load_fast()).gather(X, route)
        if r is not NotImplemented:
            return r
    tokens, top = _check_route(route)
    dt, rows, d, ld = _matrix(X, "X")
    if rows != tokens:
        raise ValueError(f"X has {rows} rows for {tokens} tokens")
    Xs = out if out is not None else torch.empty((tokens * top, d), dtype=X.dtype, device=X.device)
    lds = d if out is None else _matrix_like(Xs, "out", X.dtype, tokens * top, d)
    _check("gptq_expert_gather", load().gptq_expert_gather(
        X.data_ptr(), dt, tokens, d, ld, route.pos.data_ptr(), top, route.offsets.data_ptr(), route.experts, Xs.data_ptr(),
        lds, _raw_stream(stream)))
    return Xs


def gptq_expert_combine(Ys: torch.Tensor, route: Route, weights: Optional[torch.Tensor],
                        out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[t] = sum_j weights[t][j] * the row of slot (t, j), in fp32, rounded once; weights None: 1."""
    if out is None and stream is None:
        r = (_fast or _load_fast()).combine(Ys, route, weights)
        if r is not NotImplemented:
            return r
    tokens, top = _check_route(route)
    dt, rows, d, ld = _matrix(Ys, "Ys")
    if rows != tokens * top:
        raise ValueError(f"Ys has {rows} rows for {tokens} x {top} slots")
    if weights is not None:
        _dev_here(weights, torch.float32, "weights", (tokens, top))
    Y = out if out is not None else torch.empty((tokens, d), dtype=Ys.dtype, device=Ys.device)
    ldy = d if out is None else _matrix_like(Y, "out", Ys.dtype, tokens, d)
    _check("gptq_expert_combine", load().gptq_expert_combine(
        Ys.data_ptr(), dt, tokens, d, ld, route.pos.data_ptr(), top, _addr(weights), Y.data_ptr(), ldy, _raw_stream(stream)))
    return Y


def gptq_expert_gather_grad(dXs: torch.Tensor, route: Route, out: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """The gradient of gptq_expert_gather's input: each token's rows of dXs summed."""
    return gptq_expert_combine(dXs, route, None, out, stream)


def gptq_expert_combine_grad(dY: torch.Tensor, Ys: torch.Tensor, route: Route, weights: torch.Tensor,
                             out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gradients of gptq_expert_combine: (dYs, dweights)."""
    if out is None and stream is None:
        r = (_fast or _load_fast()).combine_grad(dY, Ys, route, weights)
        if r is not NotImplemented:
            return r
    tokens, top = _check_route(route)
    dt, rows, d, ld = _matrix(Ys, "Ys")
    if rows != tokens * top:
        raise ValueError(f"Ys has {rows} rows for {tokens} x {top} slots")
    lddy = _matrix_like(dY, "dY", Ys.dtype, tokens, d)
    _dev_here(weights, torch.float32, "weights", (tokens, top))
    dYs, dW = out if out is not None else (torch.empty((rows, d), dtype=Ys.dtype, device=Ys.device), torch.empty_like(weights))
    lds = d if out is None else _matrix_like(dYs, "out[0]", Ys.dtype, rows, d)
    if out is not None:
        _dev_here(dW, torch.float32, "out[1]", (tokens, top))
    _check("gptq_expert_combine_grad", load().gptq_expert_combine_grad(
        dY.data_ptr(), lddy, Ys.data_ptr(), ld, dt, tokens, d, route.pos.data_ptr(), top, route.offsets.data_ptr(),
        route.experts, weights.data_ptr(), dYs.data_ptr(), lds, dW.data_ptr(), _raw_stream(stream)))
    return dYs, dW


class Balance(NamedTuple):
    """What gptq_expert_balance leaves: loss fp32 (1), counts int32 (experts + 1: each expert's slots, then the
    tokens that count) and the slots per token."""
    loss: torch.Tensor
    counts: torch.Tensor
    top: int


def gptq_expert_balance_workspace_bytes(tokens: int, experts: int) -> int:
    return int(load().gptq_expert_balance_workspace_bytes(tokens, experts))


def _check_mask(mask: Optional[torch.Tensor], tokens: int) -> None:
    if mask is not None:
        _dev_here(mask, torch.uint8 if mask.dtype is torch.uint8 else torch.bool, "mask", (tokens,))


def gptq_expert_balance(logits: torch.Tensor, ids: torch.Tensor, mask: Optional[torch.Tensor] = None,
                        out: Optional[Balance] = None, ws: Optional[torch.Tensor] = None, stream=None) -> Balance:
    """The balance loss experts / (top n^2) sum_e c[e] sum_t softmax(logits[t])[e] of a router's logits (tokens,
    experts; bf16 or fp32) and choice ids (tokens, top; int32, negative: dropped), with c[e] the slots of expert e
    and n the tokens that count; mask (bool or uint8; None: all) says which do."""
    if out is None and ws is None and stream is None:
        r = (_fast or _load_fast()).balance(logits, ids, mask)
        if r is not NotImplemented:
            return r
    dt, tokens, experts, ld = _matrix(logits, "logits")
    _dev_here(ids, torch.int32, "ids")
    if ids.dim() != 2 or ids.shape[0] != tokens:
        raise ValueError("ids must be (tokens, top)")
    _check_mask(mask, tokens)
    dev, top = logits.device, ids.shape[1]
    if out is None:
        out = Balance(torch.empty((1,), dtype=torch.float32, device=dev), torch.empty((experts + 1,), dtype=torch.int32, device=dev), top)
    else:
        _dev_here(out.loss, torch.float32, "out.loss", (1,))
        _dev_here(out.counts, torch.int32, "out.counts", (experts + 1,))
        out = out._replace(top=top)
    lib = load()
    ws, nb = _workspace(ws, int(lib.gptq_expert_balance_workspace_bytes(tokens, experts)), dev, stream)
    _check("gptq_expert_balance", lib.gptq_expert_balance(
        logits.data_ptr(), dt, tokens, experts, ld, ids.data_ptr(), top, _addr(mask), out.loss.data_ptr(), out.counts.data_ptr(),
        _addr(ws), nb, _raw_stream(stream)))
    return out


def gptq_expert_balance_grad(dloss: Optional[torch.Tensor], logits: torch.Tensor, balance: Balance,
                             mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of gptq_expert_balance's logits (the counts are constants), zeros in rows that do not count;
    dloss: the loss's gradient, one fp32 (None: 1). out may be logits itself."""
    if out is None and stream is None:
        r = (_fast or _load_fast()).balance_grad(dloss, logits, balance, mask)
        if r is not NotImplemented:
            return r
    dt, tokens, experts, ld = _matrix(logits, "logits")
    if dloss is not None:
        _dev_here(dloss, torch.float32, "dloss")
        if dloss.numel() != 1:
            raise ValueError("dloss must hold one number")
    _dev_here(balance.counts, torch.int32, "balance.counts", (experts + 1,))
    _check_mask(mask, tokens)
    dZ = out if out is not None else torch.empty((tokens, experts), dtype=logits.dtype, device=logits.device)
    lddz = experts if out is None else _matrix_like(dZ, "out", logits.dtype, tokens, experts)
    _check("gptq_expert_balance_grad", load().gptq_expert_balance_grad(
        _addr(dloss), logits.data_ptr(), dt, tokens, experts, ld, balance.counts.data_ptr(), balance.top, _addr(mask), dZ.data_ptr(),
        lddz, _raw_stream(stream)))
    return dZ


def gptq_expert_mlp(X: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, W_up, W_down,
                    up_scale: Optional[torch.Tensor] = None, down_scale: Optional[torch.Tensor] = None):
    """A layer of experts on microscaled 4-bit weights (Fp4) or on 8-bit integers (Int8): y[t] = sum_j
    weights[t][j] * W_down[e] relu(W_up[e] x[t]) with e = ids[t][j] (negative: dropped), activations quantised
    to the weights' format before each product. X (tokens, d) bf16 or fp32; W_up, W_down: one
    matrix per expert, both Fp4 or both Int8; up_scale, down_scale: the activations' "nv" tensor scales (None: taken
    from the activations). Returns (y bf16, route, the experts' rows ys bf16), what
    gptq_expert_combine_grad needs for the gradients of the router's weights. Host
    orchestration only: every step runs in the library, on the current stream."""
    if isinstance(W_up, Int8) != isinstance(W_down, Int8):
        raise ValueError("W_up and W_down must both be Fp4 or both be Int8")
    route = gptq_expert_sort(ids, W_up.codes.shape[0])
    top = ids.shape[1]
    if isinstance(W_up, Int8):
        if up_scale is not None or down_scale is not None:
            raise ValueError("up_scale and down_scale are tensor scales of the 4-bit form")
        xs = gptq_int8_quantize(X, index=route.src, per=top)
        h = gptq_int8_matmul(xs, W_up, offsets=route.offsets, relu=True, out_dtype=torch.bfloat16)
        ys = gptq_int8_matmul(gptq_int8_quantize(h), W_down, offsets=route.offsets, out_dtype=torch.bfloat16)
        return gptq_expert_combine(ys, route, weights), route, ys
    if W_up.format == "nv" and up_scale is None:
        up_scale = gptq_fp4_tensor_scale(X)
    xs = gptq_fp4_quantize(X, W_up.format, up_scale, index=route.src, per=top)
    h = gptq_fp4_matmul(xs, W_up, offsets=route.offsets, relu=True, out_dtype=torch.bfloat16)
    hs = gptq_fp4_quantize(h, W_down.format, down_scale)
    ys = gptq_fp4_matmul(hs, W_down, offsets=route.offsets, out_dtype=torch.bfloat16)
    return gptq_expert_combine(ys, route, weights), route, ys


def gptq_status_string(status: int) -> str:
    return _str(status)


# ------------------------------------------------------------------------- instrumentation

def gptq_launch_count() -> int:
    return int(load().gptq_launch_count())


def gptq_profile_enable(on: bool = True) -> None:
    load().gptq_profile_enable(1 if on else 0)


def gptq_profile_read() -> Dict[str, Tuple[int, float]]:
    """{kernel class: (launches, total ms)} for the launches recorded since the last read."""
    lib = load()
    n = lib.gptq_profile_kernel_count()
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_ulonglong * n)()
    _check("gptq_profile_read", lib.gptq_profile_read(ms, cnt, n))
    return {lib.gptq_profile_kernel_name(i).decode(): (int(cnt[i]), float(ms[i])) for i in range(n) if cnt[i]}


__all__ = [
    "load", "Hessian", "GptqError", "QConfig", "qconfig", "gptq_hessian_create", "gptq_hessian_accumulate",
    "gptq_hessian_finalize", "gptq_prepare", "gptq_prepare_workspace_bytes", "gptq_quantize",
    "gptq_quantize_workspace_bytes", "rtn_quantize", "gptq_pack", "gptq_packed_words_per_row",
    "gptq_dequant_matmul", "gptq_layerwise", "gptq_status_string", "gptq_launch_count", "gptq_profile_enable", "gptq_profile_read",
    "Fp4", "MXFP4", "NVFP4", "gptq_fp4_code_pitch", "gptq_fp4_scale_bytes", "gptq_fp4_tensor_scale", "gptq_fp4_quantize",
    "gptq_fp4_dequantize", "gptq_fp4_tile_scales", "gptq_fp4_matmul", "Route", "gptq_expert_sort",
    "gptq_expert_sort_workspace_bytes", "gptq_expert_gather", "gptq_expert_gather_grad", "gptq_expert_combine",
    "gptq_expert_combine_grad", "Balance", "gptq_expert_balance", "gptq_expert_balance_workspace_bytes", "gptq_expert_balance_grad",
    "gptq_expert_mlp", "Int8", "gptq_int8_pitch", "gptq_int8_quantize", "gptq_int8_dequantize", "gptq_int8_rms_norm",
    "gptq_int8_rms_norm_grad", "gptq_int8_rms_norm_grad_workspace_bytes", "gptq_int8_matmul",
    "set_status_mode", "status_sync", "deferred_status", "STATUS_SYNC", "STATUS_DEFERRED",
    "EXPORTS", "LIB_PATH",
]

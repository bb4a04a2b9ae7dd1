"""Python binding of libpwq (ctypes): argument marshalling only.

Each function takes torch tensors that live on the GPU, checks shapes and dtypes,
allocates outputs and the workspace with torch (device memory and streams are all torch
is used for), and calls the C entry point of the same name on the current stream.  Every
step of the computation runs in the HIP kernels of libpwq.so; if the library is missing
the import fails loudly instead of falling back to anything.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpwq.so")

PWQ_OK, PWQ_EINVAL, PWQ_EDTYPE, PWQ_EWORKSPACE, PWQ_EHIP = 0, 1, 2, 3, 4
PWQ_F32, PWQ_F16, PWQ_BF16 = 0, 1, 2

_c_void_p, _i64, _i32, _sz, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float


class PwqParams(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("act_order", ctypes.c_int32)]


_SIGS = {
    "pwq_version": (ctypes.c_int, []),
    "pwq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "pwq_last_hip_error": (ctypes.c_int, []),
    "pwq_hessian_workspace_size": (_sz, [_i64, _i64, ctypes.c_int]),
    "pwq_hessian_accumulate": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "pwq_hessian_damp": (ctypes.c_int, [_c_void_p, _i64, _f32, _c_void_p, _c_void_p]),
    "pwq_act_order_perm": (ctypes.c_int, [_c_void_p, _i64, _c_void_p, _c_void_p]),
    "pwq_chol_workspace_size": (_sz, [_i64]),
    "pwq_chol_inverse_upper": (ctypes.c_int, [_c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "pwq_gptq_workspace_size": (_sz, [_i64, _i64, ctypes.POINTER(PwqParams)]),
    "pwq_gptq_quantize_layer": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p, _c_void_p,
                                               ctypes.POINTER(PwqParams), _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                               _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "pwq_rtn_quantize": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _i32, _i32, _c_void_p, _c_void_p,
                                        _c_void_p, _c_void_p, _c_void_p]),
    "pwq_dequant": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _i64, _i32, _i32, _c_void_p,
                                   ctypes.c_int, _c_void_p]),
    "pwq_gptq_quantize_layer_zp": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p, _c_void_p,
                                                  ctypes.POINTER(PwqParams), _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                  _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _sz,
                                                  _c_void_p]),
    "pwq_rtn_quantize_zp": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _i32, _i32, _c_void_p, _c_void_p,
                                           _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "pwq_dequant_zp": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _i64, _i32, _i32,
                                      _c_void_p, ctypes.c_int, _c_void_p]),
    "pwq_recon_mse_zp": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p, ctypes.c_int, _i64,
                                        _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i32,
                                        _c_void_p, _c_void_p, _sz, _c_void_p]),
    "pwq_channel_abs_mean_workspace_size": (_sz, [_i64, _i64]),
    "pwq_channel_abs_mean": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p, _c_void_p, _sz,
                                            _c_void_p]),
    "pwq_awq_search_workspace_size": (_sz, [_i64, _i64]),
    "pwq_awq_search": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p, _i64, _c_void_p, _i32, _i32,
                                      _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                      _c_void_p, _c_void_p, _sz, _c_void_p]),
    "pwq_tensor_scales_workspace_size": (_sz, []),
    "pwq_tensor_scales": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _i32, _c_void_p, _c_void_p,
                                         _c_void_p, _sz, _c_void_p]),
    "pwq_quantized_matmul_workspace_size": (_sz, [_i64, _i64, _i64]),
    "pwq_quantized_matmul": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p,
                                            _i64, _i32, _c_void_p, ctypes.c_int, _i64, _c_void_p, _sz, _c_void_p]),
    "pwq_recon_mse_hessian_workspace_size": (_sz, [_i64, _i64]),
    "pwq_recon_mse_hessian": (ctypes.c_int, [_c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, ctypes.c_int, _i64,
                                             _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i32,
                                             _c_void_p, _c_void_p, _sz, _c_void_p]),
    "pwq_quantized_matmul_noalloc": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p, _c_void_p,
                                                    _c_void_p, _i64, _i32, _c_void_p, ctypes.c_int, _i64, _c_void_p]),
    "pwq_quantize_tokens": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p, _c_void_p, _i64, _c_void_p,
                                           _c_void_p, _c_void_p]),
    "pwq_rms_norm_quantize": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p, _i64, _c_void_p,
                                             ctypes.c_int, ctypes.c_double, _c_void_p, _i64, _c_void_p, _i64, _c_void_p,
                                             _c_void_p, _c_void_p, ctypes.c_int, _i64, _c_void_p]),
    "pwq_quantized_matmul_int8_workspace_size": (_sz, [_i64, _i64, _i64]),
    "pwq_quantized_matmul_int8": (ctypes.c_int, [_c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                 _c_void_p, _i64, _c_void_p, ctypes.c_int, _i64, _c_void_p, _sz,
                                                 _c_void_p]),
    "pwq_profile_enable": (ctypes.c_int, [ctypes.c_int]),
    "pwq_profile_read": (ctypes.c_int, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double),
                                        ctypes.POINTER(ctypes.c_int64), ctypes.c_int]),
    "pwq_recon_mse_workspace_size": (_sz, [_i64, _i64, _i64]),
    "pwq_recon_mse": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p, ctypes.c_int, _i64,
                                     _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i32, _c_void_p,
                                     _c_void_p, _sz, _c_void_p]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libpwq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first (post_weight_quantization_27_amd.build_lib.build())")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


class PwqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib().pwq_status_string(status).decode()
        if status == PWQ_EHIP:
            msg += f" (hipError {lib().pwq_last_hip_error()})"
        super().__init__(f"{fn}: {msg}")
        self.status = status


def _check(fn: str, status: int):
    if status != PWQ_OK:
        raise PwqError(fn, status)


def _dtype_code(t: torch.Tensor) -> int:
    return {torch.float32: PWQ_F32, torch.float16: PWQ_F16, torch.bfloat16: PWQ_BF16}[t.dtype]


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _rows(t: torch.Tensor, name: str) -> int:
    """Leading dimension of a row-major 2-D device tensor (unit column stride)."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name}: expected a 2-D GPU tensor")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name}: columns must be contiguous")
    return max(t.stride(0), t.shape[1])


def _ws(nbytes: int, dev) -> Optional[torch.Tensor]:
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=dev) if nbytes else None


def _need(t: torch.Tensor, dtype, shape, name):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous GPU {dtype} of shape {tuple(shape)}")


# ------------------------------------------------------------------ Hessian
def hessian_accumulate(X: torch.Tensor, H: torch.Tensor) -> torch.Tensor:
    """H += 2 X^T X (X: tokens x d_in, float32 or bfloat16; H float32 d_in x d_in)."""
    ldx = _rows(X, "X")
    n_tok, d_in = X.shape
    _need(H, torch.float32, (d_in, d_in), "H")
    code = _dtype_code(X)
    nb = lib().pwq_hessian_workspace_size(n_tok, d_in, code)
    ws = _ws(nb, X.device)
    _check("pwq_hessian_accumulate", lib().pwq_hessian_accumulate(_p(X), code, n_tok, d_in, ldx, _p(H), _p(ws), nb, _stream(X)))
    return H


def hessian_damp(H: torch.Tensor, damp: float, lambda_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    _need(H, torch.float32, (H.shape[0], H.shape[0]), "H")
    _check("pwq_hessian_damp", lib().pwq_hessian_damp(_p(H), H.shape[0], float(damp), _p(lambda_out), _stream(H)))
    return H


def act_order_perm(H: torch.Tensor) -> torch.Tensor:
    n = H.shape[0]
    _need(H, torch.float32, (n, n), "H")
    perm = torch.empty(n, dtype=torch.int32, device=H.device)
    _check("pwq_act_order_perm", lib().pwq_act_order_perm(_p(H), n, _p(perm), _stream(H)))
    return perm


# ------------------------------------------------------------------ factor
def chol_inverse_upper(H: torch.Tensor, perm: Optional[torch.Tensor] = None, U: Optional[torch.Tensor] = None,
                       info: Optional[torch.Tensor] = None):
    """(U, info): U upper with H^-1 = U^T U (of H[perm][:, perm] if perm); info int32 on device."""
    n = H.shape[0]
    _need(H, torch.float32, (n, n), "H")
    if U is None:
        U = torch.empty((n, n), dtype=torch.float32, device=H.device)
    if info is None:
        info = torch.empty(1, dtype=torch.int32, device=H.device)
    nb = lib().pwq_chol_workspace_size(n)
    ws = _ws(nb, H.device)
    _check("pwq_chol_inverse_upper", lib().pwq_chol_inverse_upper(_p(H), n, _p(perm), _p(U), _p(info), _p(ws), nb, _stream(H)))
    return U, info


# ------------------------------------------------------------------ GPTQ / RTN
def _n_groups(d_in: int, group_size: int) -> int:
    return 1 if group_size == 0 else -(-d_in // group_size)


def gptq_quantize_layer(W: torch.Tensor, U: torch.Tensor, info: torch.Tensor, bits: int = 4, group_size: int = 128,
                        block_size: int = 128, perm: Optional[torch.Tensor] = None,
                        scales_in: Optional[torch.Tensor] = None, want_codes: bool = True, want_packed: bool = True,
                        out: Optional[dict] = None) -> dict:
    """GPTQ column loop.  Returns {codes (int8, original order), packed (uint8), scales (float16,
    groups in processing order), g_idx (int32, act-order only)}."""
    return _gptq(W, U, info, bits, group_size, block_size, perm, scales_in, None, want_codes, want_packed, out, False)


def gptq_quantize_layer_zp(W: torch.Tensor, U: torch.Tensor, info: torch.Tensor, bits: int = 4, group_size: int = 128,
                           block_size: int = 128, perm: Optional[torch.Tensor] = None,
                           scales_in: Optional[torch.Tensor] = None, zeros_in: Optional[torch.Tensor] = None,
                           want_codes: bool = True, want_packed: bool = True, out: Optional[dict] = None) -> dict:
    """GPTQ with zero-points.  As gptq_quantize_layer, with codes uint8 and zeros (uint16 as
    int16 storage, like the scales) in the result."""
    return _gptq(W, U, info, bits, group_size, block_size, perm, scales_in, zeros_in, want_codes, want_packed, out, True)


def _gptq(W, U, info, bits, group_size, block_size, perm, scales_in, zeros_in, want_codes, want_packed, out, zp):
    ldw = _rows(W, "W")
    d_out, d_in = W.shape
    act = perm is not None
    prm = PwqParams(bits, group_size, block_size, 1 if act else 0)
    dev = W.device
    ng = _n_groups(d_in, group_size)
    o = out if out is not None else {}
    if want_codes and o.get("codes") is None:
        o["codes"] = torch.empty((d_out, d_in), dtype=torch.uint8 if zp else torch.int8, device=dev)
    if want_packed and o.get("packed") is None:
        o["packed"] = torch.empty((d_out, d_in // 2), dtype=torch.uint8, device=dev)
    if o.get("scales") is None:
        o["scales"] = torch.empty((d_out, ng), dtype=torch.float16, device=dev)
    if zp and o.get("zeros") is None:
        o["zeros"] = torch.empty((d_out, ng), dtype=torch.int16, device=dev)
    if act and o.get("g_idx") is None:
        o["g_idx"] = torch.empty(d_in, dtype=torch.int32, device=dev)
    nb = lib().pwq_gptq_workspace_size(d_out, d_in, ctypes.byref(prm))
    ws = o.get("_ws")
    if ws is None or ws.numel() < nb:
        ws = _ws(nb, dev)
        o["_ws"] = ws
    codes = _p(o.get("codes") if want_codes else None)
    packed = _p(o.get("packed") if want_packed else None)
    g_idx = _p(o.get("g_idx") if act else None)
    if zp:
        _check("pwq_gptq_quantize_layer_zp", lib().pwq_gptq_quantize_layer_zp(
            _p(W), _dtype_code(W), d_out, d_in, ldw, _p(U), _p(info), ctypes.byref(prm), _p(perm), _p(scales_in),
            _p(zeros_in), codes, packed, _p(o["scales"]), _p(o["zeros"]), g_idx, _p(ws), nb, _stream(W)))
    else:
        _check("pwq_gptq_quantize_layer", lib().pwq_gptq_quantize_layer(
            _p(W), _dtype_code(W), d_out, d_in, ldw, _p(U), _p(info), ctypes.byref(prm), _p(perm), _p(scales_in),
            codes, packed, _p(o["scales"]), g_idx, _p(ws), nb, _stream(W)))
    return o


def rtn_quantize(W: torch.Tensor, bits: int = 4, group_size: int = 128, scales_in: Optional[torch.Tensor] = None,
                 want_codes: bool = True, want_packed: bool = True, out: Optional[dict] = None) -> dict:
    return _rtn(W, bits, group_size, scales_in, None, want_codes, want_packed, out, False)


def rtn_quantize_zp(W: torch.Tensor, bits: int = 4, group_size: int = 128, scales_in: Optional[torch.Tensor] = None,
                    zeros_in: Optional[torch.Tensor] = None, want_codes: bool = True, want_packed: bool = True,
                    out: Optional[dict] = None) -> dict:
    """RTN with zero-points: codes uint8, zeros (uint16 bits in int16 storage) per row and group."""
    return _rtn(W, bits, group_size, scales_in, zeros_in, want_codes, want_packed, out, True)


def _rtn(W, bits, group_size, scales_in, zeros_in, want_codes, want_packed, out, zp):
    ldw = _rows(W, "W")
    d_out, d_in = W.shape
    dev = W.device
    ng = _n_groups(d_in, group_size)
    o = out if out is not None else {}
    if want_codes and o.get("codes") is None:
        o["codes"] = torch.empty((d_out, d_in), dtype=torch.uint8 if zp else torch.int8, device=dev)
    if want_packed and o.get("packed") is None:
        o["packed"] = torch.empty((d_out, d_in // 2), dtype=torch.uint8, device=dev)
    if o.get("scales") is None:
        o["scales"] = torch.empty((d_out, ng), dtype=torch.float16, device=dev)
    if zp and o.get("zeros") is None:
        o["zeros"] = torch.empty((d_out, ng), dtype=torch.int16, device=dev)
    codes = _p(o.get("codes") if want_codes else None)
    packed = _p(o.get("packed") if want_packed else None)
    if zp:
        _check("pwq_rtn_quantize_zp", lib().pwq_rtn_quantize_zp(
            _p(W), _dtype_code(W), d_out, d_in, ldw, bits, group_size, _p(scales_in), _p(zeros_in), codes, packed,
            _p(o["scales"]), _p(o["zeros"]), _stream(W)))
    else:
        _check("pwq_rtn_quantize", lib().pwq_rtn_quantize(
            _p(W), _dtype_code(W), d_out, d_in, ldw, bits, group_size, _p(scales_in), codes, packed, _p(o["scales"]),
            _stream(W)))
    return o


def dequant(scales: torch.Tensor, d_in: int, bits: int = 4, group_size: int = 128, packed: Optional[torch.Tensor] = None,
            codes: Optional[torch.Tensor] = None, g_idx: Optional[torch.Tensor] = None, out_dtype=torch.float16,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    d_out = scales.shape[0]
    src = packed if packed is not None else codes
    if out is None:
        out = torch.empty((d_out, d_in), dtype=out_dtype, device=src.device)
    _check("pwq_dequant", lib().pwq_dequant(_p(packed), _p(codes), _p(scales), _p(g_idx), d_out, d_in, bits, group_size,
                                            _p(out), _dtype_code(out), _stream(src)))
    return out


def dequant_zp(scales: torch.Tensor, zeros: torch.Tensor, d_in: int, bits: int = 4, group_size: int = 128,
               packed: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
               g_idx: Optional[torch.Tensor] = None, out_dtype=torch.float16,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """What = S (code - Z) from unsigned codes or nibbles, scales and zeros."""
    d_out = scales.shape[0]
    src = packed if packed is not None else codes
    if out is None:
        out = torch.empty((d_out, d_in), dtype=out_dtype, device=src.device)
    _check("pwq_dequant_zp", lib().pwq_dequant_zp(_p(packed), _p(codes), _p(scales), _p(zeros), _p(g_idx), d_out, d_in,
                                                  bits, group_size, _p(out), _dtype_code(out), _stream(src)))
    return out


def recon_mse(X: torch.Tensor, W: torch.Tensor, scales: torch.Tensor, bits: int = 4, group_size: int = 128,
              packed: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
              g_idx: Optional[torch.Tensor] = None, mse: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = None, zeros: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Device float64 scalar: mean over tokens x outputs of (X (W - What)^T)^2.  With
    ``zeros``, the codes are those of the zero-point form (pwq_recon_mse_zp)."""
    ldx, ldw = _rows(X, "X"), _rows(W, "W")
    n_tok, d_in = X.shape
    d_out = W.shape[0]
    if mse is None:
        mse = torch.empty(1, dtype=torch.float64, device=X.device)
    nb = lib().pwq_recon_mse_workspace_size(n_tok, d_in, d_out)
    if ws is None or ws.numel() < nb:
        ws = _ws(nb, X.device)
    if zeros is not None:
        _check("pwq_recon_mse_zp", lib().pwq_recon_mse_zp(
            _p(X), _dtype_code(X), n_tok, d_in, ldx, _p(W), _dtype_code(W), ldw, _p(packed), _p(codes), _p(scales),
            _p(zeros), _p(g_idx), d_out, bits, group_size, _p(mse), _p(ws), nb, _stream(X)))
    else:
        _check("pwq_recon_mse", lib().pwq_recon_mse(
            _p(X), _dtype_code(X), n_tok, d_in, ldx, _p(W), _dtype_code(W), ldw, _p(packed), _p(codes), _p(scales),
            _p(g_idx), d_out, bits, group_size, _p(mse), _p(ws), nb, _stream(X)))
    return mse


def recon_mse_hessian(H: torch.Tensor, n_tok: int, W: torch.Tensor, scales: torch.Tensor, bits: int = 4,
                      group_size: int = 128, packed: Optional[torch.Tensor] = None,
                      codes: Optional[torch.Tensor] = None, g_idx: Optional[torch.Tensor] = None,
                      zeros: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
                      mse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Device float64 scalar: the same mean square as recon_mse, through H = 2 X^T X formed over
    n_tok tokens (pwq_recon_mse_hessian); ``shift`` (device float32, e.g. hessian_damp's
    lambda_out) is what damping added to H's diagonal."""
    ldh, ldw = _rows(H, "H"), _rows(W, "W")
    d_in = H.shape[0]
    d_out = W.shape[0]
    if H.dtype != torch.float32 or H.shape != (d_in, d_in) or W.shape[1] != d_in:
        raise ValueError("H: float32 d_in x d_in matching W's columns")
    if mse is None:
        mse = torch.empty(1, dtype=torch.float64, device=W.device)
    nb = lib().pwq_recon_mse_hessian_workspace_size(d_in, d_out)
    if ws is None or ws.numel() < nb:
        ws = _ws(nb, W.device)
    _check("pwq_recon_mse_hessian", lib().pwq_recon_mse_hessian(
        _p(H), ldh, d_in, int(n_tok), _p(shift), _p(W), _dtype_code(W), ldw, _p(packed), _p(codes), _p(scales),
        _p(zeros), _p(g_idx), d_out, bits, group_size, _p(mse), _p(ws), nb, _stream(W)))
    return mse


# ------------------------------------------------------------------ activation-aware scaling
def channel_abs_mean(X: torch.Tensor) -> torch.Tensor:
    """float32 d_in: mean over tokens of |X| per input channel."""
    ldx = _rows(X, "X")
    n_tok, d_in = X.shape
    a = torch.empty(d_in, dtype=torch.float32, device=X.device)
    nb = lib().pwq_channel_abs_mean_workspace_size(n_tok, d_in)
    ws = _ws(nb, X.device)
    _check("pwq_channel_abs_mean", lib().pwq_channel_abs_mean(_p(X), _dtype_code(X), n_tok, d_in, ldx, _p(a), _p(ws), nb,
                                                              _stream(X)))
    return a


def awq_search(W: torch.Tensor, H: torch.Tensor, n_tok: int, abs_mean: torch.Tensor, bits: int = 4,
               group_size: int = 128, n_alpha: int = 21, zero_point: bool = False, want_codes: bool = True,
               want_packed: bool = True) -> dict:
    """Grid search of s = abs_mean^alpha (H undamped).  Returns {mse (float64 n_alpha), best (int32),
    s (float32 d_in), codes, packed, scales, zeros} with the RTN result of W diag(s)."""
    ldw = _rows(W, "W")
    d_out, d_in = W.shape
    # the library reads H as a dense d_in x d_in float32 matrix (row pitch d_in) and abs_mean
    # as d_in float32 values
    _need(H, torch.float32, (d_in, d_in), "H")
    _need(abs_mean, torch.float32, (d_in,), "abs_mean")
    dev = W.device
    ng = _n_groups(d_in, group_size)
    o = {"mse": torch.empty(n_alpha, dtype=torch.float64, device=dev),
         "best": torch.empty(1, dtype=torch.int32, device=dev),
         "s": torch.empty(d_in, dtype=torch.float32, device=dev),
         "scales": torch.empty((d_out, ng), dtype=torch.float16, device=dev)}
    if want_codes:
        o["codes"] = torch.empty((d_out, d_in), dtype=torch.uint8 if zero_point else torch.int8, device=dev)
    if want_packed:
        o["packed"] = torch.empty((d_out, d_in // 2), dtype=torch.uint8, device=dev)
    if zero_point:
        o["zeros"] = torch.empty((d_out, ng), dtype=torch.int16, device=dev)
    nb = lib().pwq_awq_search_workspace_size(d_out, d_in)
    ws = _ws(nb, dev)
    _check("pwq_awq_search", lib().pwq_awq_search(
        _p(W), _dtype_code(W), d_out, d_in, ldw, _p(H), n_tok, _p(abs_mean), bits, group_size, n_alpha,
        1 if zero_point else 0, _p(o["mse"]), _p(o["best"]), _p(o["s"]), _p(o.get("codes")), _p(o.get("packed")),
        _p(o["scales"]), _p(o.get("zeros")), _p(ws), nb, _stream(W)))
    return o


# ------------------------------------------------------------------ per-tensor quantizer
def tensor_scales(W: torch.Tensor, bits: int = 4, zero_point: bool = False):
    """(scales d_out x 1 float16, zeros d_out x 1 int16 or None): one quantizer for the whole
    matrix, replicated per row; pass them as fixed scales (and zeros) with group_size 0."""
    ldw = _rows(W, "W")
    d_out, d_in = W.shape
    scales = torch.empty((d_out, 1), dtype=torch.float16, device=W.device)
    zeros = torch.empty((d_out, 1), dtype=torch.int16, device=W.device) if zero_point else None
    nb = lib().pwq_tensor_scales_workspace_size()
    ws = _ws(nb, W.device)
    _check("pwq_tensor_scales", lib().pwq_tensor_scales(_p(W), _dtype_code(W), d_out, d_in, ldw, bits, _p(scales),
                                                        _p(zeros), _p(ws), nb, _stream(W)))
    return scales, zeros


# ------------------------------------------------------------------ product with What
def quantized_matmul(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, group_size: int = 128,
                     zeros: Optional[torch.Tensor] = None, out_dtype=torch.float16, out: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = X What^T (X float16 tokens x d_in; What from packed nibbles, scales and optional zeros)."""
    ldx = _rows(X, "X")
    n_tok, d_in = X.shape
    d_out = packed.shape[0]
    if out is None:
        out = torch.empty((n_tok, d_out), dtype=out_dtype, device=X.device)
    ldy = _rows(out, "Y") if n_tok > 0 else d_out
    nb = lib().pwq_quantized_matmul_workspace_size(n_tok, d_in, d_out)
    if nb and (ws is None or ws.numel() < nb):
        ws = _ws(nb, X.device)
    _check("pwq_quantized_matmul", lib().pwq_quantized_matmul(
        _p(X), _dtype_code(X), n_tok, d_in, ldx, _p(packed), _p(scales), _p(zeros), d_out, group_size, _p(out),
        _dtype_code(out), ldy, _p(ws) if nb else None, nb, _stream(X)))
    return out


def quantized_matmul_noalloc(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, out: torch.Tensor,
                             group_size: int = 128, zeros: Optional[torch.Tensor] = None) -> torch.Tensor:
    """quantized_matmul into a caller-given ``out`` through the allocation-free entry point
    (the library's static scratch array holds the partial sums; nothing is allocated)."""
    ldx = _rows(X, "X")
    n_tok, d_in = X.shape
    d_out = packed.shape[0]
    ldy = _rows(out, "Y") if n_tok > 0 else d_out
    _check("pwq_quantized_matmul_noalloc", lib().pwq_quantized_matmul_noalloc(
        _p(X), _dtype_code(X), n_tok, d_in, ldx, _p(packed), _p(scales), _p(zeros), d_out, group_size, _p(out),
        _dtype_code(out), ldy, _stream(X)))
    return out


# ------------------------------------------------------------------ 8-bit activations
# One token's calls cost less on the GPU than here, so these marshal with few torch calls: plain
# integers for pointers, the raw stream, a device switch only where another is current, and
# checks of given tensors alone.
_CODES = {torch.float32: PWQ_F32, torch.float16: PWQ_F16, torch.bfloat16: PWQ_BF16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _bad(name: str, want: str):
    raise ValueError(f"{name}: expected {want}")


def _pitch(t: torch.Tensor, name: str, dtypes, dev, shape=None) -> int:
    """Leading dimension of a matrix of `dtypes` on dev (of `shape`) whose rows do not overlap."""
    sh = t.shape
    if t.dtype not in dtypes or t.device != dev or len(sh) != 2 or (shape is not None and sh != shape):
        _bad(name, f"a {'matrix' if shape is None else tuple(shape)} of {' / '.join(map(str, dtypes))} on {dev}")
    s0, s1 = t.stride()
    if s1 != 1 and sh[1] > 1:
        _bad(name, "contiguous columns")
    if s0 < sh[1]:
        if sh[0] > 1:
            _bad(name, f"rows that do not overlap (stride {s0})")
        return sh[1]
    return s0


def _vec(t: torch.Tensor, name: str, dtypes, dev, n: int) -> int:
    """Address of a contiguous vector of n values (n or n x 1) on dev."""
    if t.dtype not in dtypes or t.device != dev or t.shape not in ((n,), (n, 1)) or not t.is_contiguous():
        _bad(name, f"{n} contiguous {' / '.join(map(str, dtypes))} on {dev}")
    return t.data_ptr()


def _on(X: torch.Tensor, call, *args):
    """call(*args) with X's device current and its current stream as the last argument."""
    dev = X.device
    if dev.type != "cuda":
        _bad("X", "a GPU tensor")
    if torch.cuda.current_device() == dev.index:
        return call(*args, _raw_stream(dev.index))
    with torch.cuda.device(dev):
        return call(*args, _raw_stream(dev.index))


def _token_outputs(o: dict, T: int, d: int, dev, want_sums: bool):
    """(codes, its pitch, scales, sums): addresses in o's tensors, which are made where missing."""
    q, ldq = o.get("codes"), d
    if q is None:
        q = o["codes"] = torch.empty(T, d, dtype=torch.int8, device=dev)
    else:
        ldq = _pitch(q, "codes", (torch.int8,), dev, (T, d))
    s = o.get("scales")
    if s is None:
        s = o["scales"] = torch.empty(T, dtype=torch.float32, device=dev)
    else:
        _vec(s, "scales", (torch.float32,), dev, T)
    n = o.get("sums")
    if n is None and want_sums:
        n = o["sums"] = torch.empty(T, dtype=torch.int32, device=dev)
    if n is not None:
        n = _vec(n, "sums", (torch.int32,), dev, T)
    return q.data_ptr(), ldq, s.data_ptr(), n


def quantize_tokens(X: torch.Tensor, channel_scale: Optional[torch.Tensor] = None, want_sums: bool = False,
                    out: Optional[dict] = None) -> dict:
    """int8 codes of activations with one float32 scale per token: {codes (tokens x d), scales
    (tokens), sums (int32, with want_sums)}.  ``channel_scale`` (float32, d): X is divided by it
    column-wise first (awq_search's ``s``).  ``out`` may hold tensors to write into (every one of
    these names that is there is written)."""
    dev = X.device
    if dev.type != "cuda":
        _bad("X", "a GPU tensor")
    ldx = _pitch(X, "X", _CODES, dev)
    T, d = X.shape
    c = None if channel_scale is None else _vec(channel_scale, "channel_scale", (torch.float32,), dev, d)
    o = out if out is not None else {}
    q, ldq, s, n = _token_outputs(o, T, d, dev, want_sums)
    _check("pwq_quantize_tokens", _on(X, lib().pwq_quantize_tokens, X.data_ptr(), _CODES[X.dtype], T, d, ldx, c, q, ldq, s, n))
    return o


def rms_norm_quantize(X: torch.Tensor, gain: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                      eps: float = 1e-5, want_codes: bool = True, want_sums: bool = False, y_dtype=None,
                      out: Optional[dict] = None) -> dict:
    """y = h * gain / sqrt(mean(h^2) + eps) with h = X + residual: {codes, scales, sums (with
    want_sums)} as quantize_tokens gives them for y, h (the sum, in X's type, with a residual;
    ``out={"h": residual}`` updates it in place), y (with ``y_dtype``: y rounded to that type,
    e.g. the float16 input of quantized_matmul; ``want_codes=False`` for y alone).  Every tensor of
    ``out`` with one of these names is written; one that shares memory with an input is refused,
    but for h as X or the residual itself."""
    dev = X.device
    if dev.type != "cuda":
        _bad("X", "a GPU tensor")
    ldx = _pitch(X, "X", _CODES, dev)
    T, d = X.shape
    o = out if out is not None else {}
    if not want_codes and (want_sums or any(o.get(k) is not None for k in ("codes", "scales", "sums"))):
        _bad("want_codes", "True, with sums or tensors for them")
    if residual is None and o.get("h") is not None:
        _bad("h", "no tensor without a residual")
    if y_dtype is None and o.get("y") is not None:
        y_dtype = o["y"].dtype
    g = None if gain is None else _vec(gain, "gain", _CODES, dev, d)
    r = h = q = s = n = y = None
    ldr = ldh = ldq = ldy = 0
    if residual is not None:
        ldr = _pitch(residual, "residual", (X.dtype,), dev, (T, d))
        r, t, ldh = residual.data_ptr(), o.get("h"), d
        if t is None:
            t = o["h"] = torch.empty(T, d, dtype=X.dtype, device=dev)
        else:
            ldh = _pitch(t, "h", (X.dtype,), dev, (T, d))
        h = t.data_ptr()
    if want_codes:
        q, ldq, s, n = _token_outputs(o, T, d, dev, want_sums)
    if y_dtype is not None:
        t, ldy = o.get("y"), d
        if t is None:
            t = o["y"] = torch.empty(T, d, dtype=y_dtype, device=dev)
        else:
            ldy = _pitch(t, "y", (y_dtype,), dev, (T, d))
        y = t.data_ptr()
    _check("pwq_rms_norm_quantize", _on(
        X, lib().pwq_rms_norm_quantize, X.data_ptr(), _CODES[X.dtype], T, d, ldx, r, ldr, g,
        PWQ_F32 if gain is None else _CODES[gain.dtype], eps, h, ldh, q, ldq, s, n, y,
        PWQ_F32 if y_dtype is None else _CODES.get(y_dtype, -1), ldy))
    return o


def quantized_matmul_int8(X: torch.Tensor, x_scales: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                          zeros: Optional[torch.Tensor] = None, x_sums: Optional[torch.Tensor] = None,
                          out_dtype=torch.float16, out: Optional[torch.Tensor] = None,
                          ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = (x_scales X) What^T in 8-bit integers: X, x_scales (and x_sums, with zeros) from
    quantize_tokens or rms_norm_quantize; codes, scales (and zeros) from the RTN or GPTQ calls
    with group_size 0 (int8 codes, or uint8 codes with zeros)."""
    dev = X.device
    if dev.type != "cuda":
        _bad("X", "a GPU tensor")
    ldx = _pitch(X, "X", (torch.int8,), dev)
    T, d_in = X.shape
    sh = codes.shape
    if (len(sh) != 2 or sh[1] != d_in or codes.dtype != (torch.int8 if zeros is None else torch.uint8) or
            codes.device != dev or not codes.is_contiguous()):
        _bad("codes", f"contiguous d_out x {d_in} int8 (uint8 with zeros) on {dev}")
    m = sh[0]
    sx, sw = _vec(x_scales, "x_scales", (torch.float32,), dev, T), _vec(scales, "scales", (torch.float16,), dev, m)
    z = n = w = None
    if zeros is not None:
        z = _vec(zeros, "zeros", (torch.int16,), dev, m)
        if x_sums is None:
            _bad("x_sums", "the token sums, with zeros")
        n = _vec(x_sums, "x_sums", (torch.int32,), dev, T)
    ldy = m
    if out is None:
        out = torch.empty(T, m, dtype=out_dtype, device=dev)
    else:
        ldy = _pitch(out, "out", _CODES, dev, (T, m))
    L = lib()
    nb = L.pwq_quantized_matmul_int8_workspace_size(T, d_in, m)
    if nb:
        if ws is None:
            ws = _ws(nb, dev)
        elif ws.device != dev or not ws.is_contiguous():
            _bad("ws", f"contiguous bytes on {dev}")
        w = ws.data_ptr()
        nb = ws.numel() * ws.element_size()
    _check("pwq_quantized_matmul_int8", _on(
        X, L.pwq_quantized_matmul_int8, X.data_ptr(), T, d_in, ldx, sx, n, codes.data_ptr(), sw, z, m, out.data_ptr(),
        _CODES.get(out.dtype, -1), ldy, w, nb))
    return out


# ------------------------------------------------------------------ one layer, end to end
def gptq_layer(W: torch.Tensor, X: torch.Tensor, bits: int = 4, group_size: int = 128, block_size: int = 128,
               damp: float = 0.01, act_order: bool = False, want_codes: bool = True, want_packed: bool = True,
               sym: bool = True) -> dict:
    """The calls of one layer in order: Hessian, damping, [act-order], factor, GPTQ
    (``sym=False``: the zero-point form)."""
    d_in = W.shape[1]
    H = torch.zeros((d_in, d_in), dtype=torch.float32, device=W.device)
    hessian_accumulate(X, H)
    lam = torch.empty(1, dtype=torch.float32, device=W.device)
    hessian_damp(H, damp, lambda_out=lam)
    perm = act_order_perm(H) if act_order else None
    U, info = chol_inverse_upper(H, perm)
    q = gptq_quantize_layer if sym else gptq_quantize_layer_zp
    res = q(W, U, info, bits, group_size, block_size, perm=perm, want_codes=want_codes, want_packed=want_packed)
    res.update({"H": H, "lambda": lam, "U": U, "info": info, "perm": perm})
    return res


# ------------------------------------------------------------------ kernel timing
PROF_CLASSES = ("xtx", "update", "columns", "rtn", "dequant", "update_split")


def profile_enable(on: bool = True) -> None:
    """Start (or stop) recording HIP events around the library's large kernels."""
    _check("pwq_profile_enable", lib().pwq_profile_enable(1 if on else 0))


def profile_read() -> dict:
    """{class: (milliseconds, algorithmic work, launches)} summed since profile_enable; clears the record."""
    n = len(PROF_CLASSES)
    ms, work, cnt = (ctypes.c_double * n)(), (ctypes.c_double * n)(), (ctypes.c_int64 * n)()
    _check("pwq_profile_read", lib().pwq_profile_read(ms, work, cnt, n))
    return {c: (ms[i], work[i], int(cnt[i])) for i, c in enumerate(PROF_CLASSES)}


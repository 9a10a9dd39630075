"""ctypes binding of the experts' step of libmoe_route.so (include/moe_experts.h):
MXFP4 quantization and the grouped product on it, the whole step for a few tokens,
SwiGLU with its 8-bit checkpoint, and its gradient.  Argument marshalling only; the
library's checks raise MoeError, and what only the tensors can show (type, shape,
contiguity, device) raises ValueError before the call.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from ._lib import MOE_BF16, MOE_FP4_E2M1, MOE_FP8_E4M3, load, ptr
from ._train import _FLOAT, _QUANT, _call_fn, _dim, _gpu, _need, _tensor

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "moe_mxfp4_quantize": [_P, _I32, _I64, _I64, _P, _P, _P],
    "moe_mxfp4_dequantize": [_P, _P, _I64, _I64, _P, _I32, _P],
    "moe_expert_product_mxfp4": [_P, _P, _I64, _I64, _P, _P, _I64, _P, _P, _I32, _I32, _P, _I32, _P],
    "moe_experts_decode": [_P, _I64, _I64, _P, _P, _I32, _I32, _I64, _P, _P, _P, _P, _I32, _P, _I32,
                           _P, _SZ, _P],
    "moe_swiglu": [_P, _I32, _I64, _I64, _P, _P, _I32, _P, _I32, _P, _P, _P],
    "moe_swiglu_backward": [_P, _I32, _P, _I32, _P, _I64, _I64, _P, _P, _I32, _P, _P, _I32, _P],
}

_BYTE = (torch.uint8,)
_bound = None


def _lib() -> ctypes.CDLL:
    """The library with the signatures of the experts' step set (once)."""
    global _bound
    if _bound is None:
        lib = load()
        for name, args in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        lib.moe_experts_decode_workspace_size.argtypes = [_I64, _I32, _I64, _I64]
        lib.moe_experts_decode_workspace_size.restype = _SZ
        _bound = lib
    return _bound


def _call(name: str, dev: int, *args) -> None:
    _call_fn(getattr(_bound or _lib(), name), dev, *args)


def _segments(packed_cnt, packed_off, dev: int) -> int:
    """E of the segments, 0 if there are none."""
    _need((packed_cnt is None) == (packed_off is None), "packed_cnt and packed_off go together")
    if packed_cnt is None:
        return 0
    E = _dim("packed_cnt", packed_cnt, 1, 0)
    _tensor("packed_cnt", packed_cnt, (E,), (torch.int32,), dev)
    _tensor("packed_off", packed_off, (E + 1,), (torch.int32,), dev)
    return E


def mxfp4_quantize(x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                   scales: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [rows,H] (bf16 or f32, H % 32 == 0) as MXFP4: uint8 codes [rows,H/2], two e2m1
    codes per byte, and uint8 scales [rows,H/32], the e8m0 exponents of the blocks of 32.
    Expert weights [E,N,H] go as w.view(E * N, H)."""
    dev = _gpu("x", x, 2)
    rows, H = x.shape
    _tensor("x", x, (rows, H), _FLOAT, dev)
    if codes is None:
        codes = torch.empty((rows, H // 2), dtype=torch.uint8, device=dev)
    else:
        _tensor("codes", codes, (rows, H // 2), _BYTE, dev)
    if scales is None:
        scales = torch.empty((rows, H // 32), dtype=torch.uint8, device=dev)
    else:
        _tensor("scales", scales, (rows, H // 32), _BYTE, dev)
    _call("moe_mxfp4_quantize", dev, ptr(x), _FLOAT[x.dtype], rows, H, ptr(codes), ptr(scales))
    return codes, scales


def mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor,
                     out_dtype: torch.dtype = torch.bfloat16,
                     y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values [rows,H] (bf16 or f32) of MXFP4 codes [rows,H/2] and scales [rows,H/32]."""
    dev = _gpu("codes", codes, 2)
    rows, H = codes.shape[0], 2 * codes.shape[1]
    _tensor("codes", codes, (rows, H // 2), _BYTE, dev)
    _tensor("scales", scales, (rows, H // 32), _BYTE, dev)
    if y is None:
        y = torch.empty((rows, H), dtype=out_dtype, device=dev)
    _tensor("y", y, (rows, H), _FLOAT, dev)
    _call("moe_mxfp4_dequantize", dev, ptr(codes), ptr(scales), rows, H, ptr(y), _FLOAT[y.dtype])
    return y


def expert_product_mxfp4(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor,
                         w_scales: torch.Tensor, packed_cnt: torch.Tensor,
                         packed_off: torch.Tensor, swiglu: bool = False,
                         y: Optional[torch.Tensor] = None,
                         out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """y [rows,N]: every packed row times its expert's weights, both MXFP4: a uint8
    [rows,H/2] with a_scales [rows,H/32], w uint8 [E,N,H/2] with w_scales [E,N,H/32].
    swiglu=True: w holds N/2 gate rows and then N/2 up rows of each expert, and y
    [rows,N/2] is silu(gate) * up.  Rows that no expert owns (packed_cnt, packed_off as
    the dispatch wrote them) are not written: give y where they must hold something."""
    dev = _gpu("a", a, 2)
    rows, H = a.shape[0], 2 * a.shape[1]
    E, N = _dim("w", w, 3, 0), w.shape[1]
    _tensor("a", a, (rows, H // 2), _BYTE, dev)
    _tensor("a_scales", a_scales, (rows, H // 32), _BYTE, dev)
    _tensor("w", w, (E, N, H // 2), _BYTE, dev)
    _tensor("w_scales", w_scales, (E, N, H // 32), _BYTE, dev)
    _tensor("packed_cnt", packed_cnt, (E,), (torch.int32,), dev)
    _tensor("packed_off", packed_off, (E + 1,), (torch.int32,), dev)
    cols = N // 2 if swiglu else N
    if y is None:
        y = torch.empty((rows, cols), dtype=out_dtype, device=dev)
    _tensor("y", y, (rows, cols), _FLOAT, dev)
    _call("moe_expert_product_mxfp4", dev, ptr(a), ptr(a_scales), rows, H, ptr(w), ptr(w_scales), N,
          ptr(packed_cnt), ptr(packed_off), E, int(swiglu), ptr(y), _FLOAT[y.dtype])
    return y


def experts_decode_workspace_size(T: int, K: int, I: int, H: int = 8192) -> int:
    return int(_lib().moe_experts_decode_workspace_size(T, K, H, I))


def experts_decode_workspace(T: int, K: int, I: int, H: int = 8192, device="cuda") -> torch.Tensor:
    """A device workspace of experts_decode for these sizes, and for any smaller ones: a
    program keeps one for its largest batch and layer (256-byte aligned, needs no
    initialisation).  The default H covers token rows of up to 8192 elements."""
    n = max(experts_decode_workspace_size(T, K, I, H), 1)
    buf = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + n]


def experts_decode(x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor, w13: torch.Tensor,
                   w2: torch.Tensor, w13_scales: Optional[torch.Tensor] = None,
                   w2_scales: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   out_dtype: torch.dtype = torch.bfloat16,
                   ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The whole experts' step of a few tokens (T*K <= 1024): out [T,H] = sum over k of
    w[t,k] * W2[e] (silu(W1[e] x[t]) * (W3[e] x[t])) with e = idx[t,k].  x bf16 [T,H], idx
    int32 and w f32 [T,K] as the gate makes them; w13 [E,2I,H] (W1's rows, then W3's) and w2
    [E,H,I] in bf16, or as MXFP4 codes [E,2I,H/2] and [E,H,I/2] with their scales."""
    dev = _gpu("x", x, 2)
    T, H = x.shape
    K = _dim("idx", idx, 2, 1)
    E, I = _dim("w13", w13, 3, 0), w13.shape[1] // 2
    _tensor("x", x, (T, H), (torch.bfloat16,), dev)
    _tensor("idx", idx, (T, K), (torch.int32,), dev)
    _tensor("w", w, (T, K), (torch.float32,), dev)
    mx = w13_scales is not None
    _need(mx == (w2_scales is not None), "w13_scales and w2_scales go together")
    pack = 2 if mx else 1
    types = _BYTE if mx else (torch.bfloat16,)
    _tensor("w13", w13, (E, 2 * I, H // pack), types, dev)
    _tensor("w2", w2, (E, H, I // pack), types, dev)
    if mx:
        _tensor("w13_scales", w13_scales, (E, 2 * I, H // 32), _BYTE, dev)
        _tensor("w2_scales", w2_scales, (E, H, I // 32), _BYTE, dev)
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=dev)
    _tensor("out", out, (T, H), _FLOAT, dev)
    if ws is None:
        ws = experts_decode_workspace(T, K, I, H, torch.device("cuda", dev))
    else:
        _need(ws.dtype == torch.uint8 and ws.is_contiguous() and ws.is_cuda and ws.get_device() == dev,
              f"ws must be contiguous uint8 on cuda:{dev}")
    _call("moe_experts_decode", dev, ptr(x), T, H, ptr(idx), ptr(w), K, E, I, ptr(w13),
          ptr(w13_scales), ptr(w2), ptr(w2_scales), MOE_FP4_E2M1 if mx else MOE_BF16, ptr(out),
          _FLOAT[out.dtype], ptr(ws), ws.numel())
    return out


def swiglu(gu: torch.Tensor, packed_cnt: Optional[torch.Tensor] = None,
           packed_off: Optional[torch.Tensor] = None, save: bool = False,
           h: Optional[torch.Tensor] = None, h_dtype: Optional[torch.dtype] = None,
           codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
    """h [rows,I] = silu(gu[:, :I]) * gu[:, I:], of gu's type unless h or h_dtype says
    otherwise.  save=True returns (h, codes, scales) with the 8-bit checkpoint of gu that
    swiglu_backward takes: uint8 e4m3 codes [rows,2I] and f32 scales [rows,2I/128]
    (I % 128 == 0; fp8_dequant gives its values).  With the dispatch's packed_cnt and
    packed_off only rows that an expert owns are read and written."""
    dev = _gpu("gu", gu, 2)
    rows, I = gu.shape[0], gu.shape[1] // 2
    _tensor("gu", gu, (rows, 2 * I), _FLOAT, dev)
    E = _segments(packed_cnt, packed_off, dev)
    if h is None:
        h = torch.empty((rows, I), dtype=h_dtype or gu.dtype, device=dev)
    _tensor("h", h, (rows, I), _FLOAT, dev)
    _need(save or (codes is None and scales is None), "codes and scales need save=True")
    if save:
        if codes is None:
            codes = torch.empty((rows, 2 * I), dtype=torch.uint8, device=dev)
        else:
            _tensor("codes", codes, (rows, 2 * I), _BYTE, dev)
        if scales is None:
            scales = torch.empty((rows, 2 * I // 128), dtype=torch.float32, device=dev)
        else:
            _tensor("scales", scales, (rows, 2 * I // 128), (torch.float32,), dev)
    if rows:    # an empty tensor has no address
        _call("moe_swiglu", dev, ptr(gu), _FLOAT[gu.dtype], rows, I, ptr(packed_cnt),
              ptr(packed_off), E, ptr(h), _FLOAT[h.dtype], ptr(codes), ptr(scales))
    return (h, codes, scales) if save else h


def swiglu_backward(dh: torch.Tensor, gu: torch.Tensor, scales: Optional[torch.Tensor] = None,
                    packed_cnt: Optional[torch.Tensor] = None,
                    packed_off: Optional[torch.Tensor] = None,
                    dgu: Optional[torch.Tensor] = None, dgu_dtype: Optional[torch.dtype] = None,
                    h: Optional[torch.Tensor] = None, want_h: bool = True
                    ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradient of swiglu: (dgu [rows,2I], h [rows,I]) from dh [rows,I] and gu, which is
    what swiglu read (bf16 or f32) or its checkpoint (uint8 codes, with scales).  dgu has
    dh's type unless dgu or dgu_dtype says otherwise; h, of dgu's type, is the activation
    again, for the gradient of the second product (want_h=False leaves it out)."""
    dev = _gpu("dh", dh, 2)
    rows, I = dh.shape
    _tensor("dh", dh, (rows, I), _FLOAT, dev)
    quant = gu.dtype in _QUANT
    _tensor("gu", gu, (rows, 2 * I), _QUANT if quant else _FLOAT, dev)
    _need(quant == (scales is not None), "scales go with uint8 codes, and with nothing else")
    if quant:
        _tensor("scales", scales, (rows, 2 * I // 128), (torch.float32,), dev)
    E = _segments(packed_cnt, packed_off, dev)
    if dgu is None:
        dgu = torch.empty((rows, 2 * I), dtype=dgu_dtype or dh.dtype, device=dev)
    _tensor("dgu", dgu, (rows, 2 * I), _FLOAT, dev)
    _need(want_h or h is None, "h is given, but want_h=False")
    if want_h and h is None:
        h = torch.empty((rows, I), dtype=dgu.dtype, device=dev)
    if h is not None:
        _tensor("h", h, (rows, I), (dgu.dtype,), dev)
    if rows:
        _call("moe_swiglu_backward", dev, ptr(dh), _FLOAT[dh.dtype], ptr(gu),
              MOE_FP8_E4M3 if quant else _FLOAT[gu.dtype], ptr(scales), rows, I, ptr(packed_cnt),
              ptr(packed_off), E, ptr(dgu), ptr(h), _FLOAT[dgu.dtype])
    return dgu, h

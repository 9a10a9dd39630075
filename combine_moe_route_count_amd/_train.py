"""ctypes binding of the training side of libmoe_route.so (include/moe_train.h):
the top-k gate, the embedding lookup and the gradients of gate, dispatch, combine
and lookup.  Argument marshalling only; the library's checks raise MoeError, and
what only the tensors can show (type, shape, contiguity, device) raises ValueError
before the call.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from ._lib import (MOE_BF16, MOE_F32, MOE_FP4_E2M1, MOE_FP8_E4M3, _check, _raw_stream, load, ptr)

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int
_F32 = ctypes.c_float
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "moe_gate": [_P, _I32, _I64, _I32, _I32, _I32, _F32, _P, _P, _P],
    "moe_gate_backward": [_P, _I32, _I64, _I32, _I32, _I32, _F32, _P, _P, _P, _P],
    "moe_combine_backward": [_P, _I32, _P, _I64, _I64, _P, _I32, _P, _I64, _P, _P, _I32, _P, _I32,
                             _P, _P, _I32, _P, _P],
    "moe_dispatch_backward": [_P, _I32, _I64, _I64, _P, _I64, _I32, _P, _P, _I32, _P],
    "moe_embedding": [_P, _I32, _I64, _I64, _P, _I32, _I64, _F32, _P, _I32, _P, _P],
    "moe_embedding_backward": [_P, _I32, _P, _I32, _I64, _I64, _I64, _F32, _I32, _P, _I32, _P, _SZ,
                               _P],
}

_bound = None


def _lib() -> ctypes.CDLL:
    """The library with the training-side signatures set (once)."""
    global _bound
    if _bound is None:
        lib = load()
        for name, args in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        lib.moe_embedding_workspace_size.argtypes = [_I64, _I64, _I64]
        lib.moe_embedding_workspace_size.restype = _SZ
        _bound = lib
    return _bound


_FLOAT = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}
_QUANT = (torch.uint8, torch.float8_e4m3fn)
_IDS = {torch.int32: 4, torch.int64: 8}


def _need(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


# The checks run on every call, and the smallest calls take a few microseconds on
# the GPU: one expression decides, and the reason is only looked for when it fails.
# dev is a device index.
def _tensor(name: str, t: torch.Tensor, shape, dtypes, dev: int) -> None:
    """t is a contiguous tensor of this shape, one of these types, on GPU dev."""
    if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return   # (a tensor off the GPU has device -1)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has type {t.dtype}, not one of {[str(d) for d in dtypes]}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")


def _gpu(name: str, t: torch.Tensor, dim: int) -> int:
    """The index of the GPU that t, of dim dimensions, is on."""
    if not t.is_cuda:
        raise ValueError(f"{name} is not on a GPU")
    if t.dim() != dim:
        raise ValueError(f"{name} has {t.dim()} dimensions, not {dim}")
    return t.get_device()


def _dim(name: str, t: torch.Tensor, dims: int, which: int) -> int:
    """Size `which` of t, which has `dims` dimensions."""
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} has {len(shape)} dimensions, not {dims}")
    return shape[which]


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_of(dev: int):
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _call(name: str, dev: int, *args) -> None:
    """The library call on GPU dev's current stream, with dev current."""
    fn = getattr(_bound or _lib(), name)
    if dev == _current_device():
        status = fn(*args, _stream_of(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _stream_of(dev))
    if status:
        _check(status)


def gate(logits: torch.Tensor, K: int, renormalize: bool = True, scale: float = 1.0,
         idx: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None
         ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The K largest logits of each token (ties to the lowest id; -inf is never
    chosen, -1 fills up) and their softmax weights times scale: idx int32 [T,K],
    w f32 [T,K], as dispatch and combine take them.  renormalize: softmax over the
    chosen logits, otherwise over all E."""
    dev = _gpu("logits", logits, 2)
    T, E = logits.shape
    _tensor("logits", logits, (T, E), _FLOAT, dev)
    if idx is None:
        idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    else:
        _tensor("idx", idx, (T, K), (torch.int32,), dev)
    if w is None:
        w = torch.empty((T, K), dtype=torch.float32, device=dev)
    else:
        _tensor("w", w, (T, K), (torch.float32,), dev)
    _call("moe_gate", dev, ptr(logits), _FLOAT[logits.dtype], T, E, K, int(renormalize), scale,
          ptr(idx), ptr(w))
    return idx, w


def gate_backward(logits: torch.Tensor, idx: torch.Tensor, dw: torch.Tensor,
                  renormalize: bool = True, scale: float = 1.0,
                  dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of gate's weights with respect to the logits, the choice idx held
    fixed: dlogits [T,E] of the logits' type."""
    dev = _gpu("logits", logits, 2)
    T, E = logits.shape
    K = _dim("idx", idx, 2, 1)
    _tensor("logits", logits, (T, E), _FLOAT, dev)
    _tensor("idx", idx, (T, K), (torch.int32,), dev)
    _tensor("dw", dw, (T, K), (torch.float32,), dev)
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    else:
        _tensor("dlogits", dlogits, (T, E), (logits.dtype,), dev)
    _call("moe_gate_backward", dev, ptr(logits), _FLOAT[logits.dtype], T, E, K, int(renormalize),
          scale, ptr(idx), ptr(dw), ptr(dlogits))
    return dlogits


def combine_backward(dout: torch.Tensor, y: Optional[torch.Tensor], tok_map: torch.Tensor,
                     w: Optional[torch.Tensor], y_scales: Optional[torch.Tensor] = None,
                     fp4: bool = False, dout_weights: Optional[torch.Tensor] = None,
                     packed_cnt: Optional[torch.Tensor] = None,
                     packed_off: Optional[torch.Tensor] = None,
                     dy: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                     dy_dtype: Optional[torch.dtype] = None, want_dy: bool = True,
                     want_dw: bool = True
                     ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients (dy, dw) of combine, combine_fp8 and combine_fp4.  y [rows,H] is
    what the combine read: bf16, f32, or uint8 e4m3 codes (fp4: e2m1, [rows,H/2])
    with y_scales.  dy [rows,H] (dout's type unless dy or dy_dtype says otherwise)
    is w * dout in the rows of tok_map; with the dispatch's packed_cnt and
    packed_off the rows no entry owns are zeroed, without them they are not
    written.  want_dy / want_dw leave one of the two out (y may be None without dw
    if dy is given, w without dy)."""
    dev = _gpu("dout", dout, 2)
    T, H = dout.shape
    K = _dim("tok_map", tok_map, 2, 1)
    _need(want_dy or want_dw, "neither dy nor dw is wanted")
    _tensor("dout", dout, (T, H), _FLOAT, dev)
    _tensor("tok_map", tok_map, (T, K), (torch.int64,), dev)
    y_dt, rows = MOE_BF16, 0
    if y is not None:
        rows = _dim("y", y, 2, 0)
        quant = y.dtype in _QUANT
        _need(y.dtype == torch.uint8 or not fp4, "fp4 rows are uint8 codes")
        _tensor("y", y, (rows, H // 2 if fp4 else H), _QUANT if quant else _FLOAT, dev)
        y_dt = MOE_FP4_E2M1 if fp4 else (MOE_FP8_E4M3 if quant else _FLOAT[y.dtype])
    elif dy is not None:
        rows = _dim("dy", dy, 2, 0)
    _need(y is not None or not want_dw, "dw needs y")
    _need(y is not None or dy is not None, "without y, dy must be given")
    if y_scales is not None:
        _tensor("y_scales", y_scales, (rows, H // 128), (torch.float32,), dev)
    if dout_weights is not None:
        _tensor("dout_weights", dout_weights, (T,), (torch.float32,), dev)
    _need((packed_cnt is None) == (packed_off is None), "packed_cnt and packed_off go together")
    E = 0
    if packed_cnt is not None:
        E = _dim("packed_cnt", packed_cnt, 1, 0)
        _tensor("packed_cnt", packed_cnt, (E,), (torch.int32,), dev)
        _tensor("packed_off", packed_off, (E + 1,), (torch.int32,), dev)
    if want_dy:
        _need(w is not None, "dy needs w")
        if dy is None:
            dy = torch.empty((rows, H), dtype=dy_dtype or dout.dtype, device=dev)
        _tensor("dy", dy, (rows, H), _FLOAT, dev)
    else:
        dy = None
    if w is not None:
        _tensor("w", w, (T, K), (torch.float32,), dev)
    if want_dw:
        if dw is None:
            dw = torch.empty((T, K), dtype=torch.float32, device=dev)
        else:
            _tensor("dw", dw, (T, K), (torch.float32,), dev)
    else:
        dw = None
    # an empty tensor has no address; with nothing to write there is nothing to call
    if not ((dy is not None and dy.numel()) or (dw is not None and dw.numel())):
        return dy, dw
    _call("moe_combine_backward", dev, ptr(dout), _FLOAT[dout.dtype], ptr(dout_weights), T, H,
          ptr(y), y_dt, ptr(y_scales), rows, ptr(tok_map), ptr(w), K, ptr(dy),
          _FLOAT[dy.dtype] if dy is not None else MOE_BF16, ptr(packed_cnt), ptr(packed_off), E,
          ptr(dw))
    return dy, dw


def dispatch_backward(dpacked: torch.Tensor, tok_map: torch.Tensor,
                      residual: Optional[torch.Tensor] = None,
                      dx: Optional[torch.Tensor] = None,
                      dx_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Gradient of the dispatches with respect to the token rows: dx [T,H] =
    residual + sum over k ascending of dpacked[tok_map[t,k]], in f32.  dx has
    residual's type, or dpacked's, unless dx or dx_dtype says otherwise; residual
    may be dx itself."""
    dev = _gpu("dpacked", dpacked, 2)
    rows, H = dpacked.shape
    T, K = _dim("tok_map", tok_map, 2, 0), tok_map.shape[1]
    _tensor("dpacked", dpacked, (rows, H), _FLOAT, dev)
    _tensor("tok_map", tok_map, (T, K), (torch.int64,), dev)
    if dx is None:
        dt = dx_dtype or (residual.dtype if residual is not None else dpacked.dtype)
        dx = torch.empty((T, H), dtype=dt, device=dev)
    _tensor("dx", dx, (T, H), _FLOAT, dev)
    if residual is not None:
        _tensor("residual", residual, (T, H), (dx.dtype,), dev)
    _call("moe_dispatch_backward", dev, ptr(dpacked), _FLOAT[dpacked.dtype], rows, H, ptr(tok_map),
          T, K, ptr(residual), ptr(dx), _FLOAT[dx.dtype])
    return dx


def embedding(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0,
              out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
              stats: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [N,H] = scale * table[ids]; ids [N] int32 or int64, a zero row for ids
    outside the table (-1 is "no token"; any other is counted into stats int32 [1]
    if given)."""
    dev = _gpu("table", table, 2)
    V, H = table.shape
    N = _dim("ids", ids, 1, 0)
    _tensor("table", table, (V, H), _FLOAT, dev)
    _tensor("ids", ids, (N,), _IDS, dev)
    if out is None:
        out = torch.empty((N, H), dtype=out_dtype or table.dtype, device=dev)
    _tensor("out", out, (N, H), _FLOAT, dev)
    if stats is not None:
        _tensor("stats", stats, (1,), (torch.int32,), dev)
    _call("moe_embedding", dev, ptr(table), _FLOAT[table.dtype], V, H, ptr(ids), _IDS[ids.dtype], N,
          scale, ptr(out), _FLOAT[out.dtype], ptr(stats))
    return out


def embedding_workspace_size(N: int, V: int, H: int) -> int:
    return int(_lib().moe_embedding_workspace_size(N, V, H))


def embedding_workspace(N: int, V: int, H: int, device="cuda") -> torch.Tensor:
    """A device workspace of embedding_backward for these sizes, and for any smaller N
    and V of the same H (256-byte aligned, needs no initialisation)."""
    n = max(embedding_workspace_size(N, V, H), 1)
    buf = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + n]


def embedding_backward(dout: torch.Tensor, ids: torch.Tensor, V: int, scale: float = 1.0,
                       accumulate: bool = False, dtable: Optional[torch.Tensor] = None,
                       dtable_dtype: torch.dtype = torch.float32,
                       ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of embedding with respect to the table: dtable [V,H] = scale * sum
    of dout[n] over ids[n] = v, n ascending, zeros for tokens that do not occur.
    accumulate=True adds to dtable (which must be given) and leaves the rows of
    tokens that do not occur alone."""
    dev = _gpu("dout", dout, 2)
    N, H = dout.shape
    _dim("ids", ids, 1, 0)
    _tensor("dout", dout, (N, H), _FLOAT, dev)
    _tensor("ids", ids, (N,), _IDS, dev)
    _need(dtable is not None or not accumulate, "accumulate needs dtable")
    if dtable is None:
        dtable = torch.empty((V, H), dtype=dtable_dtype, device=dev)
    _tensor("dtable", dtable, (V, H), _FLOAT, dev)
    if ws is None:
        ws = embedding_workspace(N, V, H, torch.device("cuda", dev))
    else:
        _need(ws.dtype == torch.uint8 and ws.is_contiguous() and ws.is_cuda and ws.get_device() == dev,
              f"ws must be contiguous uint8 on cuda:{dev}")
    _call("moe_embedding_backward", dev, ptr(dout), _FLOAT[dout.dtype], ptr(ids), _IDS[ids.dtype],
          N, V, H, scale, int(accumulate), ptr(dtable), _FLOAT[dtable.dtype], ptr(ws), ws.numel())
    return dtable

"""Operators of the recurrent layer around the solver (libpararnn_layer.so) and
of a delta-rule layer (libpararnn_delta.so).

  norm_residual   root-mean-square norm with the residual's addition, in the
                  input's type or in 8 bits with scales, and its adjoint
  matmul_fp8      product of 8-bit matrices with a scale for each block of 128:
                  the projection that makes the gate inputs u
  gated_scan      gated linear recurrence over the sequence, its adjoint, and
                  gated_step, its form for single tokens
  delta_scan      gated delta rule over the sequence, a matrix of state per head,
                  its adjoint, and delta_step, its form for single tokens
  norm_block      the norms before and after a block with the gate and the
                  residual's scale between them, and their adjoint
  matmul_int8     product of 8-bit integer matrices with a scale for each row of
                  both

Like `binding`, this module checks tensors, allocates outputs and workspace
with torch and passes raw device pointers plus torch's current HIP stream to
the C entry points of include/pararnn_layer.h, whose comments define the
operators (include/pararnn_delta.h for the delta-rule layer's). Every tensor
must be contiguous, except where a call says that it takes views, and on the
same ROCm device; a wrong type, shape or placement raises PararnnError. There is
no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import re
from typing import Optional

import torch

from .binding import BF16, F32, PKG, PararnnError, strerror

LIB_PATH = PKG / "libpararnn_layer.so"
HEADER = PKG.parent / "include" / "pararnn_layer.h"
DELTA_LIB_PATH = PKG / "libpararnn_delta.so"
DELTA_HEADER = PKG.parent / "include" / "pararnn_delta.h"

_DTYPE = {torch.float32: F32, torch.bfloat16: BF16}


class GatedOpts(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32),
        ("L", ctypes.c_int32),
        ("D", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("c", ctypes.c_float),
        ("lengths", ctypes.c_void_p),
        ("reset", ctypes.c_void_p),
    ]


class NormOpts(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int64),
        ("D", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("out", ctypes.c_int32),
        ("eps", ctypes.c_float),
    ]


class MatmulOpts(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "w_rows", "scale", "y_dtype")]


NORM_SAME, NORM_FP8, NORM_FP8_E8M0 = 0, 1, 2
BLOCK = 128  # columns that share a scale


class View(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("batch", ctypes.c_int64), ("token", ctypes.c_int64)]


class DeltaOpts(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "L", "H", "HV", "dk", "dv", "dtype")] + [
        (n, ctypes.c_float) for n in ("c", "eps", "scale")] + [("lengths", ctypes.c_void_p), ("reset", ctypes.c_void_p)]


class NormBlockOpts(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in ("D", "group", "dtype", "out")] + [
        ("eps", ctypes.c_float)] + [(n, ctypes.c_int64) for n in ("x_row", "gate_row", "residual_row")]


class Int8Opts(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "y_dtype")]


NORM_BLOCK_SAME, NORM_BLOCK_INT8 = 0, 1


def header_functions(header=HEADER) -> list[str]:
    """Names of the functions declared in include/pararnn_layer.h (or pararnn_delta.h)."""
    return re.findall(r"^\s*[a-z_0-9]+\s+(pararnn_[a-z_0-9]+)\s*\(", header.read_text(), re.M)


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise PararnnError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(str(LIB_PATH))
        P, I32, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
        G = ctypes.POINTER(GatedOpts)
        L.pararnn_gated_workspace_bytes.argtypes = [I32, G, ctypes.POINTER(SZ)]
        L.pararnn_gated_workspace_bytes.restype = I32
        L.pararnn_gated_saved_rows.argtypes = [I32]
        L.pararnn_gated_saved_rows.restype = I32
        L.pararnn_gated_scan.argtypes = [P, P, P, P, P, P, P, SZ, G, P]
        L.pararnn_gated_scan.restype = I32
        L.pararnn_gated_scan_adjoint.argtypes = [P, P, P, P, P, P, P, P, P, SZ, G, P]
        L.pararnn_gated_scan_adjoint.restype = I32
        L.pararnn_gated_step.argtypes = [P, P, P, P, P, I32, I32, I32, I32, F, P]
        L.pararnn_gated_step.restype = I32
        N = ctypes.POINTER(NormOpts)
        L.pararnn_norm_residual.argtypes = [P, P, P, P, P, P, N, P]
        L.pararnn_norm_residual.restype = I32
        L.pararnn_norm_workspace_bytes.argtypes = [N]
        L.pararnn_norm_workspace_bytes.restype = SZ
        L.pararnn_norm_residual_adjoint.argtypes = [P, P, P, P, P, P, P, SZ, N, P]
        L.pararnn_norm_residual_adjoint.restype = I32
        M = ctypes.POINTER(MatmulOpts)
        L.pararnn_matmul_fp8.argtypes = [P, P, P, P, P, P, M, P]
        L.pararnn_matmul_fp8.restype = I32
        _lib = L
    return _lib


_delta = None


def delta_lib():
    global _delta
    if _delta is None:
        if not DELTA_LIB_PATH.exists():
            raise PararnnError(f"{DELTA_LIB_PATH} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(str(DELTA_LIB_PATH))
        P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        D, V = ctypes.POINTER(DeltaOpts), ctypes.POINTER(View)
        L.pararnn_delta_workspace_bytes.argtypes = [I32, D, ctypes.POINTER(SZ)]
        L.pararnn_delta_saved_bytes.argtypes = [D, ctypes.POINTER(SZ)]
        L.pararnn_delta_scan.argtypes = [V, V, V, V, P, P, P, P, P, P, SZ, D, P]
        L.pararnn_delta_scan_adjoint.argtypes = [V, V, V, V, P, P, P, P, V, V, V, V, P, P, P, SZ, D, P]
        L.pararnn_delta_step.argtypes = [V, V, V, V, P, P, P, P, I32, D, P]
        N = ctypes.POINTER(NormBlockOpts)
        L.pararnn_norm_block.argtypes = [P] * 9 + [N, P]
        L.pararnn_norm_block_workspace_bytes.argtypes = [N, I32, ctypes.POINTER(SZ)]
        L.pararnn_norm_block_adjoint.argtypes = [P] * 15 + [SZ, N, P]
        L.pararnn_matmul_int8.argtypes = [P] * 6 + [ctypes.POINTER(Int8Opts), P]
        for n in header_functions(DELTA_HEADER):
            getattr(L, n).restype = I32
        _delta = L
    return _delta


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dev(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape: tuple, device: torch.device):
    """Checks an argument that may be None."""
    if t is None:
        return
    if (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise PararnnError(f"{name} must be a device tensor")
    if t.device != device:
        raise PararnnError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise PararnnError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise PararnnError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise PararnnError(f"{name} must be contiguous")


def _like(t, name: str, dtype: torch.dtype, shape: tuple, device: torch.device):
    """Checks an argument but for how it lies in memory."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise PararnnError(f"{name} must be a device tensor")
    if t.device != device:
        raise PararnnError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise PararnnError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise PararnnError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


_INT32 = 0x7fffffff


def _sizes32(*sizes: int):
    for n in sizes:
        if n > _INT32:
            raise PararnnError(f"every size must be at most {_INT32}, got {n}")


def _int32(*tensors: torch.Tensor):
    """Sizes go to the library as 32-bit numbers, which would be the low bits of larger ones."""
    for t in tensors:
        if t.numel() > _INT32:  # none is larger than all of them together
            _sizes32(*t.shape)


def _first(t, name: str, dims: int) -> torch.device:
    """The device of a call, from its first tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise PararnnError(f"{name} must be a device tensor")
    if t.dim() != dims:
        raise PararnnError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if not t.is_contiguous():
        raise PararnnError(f"{name} must be contiguous")
    return t.device


_get_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _launch(what: str, device: torch.device, *args):
    """The C call on torch's current stream of the tensors' device, which is
    made current for it where it is not."""
    _run(getattr(lib(), what), what, device, args)


def _launch_delta(what: str, device: torch.device, *args):
    _run(getattr(delta_lib(), what), what, device, args)


def _run(fn, what, device, args):
    i = device.index
    if _get_device() == i:
        st = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            st = fn(*args, _raw_stream(i))
    if st != 0:
        raise PararnnError(f"{what} failed: {st} ({strerror(st)})")


def _workspace(ws, need: int, device):
    """The workspace of a call and its size: the caller's, a new one, or none."""
    if ws is None:
        if need == 0:
            return None, 0
        return torch.empty(need, dtype=torch.uint8, device=device), need
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.device != device or not ws.is_contiguous() or ws.dtype != torch.uint8:
        raise PararnnError("ws must be a contiguous uint8 tensor on the inputs' device")
    return ws, ws.numel()


# ---------------------------------------------------------------------------
# gated linear recurrence

@functools.lru_cache(maxsize=1024)
def _gated_bytes(adjoint: int, B: int, L: int, D: int, dtype: int, c: float) -> int:
    n = ctypes.c_size_t()
    st = lib().pararnn_gated_workspace_bytes(adjoint, ctypes.byref(GatedOpts(B, L, D, dtype, c, None, None)),
                                             ctypes.byref(n))
    if st != 0:
        raise PararnnError(f"pararnn_gated_workspace_bytes failed: {st} ({strerror(st)})")
    return n.value


@functools.lru_cache(maxsize=1024)
def _saved_rows(L: int) -> int:
    return lib().pararnn_gated_saved_rows(L)


def _gated_opts(u, lam, c, lengths, reset):
    dev = _first(u, "u", 4)
    B, L, G, D = u.shape
    if G != 3:
        raise PararnnError("u must be [B][L][3][D]")
    _int32(u)
    if u.dtype not in _DTYPE:
        raise PararnnError(f"u must be float32 or bfloat16, got {u.dtype}")
    _dev(lam, "lam", torch.float32, (D,), dev)
    _dev(lengths, "lengths", torch.int32, (B,), dev)
    if isinstance(reset, torch.Tensor) and reset.dtype == torch.bool:
        reset = reset.view(torch.uint8)
    _dev(reset, "reset", torch.uint8, (B, L), dev)
    o = GatedOpts(B, L, D, _DTYPE[u.dtype], c, _ptr(lengths), _ptr(reset))
    return o, dev, B, L, D


def gated_scan(u: torch.Tensor, lam: torch.Tensor, *, c: float = 8.0, h0: Optional[torch.Tensor] = None,
               lengths: Optional[torch.Tensor] = None, reset: Optional[torch.Tensor] = None, save: bool = False,
               out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> dict:
    """h_t = a_t h_{t-1} + sqrt(1 - a_t^2) s(u_i) x_t, log a_t = -c softplus(lam) s(u_r).

    u [B][L][3][D] (gates r, i, x) bf16 or fp32, lam [D] fp32, h0 [B][D] fp32 or
    None (zero), lengths [B] int32 (steps of each row), reset [B][L] uint8 or
    bool (document starts). Returns dict(h [B][L][D] in u's type, hT [B][D]
    fp32 state after the last step, saved (with save=True, for the adjoint), ws).
    """
    o, dev, B, L, D = _gated_opts(u, lam, c, lengths, reset)
    _dev(h0, "h0", torch.float32, (B, D), dev)
    if out is None:
        out = torch.empty(B, L, D, dtype=u.dtype, device=dev)
    else:
        _dev(out, "out", u.dtype, (B, L, D), dev)
    ws, nws = _workspace(ws, _gated_bytes(0, B, L, D, o.dtype, c), dev)
    hT = torch.empty(B, D, dtype=torch.float32, device=dev)
    saved = (torch.empty(_saved_rows(L), B, D, dtype=torch.float32, device=dev)
             if save else None)
    _launch("pararnn_gated_scan", dev, _ptr(u), _ptr(lam), _ptr(h0), _ptr(out), _ptr(hT), _ptr(saved), _ptr(ws),
            nws, ctypes.byref(o))
    return {"h": out, "hT": hT, "saved": saved, "ws": ws}


def gated_scan_adjoint(u: torch.Tensor, lam: torch.Tensor, dh: torch.Tensor, saved: torch.Tensor, *,
                       c: float = 8.0, dhT: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                       reset: Optional[torch.Tensor] = None, want_dlam: bool = True, want_dh0: bool = False,
                       du: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> dict:
    """Adjoint of gated_scan for dh = dL/dh [B][L][D] (u's type) and dhT = dL/dhT
    [B][D] fp32 or None; `saved` and the options are those of the forward call.
    Returns dict(du [B][L][3][D] in u's type, dlam [D], dh0 [B][D], ws)."""
    o, dev, B, L, D = _gated_opts(u, lam, c, lengths, reset)
    _dev(dh, "dh", u.dtype, (B, L, D), dev)
    _dev(saved, "saved", torch.float32, (_saved_rows(L), B, D), dev)
    if saved is None:
        raise PararnnError("the adjoint needs the states saved by gated_scan(save=True)")
    _dev(dhT, "dhT", torch.float32, (B, D), dev)
    if du is None:
        du = torch.empty(B, L, 3, D, dtype=u.dtype, device=dev)
    else:
        _dev(du, "du", u.dtype, (B, L, 3, D), dev)
    ws, nws = _workspace(ws, _gated_bytes(1, B, L, D, o.dtype, c), dev)
    dlam = torch.empty(D, dtype=torch.float32, device=dev) if want_dlam else None
    dh0 = torch.empty(B, D, dtype=torch.float32, device=dev) if want_dh0 else None
    _launch("pararnn_gated_scan_adjoint", dev, _ptr(u), _ptr(lam), _ptr(saved), _ptr(dh), _ptr(dhT), _ptr(du),
            _ptr(dlam), _ptr(dh0), _ptr(ws), nws, ctypes.byref(o))
    return {"du": du, "dlam": dlam, "dh0": dh0, "ws": ws}


def gated_step(u: torch.Tensor, lam: torch.Tensor, state: torch.Tensor, *, c: float = 8.0,
               slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One step for each of B requests, u [B][3][D]: updates the rows slots[b]
    (int32 [B]; None: row b) of the pool `state` [S][D] fp32 in place and
    returns h [B][D] in u's type. A slot outside 0..S-1 (-1, say) is a row
    without a request: h = 0. The slots must differ from each other."""
    dev = _first(u, "u", 3)
    B, G, D = u.shape
    if G != 3:
        raise PararnnError("u must be [B][3][D]")
    if u.dtype not in _DTYPE:
        raise PararnnError(f"u must be float32 or bfloat16, got {u.dtype}")
    _dev(lam, "lam", torch.float32, (D,), dev)
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise PararnnError("state must be [S][D]")
    S = state.shape[0]
    _int32(u, state)
    _dev(state, "state", torch.float32, (S, D), dev)
    _dev(slots, "slots", torch.int32, (B,), dev)
    if out is None:
        out = torch.empty(B, D, dtype=u.dtype, device=dev)
    else:
        _dev(out, "out", u.dtype, (B, D), dev)
    _launch("pararnn_gated_step", dev, _ptr(u), _ptr(lam), _ptr(slots), _ptr(state), _ptr(out), B, D, S,
            _DTYPE[u.dtype], c)
    return out


# ---------------------------------------------------------------------------
# norm

@functools.lru_cache(maxsize=1024)
def _norm_bytes(N: int, D: int, dtype: int) -> int:
    return lib().pararnn_norm_workspace_bytes(ctypes.byref(NormOpts(N, D, dtype, NORM_SAME, 0.0)))


def norm_residual(x: torch.Tensor, w: torch.Tensor, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  scale_dtype: Optional[torch.dtype] = None) -> dict:
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * w over the last of the
    two dimensions of x [N][D] (bf16 or fp32); w [D] fp32.

    scale_dtype None: y in x's type. torch.float32 or torch.float8_e8m0fnu: y in
    float8_e4m3fn with one scale of that type per row and 128 columns, laid out
    [ceil(D/128)][N] as matmul_fp8 takes them. Returns dict(y, s, scale); s is x
    itself without a residual.
    """
    dev = _first(x, "x", 2)
    N, D = x.shape
    _sizes32(D)
    if x.dtype not in _DTYPE:
        raise PararnnError(f"x must be float32 or bfloat16, got {x.dtype}")
    _dev(residual, "residual", x.dtype, (N, D), dev)
    _dev(w, "w", torch.float32, (D,), dev)
    scale = None
    if scale_dtype is None:
        out = NORM_SAME
        y = torch.empty_like(x)
    else:
        if scale_dtype not in (torch.float32, torch.float8_e8m0fnu):
            raise PararnnError(f"scale_dtype must be float32 or float8_e8m0fnu, got {scale_dtype}")
        out = NORM_FP8 if scale_dtype == torch.float32 else NORM_FP8_E8M0
        y = torch.empty(N, D, dtype=torch.float8_e4m3fn, device=dev)
        scale = torch.empty(-(-D // BLOCK), N, dtype=scale_dtype, device=dev)
    s = x if residual is None else torch.empty_like(x)
    o = NormOpts(N, D, _DTYPE[x.dtype], out, eps)
    _launch("pararnn_norm_residual", dev, _ptr(x), _ptr(residual), _ptr(w), None if s is x else _ptr(s), _ptr(y),
            _ptr(scale), ctypes.byref(o))
    return {"y": y, "s": s, "scale": scale}


def norm_residual_adjoint(s: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, *, ds: Optional[torch.Tensor] = None,
                          eps: float = 1e-6, want_dw: bool = True, ws: Optional[torch.Tensor] = None) -> dict:
    """Adjoint of norm_residual at its sum s [N][D], for dy = dL/dy and ds, the
    gradient that reaches s by its other uses (None: zero). Returns dict(dx, the
    gradient of x and of the residual, in s's type, dw [D] fp32, ws)."""
    dev = _first(s, "s", 2)
    N, D = s.shape
    _sizes32(D)
    if s.dtype not in _DTYPE:
        raise PararnnError(f"s must be float32 or bfloat16, got {s.dtype}")
    _dev(w, "w", torch.float32, (D,), dev)
    _dev(dy, "dy", s.dtype, (N, D), dev)
    _dev(ds, "ds", s.dtype, (N, D), dev)
    o = NormOpts(N, D, _DTYPE[s.dtype], NORM_SAME, eps)
    dw, nws = None, 0
    if want_dw:
        need = _norm_bytes(N, D, o.dtype)
        if need == 0:
            raise PararnnError("invalid sizes (norm_residual takes at most 16384 columns)")
        ws, nws = _workspace(ws, need, dev)
        dw = torch.empty(D, dtype=torch.float32, device=dev)
    dx = torch.empty_like(s)
    _launch("pararnn_norm_residual_adjoint", dev, _ptr(s), _ptr(w), _ptr(dy), _ptr(ds), _ptr(dx), _ptr(dw),
            _ptr(ws), nws, ctypes.byref(o))
    return {"dx": dx, "dw": dw, "ws": ws}


# ---------------------------------------------------------------------------
# 8-bit product

_SCALE = {torch.float32: 0, torch.float8_e8m0fnu: 1}


def quantize_weight(w: torch.Tensor, *, rows: int = 128, scale_dtype: torch.dtype = torch.float32):
    """Lays out a weight matrix [N][K] for matmul_fp8, once: (w in
    float8_e4m3fn, sw [ceil(N/rows)][ceil(K/128)]) with scale = max(max|w|,
    2^-100) / 448 over each rows x 128 block (rows 128 or 1), or the next power
    of two at or above it for scale_dtype float8_e8m0fnu. Works on any device."""
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or not w.is_floating_point():
        raise PararnnError("w must be a floating-point matrix [N][K]")
    if rows not in (1, BLOCK):
        raise PararnnError(f"rows must be 1 or {BLOCK}, got {rows}")
    if scale_dtype not in _SCALE:
        raise PararnnError(f"scale_dtype must be float32 or float8_e8m0fnu, got {scale_dtype}")
    N, K = w.shape
    nb, kb = -(-N // rows), -(-K // BLOCK)
    v = torch.nn.functional.pad(w.float(), (0, kb * BLOCK - K, 0, nb * rows - N)).view(nb, rows, kb, BLOCK)
    scale = v.abs().amax(dim=(1, 3)).clamp_min(2.0 ** -100)
    scale = scale / scale.new_full((), 448.0)  # by a Python number the card multiplies by a rounded reciprocal
    sw = scale
    if scale_dtype != torch.float32:
        m, e = torch.frexp(scale)
        e = torch.where(m == 0.5, e - 1, e)
        sw = torch.where(torch.isfinite(scale), e + 127, 255).to(torch.uint8).view(scale_dtype)
        scale = scale_values(sw)  # torch.ldexp on the card is a power, and good to an ulp only
    q = (v / scale[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    q = q.reshape(nb * rows, kb * BLOCK)[:N, :K].contiguous().view(torch.float8_e4m3fn)
    return q, sw.contiguous()


def scale_values(scale: torch.Tensor) -> torch.Tensor:
    """The fp32 values of scales of either type (exact: every e8m0 value is one)."""
    return scale.float()


def matmul_fp8(a: torch.Tensor, sa: torch.Tensor, w: torch.Tensor, sw: torch.Tensor, *,
               bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a w^T with the blocks' scales, plus bias: a [M][K] and w [N][K]
    float8_e4m3fn, sa [ceil(K/128)][M] and sw [ceil(N/128)][ceil(K/128)] or
    [N][ceil(K/128)], both float32 or both float8_e8m0fnu, bias [N] fp32.
    Returns [M][N] in out_dtype (bfloat16 or float32)."""
    dev = _first(a, "a", 2)
    M, K = a.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise PararnnError("w must be [N][K]")
    N = w.shape[0]
    _int32(a, w)
    _dev(a, "a", torch.float8_e4m3fn, (M, K), dev)
    _dev(w, "w", torch.float8_e4m3fn, (N, K), dev)
    KB = -(-K // BLOCK)
    if not isinstance(sa, torch.Tensor) or sa.dtype not in _SCALE:
        raise PararnnError("sa must be float32 or float8_e8m0fnu")
    _dev(sa, "sa", sa.dtype, (KB, M), dev)
    if not isinstance(sw, torch.Tensor):
        raise PararnnError("sw must be a device tensor")
    rows = 1 if N > 1 and sw.shape == (N, KB) else BLOCK
    _dev(sw, "sw", sa.dtype, (-(-N // rows), KB), dev)
    _dev(bias, "bias", torch.float32, (N,), dev)
    if out_dtype not in _DTYPE:
        raise PararnnError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=dev)
    else:
        _dev(out, "out", out_dtype, (M, N), dev)
    o = MatmulOpts(M, N, K, rows, _SCALE[sa.dtype], _DTYPE[out_dtype])
    _launch("pararnn_matmul_fp8", dev, _ptr(a), _ptr(sa), _ptr(w), _ptr(sw), _ptr(bias), _ptr(out), ctypes.byref(o))
    return out


# ---------------------------------------------------------------------------
# gated delta rule

def _view(t, name: str, dtype, shape: tuple, device) -> View:
    """A tensor [B][L][...] (or [B][...] of a step) that is packed from its third
    (second) dimension on; its rows and tokens may lie further apart."""
    _like(t, name, dtype, shape, device)
    lead = len(shape) - 2  # [B] or [B][L]
    size, n = shape, shape[-1] * shape[-2]
    if t.is_contiguous():
        return View(t.data_ptr(), n * shape[1] if lead == 2 else n, n)
    stride = t.stride()
    packed = (size[-1] == 1 or stride[-1] == 1) and (size[-2] == 1 or stride[-2] == size[-1])
    token = stride[1] if lead == 2 and size[1] > 1 else n
    batch = stride[0] if size[0] > 1 else token * (size[1] if lead == 2 else 1)
    if not packed or token < n or batch < (token * (size[1] - 1) + n if lead == 2 else n):
        raise PararnnError(f"{name} must be packed in its last two dimensions, its rows and tokens apart")
    return View(t.data_ptr(), batch, token)


def _delta_opts(q, k, v, gates, lam, c, eps, scale, lead, lengths=None, reset=None):
    """Options, views and device of a call; lead: dimensions in front of the heads."""
    for t, name in ((q, "q"), (v, "v")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise PararnnError(f"{name} must be a device tensor")
        if t.dim() != lead + 2:
            raise PararnnError(f"{name} must have {lead + 2} dimensions, got {t.dim()}")
    if q.dtype not in _DTYPE:
        raise PararnnError(f"q must be float32 or bfloat16, got {q.dtype}")
    dev, at = q.device, tuple(q.shape[:lead])
    H, dk = q.shape[lead:]
    HV, dv = v.shape[lead:]
    if 0 in q.shape or 0 in v.shape or HV % H:
        raise PararnnError("q, k and v must not be empty, and v's heads a multiple of q's")
    _int32(q, v)
    dt, qk = q.dtype, (*at, H, dk)
    views = (_view(q, "q", dt, qk, dev), _view(k, "k", dt, qk, dev), _view(v, "v", dt, (*at, HV, dv), dev),
             _view(gates, "gates", dt, (*at, 2, HV), dev))
    _dev(lam, "lam", torch.float32, (HV,), dev)
    if lam is None:
        raise PararnnError("lam must be a device tensor")
    B, L = at[0], at[1] if lead == 2 else 1
    _dev(lengths, "lengths", torch.int32, (B,), dev)
    if isinstance(reset, torch.Tensor) and reset.dtype == torch.bool:
        reset = reset.view(torch.uint8)
    _dev(reset, "reset", torch.uint8, (B, L), dev)
    o = DeltaOpts(B, L, H, HV, dk, dv, _DTYPE[q.dtype], c, eps, dk ** -0.5 if scale is None else scale,
                  _ptr(lengths), _ptr(reset))
    return o, views, dev


@functools.lru_cache(maxsize=1024)
def _delta_bytes(kind: int, B: int, L: int, H: int, HV: int, dk: int, dv: int, dtype: int) -> int:
    """Workspace of the forward (0) and the adjoint (1), bytes of `saved` (2)."""
    n = ctypes.c_size_t()
    o = DeltaOpts(B, L, H, HV, dk, dv, dtype, 1.0, 1.0, 1.0, None, None)
    L_ = delta_lib()
    st = (L_.pararnn_delta_saved_bytes(ctypes.byref(o), ctypes.byref(n)) if kind == 2
          else L_.pararnn_delta_workspace_bytes(kind, ctypes.byref(o), ctypes.byref(n)))
    if st != 0:
        raise PararnnError(f"invalid sizes (dk at most 128, dv at most 512): {st} ({strerror(st)})")
    return n.value


def delta_scan(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gates: torch.Tensor, lam: torch.Tensor, *,
               c: float = 8.0, eps: float = 1e-6, scale: Optional[float] = None, s0: Optional[torch.Tensor] = None,
               lengths: Optional[torch.Tensor] = None, reset: Optional[torch.Tensor] = None, save: bool = False,
               out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> dict:
    """S_t = a S_{t-1} + k b (v - a S_{t-1}^T k)^T, o_t = scale S_t^T q for unit q
    and k; log a = -c softplus(lam) s(gate_0), b = s(gate_1).

    q, k [B][L][H][dk] (any lengths; made unit here), v [B][L][HV][dv] and gates
    [B][L][2][HV], all bf16 or all fp32, views whose last two dimensions are
    packed (columns of one product, say); value head v takes head v // (HV // H) of
    q and k. lam [HV] fp32, s0 [B][HV][dk][dv] fp32 or None (zero), lengths and
    reset as in gated_scan (but an infinity or a NaN among a row's steps reaches those
    after it, over a start too, and in the adjoint those in front of it); scale None:
    dk^-1/2. dk at most 128, dv at most 512.
    Returns dict(o [B][L][HV][dv], sT [B][HV][dk][dv] fp32 state after the last
    step, saved (with save=True, for the adjoint), ws). saved is the fp32 state in
    front of every 64 steps and the values between: 4 dv (dk + 64) bytes of each value
    head (dk, dv up to multiples of 32), 0.4 GB for B = 8 L = 4096 and 8 heads of 128 x
    128; ws 0.16 GB there, the adjoint's 0.56.
    """
    o, views, dev = _delta_opts(q, k, v, gates, lam, c, eps, scale, 2, lengths, reset)
    B, L, H, HV, dk, dv = o.B, o.L, o.H, o.HV, o.dk, o.dv
    _dev(s0, "s0", torch.float32, (B, HV, dk, dv), dev)
    if out is None:
        out = torch.empty(B, L, HV, dv, dtype=q.dtype, device=dev)
    else:
        _dev(out, "out", q.dtype, (B, L, HV, dv), dev)
    ws, nws = _workspace(ws, _delta_bytes(0, B, L, H, HV, dk, dv, o.dtype), dev)
    sT = torch.empty(B, HV, dk, dv, dtype=torch.float32, device=dev)
    saved = (torch.empty(_delta_bytes(2, B, L, H, HV, dk, dv, o.dtype), dtype=torch.uint8, device=dev)
             if save else None)
    _launch_delta("pararnn_delta_scan", dev, *map(ctypes.byref, views), _ptr(lam), _ptr(s0), _ptr(out), _ptr(sT),
                  _ptr(saved), _ptr(ws), nws, ctypes.byref(o))
    return {"o": out, "sT": sT, "saved": saved, "ws": ws}


def delta_scan_adjoint(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gates: torch.Tensor, lam: torch.Tensor,
                       do: torch.Tensor, saved: torch.Tensor, *, c: float = 8.0, eps: float = 1e-6,
                       scale: Optional[float] = None, dsT: Optional[torch.Tensor] = None,
                       lengths: Optional[torch.Tensor] = None, reset: Optional[torch.Tensor] = None,
                       want_dlam: bool = True, want_ds0: bool = False, out: Optional[dict] = None,
                       ws: Optional[torch.Tensor] = None) -> dict:
    """Adjoint of delta_scan for do = dL/do [B][L][HV][dv] (q's type) and dsT =
    dL/dsT [B][HV][dk][dv] fp32 or None; `saved` and the options are those of the
    forward call. out: a dict of tensors or views dq, dk, dv, dgates to write to.
    Returns dict(dq, dk, dv, dgates in the inputs' shapes and type, dlam [HV], ds0
    [B][HV][dk][dv] fp32, ws)."""
    o, views, dev = _delta_opts(q, k, v, gates, lam, c, eps, scale, 2, lengths, reset)
    B, L, H, HV, dk, dv = o.B, o.L, o.H, o.HV, o.dk, o.dv
    _dev(do, "do", q.dtype, (B, L, HV, dv), dev)
    _dev(saved, "saved", torch.uint8, (_delta_bytes(2, B, L, H, HV, dk, dv, o.dtype),), dev)
    if saved is None or do is None:
        raise PararnnError("the adjoint needs do and the states saved by delta_scan(save=True)")
    _dev(dsT, "dsT", torch.float32, (B, HV, dk, dv), dev)
    g = {}
    for n, t in (("dq", q), ("dk", k), ("dv", v), ("dgates", gates)):
        g[n] = (out or {}).get(n)
        if g[n] is None:
            g[n] = torch.empty(t.shape, dtype=q.dtype, device=dev)
    outs = tuple(_view(g[n], n, q.dtype, t.shape, dev) for n, t in (("dq", q), ("dk", k), ("dv", v), ("dgates", gates)))
    ws, nws = _workspace(ws, _delta_bytes(1, B, L, H, HV, dk, dv, o.dtype), dev)
    dlam = torch.empty(HV, dtype=torch.float32, device=dev) if want_dlam else None
    ds0 = torch.empty(B, HV, dk, dv, dtype=torch.float32, device=dev) if want_ds0 else None
    _launch_delta("pararnn_delta_scan_adjoint", dev, *map(ctypes.byref, views), _ptr(lam), _ptr(saved), _ptr(do),
                  _ptr(dsT), *map(ctypes.byref, outs), _ptr(dlam), _ptr(ds0), _ptr(ws), nws, ctypes.byref(o))
    return {**g, "dlam": dlam, "ds0": ds0, "ws": ws}


def delta_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gates: torch.Tensor, lam: torch.Tensor,
               state: torch.Tensor, *, c: float = 8.0, eps: float = 1e-6, scale: Optional[float] = None,
               slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One step for each of B requests, q, k [B][H][dk], v [B][HV][dv], gates
    [B][2][HV] (views as in delta_scan): updates the entries slots[b] (int32 [B];
    None: entry b) of the pool `state` [S][HV][dk][dv] fp32 in place and returns o
    [B][HV][dv]. A slot outside 0..S-1 (-1, say) is a row without a request: o =
    0. The slots must differ from each other."""
    o, views, dev = _delta_opts(q, k, v, gates, lam, c, eps, scale, 1)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise PararnnError("state must be [S][HV][dk][dv]")
    S = state.shape[0]
    _int32(state)
    _dev(state, "state", torch.float32, (S, o.HV, o.dk, o.dv), dev)
    _dev(slots, "slots", torch.int32, (o.B,), dev)
    if out is None:
        out = torch.empty(o.B, o.HV, o.dv, dtype=q.dtype, device=dev)
    else:
        _dev(out, "out", q.dtype, (o.B, o.HV, o.dv), dev)
    _launch_delta("pararnn_delta_step", dev, *map(ctypes.byref, views), _ptr(lam), _ptr(slots), _ptr(state), _ptr(out),
                  S, ctypes.byref(o))
    return out


# ---------------------------------------------------------------------------
# norms around a block

def _rows_of(t, name: str, dtype, shape: tuple, device) -> int:
    """Checks [N][D] whose rows may lie apart; the elements from row to row."""
    _like(t, name, dtype, shape, device)
    N, D = shape
    row = t.stride(0) if N > 1 else D
    if (D > 1 and t.stride(1) != 1) or row < D:
        raise PararnnError(f"{name} must have contiguous rows that do not overlap")
    return row


def _norm_block_opts(x, w, gate, group, alpha, w_next, eps, residual: bool):
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 2:
        raise PararnnError("x must be a device tensor [N][D]")
    dev, (N, D) = x.device, x.shape
    if x.dtype not in _DTYPE:
        raise PararnnError(f"x must be float32 or bfloat16, got {x.dtype}")
    if 0 in x.shape:
        raise PararnnError("x must not be empty")
    _sizes32(D)
    group = D if group is None else group
    if not isinstance(group, int) or group < 1 or D % group:
        raise PararnnError(f"group must be a divisor of {D}, got {group}")
    if not residual and (alpha is not None or w_next is not None):
        raise PararnnError("alpha and w_next go with a residual")
    if residual and w_next is None:
        raise PararnnError("a residual needs w_next")
    if not residual and w is None:
        raise PararnnError("w or a residual must be given")
    _dev(w, "w", torch.float32, (group,), dev)
    _dev(alpha, "alpha", torch.float32, (D,), dev)
    _dev(w_next, "w_next", torch.float32, (D,), dev)
    o = NormBlockOpts(N, D, group, _DTYPE[x.dtype], NORM_BLOCK_SAME, eps, _rows_of(x, "x", x.dtype, (N, D), dev), D, D)
    if gate is not None:
        o.gate_row = _rows_of(gate, "gate", x.dtype, (N, D), dev)
    return o, dev, N, D


def norm_block(x: torch.Tensor, *, w: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
               group: Optional[int] = None, residual: Optional[torch.Tensor] = None,
               alpha: Optional[torch.Tensor] = None, w_next: Optional[torch.Tensor] = None, eps: float = 1e-6,
               out_dtype: Optional[torch.dtype] = None) -> dict:
    """p = x / sqrt(mean(x^2) + eps) * w * gate * s(gate); with a residual s =
    residual + alpha p and y = s / sqrt(mean(s^2) + eps) * w_next, else y = p.

    x, gate, residual [N][D] bf16 or fp32, rows may lie apart (columns of a wider
    matrix); w [group] fp32 norms groups of that many columns (None: all D; w None:
    x is not normed), alpha (None: ones) and w_next [D] fp32. out_dtype torch.int8:
    y in 8-bit integers with a scale per row, as matmul_int8 takes them. Groups of
    less than D beside a residual or an 8-bit y: 8, 16, 32, ... 512 columns.
    Returns dict(y, s (None without a residual), scale [N] fp32 or None).
    """
    o, dev, N, D = _norm_block_opts(x, w, gate, group, alpha, w_next, eps, residual is not None)
    s = scale = None
    if residual is not None:
        o.residual_row = _rows_of(residual, "residual", x.dtype, (N, D), dev)
        s = torch.empty(N, D, dtype=x.dtype, device=dev)
    if out_dtype is None or out_dtype == x.dtype:
        y = torch.empty(N, D, dtype=x.dtype, device=dev)
    elif out_dtype == torch.int8:
        o.out = NORM_BLOCK_INT8
        y = torch.empty(N, D, dtype=torch.int8, device=dev)
        scale = torch.empty(N, dtype=torch.float32, device=dev)
    else:
        raise PararnnError(f"out_dtype must be {x.dtype} or int8, got {out_dtype}")
    _launch_delta("pararnn_norm_block", dev, _ptr(x), _ptr(gate), _ptr(residual), _ptr(w), _ptr(alpha), _ptr(w_next),
                  _ptr(s), _ptr(y), _ptr(scale), ctypes.byref(o))
    return {"y": y, "s": s, "scale": scale}


@functools.lru_cache(maxsize=1024)
def _norm_block_bytes(N: int, D: int, group: int, dtype: int, residual: bool) -> int:
    n = ctypes.c_size_t()
    o = NormBlockOpts(N, D, group, dtype, 0, 0.0, D, D, D)
    st = delta_lib().pararnn_norm_block_workspace_bytes(ctypes.byref(o), int(residual), ctypes.byref(n))
    if st != 0:
        raise PararnnError(f"invalid sizes (norm_block takes at most 16384 columns): {st} ({strerror(st)})")
    return n.value


def norm_block_adjoint(x: torch.Tensor, dy: torch.Tensor, *, w: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None, group: Optional[int] = None,
                       s: Optional[torch.Tensor] = None, ds: Optional[torch.Tensor] = None,
                       alpha: Optional[torch.Tensor] = None, w_next: Optional[torch.Tensor] = None,
                       eps: float = 1e-6, want_params: bool = True, ws: Optional[torch.Tensor] = None) -> dict:
    """Adjoint of norm_block for dy = dL/dy [N][D] and, with a residual, ds = dL/ds
    of the other uses of s (None: zero); s is the forward call's. The other
    arguments are those of the forward call. Returns dict(dx, dgate, dresidual in
    x's type, dw [group], dalpha, dw_next [D] fp32, ws); None where there is no such
    input, and dw, dalpha, dw_next only with want_params."""
    o, dev, N, D = _norm_block_opts(x, w, gate, group, alpha, w_next, eps, s is not None)
    _dev(dy, "dy", x.dtype, (N, D), dev)
    if dy is None:
        raise PararnnError("dy must be a device tensor")
    _dev(s, "s", x.dtype, (N, D), dev)
    _dev(ds, "ds", x.dtype, (N, D), dev)
    if ds is not None and s is None:
        raise PararnnError("ds goes with a residual")
    new = lambda *shape: torch.empty(*shape, dtype=torch.float32, device=dev)  # noqa: E731
    rows = lambda on: torch.empty(N, D, dtype=x.dtype, device=dev) if on else None  # noqa: E731
    dx, dgate, dresidual = rows(True), rows(gate is not None), rows(s is not None)
    dw = new(o.group) if want_params and w is not None else None
    dalpha = new(D) if want_params and alpha is not None else None
    dw_next = new(D) if want_params and s is not None else None
    nws = 0
    if dw is not None or dw_next is not None:
        ws, nws = _workspace(ws, _norm_block_bytes(N, D, o.group, o.dtype, s is not None), dev)
    _launch_delta("pararnn_norm_block_adjoint", dev, _ptr(x), _ptr(gate), _ptr(s), _ptr(w), _ptr(alpha), _ptr(w_next),
                  _ptr(dy), _ptr(ds), _ptr(dx), _ptr(dgate), _ptr(dresidual), _ptr(dw), _ptr(dalpha), _ptr(dw_next),
                  _ptr(ws), nws, ctypes.byref(o))
    return {"dx": dx, "dgate": dgate, "dresidual": dresidual, "dw": dw, "dalpha": dalpha, "dw_next": dw_next, "ws": ws}


# ---------------------------------------------------------------------------
# 8-bit integer product

def quantize_weight_int8(w: torch.Tensor):
    """Lays out a weight matrix [N][K] for matmul_int8, once: (w in int8, sw [N])
    with scale = max(max|w|, 2^-100) / 127 over each row. Works on any device."""
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or not w.is_floating_point():
        raise PararnnError("w must be a floating-point matrix [N][K]")
    v = w.float()
    sw = v.abs().amax(dim=1).clamp_min(2.0 ** -100)
    sw = sw / sw.new_full((), 127.0)  # by a Python number the card multiplies by a rounded reciprocal
    return torch.round(v / sw[:, None]).clamp(-127, 127).nan_to_num(0.0).to(torch.int8), sw


def matmul_int8(a: torch.Tensor, sa: torch.Tensor, w: torch.Tensor, sw: torch.Tensor, *,
                bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """(a w^T) * sa * sw + bias for a [M][K] and w [N][K] int8, sa [M] and sw [N] fp32
    (scales of a's and w's rows), bias [N] fp32. The sum is exact; K at most
    131071. Returns [M][N] in out_dtype (bfloat16 or float32)."""
    dev = _first(a, "a", 2)
    M, K = a.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise PararnnError("w must be [N][K]")
    N = w.shape[0]
    _int32(a, w)
    _dev(a, "a", torch.int8, (M, K), dev)
    _dev(w, "w", torch.int8, (N, K), dev)
    if sa is None or sw is None:
        raise PararnnError("sa and sw must be device tensors")
    _dev(sa, "sa", torch.float32, (M,), dev)
    _dev(sw, "sw", torch.float32, (N,), dev)
    _dev(bias, "bias", torch.float32, (N,), dev)
    if out_dtype not in _DTYPE:
        raise PararnnError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=dev)
    else:
        _dev(out, "out", out_dtype, (M, N), dev)
    o = Int8Opts(M, N, K, _DTYPE[out_dtype])
    _launch_delta("pararnn_matmul_int8", dev, _ptr(a), _ptr(sa), _ptr(w), _ptr(sw), _ptr(bias), _ptr(out),
                  ctypes.byref(o))
    return out

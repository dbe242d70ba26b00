"""Operators of the recurrent layer around the solver (libpararnn_layer.so).

  norm_residual   root-mean-square norm with the residual's addition, in the
                  input's type or in 8 bits with scales, and its adjoint
  matmul_fp8      product of 8-bit matrices with a scale for each block of 128:
                  the projection that makes the gate inputs u
  gated_scan      gated linear recurrence over the sequence, its adjoint, and
                  gated_step, its form for single tokens

Like `binding`, this module checks tensors, allocates outputs and workspace
with torch and passes raw device pointers plus torch's current HIP stream to
the C entry points of include/pararnn_layer.h, whose comments define the
operators. Every tensor must be contiguous and on the same ROCm device; a
wrong type, shape or placement raises PararnnError. There is no fallback.
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


def header_functions() -> list[str]:
    """Names of the functions declared in include/pararnn_layer.h."""
    return re.findall(r"^\s*[a-z_0-9]+\s+(pararnn_[a-z_0-9]+)\s*\(", HEADER.read_text(), re.M)


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
    i = device.index
    fn = getattr(lib(), what)
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

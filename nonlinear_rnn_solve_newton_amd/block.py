"""A recurrent layer out of the library's operators, for training, prefill and
decoding:

  s = x + residual                      (the new residual stream)
  y = rms_norm(s) * norm_w              in 8 bits, a scale per row and 128 columns
  u = y W^T + bias                      8-bit product: the gate inputs [B][L][G][D]
  h = recurrence(u)                     gated scan, or the Newton solve of a
                                        ParaGRU / ParaLSTM cell

`RecurrentBlock` keeps the weights as the product takes them (w8 and sw of
layer.quantize_weight, which may be replaced or written between calls) and
runs the calls in order on torch's current stream. The backward pass
of the gated cell goes straight through the roundings to 8 bits; its two
products with the weights (dy = du W and dW = du^T y) are plain matrix products
in bf16.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import binding, layer
from .binding import PararnnError

GATES = {"gated": 3, "gru": 3, "lstm": 4}


class RecurrentBlock:
    """norm_w [E] fp32, w [G*D][E] (any float type; quantized here), bias [G*D]
    fp32 or None; coef: lam [D] for the gated cell, the recurrent coefficients
    a [G][D] for "gru" and "lstm". x and residual have E columns."""

    def __init__(self, cell: str, norm_w: torch.Tensor, w: torch.Tensor, coef: torch.Tensor, *,
                 bias: Optional[torch.Tensor] = None, c: float = 8.0, eps: float = 1e-6, iters: int = 3,
                 scale_dtype: torch.dtype = torch.float8_e8m0fnu):
        if cell not in GATES:
            raise PararnnError(f"cell must be one of {sorted(GATES)}, got {cell!r}")
        G = GATES[cell]
        if not all(isinstance(t, torch.Tensor) for t in (norm_w, w, coef)) or norm_w.dim() != 1:
            raise PararnnError("norm_w, w and coef must be tensors, norm_w of one dimension")
        if w.dim() != 2 or w.shape[0] % G or w.shape[1] != norm_w.shape[0]:
            raise PararnnError(f"w must be [{G}*D][{norm_w.shape[0]}], got {tuple(w.shape)}")
        self.cell, self.G, self.D, self.E = cell, G, w.shape[0] // G, w.shape[1]
        self.norm_w, self.coef, self.bias = norm_w, coef, bias
        self.c, self.eps, self.iters, self.scale_dtype = c, eps, iters, scale_dtype
        self.w8, self.sw = layer.quantize_weight(w, scale_dtype=scale_dtype)

    def _weights16(self) -> torch.Tensor:
        """The 8-bit weights' values in bf16, as dy = du W takes them. Made by each
        backward pass: a copy that is kept would miss new weights, and other streams
        and graphs than the one that made it would have to wait for it."""
        q = self.w8.to(torch.bfloat16)  # exact
        scale = self.sw.float().repeat_interleave(layer.BLOCK, 0)[:q.shape[0]]
        whole = self.E // layer.BLOCK
        cols = whole * layer.BLOCK
        if whole:  # one fp32 product each, rounded once, in place
            v = q[:, :cols].unflatten(1, (whole, layer.BLOCK))
            torch.mul(v, scale[:, :whole, None], out=v)
        if cols < self.E:
            torch.mul(q[:, cols:], scale[:, whole:], out=q[:, cols:])
        return q

    def _rows(self, t, name: str, lead) -> torch.Tensor:
        """t [*lead][E] as rows of E. As many elements in another shape would be other rows."""
        if not isinstance(t, torch.Tensor) or t.shape != (*lead, self.E):
            raise PararnnError(f"{name} must be a tensor of shape {(*lead, self.E)}, got "
                               f"{tuple(t.shape) if isinstance(t, torch.Tensor) else type(t).__name__}")
        return t.reshape(-1, self.E)

    def _dims(self, x, n: int):
        if not isinstance(x, torch.Tensor) or x.dim() != n:
            raise PararnnError(f"x must be a tensor of {n} dimensions, the last of {self.E} columns")

    def gates(self, x: torch.Tensor, residual: Optional[torch.Tensor]):
        """Gate inputs u [..., G, D] bf16 and the new residual s of rows x [..., E]."""
        lead = x.shape[:-1] if isinstance(x, torch.Tensor) else ()
        rows = self._rows(x, "x", lead)
        if residual is not None:
            residual = self._rows(residual, "residual", lead)
        n = layer.norm_residual(rows, self.norm_w, residual=residual, eps=self.eps, scale_dtype=self.scale_dtype)
        u = layer.matmul_fp8(n["y"], n["scale"], self.w8, self.sw, bias=self.bias)
        return u.view(*x.shape[:-1], self.G, self.D), n["s"].view(x.shape)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, *, state=None,
                lengths: Optional[torch.Tensor] = None, reset: Optional[torch.Tensor] = None,
                train: bool = False) -> dict:
        """x, residual [B][L][E] bf16 (without train fp32 too). state: h0 [B][D]
        (gated, gru) or (c0, h0) (lstm), None for zero; lengths and reset as in
        layer.gated_scan (gated cell only). Returns dict(h [B][L][D], s [B][L][E], state after the last
        step, ctx for backward with train=True)."""
        self._dims(x, 3)
        if train and x.dtype != torch.bfloat16:
            raise PararnnError(f"training takes x and residual in bfloat16, got {x.dtype}")
        u, s = self.gates(x, residual)
        if self.cell == "gated":
            r = layer.gated_scan(u, self.coef, c=self.c, h0=state, lengths=lengths, reset=reset, save=train)
            ctx = (u, s, r["saved"], lengths, reset) if train else None
            return {"h": r["h"], "s": s, "state": r["hT"], "ctx": ctx}
        if lengths is not None or reset is not None or train:
            raise PararnnError("lengths, reset and train are for the gated cell")
        if self.cell == "gru":
            r = binding.solve("gru", u, self.coef, h0=state, iters=self.iters)
            return {"h": r["h"], "s": s, "state": r["h"][:, -1].contiguous(), "ctx": None}
        c0, h0 = state if state is not None else (None, None)
        r = binding.solve("lstm", u, self.coef, c0=c0, h0=h0, iters=self.iters)
        return {"h": r["h"], "s": s, "state": (r["c"][:, -1].contiguous(), r["h"][:, -1].contiguous()), "ctx": None}

    def backward(self, ctx, dh: torch.Tensor, ds: Optional[torch.Tensor] = None,
                 dstate: Optional[torch.Tensor] = None) -> dict:
        """Gradients of the gated cell's forward call for dh = dL/dh [B][L][D], ds =
        dL/ds [B][L][E] and dstate = dL/dstate [B][D]: dict(dx (of x and of the
        residual), dnorm_w, dw, dbias, dcoef, dstate0). Steps past a row's length
        (whatever x, the residual and dh hold there) add nothing to the gradients
        of the weights, and their dx is ds."""
        if ctx is None:
            raise PararnnError("backward needs the ctx of forward(train=True)")
        u, s, saved, lengths, reset = ctx
        if ds is not None:
            ds = self._rows(ds, "ds", s.shape[:-1])
        a = layer.gated_scan_adjoint(u, self.coef, dh, saved, c=self.c, dhT=dstate, lengths=lengths, reset=reset,
                                     want_dh0=True)
        du = a["du"].view(-1, self.G * self.D)
        if lengths is not None:
            # padding may hold anything, and the sums over the rows would take 0 x NaN from it:
            # rows of ones there (finite also with eps 0) add the zeros that du holds
            off = torch.arange(s.shape[1], device=s.device) >= lengths[:, None]
            s = s.masked_fill(off[:, :, None], 1.0)
        rows = s.reshape(-1, self.E)
        y = layer.norm_residual(rows, self.norm_w, eps=self.eps)["y"]
        n = layer.norm_residual_adjoint(rows, self.norm_w, du @ self._weights16(), eps=self.eps, ds=ds)
        return {"dx": n["dx"].view(s.shape), "dnorm_w": n["dw"], "dw": du.t() @ y,
                "dbias": du.sum(dim=0, dtype=torch.float32), "dcoef": a["dlam"], "dstate0": a["dh0"]}

    def step(self, x: torch.Tensor, residual: Optional[torch.Tensor], state: torch.Tensor, *,
             slots: Optional[torch.Tensor] = None):
        """One token of each of B requests, x and residual [B][E]; the gated
        cell's states are the rows slots[b] of the pool `state` [S][D] and are
        updated in place. Returns (h [B][D], s [B][E])."""
        if self.cell != "gated":
            raise PararnnError("step is for the gated cell; give forward a sequence of one step")
        self._dims(x, 2)
        u, s = self.gates(x, residual)
        return layer.gated_step(u, self.coef, state, c=self.c, slots=slots), s

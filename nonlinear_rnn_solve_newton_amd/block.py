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

`DeltaBlock` is a layer whose state is a matrix per head:

  s = residual + alpha x                (the new residual stream)
  y = rms_norm(s) * norm_w              in 8-bit integers, a scale per row
  q, k, v, z, gates = y W^T             8-bit integer product, taken as it lies
  o = delta rule(q, k, v, gates)
  h = rms_norm(o by heads) * head_w * z s(z)   in 8-bit integers, a scale per row
  x = h W_out^T                         8-bit integer product: the next block's x
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


class DeltaBlock:
    """norm_w [E] fp32, w [2 H dk + 2 HV dv + 2 HV][E] (rows of q, k, v, the output's
    gate z, the decays and the write strengths; any float type, quantized here),
    lam [HV] fp32, head_w [dv] fp32, w_out [E][HV dv]; alpha [E] fp32, the scale of
    x where it is added to the residual, or None. dk at most 128; dv one of 8, 16,
    32, ... 512, or with one value head any up to 512: the heads' norm writes 8-bit
    rows, whose groups have these sizes. E and HV dv at most 16384."""

    def __init__(self, norm_w: torch.Tensor, w: torch.Tensor, lam: torch.Tensor, head_w: torch.Tensor,
                 w_out: torch.Tensor, *, heads: int, dk: int, alpha: Optional[torch.Tensor] = None, c: float = 8.0,
                 eps: float = 1e-6):
        if not all(isinstance(t, torch.Tensor) for t in (norm_w, w, lam, head_w, w_out)) or any(
                t.dim() != 1 for t in (norm_w, lam, head_w)) or w.dim() != 2 or w_out.dim() != 2:
            raise PararnnError("norm_w, lam, head_w (vectors), w and w_out (matrices) must be tensors")
        self.H, self.HV, self.dk, self.dv, self.E = heads, lam.shape[0], dk, head_w.shape[0], norm_w.shape[0]
        if heads < 1 or dk < 1 or self.HV < 1 or self.HV % heads:
            raise PararnnError(f"lam's heads ({self.HV}) must be a multiple of heads ({heads}), dk at least 1")
        if dk > 128 or not 1 <= self.dv <= 512 or (self.HV > 1 and self.dv not in (8, 16, 32, 64, 128, 256, 512)):
            raise PararnnError(f"dk must be at most 128 and dv 8, 16, 32, ... 512 (with one value head any up to 512), "
                               f"got {dk} and {self.dv}")
        if not 1 <= self.E <= 16384 or self.HV * self.dv > 16384:
            raise PararnnError(f"E and HV dv must be at most 16384, got {self.E} and {self.HV * self.dv}")
        if alpha is not None and (not isinstance(alpha, torch.Tensor) or alpha.shape != (self.E,)):
            raise PararnnError(f"alpha must be a tensor of shape {(self.E,)}")
        self.cols = (heads * dk, heads * dk, self.HV * self.dv, self.HV * self.dv, 2 * self.HV)
        if w.shape != (sum(self.cols), self.E) or w_out.shape != (self.E, self.HV * self.dv):
            raise PararnnError(f"w must be [{sum(self.cols)}][{self.E}] and w_out [{self.E}][{self.HV * self.dv}], got "
                               f"{tuple(w.shape)} and {tuple(w_out.shape)}")
        self.norm_w, self.lam, self.head_w, self.alpha, self.c, self.eps = norm_w, lam, head_w, alpha, c, eps
        self.w8, self.sw = layer.quantize_weight_int8(w)
        self.wo8, self.swo = layer.quantize_weight_int8(w_out)

    @staticmethod
    def _weights16(w8, sw):
        return (w8.float() * sw[:, None]).to(torch.bfloat16)

    def _norm(self, rows, residual, out_dtype):
        """The norm before the block: y, its scale and the new residual stream."""
        if residual is None:
            n = layer.norm_block(rows, w=self.norm_w, eps=self.eps, out_dtype=out_dtype)
            return n["y"], n["scale"], rows
        n = layer.norm_block(rows, residual=residual, alpha=self.alpha, w_next=self.norm_w, eps=self.eps,
                             out_dtype=out_dtype)
        return n["y"], n["scale"], n["s"]

    def _project(self, x, residual):
        """Columns [rows][cols] bf16 of the first product, and the residual stream."""
        if not isinstance(x, torch.Tensor) or x.dim() < 2 or x.shape[-1] != self.E:
            raise PararnnError(f"x must be a tensor with {self.E} columns")
        if residual is not None and (not isinstance(residual, torch.Tensor) or residual.shape != x.shape):
            raise PararnnError(f"residual must be a tensor of shape {tuple(x.shape)}")
        y, scale, s = self._norm(x.reshape(-1, self.E), None if residual is None else residual.reshape(-1, self.E),
                                 torch.int8)
        return layer.matmul_int8(y, scale, self.w8, self.sw), s

    def _views(self, p, lead):
        """q, k, v, z, gates as views of the product's columns."""
        q, k, v, z, g = p.split(self.cols, dim=-1)
        heads = lambda t, n, d: t.view(*lead, n, d)  # noqa: E731
        return (heads(q, self.H, self.dk), heads(k, self.H, self.dk), heads(v, self.HV, self.dv), z,
                heads(g, 2, self.HV))

    def _head_norm(self, o, z, out_dtype=None):
        return layer.norm_block(o.view(-1, self.HV * self.dv), w=self.head_w, group=self.dv, gate=z, eps=self.eps,
                                out_dtype=out_dtype)

    def _out(self, o, z, shape):
        n = self._head_norm(o, z, torch.int8)
        return layer.matmul_int8(n["y"], n["scale"], self.wo8, self.swo).view(shape)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, *,
                state: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                reset: Optional[torch.Tensor] = None, train: bool = False) -> dict:
        """x, residual [B][L][E] bf16 (without train fp32 too); state [B][HV][dk][dv]
        fp32 in front of the first step or None; lengths and reset as in
        layer.delta_scan. Returns dict(x [B][L][E] bf16, s [B][L][E], state after the
        last step, ctx for backward with train=True). Rows past a row's length hold
        what their own x makes of them, and reach no other row."""
        if not isinstance(x, torch.Tensor) or x.dim() != 3:
            raise PararnnError(f"x must be a tensor [B][L][{self.E}]")
        if train and x.dtype != torch.bfloat16:
            raise PararnnError(f"training takes x and residual in bfloat16, got {x.dtype}")
        p, s = self._project(x, residual)
        q, k, v, z, g = self._views(p, x.shape[:2])
        r = layer.delta_scan(q, k, v, g, self.lam, c=self.c, eps=self.eps, s0=state, lengths=lengths, reset=reset,
                             save=train)
        ctx = (x, s.view(x.shape), residual is not None, p, r["o"], r["saved"], lengths, reset) if train else None
        return {"x": self._out(r["o"], z, x.shape), "s": s.view(x.shape), "state": r["sT"], "ctx": ctx}

    def backward(self, ctx, dx: torch.Tensor, ds: Optional[torch.Tensor] = None,
                 dstate: Optional[torch.Tensor] = None) -> dict:
        """Gradients of a forward call for dx = dL/dx of its result [B][L][E] bf16, ds
        = dL/ds and dstate = dL/dstate, straight through the roundings to 8 bits:
        dict(dx, dresidual (None without one), dnorm_w, dalpha, dw, dlam, dhead_w,
        dw_out, dstate0). Steps past a row's length, whatever x, the residual, dx and
        ds hold there, add nothing to the gradients of the weights, and their own dx
        and dresidual are zero (what ds holds there stops here)."""
        if ctx is None:
            raise PararnnError("backward needs the ctx of forward(train=True)")
        x, s, with_residual, p, o, saved, lengths, reset = ctx
        for t, n in ((dx, "dx"), (ds, "ds")):
            if t is not None or n == "dx":
                layer._like(t, n, x.dtype, x.shape, x.device)
        lead = x.shape[:2]
        if lengths is not None:
            # padding may hold anything, and the sums over the rows would take 0 x NaN from it
            off = (torch.arange(lead[1], device=x.device) >= lengths[:, None])[:, :, None]
            x, s = x.masked_fill(off, 1.0), s.masked_fill(off, 1.0)
            dx = dx.masked_fill(off, 0.0)
            p = p.masked_fill(off.reshape(-1, 1), 0.0)
            ds = None if ds is None else ds.masked_fill(off, 0.0)
        q, k, v, z, g = self._views(p, lead)
        dout = dx.reshape(-1, self.E)
        h = self._head_norm(o, z)["y"]
        n = layer.norm_block_adjoint(o.view(-1, self.HV * self.dv), dout @ self._weights16(self.wo8, self.swo),
                                     w=self.head_w, group=self.dv, gate=z, eps=self.eps)
        dp = torch.empty_like(p)
        dq, dk, dv, dz, dg = self._views(dp, lead)
        dz.copy_(n["dgate"])
        b = layer.delta_scan_adjoint(q, k, v, g, self.lam, n["dx"].view(o.shape), saved, c=self.c, eps=self.eps,
                                     dsT=dstate, lengths=lengths, reset=reset, want_ds0=True,
                                     out={"dq": dq, "dk": dk, "dv": dv, "dgates": dg})
        rows, srows = x.reshape(-1, self.E), s.reshape(-1, self.E)
        dy = dp @ self._weights16(self.w8, self.sw)
        dsr = None if ds is None else ds.reshape(-1, self.E)
        # the norm's result again, from the saved sum: the residual stream's rows are what it norms
        y = layer.norm_block(srows, w=self.norm_w, eps=self.eps)["y"]
        out = {"dw": dp.t() @ y, "dlam": b["dlam"], "dhead_w": n["dw"], "dw_out": dout.t() @ h, "dstate0": b["ds0"]}
        if with_residual:
            m = layer.norm_block_adjoint(rows, dy, s=srows, ds=dsr, alpha=self.alpha, w_next=self.norm_w, eps=self.eps)
            out.update(dx=m["dx"].view(x.shape), dresidual=m["dresidual"].view(x.shape), dnorm_w=m["dw_next"],
                       dalpha=m["dalpha"])
        else:
            m = layer.norm_block_adjoint(rows, dy, w=self.norm_w, eps=self.eps)
            d = m["dx"] if dsr is None else m["dx"] + dsr
            out.update(dx=d.view(x.shape), dresidual=None, dnorm_w=m["dw"], dalpha=None)
        return out

    def step(self, x: torch.Tensor, residual: Optional[torch.Tensor], state: torch.Tensor, *,
             slots: Optional[torch.Tensor] = None):
        """One token of each of B requests, x and residual [B][E]; the states are the
        entries slots[b] of the pool `state` [S][HV][dk][dv] and are updated in place.
        Returns (x [B][E], s [B][E])."""
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise PararnnError(f"x must be a tensor [B][{self.E}]")
        p, s = self._project(x, residual)
        q, k, v, z, g = self._views(p, x.shape[:1])
        o = layer.delta_step(q, k, v, g, self.lam, state, c=self.c, eps=self.eps, slots=slots)
        return self._out(o, z, x.shape), s

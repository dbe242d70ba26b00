"""Contract of include/pararnn_delta.h without a GPU: every declared function is
exported, structs have the sizes the binding assumes, sizes are computed, and
invalid arguments get their status before anything is launched. Also the 64-bit
reference of the delta rule against differences and its chunked form."""
import ctypes

import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from nonlinear_rnn_solve_newton_amd.binding import BF16, F32, PararnnError
from nonlinear_rnn_solve_newton_amd.block import DeltaBlock
from tests import delta_reference as R

P = lambda v: ctypes.c_void_p(v * 4096) if v else None  # noqa: E731  (never dereferenced)
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    if not layer.DELTA_LIB_PATH.exists():
        from nonlinear_rnn_solve_newton_amd import build
        build.build_one(build.CSRC / "delta.hip", build.DELTA_LIB, device_flags=build.DELTA_FLAGS)
    return layer.delta_lib()


def test_every_declared_symbol_is_exported(lib):
    names = layer.header_functions(layer.DELTA_HEADER)
    assert set(names) == {"pararnn_delta_workspace_bytes", "pararnn_delta_saved_bytes", "pararnn_delta_scan",
                          "pararnn_delta_scan_adjoint", "pararnn_delta_step", "pararnn_norm_block",
                          "pararnn_norm_block_workspace_bytes", "pararnn_norm_block_adjoint", "pararnn_matmul_int8"}
    for n in names:
        assert hasattr(lib, n), n


def test_struct_layouts():
    assert ctypes.sizeof(layer.View) == 24 and layer.View.token.offset == 16
    assert ctypes.sizeof(layer.DeltaOpts) == 56 and layer.DeltaOpts.lengths.offset == 40
    assert ctypes.sizeof(layer.NormBlockOpts) == 56 and layer.NormBlockOpts.x_row.offset == 32
    assert ctypes.sizeof(layer.Int8Opts) == 16


def opts(B=2, L=300, H=2, HV=4, dk=64, dv=96, dtype=BF16, c=8.0, eps=1e-6, scale=0.125, lengths=None, reset=None):
    return layer.DeltaOpts(B, L, H, HV, dk, dv, dtype, c, eps, scale, lengths, reset)


BAD = [dict(B=0), dict(L=0), dict(H=0), dict(HV=0), dict(HV=3), dict(HV=-4), dict(dk=0), dict(dk=129), dict(dv=0),
       dict(dv=513), dict(c=0.0), dict(c=float("inf")), dict(c=float("nan")), dict(eps=0.0), dict(eps=float("nan")),
       dict(scale=float("inf")), dict(scale=float("nan")), dict(L=2 ** 31 - 1), dict(B=2 ** 20, L=2 ** 20)]


def test_delta_sizes(lib):
    n = ctypes.c_size_t(7)
    for adj in (0, 1):
        assert lib.pararnn_delta_workspace_bytes(adj, ctypes.byref(opts()), ctypes.byref(n)) == 0 and n.value > 0
        for kw in BAD:
            assert lib.pararnn_delta_workspace_bytes(adj, ctypes.byref(opts(**kw)), ctypes.byref(n)) == EINVAL, kw
        assert lib.pararnn_delta_workspace_bytes(adj, ctypes.byref(opts(dtype=2)), ctypes.byref(n)) == EUNSUPPORTED
    assert lib.pararnn_delta_workspace_bytes(2, ctypes.byref(opts()), ctypes.byref(n)) == EINVAL
    assert lib.pararnn_delta_workspace_bytes(0, ctypes.byref(opts()), None) == EINVAL
    assert lib.pararnn_delta_workspace_bytes(0, None, ctypes.byref(n)) == EINVAL
    assert lib.pararnn_delta_saved_bytes(ctypes.byref(opts()), ctypes.byref(n)) == 0
    # a state in front of each of 5 chunks of 64 steps, 8 heads, and the chunk's values; tiles in pairs of 16
    assert n.value == 8 * 5 * (64 * 96 + 64 * 96) * 4
    for kw in BAD:
        assert lib.pararnn_delta_saved_bytes(ctypes.byref(opts(**kw)), ctypes.byref(n)) == EINVAL, kw
    assert lib.pararnn_delta_saved_bytes(ctypes.byref(opts(dtype=9)), ctypes.byref(n)) == EUNSUPPORTED
    assert lib.pararnn_delta_saved_bytes(None, ctypes.byref(n)) == EINVAL


def views(o, B=None):
    nk, nv = o.H * o.dk, o.HV * o.dv
    return {n: layer.View(4096 * (i + 1), o.L * t, t) for i, (n, t) in
            enumerate((("q", nk), ("k", nk), ("v", nv), ("g", 2 * o.HV)))}


# what is wrong with one view: null, tokens or rows that overlap, a token too long, an odd address
WRONG = [("p", None, EINVAL), ("token", -1, EINVAL), ("token", 1, EINVAL), ("token", (1 << 22) + 1, EINVAL),
         ("batch", 5, EINVAL), ("batch", (1 << 50) + 1, EINVAL), ("p", 4097, EUNSUPPORTED)]


def test_delta_scan_invalid_arguments(lib):
    def call(o=None, ws=20, nb=1 << 40, lam=9, out=10, off=0, saved=0, **change):
        o = o or opts()
        v = views(o)
        for n, (f, x) in change.items():
            setattr(v[n], f, x)
        r = lambda n: ctypes.byref(v[n])  # noqa: E731
        return lib.pararnn_delta_scan(r("q"), r("k"), r("v"), r("g"), P(lam), None, P(out), None,
                                      ctypes.c_void_p(saved) if saved else None,
                                      ctypes.c_void_p(4096 * ws + off) if ws else None, nb, ctypes.byref(o), None)

    for kw in BAD:
        assert call(opts(**kw)) == EINVAL, kw
    assert call(opts(dtype=3)) == EUNSUPPORTED
    for n in "qkvg":
        for f, x, want in WRONG:
            assert call(**{n: (f, x)}) == want, (n, f, x)
    assert call(lam=0) == EINVAL and call(out=0) == EINVAL and call(ws=0) == EINVAL
    assert call(nb=16) == EWORKSPACE and call(off=16) == EUNSUPPORTED and call(saved=4096 + 128) == EUNSUPPORTED
    assert lib.pararnn_delta_scan(None, None, None, None, P(1), None, P(1), None, None, P(1), 1 << 40,
                                  ctypes.byref(opts()), None) == EINVAL


def test_delta_adjoint_invalid_arguments(lib):
    def call(o=None, ws=20, nb=1 << 40, saved=11, do=12, lam=9, **change):
        o = o or opts()
        v, g = views(o), views(o)
        for n, (f, x) in change.items():
            setattr((g if n[0] == "d" else v)[n[-1]], f, x)
        r = lambda t, n: ctypes.byref(t[n])  # noqa: E731
        return lib.pararnn_delta_scan_adjoint(*(r(v, n) for n in "qkvg"), P(lam), P(saved), P(do), None,
                                              *(r(g, n) for n in "qkvg"), None, None, P(ws), nb, ctypes.byref(o), None)

    for kw in BAD:
        assert call(opts(**kw)) == EINVAL, kw
    for n in ("q", "k", "v", "g", "dq", "dk", "dv", "dg"):
        for f, x, want in WRONG:
            assert call(**{n: (f, x)}) == want, (n, f, x)
    assert call(saved=0) == EINVAL and call(do=0) == EINVAL and call(lam=0) == EINVAL and call(ws=0) == EINVAL
    assert call(nb=4096) == EWORKSPACE and call(opts(dtype=7)) == EUNSUPPORTED


def test_delta_step_invalid_arguments(lib):
    def call(o=None, S=9, slots=0, state=5, out=6, lam=7, **change):
        o = o or opts(L=1)
        v = views(o)
        for n, (f, x) in change.items():
            setattr(v[n], f, x)
        return lib.pararnn_delta_step(*(ctypes.byref(v[n]) for n in "qkvg"), P(lam), P(slots), P(state), P(out), S,
                                      ctypes.byref(o), None)

    for kw in BAD[:-2]:
        if "L" not in kw:
            assert call(opts(**{"L": 1, **kw})) == EINVAL, kw
    assert call(opts(L=2)) == EINVAL and call(S=0, slots=1) == EINVAL and call(S=1) == EINVAL
    assert call(state=0) == EINVAL and call(out=0) == EINVAL and call(lam=0) == EINVAL
    assert call(opts(L=1, dtype=4)) == EUNSUPPORTED
    for n in "qkvg":
        assert call(**{n: ("p", None)}) == EINVAL and call(**{n: ("batch", 3)}) == EINVAL
        assert call(**{n: ("p", 4097)}) == EUNSUPPORTED


def test_norm_block_invalid_arguments(lib):
    def o(N=4, D=256, group=256, dtype=BF16, out=0, eps=1e-6, x_row=256, gate_row=256, residual_row=256):
        return layer.NormBlockOpts(N, D, group, dtype, out, eps, x_row, gate_row, residual_row)

    def fwd(x=1, gate=2, residual=3, w=4, alpha=5, w_next=6, s=7, y=8, scale=9, opts=None):
        return lib.pararnn_norm_block(P(x), P(gate), P(residual), P(w), P(alpha), P(w_next), P(s), P(y), P(scale),
                                      ctypes.byref(opts or o()), None)

    assert fwd(x=0) == EINVAL and fwd(y=0) == EINVAL and fwd(w_next=0) == EINVAL and fwd(s=0) == EINVAL
    assert fwd(residual=0) == EINVAL  # alpha, w_next and s without a residual
    assert fwd(residual=0, alpha=0, w_next=0, s=0, w=0) == EINVAL
    for kw in (dict(N=0), dict(D=0), dict(D=16385, group=16385, x_row=16385), dict(group=0), dict(group=100), dict(group=512),
               dict(eps=-1.0), dict(eps=float("nan")), dict(x_row=255), dict(gate_row=0), dict(residual_row=-256),
               dict(out=2)):
        assert fwd(opts=o(**kw)) == EINVAL, kw
    assert fwd(scale=0, opts=o(out=1)) == EINVAL and fwd(opts=o(dtype=5)) == EUNSUPPORTED
    # groups beside a residual or an 8-bit y are parts of a wave
    assert fwd(opts=o(D=240, group=24)) == EUNSUPPORTED and fwd(opts=o(D=240, group=4)) == EUNSUPPORTED
    assert fwd(opts=o(D=2048, group=1024, x_row=2048, gate_row=2048, residual_row=2048)) == EUNSUPPORTED
    assert fwd(residual=0, alpha=0, w_next=0, s=0, opts=o(D=240, group=24, out=1)) == EUNSUPPORTED
    n = ctypes.c_size_t()
    for res in (0, 1):
        assert lib.pararnn_norm_block_workspace_bytes(ctypes.byref(o()), res, ctypes.byref(n)) == 0 and n.value >= 1024
    assert lib.pararnn_norm_block_workspace_bytes(ctypes.byref(o(D=0)), 0, ctypes.byref(n)) == EINVAL
    assert lib.pararnn_norm_block_workspace_bytes(ctypes.byref(o()), 0, None) == EINVAL

    def adj(x=1, gate=2, s=3, w=4, alpha=5, w_next=6, dy=7, ds=8, dx=9, dgate=10, dres=11, dw=12, dal=13, dwn=14, ws=15,
            nb=1 << 30, opts=None):
        return lib.pararnn_norm_block_adjoint(P(x), P(gate), P(s), P(w), P(alpha), P(w_next), P(dy), P(ds), P(dx),
                                              P(dgate), P(dres), P(dw), P(dal), P(dwn), P(ws), nb,
                                              ctypes.byref(opts or o()), None)

    for n in ("x", "dy", "dx", "dgate", "dres", "w_next", "ws", "gate"):
        assert adj(**{n: 0}) == EINVAL, n
    assert adj(s=0) == EINVAL and adj(w=0) == EINVAL  # dw without w
    assert adj(nb=8) == EWORKSPACE and adj(opts=o(dtype=3)) == EUNSUPPORTED


def test_matmul_int8_invalid_arguments(lib):
    def mm(M=4, N=8, K=32, dt=BF16, a=1, sa=2, w=3, sw=4, y=5, off=0):
        o = layer.Int8Opts(M, N, K, dt)
        return lib.pararnn_matmul_int8(P(a), P(sa), P(w), P(sw), None, ctypes.c_void_p(4096 * y + off) if y else None,
                                       ctypes.byref(o), None)

    for n in ("a", "sa", "w", "sw", "y", "M", "N", "K"):
        assert mm(**{n: 0}) == EINVAL, n
    assert mm(K=131072) == EINVAL and mm(M=2 ** 31 - 1, N=2 ** 31 - 1) == EINVAL
    assert mm(dt=7) == EUNSUPPORTED and mm(off=1) == EUNSUPPORTED and mm(dt=F32, off=2) == EUNSUPPORTED


def test_python_entry_points_refuse_host_tensors():
    q, v, g, lam = torch.zeros(1, 2, 2, 8), torch.zeros(1, 2, 2, 4), torch.zeros(1, 2, 2, 2), torch.zeros(2)
    m = torch.zeros(2, 8)
    for f in (lambda: layer.delta_scan(q, q, v, g, lam), lambda: layer.delta_scan(None, q, v, g, lam),
              lambda: layer.delta_scan_adjoint(q, q, v, g, lam, v, None),
              lambda: layer.delta_step(q[0], q[0], v[0], g[0], lam, torch.zeros(1, 2, 8, 4)),
              lambda: layer.norm_block(m, w=torch.ones(8)), lambda: layer.norm_block(None),
              lambda: layer.norm_block_adjoint(m, m, w=torch.ones(8)),
              lambda: layer.matmul_int8(m.to(torch.int8), lam, m.to(torch.int8), lam)):
        with pytest.raises(PararnnError):
            f()


def test_block_refuses_weights_that_do_not_fit():
    E, H, HV, dk, dv = 32, 2, 4, 16, 8
    cols = 2 * H * dk + 2 * HV * dv + 2 * HV
    ok = dict(norm_w=torch.ones(E), w=torch.randn(cols, E), lam=torch.zeros(HV), head_w=torch.ones(dv),
              w_out=torch.randn(E, HV * dv))
    blk = DeltaBlock(**ok, heads=H, dk=dk)
    assert blk.w8.shape == (cols, E) and blk.wo8.shape == (E, HV * dv)
    for kw in (dict(w=torch.randn(cols + 1, E)), dict(w_out=torch.randn(E, dv)), dict(lam=torch.zeros(3)),
               dict(norm_w=torch.ones(E + 1)), dict(w=None), dict(head_w=torch.ones(1, dv))):
        with pytest.raises(PararnnError):
            DeltaBlock(**{**ok, **kw}, heads=H, dk=dk)
    for kw in (dict(heads=0, dk=dk), dict(heads=H, dk=0), dict(heads=H, dk=dk + 1)):
        with pytest.raises(PararnnError):
            DeltaBlock(**ok, **kw)


def test_quantize_weight_int8_on_the_cpu():
    w = torch.randn(130, 200, generator=torch.Generator().manual_seed(1))
    w[7] = 0
    q, s = layer.quantize_weight_int8(w)
    assert q.dtype == torch.int8 and q.shape == w.shape and s.shape == (130,) and q.abs().max() == 127
    # half a step of the row's scale, and the quotient's own rounding
    assert ((q.float() * s[:, None] - w).abs() <= s[:, None] * (0.5 + 127 * 2.0 ** -22)).all() and (q[7] == 0).all()
    for bad in (None, w[0], q):
        with pytest.raises(PararnnError):
            layer.quantize_weight_int8(bad)


def chunked(q, k, v, gates, lam, do, *, c, eps, scale, s0, dsT):
    """The chunked formulas of forward and adjoint over one chunk, in 64 bits,
    written from the equations that the kernels use (one head, no padding)."""
    n = q.shape[0]
    rq, rk = (1 / (x.square().sum(-1) + eps).sqrt() for x in (q, k))
    qh, kh = q * rq[:, None], k * rk[:, None]
    r, b = gates.sigmoid().unbind(1)
    G = (-c * torch.nn.functional.softplus(lam) * r).cumsum(0)
    E = (G[:, None] - G).exp().tril()
    kk, qk = E * (kh @ kh.T), scale * E * (qh @ kh.T)
    T = torch.linalg.inv(torch.eye(n, dtype=q.dtype) + (kk * b).tril(-1))
    X = v - G.exp()[:, None] * (kh @ s0)
    Y = T @ X
    P = (qk * b).tril()
    tail = (G[-1] - G).exp()
    o = scale * G.exp()[:, None] * (qh @ s0) + P @ Y
    S1 = G[-1].exp() * s0 + (tail[:, None] * kh).T @ (b[:, None] * Y)
    dY = P.T @ do + (tail * b)[:, None] * (kh @ dsT)
    dX = T.T @ dY
    ds0 = G[-1].exp() * dsT + (scale * G.exp()[:, None] * qh).T @ do - (G.exp()[:, None] * kh).T @ dX
    D0 = scale * (E * b) * (do @ Y.T)
    D1 = -(E * b).tril(-1) * (dX @ Y.T)
    dq = scale * G.exp()[:, None] * (do @ s0.T) + D0 @ kh
    kr = D1 @ kh - G.exp()[:, None] * (dX @ s0.T)
    kw = D0.T @ qh + D1.T @ kh + (tail * b)[:, None] * (Y @ dsT.T)
    dG = (qh * dq).sum(1) + (kh * kr).sum(1) - (kh * kw).sum(1)
    dG[-1] += (S1 * dsT).sum()
    dl = dG.flip(0).cumsum(0).flip(0)
    dk = kr + kw
    return dict(o=o, sT=S1, dv=dX, ds0=ds0, dq=rq[:, None] * (dq - qh * (qh * dq).sum(1, keepdim=True)),
                dk=rk[:, None] * (dk - kh * (kh * dk).sum(1, keepdim=True)),
                dgates=torch.stack([dl * -c * torch.nn.functional.softplus(lam) * r * (1 - r),
                                    (kh * kw).sum(1) * (1 - b)], 1),
                dlam=-c * lam.sigmoid() * (dl * r).sum(0))


def test_chunk_formulas_against_the_step_by_step_form():
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    n, dk, dv = 23, 6, 5
    q, k, v, gates, lam = rnd(1, n, 1, dk), rnd(1, n, 1, dk), rnd(1, n, 1, dv), rnd(1, n, 2, 1), rnd(1) - 3
    do, s0, dsT = rnd(1, n, 1, dv), rnd(1, 1, dk, dv), rnd(1, 1, dk, dv)
    want = R.delta_grads(q, k, v, gates, lam, do, dsT=dsT, s0=s0)
    got = chunked(q[0, :, 0], k[0, :, 0], v[0, :, 0], gates[0, :, :, 0], lam, do[0, :, 0], c=8.0, eps=1e-6,
                  scale=dk ** -0.5, s0=s0[0, 0], dsT=dsT[0, 0])
    for name, t in got.items():
        assert torch.allclose(t.reshape(-1), want[name].reshape(-1), rtol=1e-9, atol=1e-11), name


def test_reference_gradients_against_differences():
    """Central differences in 64 bits: truncation h^2, rounding 1e-16 / h."""
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    B, L, H, HV, dk, dv = 2, 9, 1, 2, 4, 3
    x = dict(q=rnd(B, L, H, dk), k=rnd(B, L, H, dk), v=rnd(B, L, HV, dv), gates=rnd(B, L, 2, HV), lam=rnd(HV) - 3,
             s0=rnd(B, HV, dk, dv))
    do, dsT = rnd(B, L, HV, dv), rnd(B, HV, dk, dv)
    kw = dict(lengths=torch.tensor([9, 5]), reset=torch.tensor([[0, 0, 1, 0, 0, 0, 0, 1, 0], [1, 0, 0, 0, 1, 0, 0, 0, 0]]))
    out = R.delta_grads(x["q"], x["k"], x["v"], x["gates"], x["lam"], do, dsT=dsT, s0=x["s0"], **kw)

    def loss(x):
        o, sT = R.delta(x["q"], x["k"], x["v"], x["gates"], x["lam"], s0=x["s0"], **kw)
        return float((o * do).sum() + (sT * dsT).sum())

    h = 1e-5
    for name, t in x.items():
        want = out["d" + name]
        for i in torch.randperm(t.numel(), generator=g)[:6].tolist():
            at = torch.zeros(t.numel(), dtype=torch.float64)
            at[i] = h
            step = at.view(t.shape)
            d = (loss({**x, name: t + step}) - loss({**x, name: t - step})) / (2 * h)
            assert abs(d - want.reshape(-1)[i].item()) <= 1e-7 * (1 + abs(d)), (name, i)

"""Measured cases of the recurrent layer's operators.

Three operators of a recurrent language-model layer, in the order in which the
layer runs them:

  norm    root-mean-square norm with the residual's addition, written in the
          input's type or in 8 bits with one scale per 128 columns; its adjoint
  matmul  product of two 8-bit matrices with a scale for each block of 128
          (the projection that makes the gate inputs)
  scan    gated linear recurrence over the sequence, its adjoint, and its
          single-token step on a pool of states

`run` computes them in plain torch where `own` is false, and through
nonlinear_rnn_solve_newton_amd.layer where it is true.

Formulas (s: logistic sigmoid, all per channel d):
  scan    r = s(u_r), i = s(u_i), log a = -c softplus(lam) r, a = exp(log a),
          h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t;  h_{t-1} counts as zero
          where reset[t] is set; steps at or past the row's length change
          nothing and give a zero output
  norm    s = x + residual, y = s / sqrt(mean(s^2) + eps) * w
          8 bits: per 128 columns scale = max|y| / 448 (or the next power of
          two at or above it), q = round(y / scale)
  matmul  y[m, n] = sum_k a[m, k] sa[k/128, m] w[n, k] sw[.., k/128] + bias[n]
"""
import math
import random

import torch

own = False

C_DECAY = 8.0    # c of the recurrence's log decay
EPS = 1e-6       # of the norm
BLOCK = 128      # columns that share a scale
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100  # floor of a block's largest magnitude

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e8m0": torch.float8_e8m0fnu}


# ---------------------------------------------------------------------------
# the cases

def listed():
    return [
        # the smallest layer that is trained: one short fp32 sequence, latency
        {"name": "scan_train_b1_l1024_d64_f32", "op": "scan", "B": 1, "L": 1024, "D": 64, "dtype": "f32",
         "train": True, "packed": False},
        # an ordinary training batch of one layer
        {"name": "scan_train_b8_l4096_d1024", "op": "scan", "B": 8, "L": 4096, "D": 1024, "dtype": "bf16",
         "train": True, "packed": False},
        # a padded batch of packed documents, odd sizes, rows of length 0 and 1
        {"name": "scan_train_packed_b5_l1237_d1000", "op": "scan", "B": 5, "L": 1237, "D": 1000, "dtype": "bf16",
         "train": True, "packed": True},
        # prefill of one long prompt from a carried state
        {"name": "scan_prefill_b1_l65536_d2048", "op": "scan", "B": 1, "L": 65536, "D": 2048, "dtype": "bf16",
         "train": False, "packed": False},
        # one token for each of 64 requests, their states in a pool of slots
        {"name": "step_b64_d4096", "op": "step", "B": 64, "D": 4096, "S": 256, "dtype": "bf16"},
        # the norm before a projection while decoding: a few rows, latency
        {"name": "norm_fp8_n16_d4096", "op": "norm", "N": 16, "D": 4096, "dtype": "bf16", "out": "fp8",
         "scale": "f32", "train": False},
        # the same over a whole training or prefill batch (16 x 2048 tokens)
        {"name": "norm_fp8_n32768_d4096", "op": "norm", "N": 32768, "D": 4096, "dtype": "bf16", "out": "fp8",
         "scale": "e8m0", "train": False},
        # forward and adjoint in training, odd row count, a width that is not a multiple of 128
        {"name": "norm_train_n4999_d1000", "op": "norm", "N": 4999, "D": 1000, "dtype": "bf16", "out": "same",
         "scale": "f32", "train": True},
        # the gate projection of an LSTM of 4096 channels while decoding: weights read once
        {"name": "matmul_m16_n16384_k4096", "op": "matmul", "M": 16, "N": 16384, "K": 4096, "scale": "f32",
         "rows": 128, "bias": True, "out": "bf16"},
        # the same over the 16 x 2048 tokens of a batch
        {"name": "matmul_m32768_n16384_k4096", "op": "matmul", "M": 32768, "N": 16384, "K": 4096, "scale": "e8m0",
         "rows": 128, "bias": True, "out": "bf16"},
        # the three gates of 2048 channels, one sequence of 4096 tokens
        {"name": "matmul_m4096_n6144_k2048", "op": "matmul", "M": 4096, "N": 6144, "K": 2048, "scale": "f32",
         "rows": 128, "bias": False, "out": "bf16"},
        # odd sizes in every direction, a scale for each row of the weights, fp32 gate inputs
        {"name": "matmul_m777_n1000_k1333_f32", "op": "matmul", "M": 777, "N": 1000, "K": 1333, "scale": "f32",
         "rows": 1, "bias": True, "out": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["scan", "scan", "scan", "step", "norm", "norm", "matmul", "matmul", "matmul"])
    if op == "scan":
        B, D = _log(rng, 1, 16), _log(rng, 16, 4096)
        L = _log(rng, 1, min(65536, max(1, 100_000_000 // (B * D))))
        if rng.random() < 0.5:
            D = max(64, D // 64 * 64)
        return {"op": "scan", "B": B, "L": L, "D": D, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "train": rng.random() < 0.6 and B * L * D <= 33_554_432, "packed": rng.random() < 0.4}
    if op == "step":
        B = _log(rng, 1, 512)
        return {"op": "step", "B": B, "D": _log(rng, 64, 8192), "S": 2 * B + 1, "dtype": rng.choice(["bf16", "f32"])}
    if op == "norm":
        D = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            D = max(128, D // 128 * 128)
        train = rng.random() < 0.4
        return {"op": "norm", "N": _log(rng, 1, min(32768, 134_217_728 // D)), "D": D,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "out": "same" if train else rng.choice(["fp8", "fp8", "same"]),
                "scale": rng.choice(["f32", "e8m0"]), "train": train}
    M, N, K = _log(rng, 1, 32768), _log(rng, 64, 16384), _log(rng, 64, 4096)
    if rng.random() < 0.7:
        N, K = max(64, N // 64 * 64), max(64, K // 64 * 64)
    return {"op": "matmul", "M": M, "N": N, "K": K, "scale": rng.choice(["f32", "e8m0"]),
            "rows": rng.choice([128, 128, 1]), "bias": rng.random() < 0.5, "out": rng.choice(["bf16", "bf16", "f32"])}


# ---------------------------------------------------------------------------
# inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=g.device, dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=g.device, dtype=torch.float32)


def _lam(g, D):
    # exp(-c softplus(lam)) uniform in (0.9, 0.999): memories of 10 to 1000 steps
    z = -torch.log(0.9 + 0.099 * _rand(g, D)) / C_DECAY
    return torch.log(torch.expm1(z))


def _pow2(scale, dtype):
    # the next power of two at or above a positive scale, as its type holds it
    m, e = torch.frexp(scale)
    e = torch.where(m == 0.5, e - 1, e)
    return (e + 127).clamp(0, 254).to(torch.uint8).view(dtype)


def _values(scale):
    # fp32 values of scales of either type
    if scale.dtype == torch.float32:
        return scale
    return torch.ldexp(torch.ones_like(scale, dtype=torch.float32), scale.view(torch.uint8).to(torch.int32) - 127)


def _transposed(scale):
    if scale.dtype == torch.float32:
        return scale.t().contiguous()
    return scale.view(torch.uint8).t().contiguous().view(scale.dtype)


def _spread(scale, n, dim):
    # one scale per block of BLOCK entries -> one per entry of a dimension of n
    return scale.repeat_interleave(BLOCK, dim=dim).narrow(dim, 0, n)


def _blocks(x):
    # columns padded with zeros to whole blocks: [rows][blocks][BLOCK]
    n = -(-x.shape[1] // BLOCK)
    return torch.nn.functional.pad(x, (0, n * BLOCK - x.shape[1])).view(x.shape[0], n, BLOCK)


def _quantize(x, rows, scale_dtype):
    # 8-bit values and scales of x [R][K]: a scale for each rows x BLOCK block, [R/rows][K/BLOCK]
    amax = _blocks(x.abs()).amax(dim=2)
    if rows > 1:
        n = -(-x.shape[0] // rows)
        amax = torch.nn.functional.pad(amax, (0, 0, 0, n * rows - x.shape[0])).view(n, rows, -1).amax(dim=1)
    scale = amax.clamp_min(SCALE_MIN) / E4M3_MAX
    if scale_dtype != torch.float32:
        scale = _pow2(scale, scale_dtype)
    full = _spread(_values(scale), x.shape[1], 1)
    if rows > 1:
        full = full.repeat_interleave(rows, dim=0)[:x.shape[0]]
    return (x / full).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    st = {"case": dict(case)}
    if case["op"] in ("scan", "step"):
        dt, D, B = DTYPES[case["dtype"]], case["D"], case["B"]
        st["lam"] = _lam(g, D)
        if case["op"] == "step":
            st["u"] = _randn(g, B, 3, D).to(dt)
            st["state"] = 0.5 * _randn(g, case["S"], D)
            slots = torch.randperm(case["S"], generator=g, device=dev)[:B].to(torch.int32)
            if B > 2:
                slots[1] = -1  # a row of the batch without a request
            st["slots"] = slots
            return st
        L = case["L"]
        st["u"] = _randn(g, B, L, 3, D).to(dt)
        st["h0"] = 0.5 * _randn(g, B, D)
        st["lengths"] = st["reset"] = None
        if case["packed"]:
            lengths = (_rand(g, B) * (L + 1)).to(torch.int32)
            lengths[0] = L
            if B > 2:
                lengths[1], lengths[2] = 0, 1
            st["lengths"] = lengths
            st["reset"] = (_rand(g, B, L) < 0.005).to(torch.uint8)
        if case["train"]:
            st["dh"] = _randn(g, B, L, D).to(dt)
            st["dhT"] = _randn(g, B, D)
        return st
    if case["op"] == "norm":
        dt, N, D = DTYPES[case["dtype"]], case["N"], case["D"]
        st["x"] = _randn(g, N, D).to(dt)
        # a residual stream: wider than its increments, with a few strong channels
        st["residual"] = (_randn(g, N, D) * 2.0 * (1.0 + 15.0 * (_rand(g, D) < 0.01))).to(dt)
        st["w"] = 1.0 + 0.2 * _randn(g, D)
        if case["train"]:
            st["dy"] = _randn(g, N, D).to(dt)
            st["ds"] = _randn(g, N, D).to(dt)
        return st
    M, N, K, sdt = case["M"], case["N"], case["K"], DTYPES[case["scale"]]
    x = _randn(g, M, K) * (1.0 + 7.0 * (_rand(g, K) < 0.01))
    st["a"], sa = _quantize(x, 1, sdt)
    st["sa"] = _transposed(sa)
    st["w"], st["sw"] = _quantize(_randn(g, N, K) / math.sqrt(K), case["rows"], sdt)
    st["bias"] = _randn(g, N) if case["bias"] else None
    return st


# ---------------------------------------------------------------------------
# plain forms, in 32 bits

def _softplus(x):
    return torch.log1p(torch.exp(-x.abs())) + x.clamp_min(0)


def _coefficients(u, lam, r_axis):
    # gates, decay and input weight of every step in 32 bits
    r, i, x = (torch.sigmoid(u.select(r_axis, 0).float()), torch.sigmoid(u.select(r_axis, 1).float()),
               u.select(r_axis, 2).float())
    la = -C_DECAY * _softplus(lam) * r
    return r, i, x, torch.exp(la), torch.sqrt(-torch.expm1(2 * la))


def _doubling(a, b):
    # all h_t = a_t h_{t-1} + b_t along dimension 1, from zero: composites of
    # 1, 2, 4, ... steps (about log2(L) passes)
    k = 1
    while k < a.shape[1]:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], dim=1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], dim=1)
        k *= 2
    return b


def _masks(st, L):
    dev = st["u"].device
    if st["lengths"] is None:
        return None, None
    return (torch.arange(L, device=dev)[None] < st["lengths"][:, None])[:, :, None], (st["reset"] != 0)[:, :, None]


def _plain_scan(st, train):
    u, h0 = st["u"], st["h0"]
    L = u.shape[1]
    valid, reset = _masks(st, L)
    r, i, x, a, m = _coefficients(u, st["lam"], 2)
    b, A = m * i * x, a
    if valid is not None:
        A = torch.where(valid, torch.where(reset, 0.0, a), 1.0)
        b = torch.where(valid, b, 0.0)
    h = _doubling(A, torch.cat([b[:, :1] + A[:, :1] * h0[:, None], b[:, 1:]], dim=1))
    out = {"h": (h if valid is None else torch.where(valid, h, 0.0)).to(u.dtype), "hT": h[:, -1].clone()}
    if not train:
        return out
    dh = st["dh"].float()
    if valid is not None:
        dh = torch.where(valid, dh, 0.0)
    # g_t = dh_t + a_{t+1} g_{t+1}, from the end
    dh = torch.cat([dh[:, :-1], dh[:, -1:] + st["dhT"][:, None]], dim=1)
    back = torch.cat([A[:, 1:], torch.ones_like(A[:, :1])], dim=1)
    g = _doubling(back.flip(1), dh.flip(1)).flip(1)
    prev = torch.cat([h0[:, None], h[:, :-1]], dim=1)
    if reset is not None:
        prev = torch.where(reset, 0.0, prev)
    dla = g * (a * prev - i * x * a * a / m)
    if valid is not None:
        g_in, dla = torch.where(valid, g, 0.0), torch.where(valid, dla, 0.0)
    else:
        g_in = g
    du = torch.stack([-C_DECAY * _softplus(st["lam"]) * dla * r * (1 - r), g_in * m * x * i * (1 - i), g_in * m * i],
                     dim=2)
    out["du"] = du.to(u.dtype)
    out["dlam"] = (-C_DECAY * torch.sigmoid(st["lam"])) * (dla * r).sum(dim=(0, 1))
    out["dh0"] = A[:, 0] * g[:, 0]
    return out


def _plain_step(st):
    u, state, slots = st["u"], st["state"], st["slots"].long()
    _, i, x, a, m = _coefficients(u, st["lam"], 1)
    live = slots >= 0
    old = state[slots.clamp_min(0)]
    h = torch.where(live[:, None], a * old + m * i * x, 0.0)
    state[slots[live]] = h[live]
    return {"h": h.to(u.dtype), "state": state}


def _plain_norm(st, case):
    s = st["x"].float() + st["residual"].float()
    y = s * torch.rsqrt((s * s).mean(dim=1, keepdim=True) + EPS) * st["w"]
    out = {"s": s.to(st["x"].dtype)}
    if case["out"] == "fp8":
        out["y"], scale = _quantize(y, 1, DTYPES[case["scale"]])
        out["scale"] = _transposed(scale)
    else:
        out["y"] = y.to(st["x"].dtype)
    if case["train"]:
        # the adjoint takes the sum as it was written
        s, dy = out["s"].float(), st["dy"].float()
        rstd = torch.rsqrt((s * s).mean(dim=1, keepdim=True) + EPS)
        n, t = s * rstd, dy * st["w"]
        out["dx"] = (rstd * (t - n * (t * n).mean(dim=1, keepdim=True)) + st["ds"].float()).to(st["x"].dtype)
        out["dw"] = (dy * n).sum(dim=0)
    return out


def _plain_matmul(st, case):
    K, N = case["K"], case["N"]
    a = st["a"].float() * _spread(_values(st["sa"]), K, 0).t()
    w = st["w"].float() * _spread(_values(st["sw"]), K, 1).repeat_interleave(case["rows"], dim=0)[:N]
    y = a @ w.t()
    if st["bias"] is not None:
        y = y + st["bias"]
    return y.to(DTYPES[case["out"]])


def run(st):
    case = st["case"]
    if own:
        return _own(st, case)
    if case["op"] == "scan":
        return _plain_scan(st, case["train"])
    if case["op"] == "step":
        return _plain_step(st)
    if case["op"] == "norm":
        return _plain_norm(st, case)
    return _plain_matmul(st, case)


# ---------------------------------------------------------------------------
# the framework's operators, as a user's program calls them

def _own(st, case):
    from nonlinear_rnn_solve_newton_amd import layer

    if case["op"] == "scan":
        kw = dict(c=C_DECAY, lengths=st["lengths"], reset=st["reset"])
        f = layer.gated_scan(st["u"], st["lam"], h0=st["h0"], save=case["train"], **kw)
        out = {"h": f["h"], "hT": f["hT"]}
        if case["train"]:
            b = layer.gated_scan_adjoint(st["u"], st["lam"], st["dh"], f["saved"], dhT=st["dhT"], want_dh0=True, **kw)
            out.update(du=b["du"], dlam=b["dlam"], dh0=b["dh0"])
        return out
    if case["op"] == "step":
        h = layer.gated_step(st["u"], st["lam"], st["state"], c=C_DECAY, slots=st["slots"])
        return {"h": h, "state": st["state"]}
    if case["op"] == "norm":
        fp8 = case["out"] == "fp8"
        f = layer.norm_residual(st["x"], st["w"], residual=st["residual"], eps=EPS,
                                scale_dtype=DTYPES[case["scale"]] if fp8 else None)
        out = {"s": f["s"], "y": f["y"]}
        if fp8:
            out["scale"] = f["scale"]
        if case["train"]:
            b = layer.norm_residual_adjoint(f["s"], st["w"], st["dy"], ds=st["ds"], eps=EPS)
            out.update(dx=b["dx"], dw=b["dw"])
        return out
    return layer.matmul_fp8(st["a"], st["sa"], st["w"], st["sw"], bias=st["bias"], out_dtype=DTYPES[case["out"]])


# ---------------------------------------------------------------------------
# what one pass cannot do without

def work(case):
    if case["op"] == "scan":
        e, B, L, D = 2 if case["dtype"] == "bf16" else 4, case["B"], case["L"], case["D"]
        n = B * L * D
        # forward: u in, h out; the adjoint is a call of its own: u and dh in, du out
        by, fl = 4 * e * n + 4 * (2 * B * D + D), 30 * n
        if case["train"]:
            by, fl = by + 7 * e * n + 4 * (2 * B * D + 2 * D), fl + 60 * n
        if case["packed"]:
            by += (2 if case["train"] else 1) * (B * L + 4 * B)
        return {"bytes": by, "flops": fl}
    if case["op"] == "step":
        e, n = 2 if case["dtype"] == "bf16" else 4, case["B"] * case["D"]
        return {"bytes": (4 * e + 8) * n + 4 * case["D"] + 4 * case["B"], "flops": 30 * n}
    if case["op"] == "norm":
        e, n = 2 if case["dtype"] == "bf16" else 4, case["N"] * case["D"]
        # x and the residual in, the sum and the norm out
        by, fl = 3 * e * n + 4 * case["D"], 6 * n
        if case["out"] == "fp8":
            blocks = case["N"] * -(-case["D"] // BLOCK)
            by, fl = by + n + blocks * (4 if case["scale"] == "f32" else 1), fl + 3 * n
        else:
            by += e * n
        if case["train"]:
            by, fl = by + 4 * e * n + 8 * case["D"], fl + 12 * n
        return {"bytes": by, "flops": fl}
    M, N, K = case["M"], case["N"], case["K"]
    kb, sb = -(-K // BLOCK), 4 if case["scale"] == "f32" else 1
    by = M * K + N * K + sb * kb * (M + -(-N // case["rows"])) + (4 * N if case["bias"] else 0)
    return {"bytes": by + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# the same in 64 bits, step by step

def _exact_scan(st, train):
    u, lam = st["u"].double(), st["lam"].double()
    B, L, _, D = u.shape
    beta = -C_DECAY * torch.nn.functional.softplus(lam, threshold=1e9)
    r, i, x = torch.sigmoid(u[:, :, 0]), torch.sigmoid(u[:, :, 1]), u[:, :, 2]
    del u
    la = beta * r
    a = la.exp()
    b = (-(2 * la).expm1()).sqrt().mul_(i).mul_(x)
    del la
    if st["lengths"] is None:
        n = torch.full((B, 1), L, device=a.device)
        start = None
    else:
        n, start = st["lengths"].long()[:, None], st["reset"].bool()
    h = torch.empty_like(a)
    s = st["h0"].double()
    for t in range(L):
        old = s if start is None else s.masked_fill(start[:, t, None], 0.0)
        new = torch.addcmul(b[:, t], a[:, t], old)
        s = new if start is None else torch.where(t < n, new, s)
        h[:, t] = s
    seen = torch.arange(L, device=a.device)[None, :, None] < n[:, :, None]
    out = {"h": h * seen, "hT": s.clone()}
    if not train:
        return out
    du = torch.zeros(B, L, 3, D, dtype=torch.float64, device=a.device)
    dlam = torch.zeros(D, dtype=torch.float64, device=a.device)
    g, h0 = st["dhT"].double(), st["h0"].double()
    for t in range(L - 1, -1, -1):
        on = t < n
        cut = torch.zeros_like(on) if start is None else start[:, t, None]
        lt = torch.where(on, g + st["dh"][:, t].double(), g)  # gradient of h_t
        at, rt, it, xt = a[:, t], r[:, t], i[:, t], x[:, t]
        w = (1 - at) * (1 + at)
        w = torch.where(at > 0.999, -torch.expm1(2 * beta * rt), w).sqrt()
        old = (h[:, t - 1] if t else h0).masked_fill(cut, 0.0)
        d = lt * at * (old - it * xt * at / w)  # of log a_t
        d = torch.where(on, d, 0.0)
        gx = torch.where(on, lt, 0.0) * w
        du[:, t, 0], du[:, t, 1], du[:, t, 2] = d * beta * rt * (1 - rt), gx * xt * it * (1 - it), gx * it
        dlam += (d * rt).sum(0)
        g = torch.where(on, torch.where(cut, 0.0, at * lt), g)
    out["du"], out["dlam"], out["dh0"] = du, -C_DECAY * torch.sigmoid(lam) * dlam, g
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "scan":
        return _exact_scan(st, case["train"])
    if case["op"] == "step":
        u, pool = st["u"].double(), st["state"].double()
        la = -C_DECAY * torch.nn.functional.softplus(st["lam"].double(), threshold=1e9) * torch.sigmoid(u[:, 0])
        h = torch.zeros_like(u[:, 0])
        for b, slot in enumerate(st["slots"].tolist()):
            if slot >= 0:
                pool[slot] = la[b].exp() * pool[slot] + (-(2 * la[b]).expm1()).sqrt() * torch.sigmoid(u[b, 1]) * u[b, 2]
                h[b] = pool[slot]
        return {"h": h, "state": pool}
    if case["op"] == "norm":
        s = st["x"].double() + st["residual"].double()
        w = st["w"].double()
        y = s / (s.square().mean(1, keepdim=True) + EPS).sqrt() * w
        out = {"s": s, "y": y}
        if case["out"] == "fp8":
            scale = _blocks(y.abs()).amax(2).clamp_min(SCALE_MIN) / E4M3_MAX
            if case["scale"] == "e8m0":
                scale = torch.exp2(torch.ceil(torch.log2(scale)))
            out["y"], out["scale"] = y / _spread(scale, case["D"], 1), scale.t()
        if case["train"]:
            s, dy = s.to(st["x"].dtype).double(), st["dy"].double()
            var = s.square().mean(1, keepdim=True) + EPS
            t = dy * w
            out["dx"] = t / var.sqrt() - s * (t * s).mean(1, keepdim=True) / var ** 1.5 + st["ds"].double()
            out["dw"] = (dy * s / var.sqrt()).sum(0)
        return out
    a, w = st["a"].double(), st["w"].double()
    for k in range(-(-case["K"] // BLOCK)):
        sl = slice(k * BLOCK, (k + 1) * BLOCK)
        a[:, sl] *= _values(st["sa"])[k].double()[:, None]
        w[:, sl] *= _values(st["sw"])[:, k].double().repeat_interleave(case["rows"])[:case["N"], None]
    y = a @ w.t()
    return y if st["bias"] is None else y + st["bias"].double()

"""Plain 64-bit forms of the recurrent layer's operators for the tests, with a
running bound on the rounding error of a 32-bit evaluation next to each value.

The bounds follow the operations: U is the unit roundoff of fp32, KV the number
of roundings that one value (a gate, a decay, a product) collects, each of them
at most 2 U (the hardware exponential, reciprocal and square root are good to
1 ulp); an error enters a recurrence at its step and is carried on by it.
"""
import numpy as np

U = 2.0 ** -24
KV = 16.0
TINY = 1e-30  # results this small may be flushed
BF16_EPS = 2.0 ** -8  # half an ulp of bf16 (8 significant bits), relative


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def softplus(x):
    return np.logaddexp(0.0, x)


def gated(u, lam, c=8.0, h0=None, lengths=None, reset=None, dh=None, dhT=None):
    """u [B][L][3][D] etc. as float64 arrays. Returns a dict of (value, bound)
    pairs: h, hT and, with dh, du, dlam, dh0."""
    B, L, _, D = u.shape
    n = np.full(B, L) if lengths is None else np.clip(lengths, 0, L)
    cut = np.zeros((B, L), bool) if reset is None else reset != 0
    beta = -c * softplus(lam)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        r, i, x = sigmoid(u[:, :, 0]), sigmoid(u[:, :, 1]), u[:, :, 2]
        la = beta * r
        a = np.exp(la)
        m = np.sqrt(-np.expm1(2 * la))
        im = np.where(m > 0, 1.0 / m, 0.0)
        # relative error of a gate: its argument's rounding grows with it
        kg = KV + 2 * np.abs(u[:, :, 0]) + 2 * np.abs(u[:, :, 1])
        h = np.zeros((B, L, D))
        eh = np.zeros((B, L, D))
        hp = np.zeros((B, L, D))  # state before each step, as the step sees it
        ehp = np.zeros((B, L, D))
        s = np.zeros((B, D)) if h0 is None else h0.astype(np.float64).copy()
        e = np.zeros((B, D))
        for t in range(L):
            on = (t < n)[:, None]
            z = cut[:, t][:, None]
            old, eold = np.where(z, 0.0, s), np.where(z, 0.0, e)
            hp[:, t], ehp[:, t] = old, eold
            b = m[:, t] * i[:, t] * x[:, t]
            new = a[:, t] * old + b
            k = kg[:, t]
            enew = a[:, t] * eold + U * (np.abs(a[:, t] * old) * (KV + k * np.abs(la[:, t])) + k * np.abs(b)) + TINY
            s, e = np.where(on, new, s), np.where(on, enew, e)
            h[:, t], eh[:, t] = np.where(on, s, 0.0), np.where(on, e, 0.0)
        out = {"h": (h, eh), "hT": (s.copy(), e.copy())}
        if dh is None:
            return out
        du, edu = np.zeros((B, L, 3, D)), np.zeros((B, L, 3, D))
        dl, edl = np.zeros(D), np.zeros(D)
        mu = np.zeros((B, D)) if dhT is None else dhT.astype(np.float64).copy()
        emu = np.zeros((B, D))
        for t in range(L - 1, -1, -1):
            on = (t < n)[:, None]
            z = cut[:, t][:, None]
            k, at, rt, it, mt = kg[:, t], a[:, t], r[:, t], i[:, t], m[:, t]
            g = mu + dh[:, t]
            eg = emu + U * np.abs(g) * 2
            q = it * x[:, t] * at * im[:, t]
            mag = np.abs(hp[:, t]) + np.abs(q)
            dla = g * at * (hp[:, t] - q)
            edla = at * (eg * mag + np.abs(g) * (ehp[:, t] + U * (2 * k + k * np.abs(la[:, t])) * mag)) + TINY
            vals = (dla * beta * rt * (1 - rt), g * mt * x[:, t] * it * (1 - it), g * mt * it)
            # 1 - gate is good to U in absolute terms
            errs = (edla * np.abs(beta) * rt * (1 - rt) + U * np.abs(dla * beta * rt) * (2 + k * (1 - rt)),
                    np.abs(mt * x[:, t] * it) * (eg * (1 - it) + U * np.abs(g) * (2 + k * (1 - it))),
                    mt * it * (eg + U * k * np.abs(g)))
            for j in range(3):
                du[:, t, j] = np.where(on, vals[j], 0.0)
                edu[:, t, j] = np.where(on, errs[j] + TINY, 0.0)
            dl += np.where(on, dla * rt, 0.0).sum(0)
            # partial sums in 32 bits: at most 64 roundings on any path of the tree
            edl += np.where(on, edla * rt + U * (64 + k) * np.abs(dla * rt), 0.0).sum(0)
            nmu = np.where(z, 0.0, at * g)
            enmu = np.where(z, 0.0, at * eg + U * np.abs(at * g) * (KV + k * np.abs(la[:, t])) + TINY)
            mu, emu = np.where(on, nmu, mu), np.where(on, enmu, emu)
        f = -c * sigmoid(lam)
        out.update(du=(du, edu), dlam=(f * dl, np.abs(f) * edl + U * KV * np.abs(f * dl)), dh0=(mu, emu))
        return out


def blocks_max(y):
    """Largest magnitude of each 128 columns of [N][D], at least 2^-100: [N][blocks]."""
    n = -(-y.shape[1] // 128)
    p = np.pad(np.abs(y), ((0, 0), (0, n * 128 - y.shape[1]))).reshape(y.shape[0], n, 128)
    return np.maximum(p.max(2), 2.0 ** -100)


def norm(x, w, residual=None, eps=1e-6):
    """(value, bound) of s and y, float64 arrays; the sum of squares is good to
    a relative 72 roundings (a lane's 32 terms, 6 + 5 levels across lanes and
    waves, twice that for their spread), its root to half of them."""
    s = x if residual is None else x + residual
    y = s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * w
    return {"s": (s, U * np.abs(s)), "y": (y, 48 * U * np.abs(y) + TINY)}


def norm_adjoint(s, w, dy, ds=None, eps=1e-6):
    rstd = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    t, n = dy * w, s * rstd
    mean, amean = (t * n).mean(1, keepdims=True), np.abs(t * n).mean(1, keepdims=True)
    o = 0.0 if ds is None else ds
    dx = rstd * (t - n * mean) + o
    e = 96 * U * rstd * (np.abs(t) + np.abs(n) * amean) + 4 * U * np.abs(o) + TINY
    mag = np.abs(dy * n).sum(0)
    return {"dx": (dx, e), "dw": ((dy * n).sum(0), U * (96 + s.shape[0] / 256) * mag + TINY)}


def matmul(a, sa, w, sw, rows, bias=None, fp32=True):
    """y = (a sa) (w sw)^T + bias and its bound: fp32 sums of exact products, or
    products that the 8-bit matrix instructions round (2^-12.4 of a block's sum
    of magnitudes at the worst measured; 2^-11 here)."""
    K, N = a.shape[1], w.shape[0]
    A = a * np.repeat(sa, 128, axis=0)[:K].T
    W = w * np.repeat(np.repeat(sw, rows, axis=0)[:N], 128, axis=1)[:, :K]
    y, mag = A @ W.T, np.abs(A) @ np.abs(W).T
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    return y, mag * (U * (16 + 2 * sa.shape[0]) if fp32 else 2.0 ** -11) + TINY

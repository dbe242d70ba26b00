"""Plain 64-bit forms of the delta-rule layer's operators for the tests: step by
step and row by row, as the header defines them; their gradients by autograd.

Tolerances. U = 2^-24 is the unit roundoff of fp32. A value of the delta rule is
a chain of inner products over dk, dv and the chunk's 64 steps, each term of
which collects at most 8 roundings (two factors split to 2^-25, their product,
gates and decays); the state is carried by contractions, so a chunk adds its own
roundings to it and enlarges none. With n steps a result is so off by at most
8 U (dk + dv + 64 + n) times the largest magnitude of its tensor before the
rounding to its type (`delta_tol`); gradients take two such chains (twice that),
and the decays' a sum over the chunk of differences of them. Norms and products
state theirs where they are tested.
"""
import torch

U = 2.0 ** -24
# fp32 and bf16 hold nothing between 0 and 2^-149, and the matrix instructions take less than 2^-126 for 0:
# a result that is smaller may be 0 whatever it is computed with
TINY = 2.0 ** -126


def half_step(dtype):
    return 0.0 if dtype == torch.float64 else torch.finfo(dtype).eps / 2


def unit(x, eps):
    return x / (x.square().sum(-1, keepdim=True) + eps).sqrt()


def delta(q, k, v, gates, lam, *, c=8.0, eps=1e-6, scale=None, s0=None, lengths=None, reset=None):
    """[B][L][H][dk], [B][L][HV][dv], [B][L][2][HV]: o and the last state, in 64 bits."""
    B, L, H, dk = q.shape
    HV, dv = v.shape[2:]
    scale = dk ** -0.5 if scale is None else scale
    S = torch.zeros(B, HV, dk, dv, dtype=torch.float64) if s0 is None else s0
    n = torch.full((B,), L) if lengths is None else lengths.clamp(0, L)
    o = []
    for t in range(L):
        on = (t < n)[:, None]
        # a step that is not there: its inputs do not count, whatever they are
        pick = lambda x: torch.where(on[:, :, None], x, torch.ones_like(x))  # noqa: E731
        qt, kt = (unit(pick(x[:, t]), eps).repeat_interleave(HV // H, 1) for x in (q, k))
        vt, (r, b) = pick(v[:, t]), torch.where(on[:, :, None], gates[:, t], 0.0).sigmoid().unbind(1)
        a = (-c * torch.nn.functional.softplus(lam, threshold=1e9) * r).exp()
        if reset is not None:
            a = torch.where((reset[:, t] != 0)[:, None], torch.zeros_like(a), a)
        D = a[:, :, None, None] * S
        u = b[:, :, None] * (vt - (D * kt[..., None]).sum(2))
        new = D + kt[..., None] * u[:, :, None]
        S = torch.where(on[:, :, None, None], new, S)
        o.append(torch.where(on[:, :, None], scale * (S * qt[..., None]).sum(2), torch.zeros_like(vt)))
    return torch.stack(o, 1), S


def delta_grads(q, k, v, gates, lam, do, *, dsT=None, s0=None, **kw):
    """dict of o, sT and the gradients, from 64-bit leaves."""
    B, _, _, dk = q.shape
    HV, dv = v.shape[2:]
    s0 = torch.zeros(B, HV, dk, dv, dtype=torch.float64) if s0 is None else s0
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v, gates, lam, s0)]
    o, sT = delta(*leaves[:5], s0=leaves[5], **kw)
    n = kw.get("lengths")
    if n is not None:
        do = torch.where((torch.arange(q.shape[1]) < n[:, None])[:, :, None, None], do, 0.0)
    loss = (o * do).sum()
    if dsT is not None:
        loss = loss + (sT * dsT).sum()
    g = torch.autograd.grad(loss, leaves, allow_unused=True)
    g = [torch.zeros_like(x) if y is None else y for x, y in zip(leaves, g)]
    return dict(o=o.detach(), sT=sT.detach(), dq=g[0], dk=g[1], dv=g[2], dgates=g[3], dlam=g[4], ds0=g[5])


def delta_tol(name, want, dtype, dk, dv, steps):
    """(absolute, relative) bound of a result in `dtype` against 64 bits."""
    big = want.abs().max().item() if want.numel() else 0.0
    k = 8 * U * (dk + dv + 64 + steps)
    k *= 1 if name in ("o", "sT") else 2
    if name in ("dgates", "dlam"):
        k *= 4  # decays: 64 terms of three sums that partly cancel
    return k * big + TINY, half_step(dtype)


def norm_block(x, w=None, gate=None, group=None, residual=None, alpha=None, w_next=None, eps=1e-6):
    """y, s in 64 bits (s None without a residual)."""
    N, D = x.shape
    p = x
    if w is not None:
        g = x.view(N, -1, group or D)
        p = (g / (g.square().mean(-1, keepdim=True) + eps).sqrt() * w).view(N, D)
    if gate is not None:
        p = p * gate * gate.sigmoid()
    if residual is None:
        return p, None
    s = residual + (p if alpha is None else alpha * p)
    return s / (s.square().mean(-1, keepdim=True) + eps).sqrt() * w_next, s

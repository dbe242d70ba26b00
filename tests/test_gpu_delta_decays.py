"""Strong and weak decays in one chunk of the delta rule. Every key is a direction of its own and every query
reads one key, five steps before it, so that each result is one term (or a sum of terms of one sign) and its
error is a few roundings of itself, however strong the decays in front of it are."""
import pytest
import torch

from tests import delta_reference as R
from tests.helpers import say
from tests.test_gpu_delta import DT, GRADS, cuda, reference, run

pytestmark = pytest.mark.gpu
U, LAG, C = R.U, 5, 8.0


def make(dk, H, HV, dtype, strong, seed):
    """64 steps: `strong` of them with decays of up to e^-240, then weak ones of about e^-0.1, some of each among
    the others too. No state in front and no gradient of the last one's."""
    L, dv = 64, 40
    g = torch.Generator().manual_seed(seed)
    eye = torch.eye(dk)[:L]
    k = eye[None, :, None].expand(2, L, H, dk)
    q = k.roll(LAG, 1).clone()  # step t reads the key of step t - 5
    q[:, :LAG] = k[:, :LAG]  # the first ones their own
    lam = torch.tensor([2.0, 30.0])[:HV].flip(0) if HV > 1 else torch.tensor([30.0])
    gates = torch.randn(2, L, 2, HV, generator=g)
    weak = torch.arange(L) >= strong
    weak[strong // 2] = True
    weak[strong + 20] = False
    # c softplus(lam) s(gate): about 0.1 where weak
    lo = torch.logit(0.1 / (C * torch.nn.functional.softplus(lam)))
    gates[:, :, 0] = torch.where(weak[None, :, None], lo + 0.3 * gates[:, :, 0], 3.0 + gates[:, :, 0])
    one = lambda *s: (1.0 + torch.rand(*s, generator=g)).to(dtype)  # noqa: E731  (of one sign)
    return dict(q=q.to(dtype), k=k.to(dtype).contiguous(), v=one(2, L, HV, dv), gates=gates.to(dtype), lam=lam,
                s0=torch.zeros(2, HV, dk, dv), do=one(2, L, HV, dv), dsT=torch.zeros(2, HV, dk, dv), lengths=None, reset=None,
                p=None)


@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [(1, 1), (1, 2), (2, 2)], ids=str)
@pytest.mark.parametrize("dk,strong", [(64, 24), (128, 24), (64, 40), (64, 0)])
def test_decays_keep_their_digits(dk, strong, heads, dtype, reset):
    """A decay over a gap of x = sum of -log a is off by 16 U x (the sigmoid, the softplus and their products: a few
    roundings of each step's part), a result by 32 roundings beside it."""
    say(f"delta decays {dk} {strong} {heads} {dtype} {reset}")
    H, HV = heads
    x = make(dk, H, HV, DT[dtype], strong, seed=dk + strong)
    start = min(strong + 3, 60)
    if reset:
        x["reset"] = torch.zeros(2, 64, dtype=torch.uint8)
        x["reset"][:, start] = 1
    want, got = reference(x), run(cuda(x))
    la = C * torch.nn.functional.softplus(x["lam"].double(), threshold=1e9) * x["gates"][:, :, 0].double().sigmoid()
    G = la.cumsum(1)  # [B][L][HV], x of i over j: G_i - G_j
    t = torch.arange(64)
    off = lambda gap: (32 + 16 * gap) * U  # noqa: E731

    def near(name, g, w, rel, dtype=torch.float64):
        err, half = (g.cpu().double() - w).abs(), R.half_step(dtype)
        bound = rel * w.abs()
        assert (err <= bound + half * (w.abs() + bound) + R.TINY).all(), (name, (err / w.abs().clamp_min(1e-30)).max().item())

    lag = torch.where(t >= LAG, LAG, 0)
    near("o", got["o"], want["o"], off(G - G[:, t - lag])[..., None], DT[dtype])
    # row j of the last state is what step j wrote
    kept = want["sT"][:, :, :64]
    near("sT", got["sT"][:, :, :64], kept, off(G[:, -1:] - G).transpose(1, 2)[..., None])
    # dv_j comes from the step that reads it, j + 5 (and the first ones from themselves)
    late = G[:, (t + LAG).clamp_max(63)] - G
    near("dv", got["dv"], want["dv"], off(late)[..., None], DT[dtype])
    # a decay's gradient: pairs of one sign that it lies between, over at most 2 * 5 steps; 64 terms' sum beside it
    gap = G[:, (t + LAG).clamp_max(63)] - G[:, (t - LAG).clamp_min(0)]
    near("dgates", got["dgates"][:, :, 0], want["dgates"][:, :, 0], off(gap) + 64 * U, DT[dtype])
    terms = want["dgates"][:, :, 0].abs() / (1 - x["gates"][:, :, 0].double().sigmoid())  # of dlam, but for a factor
    rel = ((off(gap) + 64 * U) * terms).sum((0, 1)) / terms.sum((0, 1))
    near("dlam", got["dlam"], want["dlam"], rel + 64 * U)
    assert all(torch.isfinite(got[n]).all() for n in GRADS)

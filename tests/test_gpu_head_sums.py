"""The normalisers of the vocabulary head's losses by themselves: the scores are
exact (a row of x picks one column of Wv), so that only the sums, exponentials and
logarithms are left, against the formulas in 64 bits.

Bounds, u = 2^-24 half a step of fp32.  A row's parts of 128 (fp32: 64) columns:
a lane adds 8 values in each of 4 sums, then 2 of those, then 2 lanes away: 12
additions at most.  A merge of two parts is one exponential (2 u, its argument
rounded), one product, one addition: 4 u; there are fewer than parts, and no more
than ceil(parts / 64) of a thread, 2 of its lanes' and 15 of the waves'.  An
exponential has 2 u and the rounding of its argument, u times it, for a score's, a
part's and a row's difference from the maximum and for the constant log2(e) / tau.
The logarithm has 2 u of itself (2 u around 0) and the products behind it as much
again.  The result is rounded once: u |lse|."""
import math

import pytest
import torch

import mixture_experts_layer_permute_amd as M

from _gpu import banner, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

u = 2.0 ** -24
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}
D = 64


def given(z, dt):
    """x [T,64] and Wv [V,64] whose scores are z[t % 64] (64 rows), exactly."""
    Wv = z.to(TDT[dt]).t().contiguous().cuda()
    assert torch.equal(Wv.t().cpu().float(), z.float()), "not representable"
    return Wv


def pick(T, dt):
    x = torch.zeros(T, D, dtype=TDT[dt], device="cuda")
    t = torch.arange(T, device="cuda")
    x[t, t % D] = 1.0
    return x


def sum_error(V, dt):
    """Relative error of a row's sum of exponentials, without the arguments' part."""
    bm, pc = (256, 128) if dt == "bf16" else (128, 64)
    parts = -(-V // bm) * (bm // pc)
    return (12 + 4 * min(parts - 1, -(-parts // 64) + 17) + 2) * u


def lse_and_bound(z, V, dt, tau=1.0):
    s = z.double() / tau
    top = s.max(1, keepdim=True).values
    lse = torch.logsumexp(s, 1)
    far = (torch.softmax(s, 1) * (top - s)).sum(1)
    over = lse - top[:, 0]
    return lse, sum_error(V, dt) + u * (lse.abs() + 4 + 4 * far + 4 * over)


def off(got, want, tol):
    bad = ~((got.double() - want.cuda()).abs() <= tol.cuda())
    k = bad.flatten().nonzero()
    if len(k):
        k = int(k[0])
        return "%d of %d, first %d: %.9g for %.9g, bound %.3g" % (
            int(bad.sum()), bad.numel(), k, float(got.flatten()[k]), float(want.flatten()[k]),
            float(tol.flatten()[k]))
    return None


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(64, 100), (64, 1000), (300, 5003), (300, 40000)])
def test_lse_of_high_scores(T, V, dt):
    """Maxima from 4 to 128, spread over many parts; the loss alone and with gradients."""
    banner("head lse", T, V, dt)
    g = torch.Generator().manual_seed(V)
    z = torch.linspace(4.0, 128.0, D)[:, None] - 3.0 * torch.randn(D, V, generator=g).abs()
    z = z.to(TDT[dt]).float()
    Wv, x = given(z, dt), pick(T, dt)
    lse, tol = (t[torch.arange(T) % D] for t in lse_and_bound(z, V, dt))
    labels = z.argmax(1).to(torch.int32)[torch.arange(T) % D].cuda()
    loss = lse - z.double().max(1).values[torch.arange(T) % D]
    for res in (M.moe_head_xent(x, Wv, labels), M.moe_head_xent_grad(x, Wv, labels)):
        assert off(res["lse"], lse, tol) is None
        assert off(res["loss"], loss, tol + u * loss) is None


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(64, 700), (300, 9001)])
def test_certain_tokens(T, V, dt):
    """One score of 33 to 127, all others 30 or more below: lse is the score up to
    V e^-30 and 8 u, less than half a step of the score (32 u), so it is the score
    itself and the loss is 0, and what is left of dz at the label is 8 u of the weight."""
    banner("head certain", T, V, dt)
    g = torch.Generator().manual_seed(T)
    top = torch.linspace(33.0, 127.0, D) + torch.rand(D, generator=g) / 4
    z = top[:, None] - 30.5 - 20.0 * torch.rand(D, V, generator=g)
    at = torch.randint(0, V, (D,), generator=g)
    z[torch.arange(D), at] = top
    z = z.to(TDT[dt]).float()
    Wv, x = given(z, dt), pick(T, dt)
    i = torch.arange(T) % D
    labels = at[i].to(torch.int32).cuda()
    score = z[torch.arange(D), at][i].cuda()
    a = M.moe_head_xent(x, Wv, labels)
    b = M.moe_head_xent_grad(x, Wv, labels)
    idx = labels[:, None].contiguous()
    c = M.moe_head_distill_grad(x, Wv, (idx, torch.zeros_like(idx, dtype=torch.float32)), 0.5,
                                labels)
    for res in (a, b, c):
        assert bool((res["loss"] == 0).all()), float(res["loss"].abs().max())
        assert torch.equal(res["lse"], score)
    # p at tau 0.5 is 1 too: kd = tau^2 (ln 1 - ln p)
    assert float(c["kd"].abs().max()) <= 0.25 * 8 * u
    if dt == "f32":
        n = torch.bincount(torch.arange(T) % D, minlength=D).cuda()    # copies of a token
        lab = b["dWv"][at.cuda(), torch.arange(D, device="cuda")]
        assert bool((lab.abs() <= (8 * u + V * math.exp(-30.5)) * n).all()), float(lab.abs().max())


@pytest.mark.parametrize("tau", [0.001, 0.01, 0.05, 0.3])
@pytest.mark.parametrize("V", [150, 3001])
def test_low_temperatures(V, tau):
    """fp32, one slot (q = 1): kd and dz = tau (p - [slot]), read from dWv (x picks)."""
    banner("head low tau", V, tau)
    g = torch.Generator().manual_seed(V)
    far = 20.0
    z = torch.linspace(1.0, 60.0, D)[:, None] - tau * far * torch.rand(D, V, generator=g)
    Wv, x = given(z, "f32"), pick(D, "f32")
    idx = torch.randint(0, V, (D, 1), generator=g)
    s = z.double() / tau
    logp = torch.log_softmax(s, 1)
    span = (s.max(1).values - s.min(1).values)[:, None]
    # of ln p: the sum's and its logarithm's, and of the arguments z / tau - max
    e = sum_error(V, "f32") + u * (8 + 4 * span + 4 * logp.abs())
    res = M.moe_head_distill_grad(x, Wv, (idx.to(torch.int32).cuda(),
                                          torch.zeros(D, 1, device="cuda")), tau)
    lp = logp.gather(1, idx)[:, 0]
    assert off(res["kd"], -tau ** 2 * lp, tau ** 2 * (e.gather(1, idx)[:, 0] + 4 * u * lp.abs())) is None
    hot = torch.zeros_like(z).scatter_(1, idx, 1.0).double()
    dz = tau * (logp.exp() - hot)
    tol = tau * (logp.exp() * (e + 4 * u) + 4 * u * hot)
    assert off(res["dWv"].t(), dz, tol) is None


@pytest.mark.parametrize("tau", [0.001, 0.01, 0.05, 0.3])
@pytest.mark.parametrize("K", [2, 12, 100])
def test_low_temperatures_of_the_teacher(K, tau):
    """Several slots in fp32.  A slot's ln q has 4 u times its difference from the largest
    (the difference, the constant 1 / tau, their product) and 24 u of the exponential,
    the sum of K in a wave, the quotient and the logarithm; q has that and the sum's."""
    V, far = 400, 15.0
    banner("head low tau, slots", K, tau)
    g = torch.Generator().manual_seed(K)
    z = torch.linspace(1.0, 60.0, D)[:, None] - tau * far * torch.rand(D, V, generator=g)
    Wv, x = given(z, "f32"), pick(D, "f32")
    idx = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(D)])
    score = torch.linspace(-40.0, 16.0, D)[:, None] - tau * far * torch.rand(D, K, generator=g)
    logp = torch.log_softmax(z.double() / tau, 1)
    span = z.double().max(1, keepdim=True).values / tau - z.double() / tau
    ep = sum_error(V, "f32") + u * (8 + 4 * span.max(1, keepdim=True).values + 4 * logp.abs())
    logq = torch.log_softmax(score.double() / tau, 1)
    q = logq.exp()
    wide = (score.double().max(1, keepdim=True).values - score.double()) / tau
    eq = u * (24 + 4 * wide + 4 * wide.max(1, keepdim=True).values)
    res = M.moe_head_distill_grad(x, Wv, (idx.to(torch.int32).cuda(), score.cuda()), tau)
    lp = logp.gather(1, idx)
    kd = (q * (logq - lp)).sum(1)
    tol = (q * (eq * (1 + (logq - lp).abs()) + ep.gather(1, idx)
                + 4 * u * (logq.abs() + lp.abs()))).sum(1)
    assert off(res["kd"], tau ** 2 * kd, tau ** 2 * tol) is None
    p, qs = logp.exp(), torch.zeros(D, V, dtype=torch.float64).scatter_(1, idx, q)
    eqs = torch.zeros(D, V, dtype=torch.float64).scatter_(1, idx, q * eq)
    tol = tau * (p * ep + eqs + 4 * u * (p + qs))
    assert off(res["dWv"].t(), tau * (p - qs), tol) is None


@pytest.mark.parametrize("V", [600, 3000])
def test_gradients_of_very_high_scores(V):
    """bf16, 64 equal scores of 4000 to 64000 and all others far below (2^-64 of the
    largest at most, where the 16 bits end): dz of those is
    1/64, as dWv shows it (x picks).  1/64 has no rounding in bf16, and half a step is
    2^-9 of it (below it: 2^-10), so that it comes out exactly if the scores' 16 bits
    (3.4e-4) and what else the exponent is off by stay below that; an exponent that
    is rounded at the size of the score times log2(e) does not."""
    banner("head very high scores", V)
    g = torch.Generator().manual_seed(V)
    top = torch.linspace(4000.0, 64000.0, D).to(torch.bfloat16).float()
    z = (top[:, None] * 0.9).expand(D, V).clone()
    hot = torch.stack([torch.randperm(V, generator=g)[:64] for _ in range(D)])
    z = z.scatter_(1, hot, top[:, None].expand(D, 64)).to(torch.bfloat16).float()
    Wv, x = given(z, "bf16"), pick(D, "bf16")
    labels = hot[:, 0].to(torch.int32).cuda()
    res = M.moe_head_xent_grad(x, Wv, labels)
    want = torch.zeros(D, V).scatter_(1, hot, torch.full((D, 64), 1.0 / 64))
    want.scatter_(1, hot[:, :1], torch.full((D, 1), 1.0 / 64 - 1.0))     # 63/64: 6 bits
    bad = (~((res["dWv"].t().float().cpu() - want).abs() <= 2.0 ** -64)).nonzero()
    assert len(bad) == 0, (len(bad), bad[0], float(res["dWv"][bad[0][1], bad[0][0]]))

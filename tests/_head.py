"""The vocabulary head's losses in 64 bits, with bounds on what rounding may do
to the kernels' results, shared by the head's tests.

Bounds, per element, to first order (u: half a step of the storage type; g(n) = n
2^-23 for a sum of n terms in fp32, twice the bound of recursive summation, for
matrix instructions whose inner order and rounding are not specified):
  z      |e| <= g(d) |x| |Wv|^T                       (bf16 products are exact)
  lse    the largest e of the row + g(V) (a relative error of the sum) + 2^-20
         for exp and log + 2^-22 (|lse| + |z|max + the spread of z), the roundings
         of z - m, m + ln s and their like
  loss   e(lse) + e(z) + 2^-22 |loss|
  kd     tau^2 sum_j q_j (e(z)/tau + e(lse at tau) + 2^-19 (1 + |terms|))
  p      relative: e(z) + e(lse); for the bf16 cross entropy without a teacher also
         ln 2 * 2^-11, half a step of the 16-bit scores that dz is made from (steps
         of 2^-10 of log2: a score is off by at most 2^-11 there, its exponential
         by the factor 2^(2^-11)), plus 2^-64 of the largest p where a score lies
         64 or more below its 128 columns' largest and counts as 64
  dz     w p e(p) + u |dz|  (the rounding to the storage type)
  dx     |e(dz)| |Wv| + g(V) |dz| |Wv| + u |dx|,  dWv likewise; but in bf16
         without a teacher the label's entry of dz loses nothing in dx (what its rounding
         takes is added again in fp32: 2^-23 |dz| instead of u |dz|), and with up to 128
         tokens every entry is two terms in dWv (u^2 |dz|)
"""
import math

import torch

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}
E32 = 2.0 ** -23


def reference(x, Wv, labels=None, weight=None, teacher=None, tau=1.0, dt="bf16"):
    """-> {name: (value, bound)} for loss, lse, kd, dx, dWv, all float64 on the
    inputs' device.  Rows of x that have no loss are not looked at."""
    T, d = x.shape
    V = Wv.shape[0]
    dev = x.device
    f64 = torch.float64
    lab = torch.full((T,), -1, device=dev) if labels is None else labels.long()
    has_y = (lab >= 0) & (lab < V)
    if teacher is not None:
        idx, score = teacher[0].long(), teacher[1].to(f64)
        on = (idx >= 0) & (idx < V) & (score > -math.inf)
        has_t = on.any(1)
        K = idx.shape[1]
        # a slot whose score is -infinity makes its token one with a loss, of 0
        some = ((idx >= 0) & (idx < V)).any(1)
    else:
        has_t = some = torch.zeros(T, dtype=torch.bool, device=dev)
    act = (has_y | some).nonzero()[:, 0]
    X = torch.zeros(T, d, dtype=f64, device=dev)
    X[act] = x[act].to(f64)
    W = Wv.to(f64)
    z = X @ W.t()
    za = X.abs() @ W.abs().t()
    ez = d * E32 * za
    u = U[dt]

    def lse_of(s):
        l = torch.logsumexp(z * s, 1)
        e = (ez * s).max(1).values + V * E32 + 2.0 ** -20 + \
            2.0 ** -22 * (l.abs() + (z * s).abs().max(1).values
                          + (z * s).max(1).values - (z * s).min(1).values)
        return l, e

    out = {}
    dz = torch.zeros(T, V, dtype=f64, device=dev)
    edz = torch.zeros_like(dz)
    row = torch.arange(T, device=dev)
    if labels is not None:
        l, el = lse_of(1.0)
        at = lab.clamp(0, V - 1)
        loss = l - z[row, at]
        y = has_y.to(f64)
        out["lse"] = (l * y, el * y)
        out["loss"] = (loss * y, (el + ez[row, at] + 2.0 ** -22 * loss.abs()) * y)
        w = (torch.ones(T, dtype=f64, device=dev) if weight is None else weight.to(f64)) * y
        p = torch.exp(z - l[:, None]) * w[:, None]
        dz += p
        dz[row, at] -= w
        edz += p.abs() * (ez + el[:, None] + 2.0 ** -20)
        if dt == "bf16" and teacher is None:
            edz += p.abs() * math.log(2.0) * 2.0 ** -11 + w.abs()[:, None] * 2.0 ** -64
    if teacher is not None:
        l, el = lse_of(1.0 / tau)
        q = torch.softmax(torch.where(on, score / tau, torch.full_like(score, -math.inf)), 1)
        q = torch.where(on & has_t[:, None], q, torch.zeros_like(q))
        at = idx.clamp(0, V - 1)
        lq = torch.log(torch.where(q > 0, q, torch.ones_like(q)))
        term = lq - z.gather(1, at) / tau + l[:, None]
        out["kd"] = (tau ** 2 * (q * term).sum(1),
                     tau ** 2 * (q * (ez.gather(1, at) / tau + el[:, None]
                                      + 2.0 ** -19 * (1 + term.abs() + lq.abs() + l[:, None].abs()))
                                 ).sum(1) + 2.0 ** -120)
        tw = torch.ones(T, dtype=f64, device=dev)
        if len(teacher) > 2 and teacher[2] is not None:
            tw = teacher[2].to(f64)
        c = (tau * tw * has_t.to(f64))[:, None]
        p = torch.exp(z / tau - l[:, None]) * c
        dz += p
        dz.scatter_add_(1, at, -c * q)
        edz += p.abs() * (ez / tau + el[:, None] + 2.0 ** -20)
        edz.scatter_add_(1, at, c.abs() * q * (K * E32 + 2.0 ** -20))
    base = edz
    edz = base * (1 + u) + u * dz.abs() + 2.0 ** -126
    edw = base * (1 + u) + u * u * dz.abs() + 2.0 ** -126 if dt == "bf16" and T <= 128 else edz
    if dt == "bf16" and teacher is None:
        edz = edz.clone()
        edz[row, lab.clamp(0, V - 1)] -= (u - E32) * dz[row, lab.clamp(0, V - 1)].abs()
    dx = dz @ W
    dW = dz.t() @ X
    out["dx"] = (dx, edz @ W.abs() + V * E32 * (dz.abs() @ W.abs()) + u * dx.abs() + 2.0 ** -126)
    out["dWv"] = (dW, edw.t() @ X.abs() + T * E32 * (dz.abs().t() @ X.abs()) + u * dW.abs()
                  + 2.0 ** -126)
    return out


def check(got, ref, what=""):
    """Every result of the call within its bound (5% for second-order terms)."""
    for name, t in got.items():
        if t is None:
            continue
        val, tol = ref[name]
        err = (t.to(torch.float64) - val).abs()
        bad = ~(err <= 1.05 * tol)
        if bool(bad.any()):
            k = int(bad.flatten().nonzero()[0])
            raise AssertionError("%s %s: %d of %d off, first at %d: got %.9g want %.9g tol %.3g" % (
                what, name, int(bad.sum()), bad.numel(), k, float(t.flatten()[k]),
                float(val.flatten()[k]), float(tol.flatten()[k])))


def inputs(T, d, V, dt="bf16", masked=0.0, K=0, seed=0, device="cuda", scale=2.0):
    """x, Wv, labels, weight, teacher with values a trained head has; made on the
    CPU from the seed."""
    g = torch.Generator().manual_seed(seed)
    word = torch.randint(0, V, (T,), generator=g)
    Wv = (torch.randn(V, d, generator=g) * d ** -0.5).to(TDT[dt])
    x = torch.randn(T, d, generator=g) * scale + \
        14.0 * torch.rand(T, 1, generator=g) * Wv[word].float()
    labels = torch.where(torch.rand(T, generator=g) < masked, torch.full_like(word, -1), word)
    weight = 0.25 + torch.rand(T, generator=g)
    teacher = None
    if K:
        idx = torch.randint(0, V, (T, K), generator=g)             # entries may repeat
        idx[:, 0] = word
        idx[torch.rand(T, K, generator=g) < 0.1] = -1
        score = 4.0 * torch.randn(T, K, generator=g)
        teacher = (idx.to(torch.int32).to(device), score.to(device),
                   (0.25 + torch.rand(T, generator=g)).to(device))
    return (x.to(TDT[dt]).to(device), Wv.to(device), labels.to(torch.int32).to(device),
            weight.to(device), teacher)

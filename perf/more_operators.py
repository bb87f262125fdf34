"""The training step's loss over a vocabulary, as timed work.

A vocabulary head Wv [V,d] scores the layer's outputs x [T,d]: z = x Wv^T.
Two families of operators on these scores, none of which keeps them:

* xent:    softmax cross entropy with a label a token, alone (evaluation) or
           with the gradients of x and Wv (a training step);
* distill: the divergence from a teacher of which the K top scores a token are
           kept, at a temperature, alone or with the gradients, and with the
           cross entropy of the same scores beside it.

`own` chooses between the plain form (elementary torch operations in 32 bits,
a block of tokens at a time) and the framework's operators.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
BLOCK = 4096        # tokens of the plain form at a time


# ------------------------------------------------------------------- cases

def _case(name, T, d, V, dtype="bf16", grad=True, masked=0.0, K=0, tau=1.0, labels=True):
    """masked: the share of tokens without a label; K: the teacher's slots (0: none);
    labels: whether a distillation has the cross entropy beside it."""
    return {"name": name, "T": T, "d": d, "V": V, "dtype": dtype, "grad": grad,
            "masked": masked, "K": K, "tau": tau, "labels": labels}


def listed():
    return [
        # five tokens through the smallest fp32 layer: nothing but latency
        _case("xent_tiny_f32", 5, 64, 1000, "f32", grad=False),
        # sixteen candidates scored in a serving step: the head is read once
        _case("xent_few", 16, 4096, 128000, grad=False),
        # an evaluation batch of the 8-expert layer, a tenth of it padding
        _case("xent_eval", 8192, 1024, 50257, grad=False, masked=0.1),
        # a training step of the smallest fp32 layer
        _case("xent_grad_tiny_f32", 256, 64, 1000, "f32"),
        # a micro-batch of an odd number of tokens
        _case("xent_grad_small", 777, 1024, 32000),
        # an fp32 head with an odd vocabulary
        _case("xent_grad_f32", 1999, 1088, 8191, "f32", masked=0.05),
        # a training step of the 8-expert layer
        _case("xent_grad_moe_s", 8192, 1024, 50257),
        # fine tuning of the 16-expert layer: half the tokens are prompts, without a label
        _case("xent_grad_masked", 16384, 2048, 32000, masked=0.5),
        # a quarter of the long-context chunk, a large vocabulary
        _case("xent_grad_long", 16384, 4096, 128000),
        # how far a student is from its teacher, no gradient
        _case("distill_eval", 2048, 2048, 32000, grad=False, K=32, tau=1.0, labels=False),
        # a student's step on few tokens, fp32
        _case("distill_grad_f32", 33, 320, 5003, "f32", K=8, tau=4.0, labels=False),
        # distillation and cross entropy together, the 8-expert layer
        _case("distill_grad_moe_s", 8192, 1024, 50257, masked=0.1, K=64, tau=2.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = "bf16" if rng.random() < 0.8 else "f32"
    for _ in range(1000):
        T = _log_int(rng, 1, 16384)
        d = 64 * _log_int(rng, 1, 64)
        V = _log_int(rng, 200, 131072)
        if T * d * V <= (16384 * 4096 * 128000 if dtype == "bf16" else 2e11):
            break
    K = rng.choice([0, 0, _log_int(rng, 1, 128)])
    c = _case("", T, d, V, dtype, rng.random() < 0.7, rng.choice([0.0, 0.1, 0.5]), K,
              rng.choice([1.0, 2.0, rng.uniform(0.7, 5.0)]) if K else 1.0,
              rng.random() < 0.6 if K else True)
    del c["name"]
    return c


# ------------------------------------------------------------------- inputs

def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, d, V, K, dt = case["T"], case["d"], case["V"], case["K"], DT[case["dtype"]]
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")
    # words are about Zipf distributed; scores have a spread of 2, and that of the label
    # stands out by 0 to 16: tokens from hopeless to certain
    word = (V ** rand(T)).long().clamp_(1, V) - 1
    Wv = torch.randn((V, d), generator=g, device="cuda", dtype=dt).mul_(d ** -0.5)
    x = torch.randn((T, d), generator=g, device="cuda").mul_(2.0)
    x += 16.0 * rand(T, 1) * Wv[word].float()
    st = {"x": x.to(dt), "Wv": Wv, "labels": None, "weight": None, "teacher": None}
    if case["labels"]:
        st["labels"] = torch.where(rand(T) < case["masked"], -1, word).to(torch.int32)
        st["weight"] = (0.5 + rand(T)) / T
    if K:
        # the label first, the others one from each of K stretches of the vocabulary
        n = max(1, V // K)
        step = torch.arange(K, device="cuda") * n + (rand(T, K) * n).long().clamp_(max=n - 1)
        step[:, 0] = 0
        idx = ((word[:, None] + step) % V).to(torch.int32)
        if K > 2:                                   # some teachers kept fewer
            idx[rand(T) < 0.2, K - K // 3:] = -1
        s = 16.0 * rand(T, 1) - 1.5 * torch.arange(1, K + 1, device="cuda").float().log()
        st["teacher"] = (idx, (s + 0.3 * rand(T, K)).contiguous(), (0.5 + rand(T)) / T)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        import mixture_experts_layer_permute_amd as M
        st["head"] = M.HeadLoss(case["T"], case["d"], case["V"], DT[case["dtype"]], K=case["K"],
                                tau=case["tau"], grad=case["grad"], device="cuda")
        st["head"].bind(st["Wv"])
    return st


# --------------------------------------------------------------- plain form

def _plain(st):
    c = st["case"]
    T, V, tau = c["T"], c["V"], c["tau"]
    W = st["Wv"].float()
    out = {"loss": [], "lse": [], "kd": [], "dx": []}
    dW = torch.zeros_like(W) if c["grad"] else None
    for t0 in range(0, T, BLOCK):
        blk = slice(t0, min(T, t0 + BLOCK))
        x = st["x"][blk].float()
        z = x @ W.t()
        n = x.shape[0]
        row = torch.arange(n, device=x.device)
        top = z.max(1, keepdim=True).values
        G = None
        if st["labels"] is not None:
            lab = st["labels"][blk].long()
            ok = (lab >= 0) & (lab < V)
            lab = lab.clamp(0, V - 1)
            e = torch.exp(z - top)
            s = e.sum(1, keepdim=True)
            lse = (top + s.log())[:, 0]
            zero = torch.zeros_like(lse)
            out["lse"].append(torch.where(ok, lse, zero))
            out["loss"].append(torch.where(ok, lse - z[row, lab], zero))
            if c["grad"]:
                w = torch.where(ok, st["weight"][blk], zero)
                G = e.mul_((w[:, None] / s))
                G[row, lab] -= w
            del e
        if st["teacher"] is not None:
            idx, score, u = (t[blk] for t in st["teacher"])
            idx = idx.long()
            on = (idx >= 0) & (idx < V)
            idx = idx.clamp(0, V - 1)
            any_on = on.any(1)
            sc = torch.where(on, score / tau, torch.full_like(score, -math.inf))
            hi = sc.max(1, keepdim=True).values
            sc = torch.where(any_on[:, None], sc - hi, torch.zeros_like(sc))
            q = torch.where(on, torch.exp(sc), torch.zeros_like(sc))
            tot = q.sum(1, keepdim=True).clamp_min(1e-30)
            q = q / tot
            e = torch.exp((z - top) / tau)
            s = e.sum(1, keepdim=True)
            logp = (z.gather(1, idx) - top) / tau - s.log()
            kd = torch.where(q > 0, q * ((sc - tot.log()) - logp), torch.zeros_like(q)).sum(1)
            out["kd"].append(torch.where(any_on, kd * tau ** 2, torch.zeros_like(kd)))
            if c["grad"]:
                w = torch.where(any_on, u * tau, torch.zeros_like(u))[:, None]
                e.mul_(w / s)
                G = e if G is None else G.add_(e)
                G.scatter_add_(1, idx, -w * q)
            del e
        del z
        if c["grad"]:
            out["dx"].append((G @ W).to(st["x"].dtype))
            dW.addmm_(G.t(), x)
    res = {k: torch.cat(v) for k, v in out.items() if v}
    if c["grad"]:
        res["dWv"] = dW.to(st["Wv"].dtype)
    return res


def run(state):
    if not own:
        return _plain(state)
    c, head = state["case"], state["head"]
    if c["grad"]:
        head.step(state["x"], state["labels"], state["weight"], state["teacher"])
    else:
        head.forward(state["x"], state["labels"], state["teacher"])
    res = {}
    if c["labels"]:
        res["loss"], res["lse"] = head.loss, head.lse
    if c["K"]:
        res["kd"] = head.kd
    if c["grad"]:
        res["dx"], res["dWv"] = head.dx, head.dWv
    return res


# ------------------------------------------------------------ work and truth

def work(case):
    T, d, V, K, b = case["T"], case["d"], case["V"], case["K"], BYTES[case["dtype"]]
    # tokens that have a loss; the others need no scores
    n = T if K else T * (1.0 - case["masked"])
    small = 12 * T * case["labels"] + 8 * T * K + 4 * T * (K > 0)
    if not case["grad"]:
        return {"bytes": (n * d + V * d) * b + small, "flops": 2.0 * n * d * V}
    return {"bytes": (n * d + T * d + 2 * V * d) * b + small + 4 * T * case["labels"] +
            4 * T * (K > 0), "flops": 6.0 * n * d * V}


def exact(case, seed):
    st = _inputs(case, seed)
    T, V, tau = case["T"], case["V"], case["tau"]
    W = st["Wv"].double()
    keys = (["loss", "lse"] if case["labels"] else []) + (["kd"] if case["K"] else [])
    res = {k: torch.zeros(T, dtype=torch.float64, device="cuda") for k in keys}
    if case["grad"]:
        res["dx"] = torch.zeros(T, case["d"], dtype=torch.float64, device="cuda")
        res["dWv"] = torch.zeros_like(W)
    for blk in torch.arange(T, device="cuda").split(2048):
        x = st["x"][blk].double()
        z = x.mm(W.t())
        G = torch.zeros_like(z)
        if case["labels"]:
            lab = st["labels"][blk].long()
            t = ((lab >= 0) & (lab < V)).nonzero()[:, 0]
            lse = z[t].logsumexp(1)
            res["lse"][blk[t]] = lse
            res["loss"][blk[t]] = lse - z[t, lab[t]]
            if case["grad"]:
                w = st["weight"][blk[t]].double()
                g = (z[t] - lse[:, None]).exp() * w[:, None]
                g[torch.arange(len(t), device="cuda"), lab[t]] -= w
                G[t] += g
        if case["K"]:
            idx, score, u = (v[blk] for v in st["teacher"])
            idx = idx.long()
            keep = (idx >= 0) & (idx < V)
            t = keep.any(1).nonzero()[:, 0]
            logq = (score[t].double() / tau).masked_fill(~keep[t], -math.inf).log_softmax(1)
            q = logq.exp()
            logp = (z[t] / tau).log_softmax(1)
            at = idx[t].clamp(0, V - 1)
            term = q * (logq - logp.gather(1, at))
            res["kd"][blk[t]] = tau * tau * term.masked_fill(~keep[t], 0.0).sum(1)
            if case["grad"]:
                w = (u[t].double() * tau)[:, None]
                G[t] += (logp.exp() * w).scatter_add(1, at, -w * q)
        if case["grad"]:
            res["dx"][blk] = G.mm(W)
            res["dWv"] += G.t().mm(x)
    return res

"""The MoE layer's operators for few tokens and for the gradients, as timed work.

Two families, on the shapes of moe_inputs/configs.py or generic ones:

* few:  a whole MoE layer (gate, top-k, expert FFNs, weighted sum) for 1 to 64
        tokens, the step of a serving loop;
* norm, clip: the global L2 norm of a list of gradient tensors, and the list
        scaled to a largest norm, the step of a training loop between the
        backward pass and the optimizer.

`own` chooses between the plain form (elementary torch operations in 32 bits,
64 for the long sums and the gate's logits) and the framework's operators.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------- cases

def _few(name, T, d, f, E, k, act="gelu", dtype="bf16", renorm=1, zipf=0.0):
    return {"name": name, "op": "few", "T": T, "d": d, "f": f, "E": E, "k": k, "act": act,
            "dtype": dtype, "renorm": renorm, "zipf": zipf}


def _grad(name, op, tensors, over, zero_experts=0):
    """tensors: "dtype:s0xs1x...*count" entries, comma separated."""
    return {"name": name, "op": op, "tensors": tensors, "over": over,
            "zero_experts": zero_experts}


def listed():
    return [
        # one token through the smallest fp32 layer: nothing but latency
        _few("few_tiny_f32_t1", 1, 64, 256, 4, 1, dtype="f32"),
        # one sequence being decoded, the 8-expert GeLU layer
        _few("few_small_t1", 1, 1024, 4096, 8, 2),
        # thirteen sequences: every expert is hit, some by several tokens
        _few("few_small_t13", 13, 1024, 4096, 8, 2),
        # five drafted tokens, 16 wide experts, skewed routing
        _few("few_wide_t5", 5, 2048, 8192, 16, 2, zipf=1.2),
        # a batch of 48 sequences over 64 narrow experts, most of them hit
        _few("few_many_t48", 48, 1024, 4096, 64, 2, zipf=1.0),
        # an fp32 SwiGLU layer with odd sizes and the softmax over all experts
        _few("few_f32_t7", 7, 1088, 1984, 12, 3, act="swiglu", dtype="f32", renorm=0),
        # one token of the long-context SwiGLU layer, 32 of its experts on this GPU
        _few("few_long_t1", 1, 4096, 14336, 32, 8, act="swiglu"),
        # a full serving batch of the same layer: every weight is read
        _few("few_long_t64", 64, 4096, 14336, 32, 8, act="swiglu", zipf=0.8),
        # the gradients of the smallest layer
        _grad("clip_tiny", "clip", "f32:64x4,f32:4x64x256,f32:4x256x64", 5.0),
        # the gradients of a model of 20 small layers, 200 tensors of odd sizes, fp32 gates
        _grad("clip_list", "clip",
              "f32:520x8*20,bf16:8x520x1037*20,bf16:8x1037x520*20,bf16:520*70,f32:131*70", 2.5),
        # the gradients of the 16-expert layer, some experts without tokens
        _grad("clip_wide", "clip", "bf16:2048x16,bf16:16x2048x8192,bf16:16x8192x2048", 40.0, 3),
        # the norm alone of a 16-expert shard of the long-context layer's gradients
        _grad("norm_long", "norm", "bf16:4096x16,bf16:16x4096x14336*2,bf16:16x14336x4096", 1.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.6:
        dtype = "bf16" if rng.random() < 0.8 else "f32"
        for _ in range(1000):
            d = 64 * _log_int(rng, 1, 64)
            f = 64 * _log_int(rng, 2, 224)
            E = _log_int(rng, 2, 128)
            # weights within the largest listed case's
            if E * d * f * BYTES[dtype] <= 32 * 4096 * 14336 * 2 * (1 if dtype == "bf16" else 0.25):
                break
        k = rng.randint(1, min(8, E))
        c = _few("", _log_int(rng, 1, 64), d, f, E, k, rng.choice(["gelu", "swiglu"]), dtype,
                 rng.randint(0, 1), rng.choice([0.0, 0.8, 1.2]))
    else:
        op = "clip" if rng.random() < 0.7 else "norm"
        layers = _log_int(rng, 1, 24)
        total = 10 ** rng.uniform(4.0, 8.9)             # elements
        d = max(3, min(4096, int((total / layers / 8) ** 0.5 * rng.uniform(0.4, 1.0))))
        E = _log_int(rng, 1, 16)
        f = max(3, int(total / layers / 2 / E / d))
        t = rng.choice(["bf16", "bf16", "f32"])
        c = _grad("", op, "%s:%dx%d*%d,%s:%dx%dx%d*%d,%s:%dx%dx%d*%d,%s:%d*%d" % (
            rng.choice(["bf16", "f32"]), d, E, layers, t, E, d, f, layers, t, E, f, d, layers,
            t, d, 2 * layers), 10 ** rng.uniform(-0.5, 2.0), rng.randint(0, E - 1))
    del c["name"]
    return c


def _buckets(tensors):
    """Flat buffers, one per type in order of appearance, and views like `tensors`."""
    kinds = list(dict.fromkeys(t.dtype for t in tensors))
    flat = [torch.empty(sum(t.numel() for t in tensors if t.dtype == q), dtype=q,
                        device="cuda") for q in kinds]
    used = [0] * len(kinds)
    views = []
    for t in tensors:
        q = kinds.index(t.dtype)
        views.append(flat[q][used[q]:used[q] + t.numel()].view(t.shape))
        used[q] += t.numel()
    return flat, views


def _shapes(case):
    out = []
    for ent in case["tensors"].split(","):
        t, s = ent.split(":")
        s, n = (s.split("*") + ["1"])[:2]
        out += [(t, tuple(int(v) for v in s.split("x")))] * int(n)
    return out


# ------------------------------------------------------------------- inputs

def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, std, dtype):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)

    if case["op"] == "few":
        T, d, f, E, dt = case["T"], case["d"], case["f"], case["E"], DT[case["dtype"]]
        # Tokens in steps of 1/32 and gate weights in steps of 2^-10 or finer
        # powers of two: the logits' sums are exact in fp32, so no order of
        # summation moves a token to another expert.
        q = 2.0 ** -max(6, 4 + math.ceil(math.log2(d) / 2))
        x = (normal((T, d), 32.0, torch.float32).round_().clamp_(-192, 192) / 32).to(dt)
        Wg = (normal((d, E), d ** -0.5 / q, torch.float32).round_().clamp_(-128, 128) * q).to(dt)
        st = {"x": x, "Wg": Wg, "bias": None, "W3": None}
        if case["zipf"]:
            rank = torch.randperm(E, generator=g, device="cuda").float() + 1
            st["bias"] = (rank.log() * (-case["zipf"] * 64)).round_() / 64
        st["W1"] = normal((E, d, f), d ** -0.5, dt)
        if case["act"] == "swiglu":
            st["W3"] = normal((E, d, f), d ** -0.5, dt)
        st["W2"] = normal((E, f, d), f ** -0.5, dt)
        return st
    shapes = _shapes(case)
    n = sum(math.prod(s) for _, s in shapes)
    std = case["over"] / math.sqrt(n)                   # norm about `over` times the limit 1
    grads = []
    for t, s in shapes:
        w = normal(s, std, DT[t])
        if len(s) == 3 and case["zero_experts"]:        # experts that no token chose
            w[:min(case["zero_experts"], s[0])] = 0
        grads.append(w)
    return {"grads": grads, "max_norm": 1.0}


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if case["op"] == "clip":
        # the clipped gradients go to one bucket per type, which an optimizer
        # (or a reduction between GPUs) takes as a whole: tensor after tensor,
        # no gaps, so that odd sizes leave the next one unaligned
        st["bucket"], st["out"] = _buckets(st["grads"])
    elif case["op"] == "norm":
        st["out"] = None
    if own:
        import mixture_experts_layer_permute_amd as M
        if case["op"] == "few":
            st["layer"] = M.FewTokenMoELayer(case["T"], case["d"], case["f"], case["E"],
                                             case["k"], case["act"], DT[case["dtype"]],
                                             case["renorm"], "cuda")
            st["layer"].bind(st["Wg"], st["W1"], st["W2"], st["W3"], st["bias"])
        else:
            st["clip"] = M.GradClip(st["grads"], st["out"])
    return st


# --------------------------------------------------------------- plain form

def _plain_ffn(x, W1, W3, W2):
    """One expert on the rows of x, all fp32."""
    h = x @ W1.float()
    if W3 is None:
        a = 0.5 * h * (1.0 + torch.erf(h * math.sqrt(0.5)))
    else:
        a = h / (1.0 + torch.exp(-h)) * (x @ W3.float())
    return a @ W2.float()


def _plain_few(st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = st["x"].float()
    logits = st["x"].double() @ st["Wg"].double()
    if st["bias"] is not None:
        logits = logits + st["bias"].double()
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    p = torch.exp((top - top[:, :1]).float())
    w = p[:, :k] / (p[:, :k] if c["renorm"] else p).sum(1, keepdim=True)
    idx = idx[:, :k]
    y = torch.zeros(T, c["d"], dtype=torch.float32, device=x.device)
    if T * k < E:                           # the chosen experts' weights, pair by pair
        for t in range(T):
            for j in range(k):
                W = [None if m is None else m.index_select(0, idx[t, j:j + 1])[0]
                     for m in (st["W1"], st["W3"], st["W2"])]
                y[t:t + 1] += w[t, j] * _plain_ffn(x[t:t + 1], *W)
    else:                                   # every expert on every token, weighted by 0 or w
        for e in range(E):
            we = (w * (idx == e)).sum(1, keepdim=True)
            y += we * _plain_ffn(x, st["W1"][e], None if st["W3"] is None else st["W3"][e],
                                 st["W2"][e])
    return {"y": y.to(st["x"].dtype), "topk_idx": idx.to(torch.int32), "topk_w": w}


def _plain_norm(grads):
    sq = torch.zeros((), dtype=torch.float64, device="cuda")
    for t in grads:
        sq = sq + t.float().square().sum(dtype=torch.float64)
    return sq.sqrt().float()


def run(state):
    c = state["case"]
    if c["op"] == "few":
        if own:
            layer = state["layer"]
            y = layer.forward(state["x"])
            return {"y": y, "topk_idx": layer.topk_idx, "topk_w": layer.topk_w}
        return _plain_few(state)
    if c["op"] == "norm":
        return state["clip"].norm() if own else _plain_norm(state["grads"]).reshape(1)
    if own:
        return [state["clip"].clip(state["max_norm"])] + state["bucket"]
    norm = _plain_norm(state["grads"])
    coef = torch.where(norm > state["max_norm"], state["max_norm"] / norm, torch.ones_like(norm))
    for t, o in zip(state["grads"], state["out"]):
        o.copy_(t.float() * coef)
    return [norm.reshape(1)] + state["bucket"]


# ------------------------------------------------------------ work and truth

def work(case):
    if case["op"] != "few":
        n = b = 0
        for t, s in _shapes(case):
            n += math.prod(s)
            b += math.prod(s) * BYTES[t]
        return {"bytes": 4 + b * (2 if case["op"] == "clip" else 1),
                "flops": n * (3 if case["op"] == "clip" else 2)}
    T, d, f, E, k = (case[q] for q in ("T", "d", "f", "E", "k"))
    b = BYTES[case["dtype"]]
    products = 3 if case["act"] == "swiglu" else 2
    # experts hit, in expectation: the r-th most popular one is chosen with
    # probability min(1, c r^-zipf), the c that makes k choices in all
    pop = [r ** -case["zipf"] for r in range(1, E + 1)]
    lo, hi = 0.0, 1e9
    for _ in range(100):
        c = (lo + hi) / 2
        lo, hi = (c, hi) if sum(min(1.0, c * v) for v in pop) < k else (lo, c)
    hit = sum(1.0 - (1.0 - min(1.0, lo * v)) ** T for v in pop)
    return {"bytes": hit * products * d * f * b + d * E * b + 2 * T * d * b + 8 * T * k,
            "flops": 2.0 * T * k * products * d * f + 2.0 * T * d * E}


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] != "few":
        total = math.fsum(float((t.double() ** 2).sum()) for t in st["grads"])
        norm = math.sqrt(total)
        first = torch.tensor([norm], dtype=torch.float64, device="cuda")
        if case["op"] == "norm":
            return first
        scale = min(1.0, st["max_norm"] / norm) if norm > 0 else 1.0
        kinds = list(dict.fromkeys(t.dtype for t in st["grads"]))
        return [first] + [torch.cat([t.double().flatten() * scale for t in st["grads"]
                                     if t.dtype == q]) for q in kinds]
    T, E, k = case["T"], case["E"], case["k"]
    x = st["x"].double()
    logits = x.mm(st["Wg"].double())
    if st["bias"] is not None:
        logits += st["bias"].double()
    # an expert's place: how many are larger, or equal with a lower index
    a, b = logits.unsqueeze(2), logits.unsqueeze(1)
    lower = torch.ones(E, E, dtype=torch.bool, device="cuda").tril(-1)
    place = ((b > a) | ((b == a) & lower)).sum(2)
    idx = place.argsort(1)[:, :k]
    picked = logits.gather(1, idx)
    norm = torch.logsumexp(picked if case["renorm"] else logits, 1, keepdim=True)
    w = (picked - norm).exp()
    y = torch.zeros(T, case["d"], dtype=torch.float64, device="cuda")
    for e in sorted(set(idx.flatten().tolist())):
        t, j = (idx == e).nonzero(as_tuple=True)
        h = x[t].mm(st["W1"][e].double())
        if case["act"] == "swiglu":
            h = h * torch.sigmoid(h) * x[t].mm(st["W3"][e].double())
        else:
            h = h * torch.special.ndtr(h)
        y.index_add_(0, t, h.mm(st["W2"][e].double()) * w[t, j].unsqueeze(1))
    return {"y": y, "topk_idx": idx.to(torch.int32), "topk_w": w}

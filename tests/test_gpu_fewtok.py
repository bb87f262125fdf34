"""moe_layer_fwd_few and FewTokenMoELayer (the layer for 1 to 64 tokens)
against the oracle in 64 bits, element by element.

The bound of an element of y is arithmetic, not a fitted tolerance.  With
u = 2^-24 (half a step of fp32), a sum of n terms in any order is off by at
most (n + 1) u times the sum of the terms' sizes.  So, per pair:
  dH <= (d + 2) u |x| |W1|                             pre-activation
  dA <= slope * dH (+ the second factor's) + 8 u |A|   activation function
        + ra (|A| + the above)                         kept as one fp32 or two bf16
  dO <= dA |W2| + (f + 64) u |A| |W2|                  second product, chunks joined
and y = sum_j w_j O_j has dy <= sum_j w_j (dO_j + 64 u |O_j|) + r |y|, where r
is half a step of the type (bf16 2^-8, fp32 2^-24), ra = 2^-16 for bf16 and 0
for fp32 (whose values are not rounded again); GeLU's slope is at most
1.13, SiLU's 1.10, and a gate weight is right to 32 u.
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_permute_amd as M
import oracle
from moe_inputs import stage

from _gpu import (TDT, TOL, assert_equal_i, banner, dev, host, needs_gpu, rel_err)

pytestmark = [pytest.mark.gpu, needs_gpu]

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def inputs(T, d, f, E, act, dt, seed=0, bias=None):
    x = stage.normal(seed, (T, d), 1.0, dt)
    Wg = stage.normal(seed + 1, (d, E), 1 / np.sqrt(d), dt)
    W1 = stage.normal(seed + 2, (E, d, f), 1 / np.sqrt(d), dt)
    W2 = stage.normal(seed + 3, (E, f, d), 1 / np.sqrt(f), dt)
    W3 = stage.normal(seed + 4, (E, d, f), 1 / np.sqrt(d), dt) if act == "swiglu" else None
    b = None if bias is None else np.asarray(bias, np.float32)
    return x, Wg, W1, W2, W3, b


def upload(a, dt):
    x, Wg, W1, W2, W3, b = a
    g = [dev(v, dt) for v in (x, Wg, W1, W2)] + [None if W3 is None else dev(W3, dt)]
    return g + [None if b is None else torch.from_numpy(b).cuda()]


def reference(a, k, act, renorm, dt):
    """-> (oracle forward, bound of |y - oracle's y| per element)."""
    x, Wg, W1, W2, W3, b = a
    fw = oracle.layer_forward(x, Wg, W1, W2, W3, k=k, act=act, bias=b, renorm=renorm)
    T, d = x.shape
    f = W1.shape[2]
    r = HALF[dt]
    x64 = np.abs(x.astype(np.float64))
    bound = r * np.abs(fw["y"])
    for t in range(T):
        for j in range(k):
            e, row, w = fw["idx"][t, j], fw["dest"][t, j], fw["w"][t, j]
            A = np.abs(fw["A"][row])
            dH = (d + 2) * U * (x64[t] @ np.abs(W1[e].astype(np.float64)))
            if act == "swiglu":
                dH3 = (d + 2) * U * (x64[t] @ np.abs(W3[e].astype(np.float64)))
                H, H3 = fw["H"][row], np.abs(fw["H3"][row])
                dA = 1.1 * dH * (H3 + dH3) + np.abs(oracle.silu(H)) * dH3
            else:
                dA = 1.13 * dH
            dA = dA + 8 * U * A
            dA = dA + (2.0 ** -16 if dt == "bf16" else 0.0) * (A + dA)
            W2a = np.abs(W2[e].astype(np.float64))
            bound[t] += w * ((dA + (f + 64) * U * A) @ W2a + 64 * U * (A @ W2a))
    return fw, bound * 1.001 + 1e-30


def compare(got, fw, bound, dt):
    y, logits, idx, w = got
    assert_equal_i(logits.cpu().numpy().view(np.uint32), fw["logits"].view(np.uint32), "logits")
    assert_equal_i(idx, fw["idx"], "topk_idx")
    assert np.all(np.abs(host(w) - fw["w"]) <= 32 * U * fw["w"] + 1e-30), "topk_w"
    err = np.abs(host(y) - fw["y"])
    assert np.all(err <= bound), "y: off by %.2f of its bound" % float((err / bound).max())
    assert rel_err(host(y), fw["y"]) <= TOL[dt]


CASES = [
    # T, d, f, E, k, act, dtype, renorm: every count of token tiles, strips that
    # end inside a tile, one step of the reduction and uneven shares of it
    (1, 64, 64, 1, 1, "gelu", "bf16", 1),
    (1, 64, 64, 1, 1, "swiglu", "f32", 1),
    (1, 256, 512, 8, 2, "gelu", "bf16", 1),
    (2, 192, 320, 5, 3, "swiglu", "bf16", 0),
    (7, 320, 192, 12, 3, "swiglu", "f32", 0),
    (15, 128, 448, 3, 2, "gelu", "f32", 1),
    (16, 128, 256, 2, 1, "gelu", "bf16", 1),
    (17, 64, 704, 2, 2, "swiglu", "bf16", 1),
    (31, 256, 64, 4, 2, "gelu", "bf16", 0),
    (33, 192, 128, 2, 1, "swiglu", "bf16", 1),
    (33, 128, 192, 2, 2, "swiglu", "f32", 1),
    (48, 448, 320, 40, 6, "gelu", "bf16", 1),
    (64, 128, 384, 1, 1, "gelu", "bf16", 1),
    (64, 320, 128, 4, 4, "swiglu", "bf16", 1),
    (64, 128, 128, 3, 2, "gelu", "f32", 0),
    (64, 64, 64, 130, 64, "gelu", "bf16", 1),
    (9, 320, 64, 257, 7, "gelu", "bf16", 0),
    (2, 2112, 64, 40, 2, "swiglu", "bf16", 1),
    (5, 2048, 128, 33, 1, "gelu", "f32", 1),
    (3, 2048, 192, 20, 2, "gelu", "bf16", 0),
    (6, 192, 64, 250, 9, "gelu", "f32", 0),
    (3, 64, 128, 1024, 5, "swiglu", "bf16", 0),
    (64, 64, 64, 1000, 3, "gelu", "f32", 1),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d_d%d_f%d_E%d_k%d_%s_%s_%d" % c)
def test_against_the_oracle(case):
    T, d, f, E, k, act, dt, renorm = case
    banner("few", case)
    a = inputs(T, d, f, E, act, dt, seed=T + E)
    fw, bound = reference(a, k, act, renorm, dt)
    x, Wg, W1, W2, W3, b = upload(a, dt)
    got = M.moe_layer_fwd_few(x, Wg, W1, W2, W3, k, act, b, renorm)
    torch.cuda.synchronize()
    compare(got, fw, bound, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("E", [1, 2, 3, 7, 9, 13, 16, 20, 35, 49, 64, 71, 119])
def test_gate_rows_of_any_length_and_alignment(E, dt):
    """Gate matrices whose rows are no multiple of a load, at any element of a
    buffer that holds NaN before and behind them: the fixed-order logits' bits
    and the choice, for d of one chunk and of several, with few and more tokens."""
    for d, T in ((64, 1), (192, 6), (1088, 3)):
        banner("few gate", E, dt, d, T)
        k = min(E, 3)
        a = inputs(T, d, 64, E, "gelu", dt, seed=E + d)
        x, Wg, W1, W2, _, _ = upload(a, dt)
        want = oracle.gate_logits(a[0], a[1])
        for shift in (0, 1, 3):
            buf = torch.full((d * E + 16,), float("nan"), dtype=TDT[dt], device="cuda")
            g = buf[shift:shift + d * E].view(d, E)
            g.copy_(Wg)
            y, logits, idx, w = M.moe_layer_fwd_few(x, g, W1, W2, None, k)
            torch.cuda.synchronize()
            assert_equal_i(logits.cpu().numpy().view(np.uint32), want.view(np.uint32), "logits")
            assert_equal_i(idx, oracle.topk_select(want, k), "topk_idx")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_all_tokens_to_one_expert_others_unread(act, dt):
    """Every token's only choice is expert 5: 64 rows in one expert, and the
    other experts' weights are not read (they hold NaN)."""
    T, d, f, E = 64, 128, 192, 8
    banner("few one expert", act, dt)
    a = inputs(T, d, f, E, act, dt, seed=3, bias=[0, 0, 0, 0, 0, 1000, 0, 0])
    fw, bound = reference(a, 1, act, 1, dt)
    x, Wg, W1, W2, W3, b = upload(a, dt)
    for W in (W1, W2, W3):
        if W is not None:
            for e in range(E):
                if e != 5:
                    W[e] = float("nan")
    got = M.moe_layer_fwd_few(x, Wg, W1, W2, W3, 1, act, b)
    torch.cuda.synchronize()
    compare(got, fw, bound, dt)


def test_equal_logits_go_to_the_lower_experts():
    T, d, f, E, k = 20, 64, 64, 70, 3
    x, Wg, W1, W2, W3, _ = inputs(T, d, f, E, "gelu", "bf16", seed=9)
    Wg[:] = 0
    fw, bound = reference((x, Wg, W1, W2, None, None), k, "gelu", 1, "bf16")
    g = upload((x, Wg, W1, W2, None, None), "bf16")
    banner("few ties")
    got = M.moe_layer_fwd_few(g[0], g[1], g[2], g[3], None, k)
    torch.cuda.synchronize()
    assert_equal_i(got[2], np.tile(np.arange(k, dtype=np.int32), (T, 1)), "ties")
    compare(got, fw, bound, "bf16")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_token_that_is_not_finite_stays_alone(bad, dt):
    """One token holds NaN or infinity: the others keep their bits, whatever
    experts the bad one is sent to."""
    T, d, f, E, k = 19, 128, 256, 4, 2
    banner("few not finite", bad, dt)
    a = inputs(T, d, f, E, "swiglu", dt, seed=21)
    x, Wg, W1, W2, W3, _ = upload(a, dt)
    good = [v.clone() for v in M.moe_layer_fwd_few(x, Wg, W1, W2, W3, k, "swiglu")]
    x[6, 17] = bad
    got = M.moe_layer_fwd_few(x, Wg, W1, W2, W3, k, "swiglu")
    torch.cuda.synchronize()
    keep = [t for t in range(T) if t != 6]
    for g, v in zip(good, got):
        assert torch.equal(g[keep], v[keep])
    assert not torch.isfinite(got[0][6].float()).all()
    idx = got[2][6].tolist()
    assert len(set(idx)) == k and all(0 <= e < E for e in idx)


def test_layer_steps_of_changing_size_on_a_stream_match_the_function():
    """FewTokenMoELayer over steps of 1 to T tokens on a stream of its own:
    the function's bits, and rows behind the step's last token left alone."""
    d, f, E, k = 192, 320, 10, 2
    banner("few layer steps")
    a = inputs(40, d, f, E, "swiglu", "bf16", seed=33)
    x, Wg, W1, W2, W3, _ = upload(a, "bf16")
    layer = M.FewTokenMoELayer(40, d, f, E, k, "swiglu").bind(Wg, W1, W2, W3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for n in (40, 1, 17, 0, 33, 2, 40):
            layer._y.fill_(7)
            y = layer.forward(x[:n])
            want = M.moe_layer_fwd_few(x[:n].contiguous(), Wg, W1, W2, W3, k, "swiglu")
            side.synchronize()
            assert y.shape == (n, d) and layer.topk_idx.shape == (n, k)
            for g, v in zip((y, layer.logits, layer.topk_idx, layer.topk_w), want):
                assert torch.equal(g, v), n
            assert bool((layer._y[n:] == 7).all()), n


def test_two_layers_share_weights_on_two_streams():
    """Two steps in flight at once over the same weights, a layer each."""
    d, f, E, k = 256, 512, 8, 2
    banner("few two streams")
    a = inputs(24, d, f, E, "gelu", "bf16", seed=40)
    x, Wg, W1, W2, _, _ = upload(a, "bf16")
    want = [M.moe_layer_fwd_few(v.contiguous(), Wg, W1, W2, None, k)[0].clone()
            for v in (x[:11], x[11:])]
    ls = [M.FewTokenMoELayer(13, d, f, E, k).bind(Wg, W1, W2) for _ in range(2)]
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for l, s, v in zip(ls, ss, (x[:11], x[11:])):
            with torch.cuda.stream(s):
                l.forward(v)
    torch.cuda.synchronize()
    for l, w in zip(ls, want):
        assert torch.equal(l.y, w)


@pytest.mark.parametrize("T,E,k,dt", [(1, 8, 2, "bf16"), (20, 40, 4, "bf16"), (3, 6, 2, "f32")])
def test_graph_replays_follow_their_inputs(T, E, k, dt):
    """A captured step, replayed with other tokens in its input buffer and
    eager work between the replays: each replay has the eager call's bits."""
    d, f = 256, 384
    banner("few graph", T, E, k, dt)
    a = inputs(T, d, f, E, "swiglu", dt, seed=50)
    x, Wg, W1, W2, W3, _ = upload(a, dt)
    layer = M.FewTokenMoELayer(T, d, f, E, k, "swiglu", TDT[dt]).bind(Wg, W1, W2, W3)
    layer.forward(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(x)
    for rep in range(4):
        new = dev(stage.normal(60 + rep, (T, d), 1.0, dt), dt)
        x.copy_(new)
        layer._y.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        want = M.moe_layer_fwd_few(new, Wg, W1, W2, W3, k, "swiglu")
        torch.cuda.synchronize()
        for q, v in zip((layer.y, layer.logits, layer.topk_idx, layer.topk_w), want):
            assert torch.equal(q, v), rep


def test_agrees_with_the_training_layer():
    """The same tokens through MoELayer (grouped GEMMs): the same routing bit
    for bit, outputs within two independent roundings of each."""
    T, d, f, E, k = 50, 256, 512, 16, 2
    banner("few against MoELayer")
    a = inputs(T, d, f, E, "swiglu", "bf16", seed=70)
    x, Wg, W1, W2, W3, _ = upload(a, "bf16")
    big = M.MoELayer(T, d, f, E, k, "swiglu").bind(x, Wg, W1, W2, W3)
    big.forward()
    few = M.FewTokenMoELayer(T, d, f, E, k, "swiglu").bind(Wg, W1, W2, W3)
    few.forward(x)
    torch.cuda.synchronize()
    assert torch.equal(few.logits, big.logits) and torch.equal(few.topk_idx, big.topk_idx)
    assert rel_err(host(few.y), host(big.y)) <= TOL["bf16"]


def test_masked_experts_are_not_chosen():
    """Logit biases of minus infinity and of fp32's lowest value: the masked
    experts (weights NaN) are left out while enough others remain, and with too
    few others they come last, lower index first, with weight 0."""
    T, d, f, E, k = 9, 128, 64, 8, 2
    banner("few masks")
    low = float(np.finfo(np.float32).min)
    bias = np.array([0, -np.inf, 0, low, -np.inf, 0, low, -np.inf], np.float32)
    a = inputs(T, d, f, E, "gelu", "bf16", seed=80, bias=bias)
    fw, bound = reference(a, k, "gelu", 1, "bf16")
    x, Wg, W1, W2, _, b = upload(a, "bf16")
    for e in np.flatnonzero(bias < 0):
        W1[e] = float("nan")
    got = M.moe_layer_fwd_few(x, Wg, W1, W2, None, k, "gelu", b)
    torch.cuda.synchronize()
    compare(got, fw, bound, "bf16")
    W1 = dev(a[2], "bf16")
    got = M.moe_layer_fwd_few(x, Wg, W1, W2, None, 6, "gelu", b)
    torch.cuda.synchronize()
    idx, w = got[2].cpu().numpy(), got[3].cpu().numpy()
    assert all(set(r[:3]) == {0, 2, 5} and list(r[5:]) == [1] for r in idx)
    assert (w[:, 3:] == 0).all() and np.allclose(w.sum(1), 1, atol=1e-6)
    assert bool(torch.isfinite(got[0].float()).all())


def test_optional_outputs_may_be_left_out():
    """The C entry point without logits, topk_idx and topk_w: the same y, fused
    with the gate (one token) and not (20 tokens)."""
    from mixture_experts_layer_permute_amd import _lib
    L = _lib.load()
    d, f, E, k = 128, 192, 8, 2
    for T in (1, 20):
        banner("few optional outputs", T)
        x, Wg, W1, W2, W3, _ = upload(inputs(T, d, f, E, "swiglu", "bf16", seed=90), "bf16")
        want = M.moe_layer_fwd_few(x, Wg, W1, W2, W3, k, "swiglu")[0]
        y = torch.empty_like(want)
        nb = L.moe_layer_few_workspace_bytes(T, d, f, E, k, 1, 1)
        ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
        p = lambda t: t.data_ptr()
        assert L.moe_layer_fwd_few(p(x), p(Wg), None, p(W1), p(W3), p(W2), T, d, f, E, k, 1, 1, 1,
                                   None, None, None, p(y), p(ws), nb,
                                   torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_an_expert_past_the_32_bit_offsets(dt):
    """Weight tensors over 2^32 bytes, the last expert chosen by its bias; the
    others' weights are whatever the memory holds."""
    T, d, f, E = 3, 1024, 65536, 36 if dt == "bf16" else 18
    banner("few large", dt)
    assert E * d * f * (2 if dt == "bf16" else 4) > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=TDT[dt])
    x, Wg = r(T, d), r(d, E) * d ** -0.5
    W1 = torch.empty(E, d, f, dtype=TDT[dt], device="cuda")
    W2 = torch.empty(E, f, d, dtype=TDT[dt], device="cuda")
    W1[-1] = r(d, f) * d ** -0.5
    W2[-1] = r(f, d) * f ** -0.5
    bias = torch.zeros(E, device="cuda")
    bias[-1] = 1000
    y, _, idx, _ = M.moe_layer_fwd_few(x, Wg, W1, W2, None, 1, "gelu", bias)
    torch.cuda.synchronize()
    assert bool((idx == E - 1).all())
    h = x.double() @ W1[-1].double()
    want = (h * torch.special.ndtr(h)) @ W2[-1].double()
    assert rel_err(host(y), want.cpu().numpy()) <= TOL[dt]


def test_refusals_of_the_layer():
    layer = M.FewTokenMoELayer(4, 64, 128, 4, 2, "swiglu")
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")
    ok = (z(64, 4), z(4, 64, 128), z(4, 128, 64), z(4, 64, 128))
    for bad in ((z(64, 5),) + ok[1:], (ok[0], z(4, 64, 64)) + ok[2:], ok[:3],
                ok[:2] + (z(4, 64, 128),) + ok[3:], (ok[0].float(),) + ok[1:],
                (ok[0].cpu(),) + ok[1:], ok + (z(4, dt=torch.bfloat16),)):
        with pytest.raises(M.MoEError):
            layer.bind(*bad)
    layer.bind(*ok)
    for x in (z(5, 64), z(2, 128), z(64), z(2, 64, dt=torch.float32), z(64, 2).t(),
              torch.zeros(2, 64, dtype=torch.bfloat16)):
        with pytest.raises(M.MoEError):
            layer.forward(x)
    for bad in (dict(T=65), dict(T=0), dict(k=65, E=80), dict(d=96), dict(f=100), dict(k=5)):
        a = dict(dict(T=4, d=64, f=128, E=4, k=2), **bad)
        with pytest.raises(M.MoEError):
            M.FewTokenMoELayer(**a)


def test_workspace_of_another_type_or_device():
    x, Wg, W1, W2, _, _ = upload(inputs(2, 64, 64, 4, "gelu", "bf16", seed=95), "bf16")
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 20, device="cuda"),
               torch.empty(16, dtype=torch.uint8, device="cuda")):
        with pytest.raises(M.MoEError):
            M.moe_layer_fwd_few(x, Wg, W1, W2, None, 2, "gelu", ws=ws)


@pytest.mark.parametrize("T", [17, 33, 48, 49, 64])
@pytest.mark.parametrize("act,dt", [("gelu", "bf16"), ("swiglu", "bf16"), ("swiglu", "f32")])
def test_tall_tiles_of_wide_strips(T, act, dt):
    """Two to four tiles of rows for each of 8 experts, in sizes that give the
    widest strips, the last one half full: against the products in 64 bits on
    the device, within the bound above."""
    banner("few tall", T, act, dt)
    d, f, E = 1216, 2496, 8
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-2] ** -0.5).to(TDT[dt])
    x, Wg, W1, W2 = r(T, d) * T ** 0.5, r(d, E), r(E, d, f), r(E, f, d)
    W3 = r(E, d, f) if act == "swiglu" else None
    y, logits, idx, _ = M.moe_layer_fwd_few(x, Wg, W1, W2, W3, E, act)
    assert torch.equal(logits, M.moe_gate_topk(x, Wg, E)[0])
    assert bool((idx.sort(1).values == torch.arange(E, device="cuda")).all())
    w, x64 = logits.double().softmax(1), x.double()
    want, bound = torch.zeros_like(x64), torch.zeros_like(x64)
    for e in range(E):
        W1e, W2e = W1[e].double(), W2[e].double()
        H, dH = x64 @ W1e, (d + 2) * U * (x64.abs() @ W1e.abs())
        if act == "swiglu":
            W3e = W3[e].double()
            H3, dH3 = x64 @ W3e, (d + 2) * U * (x64.abs() @ W3e.abs())
            s = H * torch.sigmoid(H)
            A, dA = s * H3, 1.1 * dH * (H3.abs() + dH3) + s.abs() * dH3
        else:
            A, dA = H * torch.special.ndtr(H), 1.13 * dH
        dA = dA + 8 * U * A.abs()
        dA = dA + (2.0 ** -16 if dt == "bf16" else 0.0) * (A.abs() + dA)
        want += w[:, e:e + 1] * (A @ W2e)
        bound += w[:, e:e + 1] * ((dA + (f + 128) * U * A.abs()) @ W2e.abs())
    bound = (bound + HALF[dt] * want.abs()) * 1.001 + 1e-30
    err = (y.double() - want).abs()
    assert bool((err <= bound).all()), "off by %.2f of its bound" % float((err / bound).max())
    assert rel_err(host(y), want.cpu().numpy()) <= TOL[dt]


def device_reference(x, W1, W2, W3, logits, idx, renorm, dt):
    """y in 64 bits on the device from the choice idx, and the bound at the top."""
    T, d = x.shape
    f = W1.shape[2]
    z = logits.double()
    p = (z.gather(1, idx.long()) - (z.gather(1, idx.long()) if renorm else z)
         .logsumexp(1, keepdim=True)).exp()
    want = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    for e in sorted(set(idx.flatten().tolist())):
        t, j = (idx == e).nonzero(as_tuple=True)
        w, xe = p[t, j].unsqueeze(1), x[t].double()
        W1e, W2e = W1[e].double(), W2[e].double()
        H, dH = xe @ W1e, (d + 2) * U * (xe.abs() @ W1e.abs())
        if W3 is not None:
            W3e = W3[e].double()
            H3, dH3 = xe @ W3e, (d + 2) * U * (xe.abs() @ W3e.abs())
            sl = H * torch.sigmoid(H)
            A, dA = sl * H3, 1.1 * dH * (H3.abs() + dH3) + sl.abs() * dH3
        else:
            A, dA = H * torch.special.ndtr(H), 1.13 * dH
        dA = dA + 8 * U * A.abs()
        dA = dA + (2.0 ** -16 if dt == "bf16" else 0.0) * (A.abs() + dA)
        want.index_add_(0, t, w * (A @ W2e))
        bound.index_add_(0, t, w * ((dA + (f + 128) * U * A.abs()) @ W2e.abs()))
    return want, (bound + HALF[dt] * want.abs()) * 1.001 + 1e-30


@pytest.mark.parametrize("width,T", [(w, T) for w, most in (
    ("wide", 64), ("8 waves", 64), ("quarter", 16), ("with the gate", 4))
    for T in (1, 2, 5, 16, 17, 32, 33, 64) if T <= most])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_every_strip_width(width, T, act, dt):
    """Sizes that give the up product each width it has, for one, two and four
    tiles of rows: strips of 16 wide columns with 4 waves (bf16 128 columns,
    fp32 64), 64 columns with 8 waves, 32 columns (up to 16 tokens), 64 columns
    behind the gate in one launch (up to 4 tokens); the down product in both
    widths.  Strips end inside the matrix, skewed routing leaves experts with
    all tokens and with one."""
    d, f, E, k = {"wide": (704, 2496, 24, 8), "8 waves": (320, 576, 24, 8),
                  "quarter": (448, 128, 24, 8), "with the gate": (320, 320, 13, 3)}[width]
    if width == "8 waves" and T < 5 and dt == "f32":
        f = 960
    banner("few widths", T, width, act, dt, d, f, E, k)
    g = torch.Generator(device="cuda").manual_seed(1000 * T + f)
    r = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-2] ** -0.5).to(TDT[dt])
    x, Wg, W1, W2 = r(T, d) * T ** 0.5, r(d, E), r(E, d, f), r(E, f, d)
    W3 = r(E, d, f) if act == "swiglu" else None
    bias = -1.5 * torch.log(torch.randperm(E, generator=g, device="cuda").float() + 1)
    for renorm in (1, 0):
        y, logits, idx, w = M.moe_layer_fwd_few(x, Wg, W1, W2, W3, k, act, bias, renorm)
        gate = M.moe_gate_topk(x, Wg, k, bias, renorm)
        assert torch.equal(logits, gate[0]) and torch.equal(idx, gate[1])
        want, bound = device_reference(x, W1, W2, W3, logits, idx, renorm, dt)
        err = (y.double() - want).abs()
        assert bool((err <= bound).all()), "off by %.2f of its bound" % float((err / bound).max())
        assert rel_err(host(y), want.cpu().numpy()) <= TOL[dt]

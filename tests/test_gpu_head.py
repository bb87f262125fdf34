"""The vocabulary head's losses (moe_head_xent, moe_head_distill and their
gradients) against the formulas in 64 bits, within derived bounds."""
import math

import pytest
import torch

import mixture_experts_layer_permute_amd as M

from _gpu import banner, needs_gpu
from _head import check, inputs, reference

pytestmark = [pytest.mark.gpu, needs_gpu]


def run(x, Wv, labels, weight=None, teacher=None, tau=1.0, grad=True, **kw):
    if teacher is not None and grad:
        return M.moe_head_distill_grad(x, Wv, teacher, tau, labels, weight, **kw)
    if teacher is not None:
        return M.moe_head_distill(x, Wv, teacher[:2], tau, labels, **kw)
    if grad:
        return M.moe_head_xent_grad(x, Wv, labels, weight, **kw)
    return M.moe_head_xent(x, Wv, labels, **kw)


def least_ws(x, V, K, grad):
    L = M.load()
    dt = 1 if x.dtype == torch.bfloat16 else 0
    return L.moe_head_workspace_bytes(x.shape[0], x.shape[1], V, K, dt, int(grad), 1)


# T, d, V: single tokens, odd sizes, tile edges, one entry, wide, many tokens on a
# small vocabulary (the products split over the tokens) and the other way round
SIZES = [(1, 64, 1000), (3, 64, 1), (5, 128, 2), (16, 256, 63), (33, 64, 65), (64, 192, 257),
         (65, 64, 511), (200, 320, 1003), (255, 64, 256), (256, 128, 129), (257, 64, 255),
         (300, 1088, 4099), (700, 128, 513), (2500, 64, 200), (7, 64, 20011), (40, 2048, 9001)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V", SIZES)
def test_xent(T, d, V, dt):
    banner("head xent", T, d, V, dt)
    x, Wv, labels, weight, _ = inputs(T, d, V, dt, masked=0.2, seed=T + V)
    ref = reference(x, Wv, labels, weight, dt=dt)
    check(run(x, Wv, labels, grad=False), ref, "forward")
    check(run(x, Wv, labels, weight), ref, "gradient")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V,K,tau,labels", [
    (1, 64, 1000, 1, 1.0, False), (3, 64, 1, 2, 2.0, True), (33, 320, 5003, 8, 4.0, False),
    (64, 64, 257, 64, 0.7, True), (257, 128, 1003, 63, 2.0, True), (300, 64, 129, 256, 5.0, True),
    (520, 192, 2051, 65, 1.0, False), (9, 1024, 30011, 128, 3.0, True)])
def test_distill(T, d, V, K, tau, labels, dt):
    banner("head distill", T, d, V, K, tau, labels, dt)
    x, Wv, lab, weight, teacher = inputs(T, d, V, dt, masked=0.3, K=K, seed=T + K)
    if not labels:
        lab = weight = None
    ref = reference(x, Wv, lab, weight, teacher, tau, dt)
    check(run(x, Wv, lab, None, teacher, tau, grad=False), ref, "forward")
    check(run(x, Wv, lab, weight, teacher, tau), ref, "gradient")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V,K", [(1000, 64, 700, 0), (513, 128, 300, 5), (2304, 64, 129, 0)])
def test_pieces(T, d, V, K, dt):
    """A small workspace: many pieces of tokens, dWv summed over them; half the
    tokens have no loss, so that the last pieces are empty."""
    banner("head pieces", T, d, V, K, dt)
    x, Wv, labels, weight, teacher = inputs(T, d, V, dt, masked=0.5, K=K, seed=5)
    ref = reference(x, Wv, labels, weight, teacher, 2.0, dt)
    L = M.load()
    for limit in (1, 1 << 20, 1 << 21, 1 << 22):
        res = run(x, Wv, labels, weight, teacher, 2.0, limit=limit)
        check(res, ref, "limit %d" % limit)
    # the smallest workspace there is, its size as queried
    ws = torch.empty(least_ws(x, V, K, True), dtype=torch.uint8, device="cuda")
    check(run(x, Wv, labels, weight, teacher, 2.0, ws=ws), ref, "smallest")
    check(run(x, Wv, labels, None, teacher, 2.0, grad=False, limit=1), ref, "forward")


def test_unsplit_products():
    """Enough tiles for every product in one part, against the formulas on the
    device."""
    T, d, V = 4096, 4096, 1111
    banner("head unsplit", T, d, V)
    x, Wv, labels, weight, _ = inputs(T, d, V, "bf16", masked=0.1, seed=3)
    check(run(x, Wv, labels, weight), reference(x, Wv, labels, weight))


def test_labels_and_tokens_left_out():
    """Labels outside [0,V) have no loss, their rows of x are not read (they hold
    NaN), dx is 0 there; a batch without any loss gives zero gradients."""
    T, d, V = 300, 128, 777
    banner("head masked")
    x, Wv, labels, weight, _ = inputs(T, d, V, seed=9)
    labels[::3] = -1
    labels[1::7] = V
    labels[2::11] = 2 ** 31 - 1
    labels[5::13] = -2 ** 31
    off = (labels < 0) | (labels >= V)
    clean = reference(x, Wv, labels, weight)
    x[off] = float("nan")
    res = run(x, Wv, labels, weight)
    check(res, clean)
    assert bool((res["dx"][off] == 0).all()) and bool((res["loss"][off] == 0).all())
    labels[:] = -100
    res = run(x, Wv, labels, weight)
    for t in res.values():
        assert bool((t == 0).all())
    res = run(x, Wv, labels, weight, limit=1)
    for t in res.values():
        assert bool((t == 0).all())
    assert bool((run(x, Wv, labels, grad=False)["loss"] == 0).all())


def test_teacher_slots_left_out():
    """Slots outside [0,V), scores of -infinity, tokens with no slot at all, the
    same entry in every slot, the label among the slots or not."""
    T, d, V, K = 64, 64, 300, 16
    banner("head teacher slots")
    x, Wv, labels, weight, (idx, score, tw) = inputs(T, d, V, K=K, seed=4)
    idx[0] = -1                                    # label only
    idx[1] = 7                                     # one entry, 16 times
    idx[2, 1:] = V                                 # one slot
    score[3, 2:] = -math.inf
    score[4] = -math.inf                           # no probability anywhere
    idx[5] = labels[5]
    idx[6] = (labels[6] + 1) % V
    idx[7] = -1
    labels[7] = -1                                 # nothing at all
    labels[8] = -1                                 # teacher only
    score[9, idx[9] < 0] = float("nan")            # never looked at
    idx[10, :8] = idx[10, 8:]
    idx[11, 3] = -1
    score[11, 3] = float("nan")
    x[7] = float("nan")
    for lab, w in ((labels, weight), (None, None)):
        ref = reference(x, Wv, lab, w, (idx, torch.nan_to_num(score, neginf=-math.inf), tw), 1.5)
        if lab is None:                            # token 7 has no loss without a label either
            assert float(ref["kd"][0][7]) == 0.0
        res = run(x, Wv, lab, w, (idx, score, tw), 1.5)
        check(res, ref)
        assert float(res["kd"][0]) == 0.0 and float(res["kd"][4]) == 0.0
        assert bool((res["dx"][7] == 0).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_scores(dt):
    """Scores far apart (no overflow, probabilities that vanish) and equal ones."""
    T, d, V = 70, 64, 900
    banner("head large scores", dt)
    x, Wv, labels, weight, teacher = inputs(T, d, V, dt, K=9, seed=2, scale=60.0)
    x[3] = 0                                       # every score 0
    ref = reference(x, Wv, labels, weight, teacher, 0.5, dt)
    assert float(ref["lse"][0].max()) > 100.0
    assert abs(float(ref["lse"][0][3]) - math.log(V)) < 1e-9
    check(run(x, Wv, labels, weight, teacher, 0.5), ref)


def test_one_gradient_only_and_default_weights():
    T, d, V, K = 130, 128, 600, 6
    banner("head one gradient")
    x, Wv, labels, weight, teacher = inputs(T, d, V, K=K, seed=8)
    both = run(x, Wv, labels)
    check(both, reference(x, Wv, labels))
    for name in ("dx", "dWv"):
        res = run(x, Wv, labels, out={name: None})
        assert res[name] is None
        other = "dWv" if name == "dx" else "dx"
        assert torch.equal(res[other], both[other])
    t2 = teacher[:2]
    check(run(x, Wv, labels, weight, t2, 2.0), reference(x, Wv, labels, weight, t2, 2.0))


def test_same_bits_every_time_and_out_of_place():
    T, d, V, K = 515, 256, 1777, 12
    banner("head determinism")
    x, Wv, labels, weight, teacher = inputs(T, d, V, masked=0.1, K=K, seed=6)
    keep = [t.clone() for t in (x, Wv, labels, weight, *teacher)]
    a = run(x, Wv, labels, weight, teacher, 2.0)
    b = run(x, Wv, labels, weight, teacher, 2.0)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    for t, k in zip((x, Wv, labels, weight, *teacher), keep):
        assert torch.equal(t, k)


def test_gradient_by_differences():
    """dx and dWv along random directions against central differences of the loss
    itself in fp32 (a step of 2^-6 of a unit direction: the loss is smooth there;
    both the fp32 loss's rounding and the third-order term stay under the bound)."""
    T, d, V, K, tau = 40, 64, 150, 7, 2.0
    banner("head differences")
    x, Wv, labels, weight, teacher = inputs(T, d, V, "f32", K=K, seed=12)
    res = run(x, Wv, labels, weight, teacher, tau)

    def total(x_, W_):
        r = run(x_, W_, labels, None, teacher, tau, grad=False)
        return float((r["loss"].double() * weight.double()).sum()
                     + (r["kd"].double() * teacher[2].double()).sum())
    g = torch.Generator().manual_seed(1)
    h = 2.0 ** -6
    for t, grad, at in ((x, res["dx"], 0), (Wv, res["dWv"], 1)):
        for _ in range(3):
            v = torch.randn(t.shape, generator=g).cuda()
            v /= v.norm()
            pair = [total(*((t + s * h * v, Wv) if at == 0 else (x, t + s * h * v)))
                    for s in (1, -1)]
            got = float((grad.double() * v.double()).sum())
            # 2 T losses of about 20, each within 2^-20 of its size, over 2 h; the
            # third derivative along a unit direction is below sum |w| |x|^3 h^2 / 6 for
            # directions spread over all tokens, here under 2^-7 in all
            tol = 2 * T * 20 * 2.0 ** -20 / (2 * h) + 2.0 ** -7
            assert abs((pair[0] - pair[1]) / (2 * h) - got) <= tol


def test_headloss_class():
    """The preallocated form: fewer tokens than it was made for, with and without a
    teacher, other gradient buffers, the views it returns."""
    T, d, V, K = 400, 128, 1200, 8
    banner("HeadLoss")
    x, Wv, labels, weight, teacher = inputs(T, d, V, masked=0.2, K=K, seed=21)
    head = M.HeadLoss(T, d, V, K=K, tau=2.0)
    dy = torch.full((T, d), 3.0, dtype=torch.bfloat16, device="cuda")
    head.bind(Wv, dx=dy)
    for n in (T, 1, 130):
        t = tuple(v[:n].contiguous() for v in teacher)
        loss = head.step(x[:n], labels[:n], weight[:n], t)
        ref = reference(x[:n], Wv, labels[:n], weight[:n], t, 2.0)
        check({"loss": loss, "lse": head.lse, "kd": head.kd, "dx": head.dx, "dWv": head.dWv}, ref)
        assert head.dx.data_ptr() == dy.data_ptr()
        head.step(x[:n], labels[:n], weight[:n])
        check({"loss": head.loss, "dx": head.dx, "dWv": head.dWv},
              reference(x[:n], Wv, labels[:n], weight[:n]))
        kd = head.forward(x[:n], None, t)
        check({"kd": kd}, ref)
        check({"loss": head.forward(x[:n], labels[:n])}, ref)
    assert head.weight_grads()[0] is head.dWv


def test_headloss_on_another_stream_and_in_a_graph():
    T, d, V, K = 300, 128, 900, 5
    banner("HeadLoss stream and graph")
    x, Wv, labels, weight, teacher = inputs(T, d, V, masked=0.1, K=K, seed=31)
    head = M.HeadLoss(T, d, V, K=K, tau=1.5, limit=1).bind(Wv)
    head.step(x, labels, weight, teacher)
    torch.cuda.synchronize()
    names = ("loss", "lse", "kd", "dx", "dWv")
    want = {n: getattr(head, n).clone() for n in names}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for n in names:
        getattr(head, n).zero_()
    torch.cuda.synchronize()
    head.step(x, labels, weight, teacher, stream=s.cuda_stream)
    s.synchronize()
    for n in names:
        assert torch.equal(getattr(head, n), want[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        head.step(x, labels, weight, teacher)
    x0 = x.clone()
    for i in range(3):
        x.copy_(x0 * (1.0 + 0.125 * i))
        for n in names:
            getattr(head, n).fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: getattr(head, n).clone() for n in names}
        eager = run(x, Wv, labels, weight, teacher, 1.5, limit=1)
        for n in names:
            assert torch.equal(got[n], eager[n]), (i, n)


def test_a_training_step():
    """Layer forward, the head's loss and gradient straight into the layer's dy,
    layer backward, the global norm over both, clipping."""
    T, d, f, E, k, V = 512, 128, 256, 4, 2, 1000
    banner("head training step")
    g = torch.Generator().manual_seed(3)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()
    x, Wg = n(T, d), n(d, E, std=d ** -0.5)
    W1, W2 = n(E, d, f, std=d ** -0.5), n(E, f, d, std=f ** -0.5)
    Wv = n(V, d, std=0.5)
    labels = torch.randint(0, V, (T,), generator=g).to(torch.int32).cuda()
    labels[::5] = -1
    weight = torch.full((T,), 1.0 / T, device="cuda")
    layer = M.MoELayer(T, d, f, E, k)
    dy = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    layer.bind(x, Wg, W1, W2, dy=dy)
    head = M.HeadLoss(T, d, V).bind(Wv, dx=dy)
    clip = M.GradClip(layer.weight_grads() + head.weight_grads())
    layer.forward()
    loss = head.step(layer.y, labels, weight)
    layer.backward()
    torch.cuda.synchronize()
    ref = reference(layer.y, Wv, labels, weight)
    check({"loss": loss, "dx": dy, "dWv": head.dWv}, ref)
    other = M.MoELayer(T, d, f, E, k).bind(x, Wg, W1, W2, dy=dy.clone())
    other.step()
    for a, b in zip(layer.weight_grads(), other.weight_grads()):
        assert torch.equal(a, b)
    sq = sum(float((t.double() ** 2).sum()) for t in layer.weight_grads() + head.weight_grads())
    before = [t.clone() for t in head.weight_grads()]
    norm = clip.clip(0.5 * math.sqrt(sq))
    assert abs(float(norm) - math.sqrt(sq)) <= 1e-6 * math.sqrt(sq)
    # scaled by half: exact up to the factor's rounding, then one of bf16
    assert torch.allclose(head.dWv.double(), before[0].double() * 0.5, rtol=2.0 ** -8, atol=1e-30)


@pytest.mark.parametrize("K", [0, 7])
@pytest.mark.parametrize("T,n", [(128, 128), (129, 129), (200, 100), (200, 128), (1000, 1), (128, 65)])
def test_few_tokens_in_a_larger_workspace(T, n, K):
    """dz in two terms (up to 128 tokens) and in one, in the workspace of more."""
    d, V = 192, 2003
    banner("head few tokens", T, n, K)
    head = M.HeadLoss(T, d, V, torch.bfloat16, K=K, tau=2.0, device="cuda")
    x, Wv, labels, weight, teacher = inputs(n, d, V, masked=0.2, K=K, seed=T + n)
    head.bind(Wv)
    head.step(x, labels, weight, teacher)
    got = {k: getattr(head, k) for k in ("loss", "lse", "dx", "dWv") + (("kd",) if K else ())}
    check(got, reference(x, Wv, labels, weight, teacher, 2.0), "%d of %d" % (n, T))


@pytest.mark.parametrize("T", [1, 19, 300])
def test_rounding_of_the_gradients(T):
    """dx is as near to 64 bits as its own rounding: half a step, and of the entries
    beside the label's, sqrt(V) e(dz) at most, a tenth of that here (the label takes
    more than nine tenths of the squares of its row).  dWv likewise up to 128 tokens."""
    d, V = 256, 5000
    banner("head rounding", T)
    x, Wv, labels, weight, _ = inputs(T, d, V, seed=T)
    ref = reference(x, Wv, labels, weight)
    got = run(x, Wv, labels, weight)
    for name in ("dx", "dWv") if T <= 128 else ("dx",):
        val = ref[name][0]
        own = (val.to(torch.bfloat16).double() - val).norm()
        err = (got[name].double() - val).norm()
        assert err <= 1.1 * own, (name, float(err / own))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("K", [0, 3])
def test_no_tokens(K, dt):
    """T = 0: dWv is zeros, and nothing else happens."""
    d, V = 128, 77
    banner("head no tokens", K, dt)
    x, Wv, labels, weight, teacher = inputs(0, d, V, dt, K=K)
    res = run(x, Wv, labels, weight, teacher, 2.0, out={"dWv": torch.full_like(Wv, 3.0)})
    assert not bool(res["dWv"].any()) and res["dx"].shape == (0, d)
    res = run(x, Wv, labels, None, teacher, 2.0, grad=False)
    assert res["loss"].shape == (0,)


@pytest.mark.parametrize("tau", [0.05, 50.0])
def test_sharp_and_flat_temperatures(tau):
    T, d, V, K = 70, 64, 999, 9
    banner("head tau", tau)
    x, Wv, labels, weight, teacher = inputs(T, d, V, "f32", K=K, seed=3)
    ref = reference(x, Wv, labels, weight, teacher, tau, "f32")
    check(run(x, Wv, labels, weight, teacher, tau), ref, "tau %g" % tau)


def test_two_losses_at_once_on_two_streams():
    """Two calls in flight, each with a workspace of its own."""
    T, d, V = 600, 256, 4001
    banner("head two streams")
    heads, wants, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        x, Wv, labels, weight, _ = inputs(T, d, V, masked=0.1, seed=i)
        wants.append({k: v.clone() for k, v in run(x, Wv, labels, weight).items()})
        h = M.HeadLoss(T, d, V, torch.bfloat16, device="cuda")
        h.bind(Wv)
        heads.append((h, x, labels, weight))
    torch.cuda.synchronize()
    for _ in range(8):
        for (h, x, labels, weight), s in zip(heads, streams):
            with torch.cuda.stream(s):
                h.step(x, labels, weight)
    torch.cuda.synchronize()
    for (h, *_), want in zip(heads, wants):
        for k in ("loss", "lse", "dx", "dWv"):
            assert torch.equal(getattr(h, k), want[k]), k


def test_gradient_past_32_bit_offsets():
    """dz of one piece is more than 4 GB: the last rows' and entries' offsets pass 32
    bits.  The tokens repeat (weights included), so that every copy of a token has the
    first one's dx bit for bit, and dWv of a vocabulary entry at the end is checked
    against the formula."""
    T, d, V, base = 20480, 64, 131008, 256
    banner("head offsets", T, d, V)
    x, Wv, labels, weight, _ = inputs(base, d, V, seed=1)
    labels[-1] = V - 1
    got = run(x.repeat(T // base, 1), Wv, labels.repeat(T // base), weight.repeat(T // base))
    one = got["dx"][:base]
    assert torch.equal(got["dx"].view(T // base, base, d), one.expand(T // base, base, d))
    assert torch.equal(got["loss"].view(-1, base), got["loss"][:base].expand(T // base, base))
    ref = reference(x, Wv, labels, weight)
    check({k: got[k][:base] for k in ("loss", "lse", "dx")}, ref, "first copy")
    val, tol = (t[-64:] * (T // base) for t in ref["dWv"])
    assert bool(((got["dWv"][-64:].double() - val).abs() <= 1.05 * tol + T * 2.0 ** -23 * val.abs()
                 .max()).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V,K", [(12, 3712, 587, 0), (1, 4096, 1, 0), (270, 1600, 1003, 5),
                                     (130, 1536, 128, 0), (30, 2112, 668, 67), (9, 768, 3000, 2)])
def test_split_scores(T, d, V, K, dt):
    """Few tiles with a long reduction: the scores' product in parts."""
    banner("head split scores", T, d, V, K, dt)
    x, Wv, labels, weight, teacher = inputs(T, d, V, dt, masked=0.2, K=K, seed=T)
    ref = reference(x, Wv, labels, weight, teacher, 2.0, dt)
    check(run(x, Wv, labels, None, teacher, 2.0, grad=False), ref, "forward")
    check(run(x, Wv, labels, weight, teacher, 2.0), ref, "gradient")

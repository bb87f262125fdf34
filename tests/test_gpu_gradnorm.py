"""moe_grad_norm, moe_clip_grads, GradClip and the layers' clip_grads against
64-bit NumPy.

Bounds, u = 2^-24: the sum of n squares in fp64 is off by at most n 2^-53 of
itself, its root and the rounding to fp32 add u, so |norm - exact| <=
(u + n 2^-53) exact.  A clipped element is g * c with c = max_norm / norm
(norm's u, the division's u), the product rounded in fp32 (u) and, in bf16,
once more (2^-8): relative 3.001 u, plus 2^-8 for bf16, and half a step of the
type's subnormals (2^-150 for fp32, 2^-134 for bf16).
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_permute_amd as M
import oracle
from moe_inputs import device, rng, small_variant, stage

from _gpu import TOL, assert_equal_i, banner, host, needs_gpu, rel_err

pytestmark = [pytest.mark.gpu, needs_gpu]

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def tensors(spec, seed=0, std=1.0):
    """[(dtype, shape)] -> tensors of normal values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").mul_(std).to(t) for t, s in spec]


def exact_norm(ts):
    return float(np.sqrt(sum(np.sum(host64(t) ** 2) for t in ts)))


def host64(t):
    return t.detach().cpu().float().numpy().astype(np.float64)


def check_norm(got, ts):
    want = exact_norm(ts)
    n = sum(t.numel() for t in ts)
    assert got.shape == (1,) and got.dtype == F32
    assert abs(float(got[0]) - want) <= (U + n * 2.0 ** -53) * want, (float(got[0]), want)
    return want


def check_clipped(outs, ts, norm, mx):
    c = mx / norm if norm > mx else 1.0
    for o, t in zip(outs, ts):
        w = host64(t) * c
        rel, sub = (3.001 * U + 2.0 ** -8, 2.0 ** -134) if t.dtype == BF else \
            (3.001 * U, 2.0 ** -150)
        assert np.all(np.abs(host64(o) - w) <= rel * np.abs(w) + sub)


LISTS = {
    "one element": [(F32, (1,))],
    "one bf16": [(BF, (1,))],
    "odd": [(BF, (7,)), (F32, (13, 3)), (BF, (1, 1)), (F32, (0,)), (BF, (2049, 17)), (BF, (0, 4))],
    "chunk edges": [(BF, (32768,)), (BF, (32769,)), (BF, (32767,)), (F32, (16384,)),
                    (F32, (16385,)), (F32, (16383,)), (BF, (8192,)), (BF, (8193,)),
                    (F32, (4096,)), (F32, (4097,))],
    "128 tensors": [(F32, (i + 1,)) for i in range(128)],
    "129 tensors": [(BF, (i + 1,)) for i in range(129)],
    "400 tensors": [((BF, F32)[i % 2], (131 * (i % 7), 3)) for i in range(400)],
    "a layer": [(F32, (1024, 8)), (BF, (8, 1024, 520)), (BF, (8, 520, 1024))],
    "more chunks than blocks": [(BF, (70_000_001,)), (F32, (5,))],
}


@pytest.mark.parametrize("name", LISTS)
def test_norm_and_clip(name):
    banner("gradnorm", name)
    ts = tensors(LISTS[name], seed=len(name))
    check_norm(M.moe_grad_norm(ts), ts)
    keep = [t.clone() for t in ts]
    out = [torch.full_like(t, 7) for t in ts]
    want = exact_norm(ts)
    for mx in (want / 3, want * 3):
        n = M.moe_clip_grads(ts, mx, out)
        torch.cuda.synchronize()
        check_norm(n, ts)
        check_clipped(out, keep, want, np.float64(np.float32(mx)))
        for t, k in zip(ts, keep):
            assert torch.equal(t, k)                       # the inputs stay
    first = [o.clone() for o in out]
    for o, t in zip(first, ts):                            # under the limit: copies
        assert torch.equal(o, t)
    M.moe_clip_grads(ts, want * 3)                         # in place, under the limit
    torch.cuda.synchronize()
    for t, k in zip(ts, keep):
        assert torch.equal(t, k)
    M.moe_clip_grads(ts, want / 3)                         # in place: the same bits
    M.moe_clip_grads(keep, want / 3, out)
    torch.cuda.synchronize()
    for t, o in zip(ts, out):
        assert torch.equal(t, o)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shift_in,shift_out", [(0, 1), (1, 0), (3, 5), (1, 1)])
def test_views_at_any_alignment(dt, shift_in, shift_out):
    """Views of flat buffers that start at any element; what lies between and
    behind them is left alone."""
    banner("gradnorm views", dt, shift_in, shift_out)
    sizes = [1, 5, 1023, 4096, 40001]
    flat_in = tensors([(dt, (60000,))], seed=4)[0]
    flat_out = torch.full_like(flat_in, 7)
    ts, outs, at = [], [], 0
    used = torch.zeros(60000, dtype=torch.bool)
    for n in sizes:
        ts.append(flat_in[at + shift_in:at + shift_in + n])
        outs.append(flat_out[at + shift_out:at + shift_out + n])
        used[at + shift_out:at + shift_out + n] = True
        at += n + 7
    want = exact_norm(ts)
    n = M.moe_clip_grads(ts, want / 2, outs)
    torch.cuda.synchronize()
    check_norm(n, ts)
    check_clipped(outs, ts, want, np.float64(np.float32(want / 2)))
    assert bool((flat_out.cpu()[~used] == 7).all())


@pytest.mark.parametrize("scale", [1e30, 1e-30, 1e37])
def test_values_whose_squares_leave_fp32(scale):
    banner("gradnorm range", scale)
    ts = [t * scale for t in tensors([(F32, (9, 11)), (BF, (77,))], seed=5)]
    want = check_norm(M.moe_grad_norm(ts), ts)
    out = [torch.empty_like(t) for t in ts]
    M.moe_clip_grads(ts, want / 7, out)
    torch.cuda.synchronize()
    check_clipped(out, ts, want, np.float64(np.float32(want / 7)))


@pytest.mark.parametrize("mx", [3.0, 1e-3, 1e-6, 1e-20])
def test_a_factor_below_the_normal_range_of_fp32(mx):
    """max_norm / norm below 2^-126, where fp32 has few bits or none left while
    the products are ordinary numbers: the same bound as for any factor."""
    banner("gradnorm small factor", mx)
    ts = [t * 1e35 for t in tensors([(F32, (901, 11)), (BF, (30077,)), (F32, (3,))], seed=31)]
    ts[2].copy_(torch.tensor([3e38, -1e37, 1e30]))
    want = exact_norm(ts)
    assert want < 3.4e38 and mx / want < 2.0 ** -126
    out = [torch.full_like(t, 7) for t in ts]
    check_norm(M.moe_clip_grads(ts, mx, out), ts)
    torch.cuda.synchronize()
    assert abs(float(out[2][0]) / mx) > 0.5
    check_clipped(out, ts, want, np.float64(np.float32(mx)))
    M.moe_clip_grads(ts, mx)                                # in place: the same bits
    torch.cuda.synchronize()
    assert all(torch.equal(t, o) for t, o in zip(ts, out))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_scales_nothing(bad):
    banner("gradnorm not finite", bad)
    ts = tensors([(BF, (3000,)), (F32, (70000,))], seed=6)
    ts[1][69999] = bad
    keep = [t.clone() for t in ts]
    bits = lambda t: t.view(torch.int16 if t.dtype == BF else torch.int32)
    out = [torch.zeros_like(t) for t in ts]
    n = M.moe_clip_grads(ts, 0.5, out)
    m = M.moe_clip_grads(ts, 0.5)
    torch.cuda.synchronize()
    for v in (n, m):
        assert bool(torch.isnan(v[0])) if bad != bad else float(v[0]) == float("inf")
    for t, k, o in zip(ts, keep, out):
        assert torch.equal(bits(t), bits(k)) and torch.equal(bits(o), bits(k))
    # a sum beyond fp32's range is no float either
    big = [torch.full((64,), 3e38, device="cuda")]
    assert float(M.moe_clip_grads(big, 1.0)[0]) == float("inf")
    assert bool((big[0] == 3e38).all())


def test_limits_zero_and_infinity_and_empty_lists():
    banner("gradnorm limits")
    ts = tensors([(BF, (500,)), (F32, (300,))], seed=7)
    keep = [t.clone() for t in ts]
    M.moe_clip_grads(ts, float("inf"))
    torch.cuda.synchronize()
    assert all(torch.equal(t, k) for t, k in zip(ts, keep))
    M.moe_clip_grads(ts, 0.0)
    torch.cuda.synchronize()
    assert all(float(t.float().abs().max()) == 0.0 for t in ts)
    assert float(M.moe_clip_grads(ts, 0.0)[0]) == 0.0       # zero gradients stay zero
    assert float(M.moe_grad_norm([])[0]) == 0.0
    assert float(M.moe_clip_grads([], 1.0)[0]) == 0.0
    empty = torch.empty(0, device="cuda")
    assert float(M.moe_clip_grads([empty, empty], 1.0)[0]) == 0.0


def test_repeated_runs_give_the_same_bits():
    banner("gradnorm determinism")
    ts = tensors([(BF, (3, 1_000_003)), (F32, (700_001,))], seed=8)
    a = M.GradClip(ts)
    n0 = a.norm().clone()
    for _ in range(5):
        assert torch.equal(a.norm(), n0)
    assert torch.equal(M.GradClip(ts).clip(1e9), n0)


def test_two_lists_at_once_on_two_streams():
    banner("gradnorm streams")
    lists = [tensors([(BF, (2_000_001,)), (F32, (513,))], seed=9 + i) for i in range(2)]
    outs = [[torch.empty_like(t) for t in ts] for ts in lists]
    cs = [M.GradClip(ts, o) for ts, o in zip(lists, outs)]
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(cs, ss):
            with torch.cuda.stream(s):
                c.clip(1.5)
    torch.cuda.synchronize()
    for c, ts, o in zip(cs, lists, outs):
        check_norm(c.result, ts)
        check_clipped(o, ts, exact_norm(ts), 1.5)


def test_graph_replays_follow_the_gradients():
    """A captured clip of 150 tensors (two launches a pass) replayed on new
    gradients, with eager work between: the eager call's bits."""
    banner("gradnorm graph")
    spec = [((BF, F32)[i % 3 == 0], (97 * i + 1,)) for i in range(150)]
    ts = tensors(spec, seed=11)
    out = [torch.empty_like(t) for t in ts]
    c = M.GradClip(ts, out)
    c.clip(2.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.clip(2.0)
    for rep in range(4):
        for t, n in zip(ts, tensors(spec, seed=20 + rep, std=(rep + 1) * 1e-3)):
            t.copy_(n)
        for o in out:
            o.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        norm = c.result.clone()
        want = [torch.empty_like(t) for t in ts]
        assert torch.equal(M.moe_clip_grads(ts, 2.0, want), norm), rep
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), rep


@pytest.mark.parametrize("kind", ["whole", "chunked"])
@pytest.mark.parametrize("act,dt", [("swiglu", "bf16"), ("gelu", "f32")])
def test_a_training_step_then_serving(kind, act, dt):
    """Forward, backward, clip and update of the layer, then the updated
    weights' serving step: the gradients clipped as the oracle's norm says,
    and the few-token layer on the updated weights like the oracle's layer."""
    banner("train, clip, update, serve", kind, act, dt)
    cfg = small_variant("long_ctx_swiglu" if act == "swiglu" else "moe_s_like", T=200, d=128,
                        f=192, E=6, k=2, act=act, dtype=dt, zipf_s=None, alpha=0.0)
    t = device.gen_all(cfg)
    tdt = device.torch_dtype(cfg)
    args = (cfg.T, cfg.d, cfg.f, cfg.E, cfg.k, cfg.act, tdt, cfg.renorm)
    layer = M.MoELayer(*args) if kind == "whole" else \
        M.ChunkedMoELayer(*args, chunk_tokens=64)
    W = {n: t[n].clone() for n in ("Wg", "W1", "W2", "W3") if t[n] is not None}
    layer.bind(t["x"], W["Wg"], W["W1"], W["W2"], W.get("W3"), t["bias"], t["dy"])
    layer.step()
    grads = layer.weight_grads()
    assert [g.shape for g in grads] == [W[n].shape for n in ("Wg", "W1", "W3", "W2") if n in W]
    raw = [g.clone() for g in grads]
    want = exact_norm(raw)
    for _ in range(2):                                      # the second finds them clipped
        norm = layer.clip_grads(want / 4).clone()
        torch.cuda.synchronize()
        if _ == 0:
            check_norm(norm, raw)
            check_clipped(grads, raw, want, np.float64(np.float32(want / 4)))
    assert abs(float(norm[0]) / (want / 4) - 1) <= 2.0 ** -8 + 8 * U
    # the oracle's gradients have that norm, to the layer's tolerance
    hx = {n: (rng.gen(cfg, n) if n in ("x", "Wg", "dy") else rng.gen_experts(cfg, n))
          for n in ("x", "dy") + tuple(W)}
    fw = oracle.layer_forward(hx["x"], hx["Wg"], hx["W1"], hx["W2"], hx.get("W3"), k=cfg.k,
                              act=act)
    gr = oracle.layer_backward(fw, hx["dy"], hx["x"], hx["Wg"], hx["W1"], hx["W2"],
                               hx.get("W3"), act=act)
    onorm = np.sqrt(sum(np.sum(np.asarray(gr["d" + n]) ** 2) for n in W))
    assert abs(want / onorm - 1) <= TOL[dt]
    for n, g in zip([n for n in ("Wg", "W1", "W3", "W2") if n in W], grads):
        W[n].sub_(g)
    few = M.FewTokenMoELayer(5, cfg.d, cfg.f, cfg.E, cfg.k, act, tdt, cfg.renorm)
    few.bind(W["Wg"], W["W1"], W["W2"], W.get("W3"), t["bias"])
    y = few.forward(t["x"][:5])
    torch.cuda.synchronize()
    h = {n: W[n].float().cpu().numpy() for n in W}
    fw = oracle.layer_forward(hx["x"][:5], h["Wg"], h["W1"], h["W2"], h.get("W3"), k=cfg.k,
                              act=act)
    assert_equal_i(few.topk_idx, fw["idx"], "topk_idx")
    assert rel_err(host(y), fw["y"]) <= TOL[dt]


def test_overlapping_tensors_are_refused():
    flat = torch.zeros(100, device="cuda")
    a, b = flat[:60], flat[50:]
    with pytest.raises(M.MoEError):
        M.moe_clip_grads([a, b], 1.0)                       # two outputs share elements
    with pytest.raises(M.MoEError):
        M.moe_clip_grads([a, a], 1.0)
    with pytest.raises(M.MoEError):
        M.moe_clip_grads([flat[:40]], 1.0, [flat[20:60]])   # a shifted copy of itself
    with pytest.raises(M.MoEError):
        M.moe_clip_grads([flat[:40], flat[40:80]], 1.0, [flat[40:80], flat[:40]])
    with pytest.raises(M.MoEError):
        M.moe_clip_grads([flat], 1.0, [torch.zeros(100, device="cuda", dtype=BF)])
    with pytest.raises(M.MoEError):
        M.moe_clip_grads([flat], -1.0)
    with pytest.raises(M.MoEError):
        M.moe_clip_grads([flat], float("nan"))
    with pytest.raises(M.MoEError):
        M.moe_grad_norm([flat.double()])
    with pytest.raises(M.MoEError):
        M.moe_grad_norm([flat.view(10, 10).t()])
    assert float(M.moe_grad_norm([a, a])[0]) == 0.0         # only read: any list will do


@pytest.mark.parametrize("dt", [BF, F32])
def test_elements_past_the_32_bit_offsets(dt):
    """A tensor over 2^32 bytes (bf16: over 2^31 elements), zeros but for five
    elements, the last among them: the exact norm, and those five scaled."""
    n = 2 ** 31 + 12345 if dt == BF else 2 ** 30 + 12345
    banner("gradnorm large", dt)
    t = torch.zeros(n, dtype=dt, device="cuda")
    at = [0, 7, n // 2 + 3, n - 9, n - 1]
    for i in at:
        t[i] = 4.0
    t[at[2]] = 6.0                                          # 4 * 16 + 36 = 100
    c = M.GradClip([t])
    assert float(c.norm()[0]) == 10.0
    assert float(c.clip(2.5)[0]) == 10.0
    torch.cuda.synchronize()
    assert [float(t[i]) for i in at] == [1.0, 1.0, 1.5, 1.0, 1.0]
    assert int(torch.count_nonzero(t)) == 5


@pytest.mark.parametrize("kind", ["whole", "chunked"])
def test_a_layer_given_other_gradient_tensors_clips_those(kind):
    banner("clip_grads of other tensors", kind)
    layer = M.MoELayer(8, 64, 64, 2, 1) if kind == "whole" else \
        M.ChunkedMoELayer(8, 64, 64, 2, 1, chunk_tokens=4)
    for _ in range(2):
        new = tensors([(BF, g.shape) for g in layer.weight_grads()], seed=30 + _)
        layer.dWg, layer.dW1, layer.dW2 = new
        keep, want = [g.clone() for g in new], exact_norm(new)
        norm = layer.clip_grads(want / 2)
        torch.cuda.synchronize()
        check_norm(norm, keep)
        check_clipped(new, keep, want, np.float64(np.float32(want / 2)))


@pytest.mark.parametrize("kind", ["whole", "chunked"])
def test_a_layer_s_first_clip_on_a_side_stream(kind):
    """The step and the layer's first clip_grads on a stream that is not torch's
    current one, by its handle: nothing is allocated by then (such memory is
    ordered on the current stream alone), the norm is the gradients' 64-bit one,
    and the next call overwrites it."""
    banner("clip_grads on a side stream", kind)
    cfg = small_variant("moe_s_like", T=300, d=128, f=256, E=4, k=2, act="gelu", dtype="bf16",
                        zipf_s=None, alpha=0.0)
    t = device.gen_all(cfg)
    args = (cfg.T, cfg.d, cfg.f, cfg.E, cfg.k, cfg.act, BF, cfg.renorm)
    layer = M.MoELayer(*args) if kind == "whole" else M.ChunkedMoELayer(*args, chunk_tokens=128)
    layer.bind(t["x"], t["Wg"], t["W1"], t["W2"], None, t["bias"], t["dy"])
    layer.step()
    torch.cuda.synchronize()
    raw = [g.clone() for g in layer.weight_grads()]
    want = exact_norm(raw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    layer.step(side.cuda_stream)
    made = torch.cuda.memory_stats()["allocation.all.allocated"]
    norm = layer.clip_grads(want / 2, side.cuda_stream)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == made
    side.synchronize()
    check_norm(norm, raw)
    check_clipped(layer.weight_grads(), raw, want, np.float64(np.float32(want / 2)))
    again = layer.clip_grads(want, side.cuda_stream)
    side.synchronize()
    assert again.data_ptr() == norm.data_ptr()
    assert abs(float(norm[0]) / (want / 2) - 1) <= 2.0 ** -8 + 8 * U


def test_lists_with_more_partial_sums_than_one_launch_has():
    """700 tensors, some of many chunks: the norm in a launch of its own before
    the scaling.  Norm and clipped values within the bounds, the same norm from
    norm() and clip(), the same bits in place and replayed from a graph."""
    banner("gradnorm long list")
    spec = [((BF, F32)[i % 3 == 0], (17_001 + 97 * i if i % 5 else i // 5,)) for i in range(700)]
    ts = tensors(spec, seed=33)
    keep, want = [t.clone() for t in ts], exact_norm(ts)
    out = [torch.full_like(t, 7) for t in ts]
    c = M.GradClip(ts, out)
    assert c.ws.numel() > 2 * 1024 * 8
    n0 = c.norm().clone()
    check_norm(n0, ts)
    for mx in (want / 3, want * 3):
        assert torch.equal(c.clip(mx), n0)
        torch.cuda.synchronize()
        check_clipped(out, ts, want, np.float64(np.float32(mx)))
    c.clip(want / 3)
    first = [o.clone() for o in out]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.clip(want / 3)
    for _ in range(3):
        c.result.fill_(-1)
        for o in out:
            o.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.result, n0) and all(torch.equal(a, b) for a, b in zip(out, first))
    d = M.GradClip(ts)
    assert torch.equal(d.clip(want / 3), n0)
    torch.cuda.synchronize()
    assert all(torch.equal(t, o) for t, o in zip(ts, first))
    for t, k in zip(ts, keep):
        t.copy_(k)
    ts[699].view(-1)[-1] = float("nan")                     # scales nothing
    assert bool(torch.isnan(d.clip(1.0)[0]))
    assert all(torch.equal(t, k) for t, k in zip(ts[:699], keep))


def test_time_grows_with_the_list_and_not_with_its_square():
    """Four times the tensors (1 MB each), in place under the limit: 4 times the
    time, measured 4.0; 8.2 where every block added all partial sums.  Bound: 6."""
    banner("gradnorm time of long lists")
    flat = torch.zeros(5120 << 19, dtype=BF, device="cuda")
    ts = list(flat.view(5120, 1 << 19))
    took = {}
    for n in (1280, 5120):
        c = M.GradClip(ts[:n])
        for rep in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            c.clip(1.0)
            b.record()
            b.synchronize()
            took.setdefault(n, []).append(a.elapsed_time(b))
    assert min(took[5120]) < 6 * min(took[1280]), took

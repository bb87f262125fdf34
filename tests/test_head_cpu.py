"""What the vocabulary head's losses refuse before any launch, what their
workspace query answers, and the bounds that their tests use (CPU only)."""
import ctypes
import os

import pytest
import torch

import mixture_experts_layer_permute_amd as M
from mixture_experts_layer_permute_amd import _lib, build

from _head import inputs, reference

INV, WS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_WORKSPACE
OK = (_lib.MOE_ERR_HIP, _lib.MOE_ERR_UNSUPPORTED)      # valid: reaches the device check


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return M.load()


@pytest.fixture(scope="module")
def base():
    mem = ctypes.create_string_buffer(1 << 12)
    base.mem = mem
    return ctypes.addressof(mem) + (-ctypes.addressof(mem)) % 16


FAR = 1 << 40                                          # addresses apart from each other


def xent(lib, b, grad=True, T=4, d=64, V=10, dt=1, x=1, W=1, lab=1, loss=1, dx=1, dW=1, ws=1,
         wsb=1 << 30, **at):
    # each pointer: 0 NULL, 1 an address of its own, else that address
    a = {n: None if on == 0 else b + FAR * i if on == 1 else on for i, (n, on) in enumerate(
        (("x", x), ("W", W), ("lab", lab), ("loss", loss), ("dx", dx), ("dW", dW), ("ws", ws)))}
    a.update(at)
    if grad:
        return lib.moe_head_xent_grad(a["x"], a["W"], a["lab"], a.get("weight"), T, d, V, dt,
                                      a["loss"], a.get("lse"), a["dx"], a["dW"], a["ws"], wsb, None)
    return lib.moe_head_xent(a["x"], a["W"], a["lab"], T, d, V, dt, a["loss"], a.get("lse"),
                             a["ws"], wsb, None)


def distill(lib, b, K=3, tau=2.0, idx=1, score=1, kd=1, lab=0, loss=0, T=4, d=64, V=10, dt=1,
            grad=True, dx=1, dW=1):
    p = lambda i, on=1: b + FAR * i if on else None
    t = None if tau is None else ctypes.byref(ctypes.c_float(tau))
    if grad:
        return lib.moe_head_distill_grad(p(0), p(1), p(2, idx), p(3, score), None, K, t, p(4, lab),
                                         None, T, d, V, dt, p(5, kd), p(6, loss), None, p(7, dx),
                                         p(8, dW), p(9), 1 << 30, None)
    return lib.moe_head_distill(p(0), p(1), p(2, idx), p(3, score), K, t, p(4, lab), T, d, V, dt,
                                p(5, kd), p(6, loss), None, p(9), 1 << 30, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=(1 << 24) + 1), dict(d=0), dict(d=100), dict(d=65600), dict(V=0),
    dict(V=(1 << 20) + 1), dict(dt=2), dict(x=0), dict(W=0), dict(lab=0), dict(loss=0)])
@pytest.mark.parametrize("grad", [True, False])
def test_xent_refuses(lib, base, bad, grad):
    assert xent(lib, base, grad, **bad) == INV


def test_xent_refuses_pointers(lib, base):
    assert xent(lib, base, dx=0, dW=0) == INV                        # no gradient wanted
    assert xent(lib, base, x=base + 8) == INV and xent(lib, base, dx=base + 2) == INV
    assert xent(lib, base, ws=base + FAR * 6 + 4) == INV             # 16 bytes
    assert xent(lib, base, lab=base + 2) == INV and xent(lib, base, weight=base + 1) == INV
    assert xent(lib, base, lse=base + 2) == INV
    # outputs over inputs or each other
    assert xent(lib, base, dx=base) == INV                           # x
    assert xent(lib, base, dx=base + FAR + 64) == INV                # inside Wv
    assert xent(lib, base, dW=base + FAR) == INV
    assert xent(lib, base, dW=base + 4 * 64 * 2 - 16) == INV         # x's end
    assert xent(lib, base, dx=base + FAR * 5 + 16) == INV            # inside dWv
    assert xent(lib, base, wsb=255) == WS and xent(lib, base, ws=0) == WS


@pytest.mark.parametrize("bad", [
    dict(K=0), dict(K=257), dict(K=-1), dict(tau=None), dict(tau=0.0), dict(tau=-1.0),
    dict(tau=float("nan")), dict(tau=float("inf")), dict(tau=1e-4), dict(tau=2e3), dict(idx=0),
    dict(score=0), dict(kd=0), dict(lab=1, loss=0), dict(d=65), dict(V=0)])
@pytest.mark.parametrize("grad", [True, False])
def test_distill_refuses(lib, base, bad, grad):
    assert distill(lib, base, grad=grad, **bad) == INV


def test_distill_needs_a_gradient(lib, base):
    assert distill(lib, base, dx=0, dW=0) == INV


def test_valid_arguments_reach_the_device_check(lib, base):
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    assert xent(lib, base) in OK and xent(lib, base, False) in OK
    assert xent(lib, base, dx=0) in OK and xent(lib, base, dW=0) in OK
    assert xent(lib, base, T=0, x=0, lab=0, loss=0, dx=0, ws=0) in OK      # dWv is zeroed
    assert distill(lib, base) in OK and distill(lib, base, grad=False) in OK
    assert distill(lib, base, lab=1, loss=1, K=256) in OK


def test_workspace(lib):
    q = lib.moe_head_workspace_bytes
    for bad in ((-1, 64, 10, 0, 1, 1), (4, 60, 10, 0, 1, 1), (4, 64, 0, 0, 1, 1),
                (4, 64, 10, 257, 1, 1), (4, 64, 10, 0, 5, 1)):
        assert q(*bad, 0) == 0
    T, d, V = 65536, 4096, 128000
    whole = 4 * T * V                                                # the scores of every token
    assert q(T, d, V, 0, 1, 1, 0) <= 8 << 30 < whole / 3
    assert whole / 2 < q(T, d, V, 0, 1, 1, 1 << 40) < whole          # one piece: dz, bf16
    assert q(T, d, V, 0, 1, 0, 0) < whole / 30                       # the loss keeps no scores
    assert q(T, d, V, 8, 1, 1, 0) <= 8 << 30
    # a larger limit never means less; the answer serves every smaller batch
    import random
    rng = random.Random(3)
    for _ in range(400):
        d, V, K = 64 * rng.randint(1, 64), rng.randint(1, 130000), rng.choice([0, 9])
        dt, g = rng.randint(0, 1), rng.randint(0, 1)
        T = rng.randint(1, 20000)
        n = rng.randint(1, T)
        need = q(T, d, V, K, dt, g, rng.choice([0, 1, 1 << 28]))
        assert 0 < q(n, d, V, K, dt, g, need) <= need
        assert 0 < q(n, d, V, 0, dt, 0, need) <= need


def test_the_binding_refuses():
    x, Wv, labels, weight, teacher = inputs(4, 64, 10, K=2, device="cpu")
    for call in (lambda: M.moe_head_xent(x, Wv, labels),
                 lambda: M.moe_head_xent_grad(x, Wv, labels, weight),
                 lambda: M.moe_head_distill(x, Wv, teacher[:2]),
                 lambda: M.moe_head_distill_grad(x, Wv, teacher)):
        with pytest.raises(M.MoEError, match="device tensors"):
            call()


def test_the_reference_against_autograd():
    """The tests' own 64-bit formulas against torch's autograd, duplicate slots and
    left-out tokens among them."""
    T, d, V, K, tau = 12, 64, 50, 6, 1.7
    x, Wv, labels, weight, (idx, score, tw) = inputs(T, d, V, "f32", masked=0.3, K=K, device="cpu",
                                                     seed=1)
    idx[2] = 5
    idx[3] = -1
    X, W = x.double().requires_grad_(), Wv.double().requires_grad_()
    z = X @ W.t()
    y = labels.long()
    ce = torch.nn.functional.cross_entropy(z, y, reduction="none", ignore_index=-1)
    kd = []
    for t in range(T):
        on = idx[t] >= 0
        if not bool(on.any()):
            kd.append(z[t, 0] * 0)
            continue
        q = torch.softmax(score[t][on].double() / tau, 0)
        lp = torch.log_softmax(z[t] / tau, 0)[idx[t][on].long()]
        kd.append(tau ** 2 * (q * (q.log() - lp)).sum())
    kd = torch.stack(kd)
    ((ce * weight.double()).sum() + (kd * tw.double()).sum()).backward()
    ref = reference(x, Wv, labels, weight, (idx, score, tw), tau, "f32")
    for got, want in ((ce, "loss"), (kd, "kd"), (X.grad, "dx"), (W.grad, "dWv")):
        assert torch.allclose(ref[want][0], got.detach(), rtol=1e-11, atol=1e-12), want

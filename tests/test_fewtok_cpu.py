"""What moe_layer_fwd_few and FewTokenMoELayer refuse, before any launch
(CPU only), and what the workspace query answers."""
import ctypes
import os

import pytest
import torch

import mixture_experts_layer_permute_amd as M
from mixture_experts_layer_permute_amd import _lib, build

INV, UNS, WS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return M.load()


@pytest.fixture(scope="module")
def mem():
    return ctypes.create_string_buffer(1 << 16)


def call(lib, mem, **kw):
    p = ctypes.addressof(mem) + (-ctypes.addressof(mem)) % 16
    a = dict(x=p, Wg=p, bias=None, W1=p, W3=None, W2=p, T=2, d=64, f=64, E=4, k=2, renorm=1,
             act=0, dt=1, logits=None, idx=None, w=None, y=p, ws=p, wsb=1 << 16)
    a.update(kw)
    return lib.moe_layer_fwd_few(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(d=0), dict(d=100), dict(d=32), dict(f=96), dict(f=0), dict(E=0),
    dict(E=1025), dict(k=0), dict(k=5), dict(act=2), dict(dt=2), dict(dt=-1), dict(x=None),
    dict(Wg=None), dict(W1=None), dict(W2=None), dict(y=None), dict(act=1),
])
def test_invalid_arguments(lib, mem, kw):
    assert call(lib, mem, **kw) == INV


def test_unaligned_rows_and_workspace(lib, mem):
    p = ctypes.addressof(mem) + (-ctypes.addressof(mem)) % 16
    for n in ("x", "W1", "W2", "y", "ws"):
        assert call(lib, mem, **{n: p + 8}) == INV, n
    assert call(lib, mem, act=1, W3=p + 8) == INV
    for n, off in (("Wg", 1), ("bias", 2), ("logits", 2), ("idx", 2), ("w", 2)):
        assert call(lib, mem, **{n: p + off}) == INV, n
    assert call(lib, mem, dt=0, Wg=p + 2) == INV


def test_more_tokens_or_pairs_than_a_few(lib, mem):
    assert call(lib, mem, T=65) == UNS
    assert call(lib, mem, T=64, E=1024, k=65) == UNS
    q = lib.moe_layer_few_workspace_bytes
    assert q(65, 64, 64, 4, 2, 0, 1) == 0 and q(64, 64, 64, 1024, 65, 0, 1) == 0
    assert q(64, 64, 64, 1024, 64, 0, 1) > 0


def test_workspace(lib, mem):
    need = lib.moe_layer_few_workspace_bytes(2, 64, 64, 4, 2, 0, 1)
    assert 0 < need < 1 << 16
    assert call(lib, mem, wsb=need - 1) == WS
    assert call(lib, mem, ws=None) == WS
    for bad in ((2, 100, 64, 4, 2, 0, 1), (2, 64, 64, 4, 5, 0, 1), (2, 64, 64, 4, 2, 7, 1),
                (2, 64, 64, 4, 2, 0, 9), (-1, 64, 64, 4, 2, 0, 1)):
        assert lib.moe_layer_few_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("layer", [(1024, 4096, 8, 2, 0, 1), (4096, 14336, 32, 8, 1, 1),
                                   (1088, 1984, 12, 3, 1, 0), (64, 64, 4, 2, 0, 1),
                                   (2048, 8192, 16, 2, 0, 1), (1024, 4096, 64, 2, 0, 0)])
def test_the_workspace_of_a_step_covers_every_smaller_step(lib, mem, layer):
    """A step of fewer tokens may be cut into more chunks; sized once for T, the
    workspace holds them all: no smaller step is refused for it."""
    need = [lib.moe_layer_few_workspace_bytes(T, *layer) for T in range(1, 65)]
    assert need == sorted(need) and need[0] > 0
    d, f, E, k, act, dt = layer
    p = ctypes.addressof(mem) + (-ctypes.addressof(mem)) % 16
    if not torch.cuda.is_available():              # the call's own check, before any launch
        for T in range(1, 65):
            got = call(lib, mem, T=T, d=d, f=f, E=E, k=k, act=act, dt=dt, W3=p if act else None,
                       wsb=need[-1])
            assert got in (_lib.MOE_ERR_HIP, UNS), T


def test_no_tokens_is_a_no_op(lib, mem):
    assert call(lib, mem, T=0, x=None, y=None, ws=None, wsb=0) == 0


def test_valid_arguments_reach_the_device_check(lib, mem):
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    assert call(lib, mem) in (_lib.MOE_ERR_HIP, UNS)


def test_the_binding_takes_device_tensors_only():
    t = torch.zeros(2, 64)
    with pytest.raises(M.MoEError):
        M.moe_layer_fwd_few(t, torch.zeros(64, 4), torch.zeros(4, 64, 64),
                            torch.zeros(4, 64, 64), k=2)


@pytest.mark.parametrize("kw", [dict(dtype=torch.float16), dict(dtype=torch.float64),
                                dict(act="relu"), dict(T=65), dict(T=0), dict(d=96), dict(k=9)])
def test_the_layer_takes_the_library_s_types_only(kw):
    """float16 buffers would be read as float32 ones, past their end."""
    a = dict(dict(T=4, d=64, f=128, E=8, k=2, device="cpu"), **kw)
    with pytest.raises(M.MoEError):
        M.FewTokenMoELayer(**a)


def test_the_layer_needs_its_weights_first():
    layer = M.FewTokenMoELayer(4, 64, 128, 8, 2, device="cpu")
    with pytest.raises(M.MoEError):
        layer.forward(torch.zeros(1, 64, dtype=torch.bfloat16))

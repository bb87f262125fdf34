"""What moe_grad_norm and moe_clip_grads refuse, before any launch (CPU only),
and what the workspace query answers."""
import ctypes
import os

import pytest
import torch

import mixture_experts_layer_permute_amd as M
from mixture_experts_layer_permute_amd import _lib, build

INV, WS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_WORKSPACE


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


def arrays(ptrs, numel, dts):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_size_t * n)(*numel),
            (ctypes.c_int32 * n)(*dts), n)


def norm(lib, base, ptrs, numel, dts, out=True, ws=True, wsb=1 << 10):
    p, c, d, n = arrays(ptrs, numel, dts)
    return lib.moe_grad_norm(p, c, d, n, base if out else None, base if ws else None, wsb, None)


def clip(lib, base, ptrs, outs, numel, dts, mx=1.0, ws=True, wsb=1 << 10, res=True):
    p, c, d, n = arrays(ptrs, numel, dts)
    o = (ctypes.c_void_p * n)(*outs)
    m = None if mx is None else ctypes.byref(ctypes.c_float(mx))
    return lib.moe_clip_grads(p, o, c, d, n, m, base if res else None, base if ws else None,
                              wsb, None)


def test_refused_lists(lib, base):
    assert norm(lib, base, [base], [4], [2]) == INV                  # unknown type
    assert norm(lib, base, [None], [4], [0]) == INV                  # elements, no pointer
    assert norm(lib, base, [base + 2], [4], [0]) == INV              # fp32 at half a float
    assert norm(lib, base, [base + 1], [4], [1]) == INV              # bf16 at an odd byte
    assert norm(lib, base, [base], [(1 << 40) + 1], [1]) == INV
    assert norm(lib, base, [base], [4], [0], out=False) == INV
    assert lib.moe_grad_norm(None, None, None, 1, base, base, 64, None) == INV
    assert lib.moe_grad_norm(None, None, None, -1, base, base, 64, None) == INV
    assert clip(lib, base, [base], [None], [4], [0]) == INV
    assert clip(lib, base, [base], [base + 2], [4], [0]) == INV
    assert clip(lib, base, [base], [base], [4], [0], res=False) == INV


@pytest.mark.parametrize("mx", [None, -1.0, float("nan"), -float("inf")])
def test_refused_limits(lib, base, mx):
    assert clip(lib, base, [base], [base], [4], [0], mx=mx) == INV


def test_workspace(lib, base):
    q = lambda numel, dts: lib.moe_grad_norm_workspace_bytes(
        (ctypes.c_size_t * len(numel))(*numel), (ctypes.c_int32 * len(dts))(*dts), len(numel))
    assert q([], []) > 0 and q([0], [0]) > 0 and q([1], [1]) > 0
    assert q([10 ** 9] * 3, [1, 0, 1]) >= 1024 * 8                   # a partial sum per block
    assert q([1] * 400, [0] * 400) >= 400 * 8                        # one chunk per tensor
    assert q([1], [2]) == 0 and q([(1 << 40) + 1], [0]) == 0
    assert lib.moe_grad_norm_workspace_bytes(None, None, 2) == 0
    assert lib.moe_grad_norm_workspace_bytes(None, None, -1) == 0
    assert norm(lib, base, [base], [4], [0], wsb=7) == WS
    assert norm(lib, base, [base], [4], [0], ws=False) == WS
    assert clip(lib, base, [base], [base], [4], [0], wsb=0) == WS


def test_valid_arguments_reach_the_device_check(lib, base):
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    ok = (_lib.MOE_ERR_HIP, _lib.MOE_ERR_UNSUPPORTED)
    assert norm(lib, base, [base + 2, None], [4, 0], [1, 0]) in ok   # bf16 at any element
    assert clip(lib, base, [base], [base], [4], [0], mx=float("inf")) in ok
    assert lib.moe_grad_norm(None, None, None, 0, base, base, 64, None) in ok


def test_the_binding_takes_device_tensors_only():
    with pytest.raises(M.MoEError):
        M.moe_grad_norm([torch.zeros(4)])
    with pytest.raises(M.MoEError):
        M.GradClip([torch.zeros(4)])

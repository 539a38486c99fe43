"""Host-side checks of the few-token entry points (no GPU): sizes and the
refusals, each before anything is launched."""
import ctypes

import pytest
import torch

from sparse_mixture_experts_renorm_b200 import MoEError, _binding as B, build as build_mod
from sparse_mixture_experts_renorm_b200 import few_workspace_size, moe_forward_few

P = ctypes.c_void_p(4096)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(4104)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


def test_workspace_size(lib):
    R = 16 * 2
    n = lib.moe_few_workspace_size(16, 4096, 8, 2, 14336, B.MOE_BF16)
    assert 2 * R * 14336 * 2 + R * 4096 * 4 <= n <= 2 * R * 28 * 1088 + 8 * R * 4096 * 4 + 8192
    assert few_workspace_size(3, 12, 4, 2, 20, torch.float32) > 0
    with pytest.raises(MoEError):
        few_workspace_size(17, 64, 4, 2, 64, torch.bfloat16)


@pytest.mark.parametrize("change,expect", [
    (dict(T=-1), B.MOE_ERR_INVALID_ARG), (dict(T=17), B.MOE_ERR_UNSUPPORTED), (dict(d=0), B.MOE_ERR_INVALID_ARG),
    (dict(d=68), B.MOE_ERR_UNSUPPORTED), (dict(I=4), B.MOE_ERR_UNSUPPORTED), (dict(I=-8), B.MOE_ERR_INVALID_ARG),
    (dict(d=66, dt=B.MOE_F32), B.MOE_ERR_UNSUPPORTED), (dict(dt=5), B.MOE_ERR_INVALID_ARG),
    (dict(E=257), B.MOE_ERR_UNSUPPORTED), (dict(k=5), B.MOE_ERR_INVALID_ARG), (dict(k=0), B.MOE_ERR_INVALID_ARG),
    (dict(E=16, k=9), B.MOE_ERR_UNSUPPORTED), (dict(renorm=2), B.MOE_ERR_INVALID_ARG),
    (dict(E=256, I=1 << 24), B.MOE_ERR_UNSUPPORTED), (dict(d=1 << 29), B.MOE_ERR_UNSUPPORTED),
    (dict(x=None), B.MOE_ERR_INVALID_ARG), (dict(out=None), B.MOE_ERR_INVALID_ARG),
    (dict(status=None), B.MOE_ERR_INVALID_ARG), (dict(w=ODD), B.MOE_ERR_INVALID_ARG),
    (dict(ws=None), B.MOE_ERR_WORKSPACE), (dict(n=100), B.MOE_ERR_WORKSPACE), (dict(ws=ODD), B.MOE_ERR_INVALID_ARG),
])
def test_refusals(lib, change, expect):
    v = dict(T=4, d=64, E=4, k=2, I=64, dt=B.MOE_BF16, renorm=1, x=P, w=P, out=P, ws=P, n=1 << 30, status=P) | change
    st = lib.moe_forward_few(v["x"], P, None, v["w"], P, P, v["T"], v["d"], v["E"], v["k"], v["I"], v["renorm"],
                             v["dt"], v["out"], P, P, None, None, v["ws"], v["n"], v["status"], None)
    assert st == expect and B.last_error_detail(lib)


def test_python_refuses_host_tensors():
    x = torch.zeros((2, 64))
    w = torch.zeros((4, 64, 64))
    with pytest.raises(ValueError, match="CUDA"):
        moe_forward_few(x, torch.zeros((4, 64)), None, w, w, w, 2, True)


def test_the_workspace_as_status_word_needs_room_for_it(lib):
    st = lib.moe_forward_few(P, P, None, P, P, P, 0, 64, 4, 2, 64, 1, B.MOE_BF16, P, P, P, None, None, P, 3, P, None)
    assert st == B.MOE_ERR_WORKSPACE and "status" in B.last_error_detail(lib)

"""Host-side checks of the MXFP4 entry points (no GPU): sizes, the documented
layout and the refusals, each before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import mx_oracle as O
from sparse_mixture_experts_renorm_b200 import MXTensor, _binding as B, build as build_mod
from sparse_mixture_experts_renorm_b200 import mx_experts, mx_matmul, mx_quantize

P = ctypes.c_void_p(4096)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(4104)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


def test_scale_bytes(lib):
    assert lib.moe_mx_scale_bytes(1, 1, 32, 0) == 2 * 1024
    assert lib.moe_mx_scale_bytes(8, 300, 288, 0) == 8 * 4 * 2 * 1024
    assert lib.moe_mx_scale_bytes(64, 1000, 256, 1) == 2 * (3 + 64) * 1024
    assert lib.moe_mx_scale_bytes(64, 5, 256, 1) == 2 * 5 * 1024
    for bad in ((0, 1, 32), (1, -1, 32), (1, 1, 0), (1, 1, 40), (1 << 20, 1 << 20, 32)):
        assert lib.moe_mx_scale_bytes(*bad, 0) == 0 and B.last_error_detail(lib)


@pytest.mark.parametrize("args,expect", [
    ((P, None, 1, 4, 64, 7, P, P, 1 << 20), B.MOE_ERR_INVALID_ARG),
    ((P, None, 1, 4, 40, B.MOE_BF16, P, P, 1 << 20), B.MOE_ERR_UNSUPPORTED),
    ((P, None, 0, 4, 64, B.MOE_BF16, P, P, 1 << 20), B.MOE_ERR_INVALID_ARG),
    ((P, None, 1, -4, 64, B.MOE_BF16, P, P, 1 << 20), B.MOE_ERR_INVALID_ARG),
    ((P, None, 1, 4, 64, B.MOE_BF16, P, P, 2047), B.MOE_ERR_INVALID_ARG),
    ((None, None, 1, 4, 64, B.MOE_BF16, P, P, 1 << 20), B.MOE_ERR_INVALID_ARG),
    ((ODD, None, 1, 4, 64, B.MOE_BF16, P, P, 1 << 20), B.MOE_ERR_INVALID_ARG),
    ((P, P, 257, 4, 64, B.MOE_BF16, P, P, 1 << 30), B.MOE_ERR_UNSUPPORTED),
])
def test_quantize_refusals(lib, args, expect):
    assert lib.moe_mx_quantize(*args, None) == expect
    x, off, g, r, c, dt, q, s, n = args
    assert lib.moe_mx_dequantize(q, s, n, off, g, r, c, dt, x, None) == expect
    assert B.last_error_detail(lib)


@pytest.mark.parametrize("change,expect", [
    (dict(N=20), B.MOE_ERR_UNSUPPORTED), (dict(N=0), B.MOE_ERR_INVALID_ARG), (dict(K=48), B.MOE_ERR_UNSUPPORTED),
    (dict(M=-1), B.MOE_ERR_INVALID_ARG), (dict(groups=0), B.MOE_ERR_INVALID_ARG),
    (dict(groups=300), B.MOE_ERR_UNSUPPORTED), (dict(dt=9), B.MOE_ERR_INVALID_ARG),
    (dict(a=None), B.MOE_ERR_INVALID_ARG), (dict(out=ODD), B.MOE_ERR_INVALID_ARG),
    (dict(status=None), B.MOE_ERR_INVALID_ARG), (dict(M=1 << 30, groups=4), B.MOE_ERR_UNSUPPORTED),
])
def test_matmul_refusals(lib, change, expect):
    v = dict(a=P, groups=1, M=8, N=16, K=64, dt=B.MOE_F32, out=P, status=P) | change
    st = lib.moe_mx_matmul(v["a"], P, P, P, None, v["groups"], v["M"], v["N"], v["K"], v["dt"], v["out"], v["status"],
                           None)
    assert st == expect and B.last_error_detail(lib)


def weights(**change):
    w = B.moe_mx_weights()
    w.struct_bytes = ctypes.sizeof(B.moe_mx_weights)
    for n, _ in B.moe_mx_weights._fields_[1:]:
        setattr(w, n, 4096)
    for n, v in change.items():
        setattr(w, n, v)
    return w


@pytest.mark.parametrize("change,expect", [
    (dict(d=40), B.MOE_ERR_UNSUPPORTED), (dict(I=48), B.MOE_ERR_UNSUPPORTED), (dict(k=5), B.MOE_ERR_INVALID_ARG),
    (dict(E=300), B.MOE_ERR_UNSUPPORTED), (dict(T=-1), B.MOE_ERR_INVALID_ARG), (dict(dt=3), B.MOE_ERR_INVALID_ARG),
    (dict(d=0), B.MOE_ERR_INVALID_ARG), (dict(ws=None), B.MOE_ERR_WORKSPACE), (dict(nb=100), B.MOE_ERR_WORKSPACE),
    (dict(ws=ctypes.c_void_p(4096 + 16)), B.MOE_ERR_INVALID_ARG), (dict(x=ODD), B.MOE_ERR_INVALID_ARG),
    (dict(w=weights(struct_bytes=8)), B.MOE_ERR_INVALID_ARG), (dict(w=weights(up=None)), B.MOE_ERR_INVALID_ARG),
    (dict(w=weights(down_scales=4100)), B.MOE_ERR_INVALID_ARG),
])
def test_experts_refusals(lib, change, expect):
    v = dict(x=P, T=8, d=64, E=4, k=2, I=64, dt=B.MOE_BF16, w=weights(), ws=P, nb=1 << 30) | change
    shape = tuple(v[n] for n in ("T", "d", "E", "k", "I"))
    st = lib.moe_mx_experts(v["x"], P, P, ctypes.byref(v["w"]), *shape, v["dt"], P, None, v["ws"], v["nb"], None, None)
    assert st == expect and B.last_error_detail(lib)
    st = lib.moe_mx_forward(v["x"], P, None, ctypes.byref(v["w"]), *shape, 1, v["dt"], P, P, P, None, None, v["ws"],
                            v["nb"], None, None)
    assert st == expect


def test_forward_refusals(lib):
    st = lib.moe_mx_forward(P, P, None, ctypes.byref(weights()), 8, 64, 4, 2, 64, 2, B.MOE_BF16, P, P, P, None, None,
                            P, 1 << 30, None, None)
    assert st == B.MOE_ERR_INVALID_ARG
    st = lib.moe_mx_forward(P, P, None, ctypes.byref(weights()), 8, 96, 4, 2, 64, 1, B.MOE_BF16, P, P, P, None, None,
                            P, 1 << 30, None, None)
    assert st == B.MOE_ERR_UNSUPPORTED  # the bf16 router's d % 64


def test_python_refusals():
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        mx_quantize(x)
    with pytest.raises(TypeError):
        mx_matmul(x, x)
    q = MXTensor(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((2048,), dtype=torch.uint8))
    assert q.shape == (4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        mx_matmul(q, q)
    with pytest.raises(ValueError, match="CUDA"):
        mx_experts(x, x, x, q, q, q)


def test_oracle_rounds_to_the_nearest_code():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((50, 64)) * np.exp2(rng.integers(-30, 30, (50, 1)))
    s = O.scale_exponents(v)
    q = O.values(O.round_codes(v, s), s)
    scale = np.repeat(np.exp2(s.astype(float)), 32, axis=-1)
    every = np.concatenate([O.GRID, -O.GRID])
    best = np.abs(v[..., None] / scale[..., None] - every).min(-1)
    assert np.allclose(np.abs(q / scale - v / scale), best, rtol=0, atol=0)
    top = np.abs(v).reshape(50, 2, 32).max(-1) / np.exp2(s.astype(float))
    assert ((top >= 4) & (top < 8)).all()
    one = np.zeros((1, 32))
    one[0, :9] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 100]  # ties to the even code; 100 sets the scale
    assert O.values(O.round_codes(one, np.zeros((1, 1), int)), np.zeros((1, 1), int))[0, :9].tolist() == [
        4, 0, 1, 1, 2, 2, 4, 4, 6]


@pytest.mark.parametrize("d,I", [(128, 160), (1024, 512)])
def test_what_four_bits_cost_on_normal_data(d, I):
    """The figures of include/moe.h, from the definition: 0.11 of a matrix's norm, 0.20 of the layer's output by the
    weights alone, 0.30 with x and the hidden rows rounded as well."""
    r = np.random.default_rng(1)
    x = r.standard_normal((64, d))
    w = [r.standard_normal(s) * 0.02 for s in ((I, d), (I, d), (d, I))]

    def layer(x, wg, wu, wd, keep):
        g = x @ wg.T
        return keep(g / (1 + np.exp(-g)) * (x @ wu.T)) @ wd.T

    want, q = layer(x, *w, lambda h: h), [O.fake(v) for v in w]
    off = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)  # noqa: E731
    assert 0.105 < off(q[0], w[0]) < 0.12
    assert 0.18 < off(layer(x, *q, lambda h: h), want) < 0.22
    assert 0.27 < off(layer(O.fake(x), *q, O.fake), want) < 0.32

"""MXFP4 on the GPU at the ends of the number range, against the 64-bit oracle
of test_mx_gpu.py (its tolerances are derived there). The experts' down product
has two kernels, for groups of few rows (at most 64 on average) and of many:
each case runs through both."""
import numpy as np
import pytest
import torch

import mx_oracle as O
from sparse_mixture_experts_renorm_b200 import MXTensor, _call, mx_dequantize, mx_experts, mx_matmul, mx_quantize
from test_mx_gpu import BF16, F32, check_experts, experts64, layer, rand

pytestmark = pytest.mark.gpu

BOTH = pytest.mark.parametrize("T", [40, 400])  # rows of 3 experts: 13 on average, and 133


def rows64(x, idx, w):
    """The experts' rows of one choice a token, in fp64."""
    one = np.ones(idx.shape)
    return experts64(O.fake(O.f64(x)), idx.cpu().numpy(), one, *(O.dense64(q) for q in w), (*x.shape, w[0].shape[1], 1))[0]


@BOTH
@pytest.mark.parametrize("top", [1.9, 1.0, 0.5, 0.24])
def test_gated_rows_up_to_the_largest_number(T, top):
    """The largest of a token's outputs is top 2^127: in [2^127, 2^128), where 2^(127 - exponent) is no normal
    fp32 number, at its border, and below. bf16 holds all of them."""
    x, idx, _, w = layer(T, 96, 3, 1, 160, 40, F32)
    x = x * 8  # outputs of some size, so that gates are below the largest fp32 number
    y = np.abs(rows64(x, idx, w)).max(1)
    g = top * 2.0**127 / y
    assert g.max() < 3.4e38
    gate = torch.tensor(g, dtype=F32, device="cuda")[:, None].contiguous()
    r = mx_experts(x, idx, gate, *w)
    assert torch.isfinite(r.out).all() and int(r.status.item()) == 0
    assert (r.out.float().abs().amax(1) > 0.9 * top * 2.0**127).all()
    check_experts(x, idx, gate, w, r.out)


@BOTH
def test_gates_of_any_value(T):
    x, idx, gate, w = layer(T, 96, 3, 2, 160, 41)
    some = torch.tensor([0.0, -0.0, -1.0, 2.0**100, -(2.0**100), 2.0**-100, 2.0**-140, 1.0, -3.7e-5, 6e4], device="cuda")
    gate = some[torch.arange(gate.numel(), device="cuda") * 7 % 10].view_as(gate).contiguous()
    gate[0], gate[1] = torch.tensor([0.0, -0.0]), torch.tensor([2.0**100, 2.0**-100])
    r = mx_experts(x, idx, gate, *w)
    assert (r.out[0] == 0).all()
    check_experts(x, idx, gate, w, r.out)


@BOTH
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["x", "gate"])
def test_what_is_not_finite_stays_in_its_token(T, bad, where):
    """A NaN or infinity among x makes its block of x NaN, and with it the token's output; a gate that is not finite
    makes the products with it infinite, or NaN (as inf times 0)."""
    x, idx, gate, w = layer(T, 96, 3, 2, 160, 42)
    want = mx_experts(x, idx, gate, *w).out.clone()
    t = T - 3
    if where == "x":
        x[t, 5] = bad
    else:
        gate[t, 1] = bad
    out = mx_experts(x, idx, gate, *w).out
    keep = torch.arange(T, device="cuda") != t
    assert torch.equal(out[keep], want[keep])
    if where == "x" or bad != bad:
        assert torch.isnan(out[t]).all()
    else:
        y = torch.tensor(rows64(x, idx[:, 1:].contiguous(), w)[t], device="cuda")
        big = y.abs() > 0.1 * y.abs().max()  # no hidden value's other code changes the sign of these
        assert big.sum() > 32 and torch.equal(out[t][big].float(), torch.sign(y[big]).float() * bad)


@BOTH
def test_a_row_with_an_infinite_block_keeps_its_other_blocks(T):
    """One weight row of w_down so large that its output overflows: that column is infinite, and the others, in its
    block of 32 columns rounded to bf16 before the sum and in the others as always, keep their values."""
    x, idx, gate, w = layer(T, 96, 3, 1, 160, 43, F32)
    gate = torch.full_like(gate, 2.0**80)
    want = mx_experts(x, idx, gate, *w).out.clone()
    v = w[2]
    r, stages = 40, 1  # output column 40 of every expert, all blocks of its 160 columns
    scales = v.scales.view(3, 2, stages, 2, 32, 4, 4)  # expert, tile row, stage, half, row % 32, row / 32, block % 4
    scales[:, r // 128, :, :, r % 32, r % 128 // 32, :] += 90
    out = mx_experts(x, idx, gate, *w).out
    cols = torch.arange(96, device="cuda")
    assert torch.isinf(out[:, r]).sum() > 0.9 * T
    other = (cols < 32) | (cols >= 64)
    assert torch.equal(out[:, other], want[:, other])
    near = (cols >= 32) & (cols < 64) & (cols != r)
    a, b = out[:, near].double(), want[:, near].double()
    # rounded to bf16 (2^-8) on one side, to fp16 with a shared exponent (2^-11, 2^-25 of the block's largest) and to
    # bf16 on the other; 1.02 for taking the rounded value in place of the value
    tol = (2 * 2.0**-8 + 2.0**-11) * b.abs() + 2.0**-25 * want.double().abs().amax(1, keepdim=True)
    assert ((a - b).abs() <= tol * 1.02).all()


@pytest.mark.parametrize("inside", [True, False])
def test_the_first_product_on_a_device_is_not_captured(inside, monkeypatch):
    """The device's status word would belong to the graph: refused on a capturing stream, be it torch's current one or
    the one that is given, and the capture goes on."""
    a, b = mx_quantize(rand((9, 64), 60)), mx_quantize(rand((16, 64), 61))
    want, st = mx_matmul(a, b), torch.zeros((1,), dtype=torch.int32, device="cuda")
    out = torch.zeros_like(want)
    monkeypatch.setattr(_call, "_status", {})
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        g.capture_begin()
        try:
            with torch.cuda.stream(s if inside else torch.cuda.default_stream()):
                with pytest.raises(RuntimeError, match="captured"):
                    mx_matmul(a, b, stream=None if inside else s)
                mx_matmul(a, b, out=out, status=st, stream=None if inside else s)
        finally:
            g.capture_end()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and int(st) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_every_code_at_every_scale(dtype):
    """Exact from 2^-128 (0.5 at the smallest scale, subnormal) up to 1.5 2^127; what passes that, at the scales 2^126
    and 2^127, is infinite, and the scale 0xFF is NaN."""
    code = torch.arange(16, dtype=torch.uint8)
    row = code[0::2] | code[1::2] << 4  # the 16 codes, and again
    data = row.repeat(2).repeat(256, 1).cuda()
    scales = torch.zeros((2048,), dtype=torch.uint8)
    r = torch.arange(256)
    scales[r // 128 * 1024 + r % 32 * 16 + r % 128 // 32 * 4] = r.to(torch.uint8)
    got = mx_dequantize(MXTensor(data, scales.cuda()), dtype).cpu().double()
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64).repeat(2)
    want = level * torch.exp2(r[:255, None].double() - 127)
    want = torch.where(want.abs() >= 2.0**128, torch.sign(want) * float("inf"), want)
    assert torch.equal(got[:255], want) and torch.equal(torch.signbit(got[:255]), torch.signbit(want))
    assert torch.isnan(got[255]).all()

"""MXFP4 on the GPU against the 64-bit oracle: quantisation and its inverse
(exact), the grouped product, and the experts.

Tolerances. A product: every term a_i b_i is exact in fp32 up to the range of
the scales, and adding n terms in fp32, rounded or truncated (at most 2^-23 of
the running value each), is off by at most n 2^-23 sum |a_i b_i|; a bf16 result
adds its rounding, 2^-8 of the value (half an eps of 2^-7)."""
import numpy as np
import pytest
import torch

import mx_oracle as O
from sparse_mixture_experts_renorm_b200 import (MXTensor, device_status, moe_forward_mx, mx_dequantize, mx_experts,
                                                mx_matmul, mx_quantize, mx_scale_bytes, mx_workspace_size)
from sparse_mixture_experts_renorm_b200 import _binding as B

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def rand(shape, seed, dtype=F32, std=1.0, spread=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda") * std
    if spread:
        x = x * torch.exp2(torch.randint(-spread, spread + 1, (*shape[:-1], 1), generator=g, device="cuda").float())
    return x.to(dtype)


# ------------------------------------------------------------ quantisation --


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 32), (1, 64), (3, 96), (129, 256), (257, 288), (40, 1056), (2, 33, 320),
                                   (5, 300, 64), (700, 2048)])
def test_quantize_is_exact(shape, dtype):
    x = rand(shape, sum(shape), dtype, spread=20)
    q = mx_quantize(x)
    v = O.f64(x)
    s = O.scale_exponents(v)
    code = O.round_codes(v, s)
    assert np.array_equal(O.unpack(q.data.cpu().numpy()), code)
    groups = [shape[-2]] * (shape[0] if len(shape) == 3 else 1)
    got = O.untile(q.scales.cpu().numpy(), shape[-1], groups)
    assert np.array_equal(got, (s + 127).reshape(got.shape))
    for dt in (BF16, F32):
        assert np.array_equal(O.f64(mx_dequantize(q, dt)), O.values(code, s))


def test_quantize_ties_borders_and_the_ends_of_the_range():
    rows = []
    for top in (4.0, 5.0, 6.0, 7.0, 7.96875):  # floor(log2 top) - 2 = 0: beyond 6 saturates
        grid = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 0.2490234375, 0.25390625, 2.484375])
        rows.append(np.concatenate([[top], grid, -grid, [0]]))
    rows.append(np.zeros(32))
    rows.append(np.full(32, -0.0))
    v = np.stack(rows)
    v = np.concatenate([v * 2.0**e for e in (0, -126, -130, 120, 124)])  # 7.97 * 2^124 is the largest there is
    for dtype in (BF16, F32):
        x = torch.tensor(v, dtype=torch.float64).to(dtype).cuda()
        w = O.f64(x)
        q = mx_quantize(x)
        s = O.scale_exponents(w)
        code = O.round_codes(w, s)
        assert np.array_equal(O.unpack(q.data.cpu().numpy()), code)
        assert np.array_equal(O.f64(mx_dequantize(q, F32)), O.values(code, s))
    x = torch.tensor([[2.0**-149] * 32, [2.0**-127] + [2.0**-149] * 31], dtype=F32, device="cuda")  # subnormal
    q = mx_quantize(x)
    assert np.array_equal(O.f64(mx_dequantize(q, F32)), O.fake(O.f64(x)))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_block_with_a_nan_or_infinity_is_nan_and_the_others_are_not(bad):
    x = rand((4, 128), 3)
    x[2, 40] = bad
    v = mx_dequantize(mx_quantize(x), F32)
    assert torch.isnan(v[2, 32:64]).all()
    v[2, 32:64] = 0
    y = x.clone()
    y[2, 32:64] = 0
    assert np.array_equal(O.f64(v), O.fake(O.f64(y)))


@pytest.mark.parametrize("offsets,rows", [([0, 5], 5), ([0, 0, 3, 3, 300, 300, 813], 813), ([0, 256, 512], 600),
                                          ([7, 7, 90], 100), ([0] * 256 + [70], 70)])
def test_quantize_ragged_groups(offsets, rows):
    x = rand((rows, 288), rows, BF16, spread=6)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    q = mx_quantize(x, off)
    assert q.scales.numel() == mx_scale_bytes(len(offsets) - 1, rows, 288, True)
    v = O.f64(x)[offsets[0]:offsets[-1]]
    s = O.scale_exponents(v)
    assert np.array_equal(O.unpack(q.data.cpu().numpy()[offsets[0]:offsets[-1]]), O.round_codes(v, s))
    assert np.array_equal(O.untile(q.scales.cpu().numpy(), 288, np.diff(offsets)), s + 127)
    out = torch.full((rows, 288), 123.0, dtype=BF16, device="cuda")
    mx_dequantize(q, BF16, off, out=out)
    want = np.full((rows, 288), 123.0)
    want[offsets[0]:offsets[-1]] = O.values(O.round_codes(v, s), s)
    assert np.array_equal(O.f64(out), want)  # rows of no group are left as they were


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_of_values_at_an_odd_multiple_of_16_bytes(dtype):
    n = 16 // torch.empty((), dtype=dtype).element_size()
    x = rand((n + 70 * 96,), 8, dtype)[n:].view(70, 96)
    assert x.data_ptr() % 32 == 16 and x.is_contiguous()
    q = mx_quantize(x)
    s = O.scale_exponents(O.f64(x))
    assert np.array_equal(O.unpack(q.data.cpu().numpy()), O.round_codes(O.f64(x), s))
    out = torch.full((n + 70 * 96,), 5.0, dtype=dtype, device="cuda")[n:].view(70, 96)
    mx_dequantize(q, dtype, out=out)
    assert np.array_equal(O.f64(out), O.fake(O.f64(x)))


def test_quantize_of_no_rows():
    q = mx_quantize(torch.empty((0, 64), device="cuda"))
    assert q.shape == (0, 64) and mx_dequantize(q).shape == (0, 64)


# ----------------------------------------------------------------- product --


def product64(a, b, offsets):
    """(value, sum of magnitudes) for a [M, K], b [G, N, K] in fp64."""
    out = np.zeros((a.shape[0], b.shape[1]))
    mag = np.zeros_like(out)
    for g in range(b.shape[0]):
        r = slice(offsets[g], offsets[g + 1])
        out[r] = a[r] @ b[g].T
        mag[r] = np.abs(a[r]) @ np.abs(b[g]).T
    return out, mag


def close(got, want, mag, n, dtype):
    tol = n * 2.0**-23 * mag + (2.0**-8 * np.abs(want) * (1 + 2.0**-7) if dtype == BF16 else 0) + 2.0**-126
    bad = np.abs(O.f64(got) - want) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), np.abs(O.f64(got) - want).max())


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [(128, 256, 64), (1, 8, 32), (128, 256, 256), (256, 256, 512), (130, 264, 96), (300, 520, 1056),
                                   (257, 128, 160), (19, 1000, 2048), (600, 264, 224), (1, 4096, 4096)])
def test_product_dense(M, N, K, out_dtype):
    a, b = mx_quantize(rand((M, K), M, spread=3)), mx_quantize(rand((N, K), N + 1, spread=3))
    got = mx_matmul(a, b, out_dtype=out_dtype)
    want, mag = product64(O.dense64(a), O.dense64(b)[None], [0, M])
    close(got, want, mag, K, out_dtype)
    assert int(device_status("cuda").item()) == 0


@pytest.mark.parametrize("G,M,N,K", [(3, 40, 72, 96), (2, 256, 256, 256), (5, 300, 136, 320)])
def test_product_dense_groups(G, M, N, K):
    a, b = mx_quantize(rand((G, M, K), 1, BF16, spread=2)), mx_quantize(rand((G, N, K), 2, BF16, spread=2))
    got = mx_matmul(a, b, out_dtype=F32)
    want, mag = product64(O.dense64(a).reshape(G * M, K), O.dense64(b), [g * M for g in range(G + 1)])
    close(got.view(G * M, N), want, mag, K, F32)


@pytest.mark.parametrize("offsets,M,N,K", [([0, 7], 7, 40, 64), ([0, 0, 1, 1, 258, 770, 770], 780, 264, 352),
                                           ([0, 300, 556], 556, 256, 512), ([5, 5, 6, 200], 260, 72, 288),
                                           ([0] * 128 + [3] * 128 + [9], 9, 64, 96), ([0, 0, 0], 4, 64, 64),
                                           # few rows on average, one group with more than a tile of them
                                           ([0] * 20 + [1, 290, 290, 291, 400, 403], 403, 264, 1056), ([2, 66], 70, 520, 224),
                                           # many
                                           ([0, 130, 131, 520], 530, 72, 544)])
def test_product_ragged(offsets, M, N, K):
    G = len(offsets) - 1
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    a, b = mx_quantize(rand((M, K), 5, spread=3), off), mx_quantize(rand((G, N, K), 6, spread=3))
    out = torch.full((M, N), 77.0, device="cuda")
    mx_matmul(a, b, off, out_dtype=F32, out=out)
    av = np.zeros((M, K))
    av[offsets[0]:offsets[-1]] = O.values(O.unpack(a.data.cpu().numpy()[offsets[0]:offsets[-1]]),
                                          O.untile(a.scales.cpu().numpy(), K, np.diff(offsets)).astype(np.int64) - 127)
    want, mag = product64(av, O.dense64(b), offsets)
    r = slice(offsets[0], offsets[-1])
    close(out[r], want[r], mag[r], K, F32)
    rest = torch.ones(M, dtype=torch.bool)
    rest[r] = False
    assert (out.cpu()[rest] == 77.0).all()  # rows of no group are left as they were


@pytest.mark.parametrize("offsets", [[0, 9, 5], [-1, 4, 8], [0, 4, 11]])
def test_product_refuses_offsets_that_are_no_partition(offsets):
    a, b = mx_quantize(rand((10, 64), 5)), mx_quantize(rand((2, 16, 64), 6))
    a = MXTensor(a.data, torch.zeros((mx_scale_bytes(2, 10, 64, True),), dtype=torch.uint8, device="cuda"))
    st = torch.zeros((1,), dtype=torch.int32, device="cuda")
    out = torch.full((10, 16), 3.0, device="cuda")
    mx_matmul(a, b, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out_dtype=F32, out=out, status=st)
    assert int(st.item()) == B.MOE_DEV_INTERNAL and (out == 3.0).all()


def test_product_nan_stays_in_its_row_and_column():
    x, w = rand((200, 128), 1), rand((40, 128), 2)
    x[3, 5], w[7, 100] = float("nan"), float("inf")
    got = mx_matmul(mx_quantize(x), mx_quantize(w), out_dtype=F32)
    bad = torch.isnan(got).cpu()
    want = torch.zeros((200, 40), dtype=torch.bool)
    want[3], want[:, 7] = True, True
    assert torch.equal(bad, want)


# ----------------------------------------------------------------- experts --


def experts64(xv, idx, gate, wg, wu, wd, dims):
    """(out, tolerance) in fp64 for quantised values xv [T, d] and weights.

    A hidden value of the kernel is off from the exact one by at most dh: the
    two products by n 2^-23 sum|terms| each, through SiLU (slope below 1.1) and
    the product of the two, plus 2^-18 of the value for the fp32 exponential,
    division and products. What that can move behind the rounding to MXFP4 is
    found by rounding both ends with both scales that the block can get. Then
    the down product's own error, each gated row's rounding (fp16, 2^-11 of the
    value or, below its normal numbers, 2^-25 of the largest of 32 columns), and
    the sum's."""
    T, d, I, k = dims
    out, tol = np.zeros((T, d)), np.zeros((T, d))
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if not 0 <= e < wg.shape[0]:
                continue
            g, u = wg[e] @ xv[t], wu[e] @ xv[t]
            dg, du = (d * 2.0**-23 * (np.abs(w[e]) @ np.abs(xv[t])) for w in (wg, wu))
            sg = g / (1 + np.exp(-g))
            h = sg * u
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(sg) * du + 2.0**-18 * np.abs(h)
            mag = np.abs(h).reshape(-1, 32), dh.reshape(-1, 32)
            q = O.fake(h)
            move = np.zeros_like(h)
            for s in (O.scale_exponents((mag[0] + mag[1]).reshape(-1)), O.scale_exponents(np.maximum(mag[0] - mag[1], 0).reshape(-1))):
                for side in (h - dh, h + dh):
                    move = np.maximum(move, np.abs(O.fake(side, s) - q))
            y = wd[e] @ q
            dy = np.abs(wd[e]) @ move + I * 2.0**-23 * (np.abs(wd[e]) @ (np.abs(q) + move))
            out[t] += gate[t, j] * y
            top = np.pad(np.abs(gate[t, j] * y) + np.abs(gate[t, j]) * dy, (0, -d % 32)).reshape(-1, 32).max(1)
            tol[t] += np.abs(gate[t, j]) * (dy + 2.0**-23 * np.abs(y)) + 2.0**-11 * 1.01 * np.abs(gate[t, j]) * (np.abs(y) + dy) + 2.0**-25 * np.repeat(top, 32)[:d] + 2.0**-126
    return out, tol + 2.0**-8 * (np.abs(out) + tol) + 2.0**-120


def layer(T, d, E, k, I, seed, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = rand((T, d), seed, dtype)
    idx = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    gate = torch.rand((T, k), generator=g, device="cuda") + 0.1
    std = 0.1
    w = [mx_quantize(rand(s, seed + i + 1, BF16, std)) for i, s in enumerate([(E, I, d), (E, I, d), (E, d, I)])]
    return x, idx, gate, w


def check_experts(x, idx, gate, w, out):
    T, d = x.shape
    I, k = w[0].shape[1], idx.shape[1]
    want, tol = experts64(O.fake(O.f64(x)), idx.cpu().numpy(), O.f64(gate), *(O.dense64(q) for q in w), (T, d, I, k))
    bad = np.abs(O.f64(out) - want) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
    # the tolerance says something: most outputs are held to a few per cent of
    # their size. (Sums over more columns may be off by as much more in the worst
    # case, which moves more of the hidden values across a border of their codes.)
    assert d > 512 or np.median(tol / (np.abs(want) + 1e-30)) < 0.1


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d,E,k,I", [(1, 32, 1, 1, 32), (1, 64, 8, 2, 96), (5, 96, 4, 4, 160), (17, 256, 8, 2, 352),
                                       (130, 160, 3, 1, 128), (260, 64, 2, 2, 64), (300, 128, 16, 8, 96),
                                       # counted by the dispatch's own blocks, per block of tokens, and by the scan
                                       (2050, 64, 5, 2, 64), (2100, 96, 7, 3, 32), (1500, 32, 9, 4, 32),
                                       (4300, 32, 256, 1, 32), (31, 2080, 4, 2, 64)])
def test_experts(T, d, E, k, I, dtype):
    x, idx, gate, w = layer(T, d, E, k, I, T + d, dtype)
    r = mx_experts(x, idx, gate, *w)
    check_experts(x, idx, gate, w, r.out)
    assert int(r.status.item()) == 0
    assert torch.equal(r.counts.long(), torch.bincount(idx.flatten().long(), minlength=E))
    assert torch.equal(r.out, mx_experts(x, idx, gate, *w).out)  # the same bits again


def test_experts_all_tokens_on_one_expert_and_one_expert_twice():
    x, idx, gate, w = layer(300, 64, 6, 2, 64, 9)
    idx[:] = 3
    r = mx_experts(x, idx, gate, *w)
    check_experts(x, idx, gate, w, r.out)
    assert r.counts.tolist() == [0, 0, 0, 600, 0, 0]


def test_experts_choices_out_of_range_are_flagged_and_add_nothing():
    x, idx, gate, w = layer(20, 64, 4, 2, 64, 10)
    idx[3, 1], idx[7, 0], idx[8] = -1, 4, 1 << 20
    r = mx_experts(x, idx, gate, *w)
    check_experts(x, idx, gate, w, r.out)
    assert int(r.status.item()) == B.MOE_DEV_INTERNAL and (r.out[8] == 0).all()


def test_experts_nan_stays_in_its_token():
    x, idx, gate, w = layer(40, 64, 4, 2, 64, 11)
    x[5, 3] = float("nan")
    r = mx_experts(x, idx, gate, *w)
    assert torch.isnan(r.out[5]).all() and int(torch.isnan(r.out).any(1).sum()) == 1


def test_experts_of_no_tokens():
    x, idx, gate, w = layer(4, 64, 4, 2, 64, 12)
    r = mx_experts(x[:0], idx[:0], gate[:0], *w)
    assert r.out.shape == (0, 64) and r.counts.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("T,dtype", [(1, BF16), (100, BF16), (150, BF16), (33, F32)])
def test_layer_with_mx_experts_is_the_router_and_then_the_experts(T, dtype):
    from sparse_mixture_experts_renorm_b200 import moe_forward

    d, E, k, I = 128, 6, 2, 64
    x, _, _, w = layer(T, d, E, k, I, 13, dtype)
    wr = rand((E, d), 14, dtype, 0.3)
    b = rand((E,), 15)
    r = moe_forward_mx(x, wr, b, *w, k, True)
    p = [rand(s, 16, dtype, 0.1) for s in ((E, I, d), (E, I, d), (E, d, I))]
    ref = moe_forward(x, wr, b, *p, k, True)
    assert torch.equal(r.topk_idx, ref.topk_idx) and torch.equal(r.topk_gate, ref.topk_gate)
    assert torch.equal(r.counts, ref.counts)
    assert abs(float(r.aux) - float(ref.aux)) < 1e-5
    assert torch.equal(r.out, mx_experts(x, r.topk_idx, r.topk_gate, *w).out)
    check_experts(x, r.topk_idx, r.topk_gate, w, r.out)


def test_experts_on_a_stream_in_a_graph_and_after_other_work_in_the_workspace():
    x, idx, gate, w = layer(70, 128, 5, 2, 96, 17)
    want = mx_experts(x, idx, gate, *w).out.clone()
    ws = torch.full((mx_workspace_size(70, 128, 5, 2, 96),), 0xFF, dtype=torch.uint8, device="cuda")  # any contents
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = mx_experts(x, idx, gate, *w, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(got.out, want)
    xs, out = torch.zeros_like(x), torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mx_experts(xs, idx, gate, *w, workspace=ws, out=out)
    for scale in (1.0, 2.0):
        xs.copy_(x * scale)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mx_experts(x * scale, idx, gate, *w).out)


def test_refusals_of_the_wrappers():
    x, idx, gate, w = layer(20, 64, 4, 2, 64, 18)
    q = mx_quantize(x)
    with pytest.raises(ValueError):
        mx_quantize(x.t())
    with pytest.raises(TypeError):
        mx_quantize(x.half())
    with pytest.raises(B.MoEError):
        mx_quantize(torch.zeros((4, 40), device="cuda"))
    with pytest.raises(ValueError):
        mx_dequantize(q, BF16, out=torch.empty((20, 64), device="cuda"))
    with pytest.raises(B.MoEError):
        mx_dequantize(MXTensor(q.data, q.scales[:100].clone()), BF16)
    with pytest.raises(ValueError):
        mx_matmul(q, MXTensor(w[0].data[0], w[0].scales[:100].clone()))
    with pytest.raises(ValueError):
        mx_matmul(q, w[0])  # one group against four
    with pytest.raises(TypeError):
        mx_matmul(x, w[0])
    with pytest.raises(TypeError):
        mx_experts(x, idx, gate, w[0], w[1], x)
    with pytest.raises(ValueError):
        mx_experts(x, idx.long(), gate, *w)
    with pytest.raises(ValueError):
        mx_experts(x, idx, gate, w[0], MXTensor(w[1].data[:, ::2], w[1].scales), w[2])
    with pytest.raises(B.MoEError):
        mx_experts(x, idx, gate, *w, workspace=torch.empty((256,), dtype=torch.uint8, device="cuda"))
    assert int(device_status("cuda").item()) == 0

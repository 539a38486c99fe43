"""The few-token and MXFP4 entry points as programs call them: prompts behind
the router, several streams, threads and graphs at once, streams as handles, and
matrices whose elements pass 32-bit numbers. Tolerances: test_mx_gpu.py and
test_few_gpu.py."""
import threading

import numpy as np
import pytest
import torch

import mx_oracle as O
import test_few_gpu as F
from sparse_mixture_experts_renorm_b200 import (few_workspace_size, moe_forward, moe_forward_few, moe_forward_mx,
                                                mx_dequantize, mx_experts, mx_matmul, mx_quantize, mx_workspace_size)
from test_mx_gpu import BF16, F32, check_experts, close, layer, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,dtype", [(2500, 64, 6, BF16), (4100, 8, 2, BF16), (2300, 20, 3, F32), (700, 16, 8, F32)])
def test_a_prompt_through_the_layer(T, E, k, dtype):
    """The dispatch behind the router, of eight tokens a block from 2048 on, against the router's own choices."""
    d, I = 128, 64
    x, _, _, w = layer(T, d, E, k, I, 70, dtype)
    wr, b = rand((E, d), 71, dtype, 0.3), rand((E,), 72)
    r = moe_forward_mx(x, wr, b, *w, k, False)
    p = [rand(s, 73, dtype, 0.1) for s in ((E, I, d), (E, I, d), (E, d, I))]
    ref = moe_forward(x, wr, b, *p, k, False)
    assert torch.equal(r.topk_idx, ref.topk_idx) and torch.equal(r.topk_gate, ref.topk_gate)
    assert torch.equal(r.counts, ref.counts) and int(r.status) == 0
    assert torch.equal(r.out, mx_experts(x, r.topk_idx, r.topk_gate, *w).out)
    some = torch.arange(0, T, T // 97, device="cuda")
    check_experts(x[some], r.topk_idx[some], r.topk_gate[some], w, r.out[some])


def several():
    """(what is called with a stream, its result when called alone) of each kind."""
    p = F.layer(7, 512, 8, 2, 768, 80, BF16)
    q = F.layer(3, 132, 5, 2, 260, 81, F32)
    x, idx, gate, w = layer(300, 256, 6, 2, 320, 82)
    y, iy, gy, v = layer(9, 256, 6, 2, 320, 83)
    wr = rand((6, 256), 84, BF16, 0.3)
    a, b = mx_quantize(rand((200, 512), 85)), mx_quantize(rand((264, 512), 86))
    word = torch.zeros((1,), dtype=torch.int32, device="cuda")
    calls = [lambda s: moe_forward_few(**p, k=2, renorm=True, stream=s).out,
             lambda s: moe_forward_few(**q, k=2, renorm=False, stream=s).out,
             lambda s: mx_experts(x, idx, gate, *w, stream=s).out,
             lambda s: mx_experts(y, iy, gy, *v, stream=s).out,
             lambda s: moe_forward_mx(x, wr, None, *w, 2, True, stream=s).out,
             lambda s: mx_matmul(a, b, status=word, stream=s),
             lambda s: mx_dequantize(mx_quantize(x, stream=s), stream=s)]
    return [(f, f(None).clone()) for f in calls], word


def test_all_of_them_on_streams_of_their_own_at_once():
    calls, word = several()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[] for _ in calls]
    for i in range(30):
        for j, (f, _) in enumerate(calls):
            got[j].append(f(streams[j] if i % 2 else streams[j].cuda_stream))
    torch.cuda.synchronize()
    for outs, (_, want) in zip(got, calls):
        assert all(torch.equal(o, want) for o in outs)
    default = torch.cuda.default_stream().cuda_stream  # 0
    assert all(torch.equal(f(default), want) for f, want in calls)
    assert int(word) == 0


def test_all_of_them_from_threads_at_once():
    calls, word = several()
    torch.cuda.synchronize()
    bad, gate = [], threading.Barrier(len(calls))

    def work(f, want):
        s = torch.cuda.Stream()
        gate.wait()
        try:
            outs = [f(s) for _ in range(30)]
            s.synchronize()
            if not all(torch.equal(o, want) for o in outs):
                bad.append("another result")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and int(word) == 0


def test_all_of_them_as_graphs_replayed_at_once():
    calls, word = several()
    torch.cuda.synchronize()
    graphs = []
    for f, want in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = [f(None) for _ in range(5)]
        graphs.append((g, outs, want, torch.cuda.Stream()))
    for _ in range(10):
        for g, _, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, outs, want, _ in graphs:
        assert all(torch.equal(o, want) for o in outs)
    assert int(word) == 0


@pytest.mark.parametrize("T,dtype", [(1, BF16), (6, F32)])
def test_one_workspace_from_call_to_call(T, dtype):
    """A server's workspace: the largest that its layers need, given to each of them in turn."""
    few = [(F.layer(T, d, E, k, I, 90 + E, dtype), k) for d, E, k, I in ((512, 8, 2, 768), (128, 40, 5, 64), (1024, 2, 1, 2048))]
    mx = [layer(T, 256, E, k, 320, 93 + E, dtype) for E, k in ((6, 2), (3, 1))]
    n = max([few_workspace_size(T, p["x"].shape[1], p["w_router"].shape[0], k, p["w_gate"].shape[1], dtype) for p, k in few]
            + [mx_workspace_size(T, 256, w[0].shape[0], idx.shape[1], 320) for _, idx, _, w in mx])
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    want = [moe_forward_few(**p, k=k, renorm=True).out for p, k in few] + [mx_experts(x, i, g, *w).out for x, i, g, w in mx]
    for _ in range(4):
        got = [moe_forward_few(**p, k=k, renorm=True, workspace=ws).out for p, k in few]
        got += [mx_experts(x, i, g, *w, workspace=ws).out for x, i, g, w in mx]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_experts_masked_by_the_lowest_number(dtype):
    """A router bias of the lowest finite number takes an expert out: it is not chosen while others are left, and
    where none are its gate is 0 (their exponentials are), renormalised or not."""
    p = F.layer(9, 256, 12, 4, 64, 104, dtype)
    p["b_router"][torch.tensor([0, 3, 4, 7, 10, 11], device="cuda")] = torch.finfo(F32).min
    for renorm in (True, False):
        r = moe_forward_few(**p, k=4, renorm=renorm)
        assert int(r.status) == 0 and set(r.topk_idx.flatten().tolist()) <= {1, 2, 5, 6, 8, 9}
        F.check_out(p, r.topk_idx, r.topk_gate, r.out, dtype)
    p["b_router"][:] = torch.finfo(F32).min
    p["b_router"][5] = 0
    for renorm in (True, False):
        r = moe_forward_few(**p, k=4, renorm=renorm)
        assert int(r.status) == 0 and (r.topk_idx[:, 0] == 5).all() and all(len(set(i)) == 4 for i in r.topk_idx.tolist())
        assert (r.topk_gate[:, 0] == 1).all() and (r.topk_gate[:, 1:] == 0).all()
        F.check_out(p, r.topk_idx, r.topk_gate, r.out, dtype)


# ------------------------------------------------ elements past 32-bit numbers --


def test_quantisation_of_more_than_2_32_elements():
    rows, cols = 65601, 65536
    x = torch.empty((rows, cols), dtype=BF16, device="cuda").normal_()
    q = mx_quantize(x)
    back = mx_dequantize(q)
    for r in (0, 32767, 32768, 65407, rows - 1):
        v = O.f64(x[r:r + 1])
        assert np.array_equal(O.f64(back[r:r + 1]), O.fake(v))
    assert torch.equal(back[-300:], mx_dequantize(mx_quantize(x[-300:])))


@pytest.mark.parametrize("M,out_dtype", [(66000, BF16), (60, F32)])
def test_a_product_with_more_than_2_32_results_or_weights(M, out_dtype):
    """66000 x 65544 results; or 60 rows (the other kernel) against 2^26 + 8 weight rows, 4.03e9 results."""
    N, K = (65544, 64) if M > 64 else ((1 << 26) + 8, 64)
    a = mx_quantize(rand((M, K), 100, spread=3))
    b = mx_quantize(torch.empty((N, K), dtype=BF16, device="cuda").normal_())
    got = mx_matmul(a, b, out_dtype=out_dtype)
    rows = sorted({0, 1, 32800 % M, M - 257 if M > 257 else 5, M - 1})
    cols = np.r_[0:300, N - 300:N]
    bv = O.values(O.unpack(b.data[cols].cpu().numpy()), untile_rows(b.scales, cols, K) - 127)
    av = O.dense64(a)[rows]
    close(got[rows][:, torch.tensor(cols, device="cuda")], av @ bv.T, np.abs(av) @ np.abs(bv).T, K, out_dtype)


def untile_rows(scales, rows, cols):
    """Scale bytes [len(rows), cols / 32] of rows of one group, cols <= 256."""
    r, b = rows[:, None], np.arange(cols // 32)[None, :]
    at = r // 128 * 1024 + b // 4 % 2 * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
    return scales[torch.tensor(at, device=scales.device)].cpu().numpy().astype(np.int64)


def test_experts_with_more_than_2_32_numbers_between_the_products():
    T, d, E, k, I = 131100, 4096, 8, 8, 32
    x, idx, gate, w = layer(T, d, E, k, I, 101)
    assert T * k * d > 1 << 32
    r = mx_experts(x, idx, gate, *w)
    assert int(r.status) == 0 and r.counts.tolist() == [T] * E
    some = [0, 65537, T - 1]
    check_experts(x[some], idx[some], gate[some], w, r.out[some])


def test_few_tokens_with_more_than_2_32_weights():
    """Only the last expert is chosen, whose weights begin past 2^32 elements; the others' are not even set."""
    T, d, E, I = 2, 16384, 17, 16384
    p = F.layer(T, d, 1, 1, I, 102, BF16)
    big = dict(p, w_router=torch.zeros((E, d), dtype=BF16, device="cuda"), b_router=torch.zeros((E,), device="cuda"))
    big["b_router"][-1] = 1
    for n in ("w_gate", "w_up", "w_down"):
        big[n] = torch.empty((E, *p[n].shape[1:]), dtype=BF16, device="cuda")
        big[n][-1] = p[n][0]
    assert (E - 1) * d * I >= 1 << 32
    r = moe_forward_few(**big, k=1, renorm=True)
    assert r.topk_idx.tolist() == [[E - 1]] * T
    F.check_out(p, torch.zeros_like(r.topk_idx), r.topk_gate, r.out, BF16)


def test_what_is_no_tensor_is_refused_as_any_wrong_argument():
    p = F.layer(4, 128, 8, 2, 64, 105, BF16)
    x, idx, gate, w = layer(4, 64, 4, 2, 64, 106)
    for name in ("x", "w_router", "w_gate", "w_up", "w_down", "b_router"):
        with pytest.raises(ValueError):
            moe_forward_few(**dict(p, **{name: p[name].tolist()}), k=2, renorm=True)
    for args in ((x.tolist(), idx, gate), (x, idx.tolist(), gate), (x, idx, gate.tolist())):
        with pytest.raises(ValueError):
            mx_experts(*args, *w)

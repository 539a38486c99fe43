"""The layer for a few tokens (moe_forward_few) against its formulas in 64 bits.

Tolerances. A sum of n products in fp32, rounded or truncated (at most 2^-23 of
the running value at each addition), is off by at most n 2^-23 sum |terms|: dl
for a logit, dg and du for the gate and up products, and likewise for the down
product. A probability is off by at most the factor exp(2 dl) (its own logit
and the sum's), and by 2^-20 for the exponentials, the sum of 256 and the
division. A hidden value is off by 1.1 dg (|u| + du) (SiLU's slope is below
1.1) + |silu| du, by c of itself for the exponential, the division and the
products (bf16: fast exponential of arguments below 20, 25 units of 2^-23, less
than 2^-18; fp32: less than 2^-20), and by its own rounding: fp32 half a step,
2^-24; bf16 keeps it in two bf16 terms, each rounded by half a step of 2^-8,
which leaves 2^-16. The last rounding adds half a step of the output."""
import numpy as np
import pytest
import torch

from sparse_mixture_experts_renorm_b200 import _binding as B
from sparse_mixture_experts_renorm_b200 import device_status, few_workspace_size, moe_forward, moe_forward_few

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def layer(T, d, E, k, I, seed, dtype, bias=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda shape, std: (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
    s = d ** -0.5
    return {"x": rand((T, d), 1.0), "w_router": rand((E, d), s), "b_router": torch.randn((E,), generator=g, device="cuda") if bias else None,
            "w_gate": rand((E, I, d), s), "w_up": rand((E, I, d), s), "w_down": rand((E, d, I), I ** -0.5)}


def logits64(p):
    x, w = f64(p["x"]), f64(p["w_router"])
    l = x @ w.T + (f64(p["b_router"]) if p["b_router"] is not None else 0)
    n = x.shape[1] + 2
    return l, n * 2.0**-23 * (np.abs(x) @ np.abs(w).T + (np.abs(f64(p["b_router"])) if p["b_router"] is not None else 0))


def check_routing(p, k, renorm, idx, gate, ties=False):
    """Choices and gates. The j-th largest of logits that are each off by at
    most dl is off by at most dl from the j-th largest exact one, and so is the
    logit of the expert chosen there from its own exact value: that value is
    within 2 dl of the j-th largest. Where all gaps are wider, as with ties, the
    choices are the exact ones."""
    l, dl = logits64(p)
    want = np.argsort(-l, axis=1, kind="stable")[:, :k]
    got = idx.cpu().numpy()
    assert ((got >= 0) & (got < l.shape[1])).all() and all(len(set(r)) == k for r in got.tolist())
    short = np.take_along_axis(l, want, 1) - np.take_along_axis(l, got, 1)
    assert (np.abs(short) <= 2 * dl.max()).all()
    assert np.array_equal(got, want) if ties else (got == want).mean() > 0.9
    want = got
    e = np.exp(l - l.max(1, keepdims=True))
    pr = e / e.sum(1, keepdims=True)
    g = np.take_along_axis(pr, want, 1)
    if renorm:
        g = g / g.sum(1, keepdims=True)
    tol = g * (np.expm1(4 * dl.max()) + 2.0**-19)
    assert (np.abs(f64(gate) - g) <= tol).all(), np.abs(f64(gate) / g - 1).max()
    return pr


def check_out(p, idx, gate, out, dtype):
    """The output for the kernel's own choices and gates."""
    x, wg, wu, wd = (f64(p[n]) for n in ("x", "w_gate", "w_up", "w_down"))
    T, d = x.shape
    I = wg.shape[1]
    half = 2.0**-8 if dtype == BF16 else 2.0**-24
    c = 2.0**-18 + 2.0**-16 if dtype == BF16 else 2.0**-20 + 2.0**-24
    idx, gate = idx.cpu().numpy(), f64(gate)
    want, tol = np.zeros((T, d)), np.zeros((T, d))
    for t in range(T):
        for j in range(idx.shape[1]):
            e = idx[t, j]
            g, u = wg[e] @ x[t], wu[e] @ x[t]
            dg, du = (d * 2.0**-23 * (np.abs(w[e]) @ np.abs(x[t])) for w in (wg, wu))
            assert np.abs(g).max() < 20
            sg = g / (1 + np.exp(-g))
            h = sg * u
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(sg) * du + c * np.abs(h) * 1.01
            y = wd[e] @ h
            dy = np.abs(wd[e]) @ dh + (I + 8) * 2.0**-23 * (np.abs(wd[e]) @ (np.abs(h) + dh))
            want[t] += gate[t, j] * y
            tol[t] += gate[t, j] * (dy + 10 * 2.0**-23 * (np.abs(y) + dy))
    tol = tol + half * (np.abs(want) + tol) + 2.0**-120
    bad = np.abs(f64(out) - want) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), np.abs(f64(out) - want).max())


def check_statistics(pr, idx, counts, aux):
    T, E = pr.shape
    n = np.bincount(idx.cpu().numpy().ravel(), minlength=E)
    assert np.array_equal(counts.cpu().numpy(), n)
    want = E * float((n / idx.numel() * pr.mean(0)).sum())
    assert abs(float(aux) - want) <= 1e-4 * want  # dl of these inputs is below 2e-5


SHAPES = [(1, 8, 1, 1, 8), (1, 64, 8, 2, 96), (2, 136, 4, 4, 40), (3, 128, 4, 2, 256), (5, 520, 13, 6, 72),
          (7, 1032, 60, 8, 24), (8, 512, 2, 1, 520), (9, 256, 16, 3, 1032), (15, 96, 128, 8, 64), (16, 264, 256, 8, 8),
          (16, 2048, 1, 1, 64), (16, 64, 2, 2, 1544), (4, 4096, 8, 2, 128)]


@pytest.mark.parametrize("T,d,E,k,I", SHAPES + [(1, 4, 3, 1, 4), (16, 2052, 5, 2, 12), (6, 12, 70, 3, 260)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layer(T, d, E, k, I, dtype):
    if dtype == BF16 and (d % 8 or I % 8):
        d, I = -(-d // 8) * 8, -(-I // 8) * 8
    for renorm in (True, False):
        p = layer(T, d, E, k, I, 7 * T + d + E, dtype, bias=renorm)
        st = torch.zeros((1,), dtype=torch.int32, device="cuda")
        n = few_workspace_size(T, d, E, k, I, dtype)
        ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # any contents
        counts, aux = torch.empty((E,), dtype=torch.int32, device="cuda"), torch.empty((1,), device="cuda")
        r = moe_forward_few(**p, k=k, renorm=renorm, status=st, workspace=ws[:n], counts=counts, aux=aux)
        assert int(st) == 0 and r.out.dtype == dtype and r.out.shape == (T, d)
        pr = check_routing(p, k, renorm, r.topk_idx, r.topk_gate)
        check_out(p, r.topk_idx, r.topk_gate, r.out, dtype)
        check_statistics(pr, r.topk_idx, counts, aux)
        assert (ws[n:] == 0xFF).all()
        again = moe_forward_few(**p, k=k, renorm=renorm)
        assert torch.equal(r.out, again.out) and torch.equal(r.topk_gate, again.topk_gate)  # the same bits


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 11, 16])
def test_all_tokens_on_the_same_experts(T, dtype):
    p = layer(T, 192, 9, 2, 320, T, dtype)
    p["b_router"] = torch.tensor([0, 0, 0, 60, 0, 0, 30, 0, 0.0], device="cuda")
    counts = torch.empty((9,), dtype=torch.int32, device="cuda")
    r = moe_forward_few(**p, k=2, renorm=False, counts=counts)
    assert counts.tolist() == [0, 0, 0, T, 0, 0, T, 0, 0]
    check_routing(p, 2, False, r.topk_idx, r.topk_gate)
    check_out(p, r.topk_idx, r.topk_gate, r.out, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_equal_logits_go_to_the_lower_expert(dtype):
    p = layer(6, 256, 40, 5, 64, 3, dtype, bias=False)
    p["w_router"][:] = p["w_router"][0]
    r = moe_forward_few(**p, k=5, renorm=True)
    assert (r.topk_idx == torch.arange(5, device="cuda", dtype=torch.int32)).all()
    check_routing(p, 5, True, r.topk_idx, r.topk_gate, ties=True)
    check_out(p, r.topk_idx, r.topk_gate, r.out, dtype)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_bad_token_is_flagged_and_stays_alone(dtype, bad):
    p = layer(7, 128, 16, 2, 96, 4, dtype)
    p["x"][3, 5] = bad
    st = torch.zeros((1,), dtype=torch.int32, device="cuda")
    r = moe_forward_few(**p, k=2, renorm=True, status=st)
    assert int(st) & B.MOE_DEV_NONFINITE
    i = r.topk_idx[3].tolist()
    assert len(set(i)) == 2 and all(0 <= e < 16 for e in i)
    keep = [0, 1, 2, 4, 5, 6]
    q = dict(p, x=p["x"][keep].contiguous())
    ref = moe_forward_few(**q, k=2, renorm=True)
    assert torch.equal(r.topk_idx[keep], ref.topk_idx) and torch.isfinite(r.out[keep]).all()
    check_out(q, ref.topk_idx, ref.topk_gate, r.out[keep], dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_same_choices_as_the_layer(dtype):
    p = layer(16, 256, 12, 3, 128, 5, dtype)
    r = moe_forward_few(**p, k=3, renorm=True)
    ref = moe_forward(**p, k=3, renorm=True)
    assert torch.equal(r.topk_idx, ref.topk_idx)
    check_out(p, ref.topk_idx, ref.topk_gate, r.out, dtype)


def test_no_tokens():
    p = layer(4, 64, 4, 2, 64, 6, BF16)
    p["x"] = p["x"][:0]
    counts = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    aux = torch.full((1,), 9.0, device="cuda")
    r = moe_forward_few(**p, k=2, renorm=True, counts=counts, aux=aux)
    assert r.out.shape == (0, 64) and counts.tolist() == [0] * 4 and float(aux) == 0


def test_two_streams_at_once_and_a_graph():
    p, q = layer(16, 1024, 8, 2, 512, 8, BF16), layer(3, 1024, 8, 2, 2048, 9, BF16)
    want = [moe_forward_few(**v, k=2, renorm=True).out.clone() for v in (p, q)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [torch.empty((few_workspace_size(v["x"].shape[0], 1024, 8, 2, v["w_gate"].shape[1], BF16),), dtype=torch.uint8, device="cuda")
          for v in (p, q)]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(40):
        for i, v in enumerate((p, q)):
            moe_forward_few(**v, k=2, renorm=True, workspace=ws[i], out=outs[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    xs, out = torch.zeros_like(p["x"]), torch.empty_like(want[0])
    idx, gate = torch.empty((16, 2), dtype=torch.int32, device="cuda"), torch.empty((16, 2), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe_forward_few(**dict(p, x=xs), k=2, renorm=True, workspace=ws[0], out=out, topk_idx=idx, topk_gate=gate)
    for scale in (1.0, 0.5):
        xs.copy_(p["x"] * scale)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, moe_forward_few(**dict(p, x=p["x"] * scale), k=2, renorm=True).out)
    assert int(device_status("cuda").item()) == 0


def test_tokens_and_output_at_an_odd_multiple_of_16_bytes():
    p = layer(5, 136, 6, 2, 200, 11, BF16)
    want = moe_forward_few(**p, k=2, renorm=True).out
    x = torch.empty((8 + 5 * 136,), dtype=BF16, device="cuda")[8:].view(5, 136)
    x.copy_(p["x"])
    out = torch.full((8 + 5 * 136 + 8,), 7.0, dtype=BF16, device="cuda")
    r = moe_forward_few(**dict(p, x=x), k=2, renorm=True, out=out[8:-8].view(5, 136))
    assert x.data_ptr() % 32 == 16 and torch.equal(r.out, want)
    assert (out[:8] == 7).all() and (out[-8:] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weights_of_experts_that_nobody_chose_are_not_read(dtype):
    p = layer(8, 128, 10, 2, 64, 12, dtype)
    p["b_router"] = torch.tensor([0, 9, 0, 0, 9, 0, 0, 0, 0, 0.0], device="cuda") * 10
    want = moe_forward_few(**p, k=2, renorm=True).out.clone()
    for n in ("w_gate", "w_up", "w_down"):
        for e in (0, 2, 3, 5, 6, 7, 8, 9):
            p[n][e] = float("nan")
    assert torch.equal(moe_forward_few(**p, k=2, renorm=True).out, want)


def test_hidden_units_and_columns_that_end_inside_a_block():
    # the rows behind an expert's last are the next expert's, or none
    for dtype, d, I in ((BF16, 24, 8), (F32, 20, 4), (F32, 12, 28)):
        p = layer(3, d, 2, 2, I, 13, dtype)
        p["w_gate"][1], p["w_up"][1], p["w_down"][1] = (p[n][1] * 1e4 for n in ("w_gate", "w_up", "w_down"))
        p["b_router"] = torch.tensor([0.0, -200.0], device="cuda")  # the second expert's gate is 0
        r = moe_forward_few(**p, k=1, renorm=True)
        assert (r.topk_idx == 0).all()
        check_out(p, r.topk_idx, r.topk_gate, r.out, dtype)


def test_more_items_than_the_joins_may_lie_behind():
    # 128 experts with a token each and 1024 blocks of columns: some 440 items for each of a block's two pipelines
    p = layer(16, 16384, 128, 8, 8, 14, BF16)
    p["b_router"] = torch.zeros_like(p["b_router"])
    r = moe_forward_few(**p, k=8, renorm=True)
    check_routing(p, 8, True, r.topk_idx, r.topk_gate)
    check_out(p, r.topk_idx, r.topk_gate, r.out, BF16)
    assert torch.equal(r.out, moe_forward_few(**p, k=8, renorm=True).out)


def test_a_prompt_through_mxfp4_experts_and_then_single_tokens():
    """As a server uses them: the experts are quantised once, the prompt and a batch of next tokens go through
    moe_forward_mx, and one user's next tokens through moe_forward_few on the weights' values."""
    from sparse_mixture_experts_renorm_b200 import moe_forward_mx, mx_dequantize, mx_experts, mx_quantize

    p = layer(90, 256, 8, 2, 320, 15, BF16)
    mx = [mx_quantize(p[n]) for n in ("w_gate", "w_up", "w_down")]
    q = dict(p, **{n: mx_dequantize(t) for n, t in zip(("w_gate", "w_up", "w_down"), mx)})
    prompt = moe_forward_mx(p["x"], p["w_router"], p["b_router"], *mx, k=2, renorm=True)
    assert int(prompt.status) == 0
    x = prompt.out[-3:].contiguous()
    for step in range(3):
        x = x / x.float().square().mean(1, keepdim=True).sqrt().to(BF16)
        few = moe_forward_few(**dict(q, x=x), k=2, renorm=True)
        batch = moe_forward_mx(x, p["w_router"], p["b_router"], *mx, k=2, renorm=True)
        assert torch.equal(few.topk_idx, batch.topk_idx)
        check_out(dict(q, x=x), few.topk_idx, few.topk_gate, few.out, BF16)
        assert torch.equal(batch.out, mx_experts(x, batch.topk_idx, batch.topk_gate, *mx).out)
        x = few.out
    assert int(device_status("cuda").item()) == 0


@pytest.mark.parametrize("change,error", [
    (dict(x=lambda p: p["x"].t().contiguous().t()), ValueError), (dict(x=lambda p: p["x"].float()), ValueError),
    (dict(x=lambda p: p["x"].half()), TypeError), (dict(x=lambda p: p["x"].cpu()), ValueError),
    (dict(w_down=lambda p: p["w_down"].transpose(1, 2)), ValueError), (dict(w_up=lambda p: p["w_up"][:, ::2]), ValueError),
    (dict(w_router=lambda p: p["w_router"][:-1]), ValueError), (dict(b_router=lambda p: p["b_router"].double()), ValueError),
    (dict(out=lambda p: torch.empty((4, 128), device="cuda")), ValueError),
    (dict(workspace=lambda p: torch.empty((64,), dtype=torch.uint8, device="cuda")), B.MoEError),
    (dict(status=lambda p: torch.zeros((2,), dtype=torch.int32, device="cuda")), ValueError),
    (dict(x=lambda p: p["x"].repeat(5, 1)), B.MoEError), (dict(k=lambda p: 9), B.MoEError), (dict(k=lambda p: 0), B.MoEError)])
def test_refusals(change, error):
    p = layer(4, 128, 8, 2, 64, 16, BF16)
    args = dict(p, k=2, renorm=True)
    args.update({n: f(p) for n, f in change.items()})
    with pytest.raises(error):
        moe_forward_few(**args)

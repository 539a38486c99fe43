"""moe_forward_few where its numbers, its queues and its callers come to their
ends; test_few_gpu.py derives the tolerances."""
import numpy as np
import pytest
import torch

from sparse_mixture_experts_renorm_b200 import _binding as B
from sparse_mixture_experts_renorm_b200 import device_status, few_workspace_size, moe_forward_few
from test_few_gpu import BF16, F32, check_out, check_routing, f64, layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 5])
def test_hidden_values_at_the_end_of_the_range(T, dtype):
    """Hidden unit i is SiLU(g_i) u_i of one column of x: exactly g_i u_i, as SiLU(90.5) is 90.5 in fp32 (e^-90.5 is
    below 2^-130). 181 * 181 has 15 bits, so 181^2 2^113, 1.9996 * 2^127, is an fp32 number between the largest of
    bf16 and that of fp32; twice that is infinite in fp32. Other tokens' outputs are zeros."""
    d = I = 64
    units = np.zeros(I)
    units[[3, 20, 41, 63]] = 181.0 * 2.0**114, -181.0 * 2.0**114, 181.0 * 2.0**113, 255.0 * 2.0**113
    down = torch.randn((1, d, I), generator=torch.Generator().manual_seed(1)).mul(2.0**-20).to(dtype)
    p = {"x": torch.zeros((T, d)), "w_router": torch.zeros((1, d)), "w_gate": torch.zeros((1, I, d)),
         "w_up": torch.zeros((1, I, d)), "w_down": down}
    p["x"][T - 1, 7] = 1
    p["w_gate"][0, :, 7] = 90.5
    p["w_up"][0, :, 7] = torch.tensor(units, dtype=F32)
    p = {n: v.to(dtype).cuda() for n, v in p.items()}
    r = moe_forward_few(**p, b_router=None, k=1, renorm=True)
    h = 90.5 * units
    assert 3.3895e38 < h[3] < 3.4028e38 and np.array_equal(f64(p["w_up"])[0, :, 7], units)
    want, mag = f64(down)[0] @ h, np.abs(f64(down)[0]) @ np.abs(h)
    # SiLU 2^-18 of the value, two bf16 terms 2^-16 (none of both in fp32, where it is 2^-20), the sum, the output
    tol = mag * ((2.0**-18 + 2.0**-16 if dtype == BF16 else 2.0**-20) + (I + 8) * 2.0**-23)
    tol += (2.0**-8 if dtype == BF16 else 2.0**-24) * (np.abs(want) + tol)
    assert (np.abs(f64(r.out[T - 1]) - want) <= tol).all()
    assert (r.out[:T - 1] == 0).all()

    p["w_up"][0, 3, 7] = 181.0 * 2.0**115  # and a unit that is infinite: so is every output it takes part in
    p["w_up"][0, 20, 7] = 0
    r = moe_forward_few(**p, b_router=None, k=1, renorm=True)
    w = down[0, :, 3].float().cuda()
    assert (w != 0).all() and torch.equal(r.out[T - 1].float(), torch.sign(w) * float("inf"))
    assert (r.out[:T - 1] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_calls_with_and_without_weights_asked_for_ahead(dtype):
    """One warp of a block asks for the experts' weights ahead of the routing where nearly all of them will be chosen
    (16 tokens, 4 experts of 6; not for 2 tokens and one), while another sets up the barriers: in turn, on one stream."""
    p, q = layer(16, 1032, 6, 4, 264, 50, dtype), layer(2, 1032, 6, 1, 264, 51, dtype)
    want = [moe_forward_few(**v, k=k, renorm=True) for v, k in ((p, 4), (q, 1))]
    for v, k, r in ((p, 4, want[0]), (q, 1, want[1])):
        check_routing(v, k, True, r.topk_idx, r.topk_gate)
        check_out(v, r.topk_idx, r.topk_gate, r.out, dtype)
    got = [[moe_forward_few(**v, k=k, renorm=True).out for v, k in ((p, 4), (q, 1))] for _ in range(100)]
    assert all(torch.equal(a, want[0].out) and torch.equal(b, want[1].out) for a, b in got)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_more_items_than_the_joins_may_lie_behind(dtype):
    """Token t chooses experts 8t .. 8t + 7, so that 128 experts have a token each: 128 * 2048 items of 16 output
    columns, on average at least three times the 256 that a pipeline's joins may lie behind its products (two
    pipelines a block in bf16), so that each one's queue goes round."""
    T, E, k, d, I = 16, 128, 8, 32768, 8
    pipelines = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    assert E * (d // 16) > 3 * 256 * pipelines
    p = layer(T, d, E, k, I, 52, dtype, bias=False)
    p["w_router"].zero_()
    p["x"][:, :T] = torch.eye(T, device="cuda").to(dtype)
    e = torch.arange(E, device="cuda")
    p["w_router"][e, e // 8] = (8 + (e % 8) / 2).to(dtype)
    r = moe_forward_few(**p, k=k, renorm=True)
    assert torch.equal(r.topk_idx.long(), e.view(T, k).flip(1))
    check_routing(p, k, True, r.topk_idx, r.topk_gate, ties=True)
    check_out(p, r.topk_idx, r.topk_gate, r.out, dtype)
    for _ in range(5):
        assert torch.equal(r.out, moe_forward_few(**p, k=k, renorm=True).out)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_call_without_a_status_word_has_its_own(dtype):
    p = layer(5, 256, 8, 2, 64, 53, dtype)
    q = dict(p, x=p["x"].clone())
    q["x"][2, 9] = float("nan")
    device_status("cuda").zero_()
    bad = moe_forward_few(**q, k=2, renorm=True)
    good = moe_forward_few(**p, k=2, renorm=True)
    again = moe_forward_few(**q, k=2, renorm=True)
    assert [int(r.status) for r in (bad, good, again)] == [B.MOE_DEV_NONFINITE, 0, B.MOE_DEV_NONFINITE]
    ws = torch.full((few_workspace_size(5, 256, 8, 2, 64, dtype),), 0xFF, dtype=torch.uint8, device="cuda")
    assert int(moe_forward_few(**p, k=2, renorm=True, workspace=ws).status) == 0
    assert int(moe_forward_few(**q, k=2, renorm=True, workspace=ws).status) == B.MOE_DEV_NONFINITE
    # a word that is given keeps what it holds
    word = torch.full((1,), 64, dtype=torch.int32, device="cuda")
    r = moe_forward_few(**q, k=2, renorm=True, workspace=ws, status=word)
    assert r.status is word and int(word) == 64 | B.MOE_DEV_NONFINITE
    # captured, each replay has its own answer; a graph needs no word made before
    x = q["x"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = moe_forward_few(**dict(p, x=x), k=2, renorm=True)
    for src, want in ((q, B.MOE_DEV_NONFINITE), (p, 0), (q, B.MOE_DEV_NONFINITE)):
        x.copy_(src["x"])
        g.replay()
        assert int(r.status) == want
    none = moe_forward_few(**dict(p, x=p["x"][:0]), k=2, renorm=True, workspace=ws.fill_(0xFF))
    assert int(none.status) == 0
    assert int(device_status("cuda").item()) == 0

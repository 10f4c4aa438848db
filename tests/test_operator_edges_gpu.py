"""Calls of the operators that their documentation allows at its ends: limits of
sizes, masks that leave nothing, several threads, autograd in a captured graph."""
import threading

import pytest
import torch

from sparse_mixture_experts_aux_b200 import (Workspace, _lib, balance_loss, balance_loss_backward,
                                             forward, matmul_fp8_block, moe_get_device_status,
                                             quantize_fp8_block, swiglu_fp8_block)
from sparse_mixture_experts_aux_b200.inputs import Workload, make_inputs
from tests.test_balance_loss_gpu import check, draw, eps_p
from tests.test_fp8_block_gpu import check_swiglu, near, operands, product, swiglu_reference
from tests.test_fp8_block_layer_gpu import quantised, run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


@pytest.mark.parametrize("T", [0, 20, 100])
def test_many_more_sequences_than_tokens(T):
    S = 30_000
    logits, idx = draw(T, 12, 2, seed=50) if T else (torch.empty(0, 12, device="cuda"),
                                                      torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    g = torch.Generator().manual_seed(51)
    cuts = torch.sort(torch.randint(0, T + 1, (S + 1,), generator=g)).values.int()
    loss, counts, tokens = balance_loss(logits, idx, cu_seqlens=cuts.cuda())
    assert torch.equal(tokens.cpu(), cuts[1:] - cuts[:-1])
    assert int(counts.sum()) == 2 * int(cuts[-1] - cuts[0])
    full = torch.nonzero(tokens).flatten().tolist()
    for s in full[:5] + full[-5:]:
        b, e = int(cuts[s]), int(cuts[s + 1])
        want = balance_loss(logits[b:e], idx[b:e])
        assert torch.equal(counts[s], want[1][0])
        assert abs(loss[s].item() - want[0].item()) <= 2.0 ** -20 * want[0].item()
    assert not loss[tokens == 0].any()


@pytest.mark.parametrize("E,k", [(8, 8), (16, 16), (32, 32), (40, 32), (1024, 32)])
def test_most_choices(E, k):
    logits, idx = draw(77, E, k, torch.bfloat16, seed=52)
    if k < E:
        check(logits, idx)
        return
    # every expert chosen by every token: f = 1/E, so the loss is the mean of sums of
    # probabilities, which are 1 to their rounding, and the gradient is zero itself
    # (the fp64 reference has 1e-18 in its place, the rounding of f - sum f p)
    loss, counts, tokens = balance_loss(logits, idx)
    d = balance_loss_backward(torch.ones(1, device="cuda"), logits, counts, tokens, k)
    assert (counts == 77).all() and not d.any()
    assert abs(loss.item() - 1.0) <= eps_p(E, 16.0)


def test_masks_that_leave_nothing():
    logits, idx = draw(5000, 30, 2, seed=53)
    cu = torch.tensor([0, 1000, 1010, 5000], dtype=torch.int32, device="cuda")
    mask = torch.zeros(5000, dtype=torch.uint8, device="cuda")
    mask[1005] = 255                              # any value but zero counts
    loss, counts, tokens, d = check(logits, idx, 0, mask, cu)
    assert tokens.tolist() == [0, 1, 0] and loss[[0, 2]].tolist() == [0, 0]
    assert torch.nonzero(d.abs().sum(1)).flatten().tolist() == [1005]


def test_rows_of_odd_addresses_and_one_expert():
    store = torch.randn(3 + 400 * 21, generator=torch.Generator().manual_seed(54)).bfloat16().cuda()
    logits = store[3:].view(400, 21)[:, :19]      # two-byte alignment, rows 21 apart
    idx = torch.topk(logits.float(), 3, dim=1).indices.int()
    a, b = check(logits, idx), check(logits.contiguous(), idx)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    one = store[:800:2].view(400, 1)              # a single expert, rows two apart
    loss, counts, tokens, d = check(one, torch.zeros(400, 1, dtype=torch.int32, device="cuda"))
    assert loss.item() == 1.0 and not d.any()


def test_autograd_in_a_captured_graph():
    # a router's step: logits, loss and backward, all replayed
    g = torch.Generator().manual_seed(55)
    x = torch.randn(700, 64, generator=g).cuda()
    W = (torch.randn(24, 64, generator=g) / 8).cuda().requires_grad_(True)
    idx = torch.topk(x @ W.detach().t(), 2, dim=1).indices.int().contiguous()

    def step():
        loss, _, _ = balance_loss(x @ W.t(), idx)
        return torch.autograd.grad(loss.sum(), W)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            want = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_inference_mode():
    with torch.inference_mode():
        logits, idx = draw(300, 16, 2, seed=56)
        loss, counts, tokens = balance_loss(logits, idx)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        again = balance_loss(logits, idx, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(again[0], loss) and torch.equal(again[1], counts)


def test_most_experts():
    # 1024 experts, a row or none each, and one with two tiles
    E, N, K = 1024, 256, 144
    lens = [i % 2 for i in range(E)]
    lens[1000] = 200
    M = sum(lens)
    cuts = [0]
    for n in lens:
        cuts.append(cuts[-1] + n)
    a, sa, w, sw = operands(M, N, K, E, seed=57)
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    near(matmul_fp8_block(a, sa, w, sw, offsets=off, out_dtype=torch.float32),
         *product(a, sa, w, sw, cuts), K)
    u = w.flip(1).contiguous()
    codes, scales = swiglu_fp8_block(a, sa, w, u, sw, sw, offsets=off)
    check_swiglu(codes, scales, *swiglu_reference(a, sa, w, sw, u, sw, cuts))
    assert moe_get_device_status() == 0


def test_threads_on_their_own_streams():
    a, sa, w, sw = operands(300, 512, 1024, 0, seed=58)
    logits, idx = draw(6000, 48, 2, seed=58)
    want = (matmul_fp8_block(a, sa, w, sw), *balance_loss(logits, idx),
            *quantize_fp8_block(logits[:, :48], 1))
    torch.cuda.synchronize()
    bad = []

    def work():
        side = torch.cuda.Stream()
        for i in range(20):
            if i % 2:
                with torch.cuda.stream(side):
                    got = (matmul_fp8_block(a, sa, w, sw), *balance_loss(logits, idx),
                           *quantize_fp8_block(logits[:, :48], 1))
            else:
                got = (matmul_fp8_block(a, sa, w, sw, stream=side),
                       *balance_loss(logits, idx, stream=side),
                       *quantize_fp8_block(logits[:, :48], 1, stream=side))
            side.synchronize()
            bad.extend(1 for x, y in zip(got, want) if not torch.equal(x, y))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and moe_get_device_status() == 0


def test_two_layer_graphs_share_a_workspace():
    ws = Workspace()
    cases = []
    for seed, T in ((60, 200), (61, 90)):         # the larger first: the buffer stays
        w = Workload("graphs", T, 256, 8, 256, 2, seed=seed)
        inp = make_inputs(w, device="cuda")
        q = quantised(inp)
        want = run(w, inp, q, ws)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out = run(w, inp, q, ws)
        cases.append((graph, out, [t.clone() for t in want], inp, q))
    for _ in range(3):
        for graph, out, want, *_ in cases:
            graph.replay()
        torch.cuda.synchronize()
        for graph, out, want, *_ in cases:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("M", [3, 200, 3000])
def test_far_scales_under_short_limits(M):
    # wherever the roles are when a limit runs out, the call ends in a status
    a, sa, w, sw = operands(M, 1040, 2048, 0, seed=62)
    sa *= 2.0 ** 70
    sw[:, ::3] *= 2.0 ** 60
    want = matmul_fp8_block(a, sa, w, sw, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert moe_get_device_status() == 0
    for limit in (1, 100, 1000, 3000, 10000):
        matmul_fp8_block(a, sa, w, sw, wait_timeout_ns=limit)
        swiglu_fp8_block(a, sa, w, w, sw, sw, wait_timeout_ns=limit)
        torch.cuda.synchronize()
        assert moe_get_device_status() in (0, _lib.MOE_ERR_DEVICE_TIMEOUT)
    again = matmul_fp8_block(a, sa, w, sw, out_dtype=torch.float32)
    assert torch.equal(again.view(torch.int32), want.view(torch.int32))   # some are inf and NaN
    assert moe_get_device_status() == 0


def test_layer_refuses_before_it_allocates_on_another_stream():
    w = Workload("refused", 16, 256, 4, 256, 2, seed=63)
    inp = make_inputs(w, device="cuda")
    with pytest.raises((TypeError, ValueError)):
        forward(inp["x"], inp["W_r"], inp["W_g"], inp["W_u"], inp["W_d"], k=2, stream="side")
    assert torch.cuda.current_stream() == torch.cuda.default_stream()

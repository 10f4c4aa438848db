"""Balance loss, per-expert counts and the loss's gradient against 64-bit references.

The reference computes each sequence by itself in fp64 and takes its gradient by
autograd (and, in one test, by differences). Tolerances:

* A probability: expf is good to 2 ulp, its argument r - max is rounded once
  (half an ulp of |r - max|, which the exponential turns into a relative error
  |r - max| 2^-24), the row's sum of E terms rounds at most E / 32 + 5 times, and
  the quotient and products a few times more. eps_p = (R + E / 32 + 16) 2^-23
  bounds the relative error, R the row's spread of logits.
* The loss is a sum of products of counts and probabilities, all positive: the
  relative error is eps_p plus the rounding of a warp's fp32 sums, one for each
  of at most `chunk` tokens, plus the final rounding.
* The gradient is c p_j (f_j - sum f_i p_i), with f less 1/E: each of the two
  terms is off by eps_p relative to its magnitude, (|f_j| + sum |f_i| p_i).
"""
import numpy as np
import pytest
import torch

from sparse_mixture_experts_aux_b200 import (Workspace, balance_loss, balance_loss_backward, forward,
                                             routing_views)
from sparse_mixture_experts_aux_b200.inputs import Workload, make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def probs64(r, gate_mode):
    empty = torch.isneginf(r).all(dim=1, keepdim=True)
    r = torch.where(empty, torch.zeros_like(r), r)  # before the softmax: its gradient would be NaN
    if gate_mode == 2:
        r = torch.nn.functional.logsigmoid(r)
    p = torch.softmax(r, dim=1)
    return torch.where(empty, torch.zeros_like(p), p)


def reference(logits, idx, gate_mode, mask, cu, dloss):
    """loss, counts, tokens, dlogits and the magnitudes behind the tolerances, in fp64 on the CPU."""
    r = logits.detach().cpu().double()
    idx = idx.cpu().long()
    T, E = r.shape
    k = idx.shape[1]
    cuts = [0, T] if cu is None else cu.cpu().tolist()
    S = len(cuts) - 1
    loss, counts, tokens = torch.zeros(S).double(), torch.zeros(S, E, dtype=torch.int32), []
    d, mag = torch.zeros(T, E).double(), torch.zeros(T, E).double()
    for s in range(S):
        live = [t for t in range(cuts[s], cuts[s + 1]) if mask is None or bool(mask[t])]
        tokens.append(len(live))
        if not live:
            continue
        n = len(live)
        flat = idx[live].reshape(-1)
        flat = flat[(flat >= 0) & (flat < E)]
        counts[s] = torch.bincount(flat, minlength=E).int()
        x = r[live].clone().requires_grad_(True)
        p = probs64(x, gate_mode)
        f = counts[s].double() / (n * k)
        value = E * (f * p.mean(dim=0)).sum()
        g, = torch.autograd.grad(value, x)
        loss[s] = value.detach()
        d[live] = g * float(dloss[s])
        p = p.detach()
        fc = (f - 1.0 / E).abs()
        mag[live] = abs(float(dloss[s])) * E / n * p * (fc + (fc * p).sum(dim=1, keepdim=True))
    return loss, counts, torch.tensor(tokens, dtype=torch.int32), d, mag


def eps_p(E, spread):
    return (spread + E / 32 + 16) * 2.0 ** -23


def check(logits, idx, gate_mode=0, mask=None, cu=None, seed=0, spread=None):
    T, E = logits.shape
    S = 1 if cu is None else cu.numel() - 1
    g = torch.Generator().manual_seed(seed)
    dloss = torch.rand(S, generator=g) + 0.5
    loss, counts, tokens = balance_loss(logits, idx, gate_mode, token_mask=mask, cu_seqlens=cu)
    d = balance_loss_backward(dloss.cuda(), logits, counts, tokens, idx.shape[1], gate_mode,
                              token_mask=mask, cu_seqlens=cu)
    torch.cuda.synchronize()
    rl, rc, rn, rd, mag = reference(logits, idx, gate_mode, mask, cu, dloss)
    assert torch.equal(counts.cpu(), rc)
    assert torch.equal(tokens.cpu(), rn)
    if spread is None:
        fin = logits.float()[torch.isfinite(logits.float())]
        spread = float(fin.max() - fin.min()) if fin.numel() else 0.0
    eps = eps_p(E, spread)
    chunk = max(32, -(-T // 148))
    assert ((loss.cpu().double() - rl).abs() <= (eps + chunk * 2.0 ** -24 + 2.0 ** -23) * rl.abs()).all()
    out_eps = torch.finfo(logits.dtype).eps / 2
    tiny = torch.finfo(logits.dtype).tiny
    err = (d.cpu().double() - rd).abs()
    assert (err <= 4 * eps * mag + out_eps * rd.abs() + tiny).all(), float((err - 4 * eps * mag).max())
    return loss, counts, tokens, d


def draw(T, E, k, dtype=torch.float32, seed=0, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn(T, E, generator=g) * scale).to(dtype)
    idx = torch.argsort(logits.float(), dim=1, descending=True, stable=True)[:, :k].int()
    return logits.cuda(), idx.contiguous().cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate_mode", [0, 1, 2])
@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 8, 2), (3, 2, 1), (31, 5, 3), (64, 8, 2), (33, 9, 2), (70, 16, 4), (129, 17, 1),
    (65, 32, 8), (100, 33, 2), (37, 64, 1), (150, 127, 6), (200, 256, 8), (41, 257, 3), (40, 512, 4),
    (35, 513, 32), (33, 1024, 2)])
def test_shapes(T, E, k, gate_mode, dtype):
    check(*draw(T, E, k, dtype, seed=T + E), gate_mode)


@pytest.mark.parametrize("T,E,k", [(5000, 8, 2), (4737, 64, 1), (9001, 256, 8), (2000, 600, 2)])
@pytest.mark.parametrize("gate_mode", [0, 2])
def test_many_chunks(T, E, k, gate_mode):
    check(*draw(T, E, k, seed=1), gate_mode)


@pytest.mark.parametrize("E,k", [(4, 2), (12, 2), (40, 3), (300, 4)])
@pytest.mark.parametrize("T,cuts", [
    (100, [0, 100]),
    (100, [0, 1, 1, 50, 50, 99, 100]),            # empty sequences between others
    (100, [0, 0, 0, 100, 100]),                   # empty at both ends
    (100, [10, 30, 60]),                          # tokens before the first and behind the last
    (6000, [0, 1, 700, 701, 701, 3000, 5900]),    # several chunks, ends inside a chunk
    (6000, list(range(0, 6001, 50))),             # many short ones
    (4736, [0, 32, 64, 64, 4736]),                # ends on chunk borders
])
def test_ragged_sequences(T, cuts, E, k):
    logits, idx = draw(T, E, k, seed=3)
    cu = torch.tensor(cuts, dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(4)
    mask = torch.rand(T, generator=g) < 0.8
    if len(cuts) > 2:
        mask[cuts[1]:cuts[2]] = False             # a sequence with every token masked
    for gate_mode in (0, 2):
        _, _, _, d = check(logits, idx, gate_mode, mask.cuda(), cu)
        outside = torch.ones(T, dtype=torch.bool)
        outside[cuts[0]:cuts[-1]] = False
        outside |= ~mask
        assert (d.cpu()[outside] == 0).all()


def test_no_tokens():
    logits = torch.empty(0, 8, device="cuda")
    idx = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    loss, counts, tokens = balance_loss(logits, idx)
    assert loss.tolist() == [0.0] and counts.tolist() == [[0] * 8] and tokens.tolist() == [0]
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    loss, counts, tokens = balance_loss(logits, idx, cu_seqlens=cu)
    assert loss.tolist() == [0.0] * 3 and not counts.any() and tokens.tolist() == [0] * 3
    d = balance_loss_backward(torch.ones(1, device="cuda"), logits, counts[:1].contiguous(),
                              tokens[:1].contiguous(), 2)
    assert d.shape == (0, 8)


def test_strided_rows():
    wide = torch.randn(300, 40, generator=torch.Generator().manual_seed(5)).cuda()
    logits = wide[:, 3:20]                        # neither dense nor 16-byte aligned
    idx = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :2].int().contiguous()
    a = check(logits, idx)
    b = check(logits.contiguous(), idx)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_unrouted_and_repeated_choices():
    logits, idx = draw(500, 12, 3, seed=6)
    idx[::3, 1] = -1                              # dropped slots
    idx[5] = -1                                   # a token without any expert
    idx[7] = 4                                    # the same expert three times
    idx[9, 0], idx[9, 1] = 12, 2 ** 30            # outside
    check(logits, idx)


@pytest.mark.parametrize("gate_mode", [0, 2])
def test_masked_places_may_hold_anything(gate_mode):
    logits, idx = draw(400, 20, 2, seed=7)
    mask = torch.ones(400, dtype=torch.bool)
    mask[10:60] = False
    clean = check(logits, idx, gate_mode, mask.cuda())
    for v in (float("nan"), float("inf"), float("-inf"), torch.finfo(torch.float32).min):
        bad = logits.clone()
        bad[10:60] = v
        loss, counts, tokens = balance_loss(bad, idx, gate_mode, token_mask=mask.cuda())
        d = balance_loss_backward(torch.ones(1, device="cuda"), bad, counts, tokens, 2, gate_mode,
                                  token_mask=mask.cuda())
        assert torch.equal(loss, clean[0]) and torch.equal(counts, clean[1])
        assert (d[10:60] == 0).all() and torch.isfinite(d).all()


@pytest.mark.parametrize("gate_mode", [0, 2])
@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min, -3e4])
def test_experts_masked_by_their_logit(gate_mode, low):
    logits, idx = draw(200, 24, 2, seed=8)
    logits[:, 5] = low                            # an expert nobody may use
    logits[3, 1:] = low                           # a row with one expert left
    check(logits, idx, gate_mode, spread=40.0)


def test_rows_of_minus_infinity_and_nan():
    logits, idx = draw(200, 24, 2, seed=9)
    logits[11] = float("-inf")
    for gate_mode in (0, 2):
        _, _, tokens, d = check(logits, idx, gate_mode)
        assert tokens.item() == 200 and (d[11] == 0).all()
    logits[11, 3] = float("nan")
    loss, counts, tokens = balance_loss(logits, idx)
    d = balance_loss_backward(torch.ones(1, device="cuda"), logits, counts, tokens, 2)
    assert torch.isnan(loss).all() and torch.isnan(d[11]).all()
    assert torch.isfinite(d[:11]).all() and torch.isfinite(d[12:]).all()


@pytest.mark.parametrize("gate_mode", [0, 2])
def test_far_logits_keep_their_ratios(gate_mode):
    # every logit of a row far below zero (sigmoid underflows) or far above
    logits, idx = draw(96, 16, 2, seed=10)
    logits[:32] -= 150.0
    logits[32:64] += 80.0
    # R: the row's own spread plus the rounding of the shifted logits, which both sides share
    check(logits, idx, gate_mode, spread=160.0)


def test_uniform_routing_is_one_and_flat():
    E, T = 8, 64
    idx = (torch.arange(T * 2) % E).int().view(T, 2).cuda()
    loss, counts, tokens = balance_loss(torch.zeros(T, E, device="cuda"), idx)
    assert loss.item() == 1.0 and (counts == 16).all()
    d = balance_loss_backward(torch.ones(1, device="cuda"), torch.randn(T, E, device="cuda"), counts,
                              tokens, 2)
    assert (d == 0).all()                         # f = 1/E for every expert


@pytest.mark.parametrize("gate_mode", [0, 2])
def test_gradient_against_differences(gate_mode):
    # central differences of the fp64 loss: the truncation error is h^2 / 6 times a
    # third derivative of order one; h = 1e-4 leaves 1e-8 of it
    logits, idx = draw(12, 6, 2, seed=11)
    loss, counts, tokens = balance_loss(logits, idx, gate_mode)
    d = balance_loss_backward(torch.ones(1, device="cuda"), logits, counts, tokens, 2, gate_mode)
    r = logits.cpu().double()
    f = counts.cpu().double()[0] / 24
    for t in range(12):
        for e in range(6):
            v = []
            for h in (1e-4, -1e-4):
                x = r.clone()
                x[t, e] += h
                v.append(6 * float((f * probs64(x, gate_mode).mean(dim=0)).sum()))
            assert abs((v[0] - v[1]) / 2e-4 - float(d[t, e])) <= 1e-6 * 6 / 12


def test_autograd():
    logits, idx = draw(300, 16, 2, seed=12)
    cu = torch.tensor([0, 100, 100, 300], dtype=torch.int32).cuda()
    logits.requires_grad_(True)
    loss, counts, tokens = balance_loss(logits, idx, cu_seqlens=cu)
    assert not counts.requires_grad and not tokens.requires_grad
    (0.01 * loss.sum()).backward()                # an expanded gradient
    want = balance_loss_backward(torch.full((3,), 0.01, device="cuda"), logits.detach(), counts,
                                 tokens, 2, cu_seqlens=cu)
    assert torch.equal(logits.grad, want)
    with torch.no_grad():
        again = balance_loss(logits, idx, cu_seqlens=cu)
    assert torch.equal(again[0], loss.detach()) and not again[0].requires_grad


def test_gradient_reaches_the_router_weights():
    # a router's training step: logits = x W_r^T + b; W_r and the bias get gradients
    g = torch.Generator().manual_seed(13)
    x = torch.randn(256, 64, generator=g).cuda()
    W = (torch.randn(8, 64, generator=g) / 8).cuda().requires_grad_(True)
    b = torch.zeros(8, device="cuda", requires_grad=True)
    logits = x @ W.t() + b
    idx = torch.argsort(logits.detach(), dim=1, descending=True, stable=True)[:, :2].int().contiguous()
    loss, counts, _ = balance_loss(logits, idx)
    loss.sum().backward()
    W64 = W.detach().double().requires_grad_(True)
    b64 = b.detach().double().requires_grad_(True)
    p = torch.softmax(x.double() @ W64.t() + b64, dim=1)
    (8 * (counts[0].double() / 512 * p.mean(dim=0)).sum()).backward()
    # the product x^T dlogits sums 256 terms in fp32: 256 2^-24 of their magnitudes, and eps_p of each
    bound = (256 + 4 * 40) * 2.0 ** -23 * float(W64.grad.abs().max()) * 16
    assert (W.grad.double() - W64.grad).abs().max() <= bound
    assert (b.grad.double() - b64.grad).abs().max() <= bound


def test_forward_then_loss_agrees_with_the_layers_statistic():
    w = Workload("balance after forward", 384, 256, 8, 256, 2, seed=5)
    inp = make_inputs(w, device="cuda:0")
    ws = Workspace()
    _, aux, counts = forward(inp["x"], inp["W_r"], inp["W_g"], inp["W_u"], inp["W_d"], k=2, workspace=ws)
    v = routing_views(ws.buf, inp["x"], inp["W_g"], 8, 2)
    loss, mine, tokens = check(v["logits"], v["topk_idx"])[:3]
    assert torch.equal(mine[0], counts) and tokens.item() == 384
    assert abs(loss.item() - aux.item()) <= (eps_p(8, 16.0) + 64 * 2.0 ** -24) * aux.item()


def test_same_bits_on_repeat_stream_workspace_and_graph():
    logits, idx = draw(9001, 64, 4, seed=14)
    cu = torch.tensor([0, 100, 4000, 9001], dtype=torch.int32).cuda()
    first = balance_loss(logits, idx, cu_seqlens=cu)
    ws = Workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = balance_loss(logits, idx, cu_seqlens=cu, workspace=ws, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    one = torch.ones(3, device="cuda")
    want = balance_loss_backward(one, logits, first[1], first[2], 4, cu_seqlens=cu)
    static = logits.clone()
    graphs, outs = [], []
    for _ in range(2):                            # two graphs, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            l, c, n = balance_loss(static, idx, cu_seqlens=cu)
            d = balance_loss_backward(one, static, c, n, 4, cu_seqlens=cu)
        graphs.append(g)
        outs.append((l, c, n, d))
    static.copy_(logits * 0.5)
    half = balance_loss(static, idx, cu_seqlens=cu)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], half[0]) and torch.equal(o[1], half[1])
    static.copy_(logits)
    for g in reversed(graphs):
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], first[0]) and torch.equal(o[3], want)


def test_two_streams_at_once():
    cases = [draw(3000 + 500 * i, 32, 2, seed=20 + i) for i in range(4)]
    want = [balance_loss(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(10):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(balance_loss(*c))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        for a, b in zip(o, want[i % 4]):
            assert torch.equal(a, b)


def test_refusals():
    logits, idx = draw(16, 8, 2)
    ok = dict(token_mask=None, cu_seqlens=None)
    with pytest.raises(RuntimeError):
        balance_loss(logits.cpu(), idx)
    with pytest.raises(TypeError):
        balance_loss(logits.half(), idx)
    with pytest.raises(TypeError):
        balance_loss(logits, idx.long())
    with pytest.raises(RuntimeError):
        balance_loss(logits, idx[:8])
    with pytest.raises(RuntimeError):
        balance_loss(logits.t(), idx[:8])
    with pytest.raises(RuntimeError):
        balance_loss(logits[0], idx)
    with pytest.raises(RuntimeError):
        balance_loss(logits, torch.zeros(16, 9, dtype=torch.int32, device="cuda"))   # k > E
    with pytest.raises(RuntimeError):
        balance_loss(logits, idx, gate_mode=3)
    with pytest.raises(RuntimeError):
        balance_loss(logits, idx, token_mask=torch.ones(15, dtype=torch.bool, device="cuda"))
    with pytest.raises(TypeError):
        balance_loss(logits, idx, token_mask=torch.ones(16, device="cuda"))
    with pytest.raises(TypeError):
        balance_loss(logits, idx, cu_seqlens=torch.tensor([0, 16], device="cuda"))
    with pytest.raises(RuntimeError):
        balance_loss(logits, idx, cu_seqlens=torch.tensor([0], dtype=torch.int32, device="cuda"))
    with pytest.raises(RuntimeError):
        balance_loss(logits.clone().requires_grad_(True), idx, stream=torch.cuda.Stream())
    loss, counts, tokens = balance_loss(logits, idx, **ok)
    with pytest.raises(RuntimeError):
        balance_loss_backward(torch.ones(2, device="cuda"), logits, counts, tokens, 2)
    with pytest.raises(RuntimeError):
        balance_loss_backward(torch.ones(1, device="cuda"), logits, counts[:, :4], tokens, 2)


def test_careless_sequence_bounds_stay_inside_the_batch():
    # values outside 0..T are read as 0 or T: [-5, 8), [8, 99)
    logits, idx = draw(16, 8, 2, seed=15)
    bad = torch.tensor([-5, 8, 99], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 8, 16], dtype=torch.int32, device="cuda")
    for a, b in zip(balance_loss(logits, idx, cu_seqlens=bad), balance_loss(logits, idx, cu_seqlens=good)):
        assert torch.equal(a, b)


def test_long_batch_sums_stay_exact():
    # 200000 tokens of equal rows: P_i is the row's probability itself, so the loss
    # is known; fp32 sums of a warp hold at most 1352 / 32 rows
    T, E = 200_000, 16
    row = torch.randn(1, E, generator=torch.Generator().manual_seed(16))
    logits = row.expand(T, E).contiguous().cuda()
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    loss, counts, tokens = balance_loss(logits, idx)
    want = E * float(torch.softmax(row.double(), dim=1)[0, 0])
    assert counts[0, 0].item() == T and tokens.item() == T
    assert abs(loss.item() - want) <= (eps_p(E, 6.0) + 43 * 2.0 ** -24) * want
    assert np.isfinite(loss.item())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate_mode", [0, 1, 2])
@pytest.mark.parametrize("E", [7, 12, 40, 300])
def test_rows_far_from_zero(E, gate_mode, dtype):
    # finite rows whose largest logit is far from zero, up to the type's last value:
    # r - max rounds by half an ulp of itself whatever max is, so eps_p holds with R
    # the differences that still count (e^-100 of the largest term is zero in fp32).
    # In the kernel's own operations: r - max and its product with log2 e round once
    # each, log2 e itself is off by 0.22 2^-24, in all 1.11 |r - max| 2^-23; what is
    # above R 2^-23 (below 10 2^-23 where the term is not zero), two ulp of 2^x, one of
    # the reciprocal and the products' halves fit into the 16 2^-23
    top = torch.finfo(dtype).max
    far = [s * v for v in (1e4, 1e9, 1e10, 1e12, 1e30, top) for s in (1.0, -1.0)]
    logits, idx = draw(4 * len(far), E, 2, dtype, seed=17)
    for i, v in enumerate(far):
        logits[4 * i] = v                         # equal logits: as likely as one another
        logits[4 * i + 1] = (logits[4 * i + 1].float() + v).clamp(-top, top).to(dtype)
        logits[4 * i + 2, 3] = v                  # one among ordinary ones
    check(logits, idx, gate_mode, spread=100.0)


def test_forward_mode_is_refused():
    # a dual tensor needs no gradient by its own account; its tangent must not vanish
    import torch.autograd.forward_ad as fwAD
    logits, idx = draw(16, 8, 2)
    loss, counts, tokens = balance_loss(logits, idx)
    one = torch.ones(1, device="cuda")
    with fwAD.dual_level():
        for t in (logits, logits.clone().requires_grad_(True)):
            dual = fwAD.make_dual(t, torch.ones_like(logits))
            with pytest.raises(RuntimeError):
                balance_loss(dual, idx)
            with pytest.raises(RuntimeError):
                balance_loss_backward(one, dual, counts, tokens, 2)
        with pytest.raises(RuntimeError):
            balance_loss_backward(fwAD.make_dual(one, one), logits, counts, tokens, 2)
        assert torch.equal(balance_loss(logits, idx)[0], loss)
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda r: balance_loss(r, idx)[0], (logits,), (torch.ones_like(logits),))


@pytest.mark.parametrize("T,E", [(1 << 26, 8), (1 << 24, 100), (1 << 22, 600)])
def test_rounding_of_the_sums_does_not_grow_with_the_batch(T, E):
    # equal rows: the mean of T probabilities is the probability, which a batch of one
    # row gives with the same rounding. 64 fp32 additions, two levels of a warp's own,
    # the probability's and the result's rounding are what may differ
    row = torch.randn(1, E, generator=torch.Generator().manual_seed(16)).to(torch.bfloat16).cuda()
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    one = balance_loss(row, idx[:1])[0].item()
    loss, counts, tokens = balance_loss(row.expand(T, E).contiguous(), idx)
    assert counts[0, 0].item() == T and tokens.item() == T
    assert abs(loss.item() - one) <= 68 * 2.0 ** -24 * one


@pytest.mark.parametrize("T,E,k", [(700_001, 12, 2), (350_003, 200, 3), (80_007, 600, 2)])
def test_chunks_of_several_spans(T, E, k):
    # sequences that hold several spans of rows, end inside one, or inside a chunk
    g = torch.Generator(device="cuda").manual_seed(18)
    logits = torch.randn(T, E, generator=g, device="cuda") * 2
    idx = torch.topk(logits, k, dim=1).indices.int()
    mask = torch.rand(T, generator=g, device="cuda") < 0.8
    cuts = [0, T // 2 + 5, T // 2 + 700, T - 3]
    loss, counts, tokens = balance_loss(logits, idx, token_mask=mask,
                                        cu_seqlens=torch.tensor(cuts, dtype=torch.int32, device="cuda"))
    for s, (b, e) in enumerate(zip(cuts[:-1], cuts[1:])):
        live = mask[b:e]
        n = int(live.sum())
        c = torch.bincount(idx[b:e][live].reshape(-1).long(), minlength=E)
        p = torch.softmax(logits[b:e][live].double(), dim=1).mean(dim=0)
        want = float(E * (c.double() / (n * k) * p).sum())
        assert tokens[s].item() == n and torch.equal(counts[s].long(), c)
        assert abs(loss[s].item() - want) <= (eps_p(E, 24.0) + 66 * 2.0 ** -24 + 2.0 ** -23) * want

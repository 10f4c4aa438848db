"""The layer on block-scaled FP8 experts (MOE_WEIGHTS_FP8_BLOCK), stage by stage
against fp64 on what the stage before left in the workspace: the routed rows'
codes bit by bit, H within the bounds of test_fp8_block_gpu.py, and y within the
roundings of its own stage; then the routing and the balance loss behind it."""
import ctypes

import pytest
import torch

from sparse_mixture_experts_aux_b200 import (Workspace, _lib, balance_loss, forward, make_dims,
                                             moe_get_device_status, quantize_fp8_block,
                                             routing_views)
from sparse_mixture_experts_aux_b200.inputs import Workload, make_inputs
from tests.test_fp8_block_gpu import (ceil, check_swiglu, product, reference_codes, sum_eps,
                                      swiglu_reference)

pytestmark = pytest.mark.gpu

CASES = [
    Workload("one token", 1, 256, 8, 192, 2, seed=1),
    Workload("decode", 32, 512, 8, 1024, 2, seed=2),
    Workload("odd widths", 77, 320, 5, 448, 3, seed=3),
    Workload("many experts", 200, 256, 64, 128, 6, seed=4, gate_mode=2, selection_bias=True),
    Workload("several tiles", 700, 384, 4, 320, 2, seed=5),
    Workload("capacity", 400, 256, 8, 256, 2, capacity_factor=0.6, zipf_bias=True, seed=6),
    Workload("raw gates", 65, 128, 16, 64, 1, seed=7, gate_mode=1),
]


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def quantised(inp):
    out, scales = {}, []
    for name in ("W_g", "W_u", "W_d"):
        out[name], s = quantize_fp8_block(inp[name], 128)
        out[name + "_s"] = s
        scales.append(s.reshape(-1))
    out["scales"] = torch.cat(scales)
    return out


def run(w, inp, q, ws, **kw):
    return forward(inp["x"], inp["W_r"], q["W_g"], q["W_u"], q["W_d"], k=w.k,
                   capacity_factor=w.capacity_factor, router_bias=inp["router_bias"],
                   selection_bias=inp["selection_bias"], gate_mode=w.gate_mode, workspace=ws,
                   weight_scales=q["scales"], fp8_block=True, **kw)


@pytest.mark.parametrize("w", CASES, ids=lambda w: w.name)
def test_stages(w):
    inp = make_inputs(w, device="cuda")
    q = quantised(inp)
    ws = Workspace()
    y, aux, counts = run(w, inp, q, ws)
    torch.cuda.synchronize()
    assert moe_get_device_status() == 0
    v = routing_views(ws.buf, inp["x"], q["W_g"], w.E, w.k, w.capacity_factor, fp8_block=True)
    pos = v["slot_pos"].long()
    kept = pos >= 0
    token = torch.arange(w.T, device="cuda")[:, None].expand(-1, w.k)[kept]
    rows, experts, gates = pos[kept], v["topk_idx"].long()[kept], v["gates"][kept]
    order = torch.argsort(rows)
    rows, experts, gates, token = rows[order], experts[order], gates[order], token[order]

    # the permuted rows are x's codes
    rc, rs = reference_codes(inp["x"][None], 1)
    assert torch.equal(v["xq"][rows].cpu(), rc[0][token.cpu()])
    assert torch.equal(v["xscale"][rows].cpu(), rs[0][token.cpu()])

    # H and y of those rows, expert by expert
    offsets = [0] + torch.cumsum(torch.bincount(experts, minlength=w.E), 0).tolist()
    xq, xs, hq, hs = (v[n][rows] for n in ("xq", "xscale", "hq", "hscale"))
    h, dh = swiglu_reference(xq, xs, q["W_g"], q["W_g_s"], q["W_u"], q["W_u_s"], offsets)
    check_swiglu(hq, hs, h, dh)
    c, mag = product(hq, hs, q["W_d"], q["W_d_s"], offsets)
    g = gates.double()[:, None]
    want = torch.zeros(w.T, w.d, dtype=torch.float64, device="cuda").index_add_(0, token, g * c)
    # each row is rounded to bf16 on its way and the sum once more, the k terms are added in fp32
    half = 2.0 ** -8
    row_err = sum_eps(w.d_e) * g * mag * (1 + half) + half * (g * c).abs()
    err = torch.zeros_like(want).index_add_(0, token, row_err + w.k * 2.0 ** -24 * (g * c).abs())
    bound = err * (1 + half) + half * want.abs() + 1e-30
    assert ((y.double() - want).abs() <= bound).all()

    # routing does not depend on the experts' format
    y2, aux2, counts2 = forward(inp["x"], inp["W_r"], inp["W_g"], inp["W_u"], inp["W_d"], k=w.k,
                                capacity_factor=w.capacity_factor, router_bias=inp["router_bias"],
                                selection_bias=inp["selection_bias"], gate_mode=w.gate_mode)
    assert torch.equal(aux, aux2) and torch.equal(counts, counts2)
    # and the balance loss takes up where the layer left its routing
    logits = v["logits"] if inp["router_bias"] is None else v["logits"] + inp["router_bias"]
    loss, mine, tokens = balance_loss(logits, v["topk_idx"], gate_mode=w.gate_mode)
    assert torch.equal(mine[0], counts) and tokens.item() == w.T
    assert abs(loss.item() - aux.item()) <= 1e-5 * aux.item()
    # four roundings to E4M3 apart from the bf16 layer: 2^-4 / sqrt(3) of a value each in the
    # mean square, six of them on the way to y (see test_experts_end_to_end)
    rel = float((y.double() - y2.double()).norm() / y2.double().norm())
    assert rel <= (2 * 1.28 ** 2 + 4) ** 0.5 * 2.0 ** -4 / 3 ** 0.5


def test_repeat_graph_and_no_alloc_give_the_same_bits():
    w = CASES[1]
    inp = make_inputs(w, device="cuda")
    q = quantised(inp)
    ws = Workspace()
    want = run(w, inp, q, ws)
    again = run(w, inp, q, Workspace())
    for a, b in zip(want, again):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, aux, counts = run(w, inp, q, ws)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(counts, want[2])
    dims = make_dims(w.T, w.d, w.d_e, dtype=_lib.MOE_BF16, weight_format=_lib.MOE_WEIGHTS_FP8_BLOCK,
                     weight_scales=q["scales"], stream=torch.cuda.current_stream().cuda_stream)
    y.zero_()
    _lib.moe_forward_no_alloc(dims, inp["x"], inp["W_r"], q["W_g"], q["W_u"], q["W_d"], None, w.E,
                              w.k, 0.0, y, aux, counts)
    torch.cuda.synchronize()
    assert torch.equal(y, want[0])


@pytest.mark.parametrize("w", [CASES[1], CASES[4], CASES[5]], ids=lambda w: w.name)
def test_debug_build_is_silent_and_bit_identical(w):
    inp = make_inputs(w, device="cuda")
    q = quantised(inp)
    ws = Workspace()
    want = run(w, inp, q, ws)
    dbg, p = _lib.load_debug(), _lib._ptr
    buf = torch.empty_like(ws.buf)
    dims = make_dims(w.T, w.d, w.d_e, 0, _lib.MOE_BF16, inp["router_bias"], buf, buf.numel(),
                     torch.cuda.current_stream().cuda_stream,
                     weight_format=_lib.MOE_WEIGHTS_FP8_BLOCK, weight_scales=q["scales"])
    got = [torch.empty_like(t) for t in want]
    st = dbg.moe_forward(ctypes.byref(dims), p(inp["x"]), p(inp["W_r"]), p(q["W_g"]), p(q["W_u"]),
                         p(q["W_d"]), None, w.E, w.k, w.capacity_factor, *map(p, got))
    assert st == _lib.MOE_OK
    torch.cuda.synchronize()
    assert dbg.moe_get_device_status() == _lib.MOE_OK
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_empty_batch():
    w = CASES[0]
    inp = make_inputs(w, device="cuda")
    q = quantised(inp)
    y, aux, counts = forward(inp["x"][:0], inp["W_r"], q["W_g"], q["W_u"], q["W_d"], k=2,
                             weight_scales=q["scales"], fp8_block=True)
    assert y.shape == (0, w.d) and aux.item() == 0 and not counts.any()


def test_timeout_is_reported():
    w = CASES[4]
    inp = make_inputs(w, device="cuda")
    q = quantised(inp)
    ws = Workspace()
    want = run(w, inp, q, ws)[0]
    torch.cuda.synchronize()
    run(w, inp, q, ws, wait_timeout_ns=1)
    torch.cuda.synchronize()
    v = routing_views(ws.buf, inp["x"], q["W_g"], w.E, w.k, fp8_block=True)
    assert int(v["status"][0]) != 0
    assert moe_get_device_status() == _lib.MOE_ERR_DEVICE_TIMEOUT
    assert torch.equal(run(w, inp, q, ws)[0], want)
    assert moe_get_device_status() == 0


def test_refusals():
    w = CASES[1]
    inp = make_inputs(w, device="cuda")
    q = quantised(inp)
    args = (inp["x"], inp["W_r"], q["W_g"], q["W_u"], q["W_d"])
    with pytest.raises(RuntimeError):
        forward(*args, k=2, weight_scales=q["scales"][:-1], fp8_block=True)
    with pytest.raises(RuntimeError):
        forward(*args, k=2, weight_scales=q["scales"], fp8_block=True, act_fp8=True)
    with pytest.raises(RuntimeError):
        forward(inp["x"], inp["W_r"], inp["W_g"], inp["W_u"], inp["W_d"], k=2,
                weight_scales=q["scales"], fp8_block=True)
    with pytest.raises(RuntimeError):
        forward(inp["x"].float(), *args[1:], k=2, weight_scales=q["scales"], fp8_block=True)
    assert ceil(w.d, 128) == 4


def test_weights_of_other_shapes_and_types_are_refused():
    w = CASES[2]                                  # d = 320, d_e = 448
    inp = make_inputs(w, device="cuda")
    q = quantised(inp)
    names = ("W_g", "W_u", "W_d")
    good = [q[n] for n in names]
    kw = dict(k=w.k, weight_scales=q["scales"], fp8_block=True)
    for i in range(3):
        for bad in (good[i][:-1], good[i][:, :-1].contiguous(), good[i].transpose(1, 2).contiguous(),
                    good[i][0], inp[names[i]], good[i].view(torch.float8_e4m3fn)):
            args = list(good)
            args[i] = bad
            with pytest.raises(RuntimeError):
                forward(inp["x"], inp["W_r"], *args, **kw)
    # codes of another type are not read as numbers of x's type, whatever the format
    with pytest.raises(RuntimeError):
        forward(inp["x"], inp["W_r"], *[t.view(torch.float8_e4m3fn) for t in good], k=w.k)


def test_group_limited_selection():
    # experts chosen from 2 of 4 groups: the layer's own choices and gates, and y
    # within the format's roundings of the bf16 layer (see test_stages)
    w = Workload("groups", 150, 256, 32, 256, 4, seed=8, gate_mode=2, selection_bias=True)
    inp = make_inputs(w, device="cuda")
    q = quantised(inp)
    ws, ws2 = Workspace(), Workspace()
    kw = dict(n_group=4, topk_group=2)
    y, aux, counts = run(w, inp, q, ws, **kw)
    y2, aux2, counts2 = forward(inp["x"], inp["W_r"], inp["W_g"], inp["W_u"], inp["W_d"], k=w.k,
                                router_bias=inp["router_bias"], selection_bias=inp["selection_bias"],
                                gate_mode=2, workspace=ws2, **kw)
    v = routing_views(ws.buf, inp["x"], q["W_g"], w.E, w.k, fp8_block=True)
    v2 = routing_views(ws2.buf, inp["x"], inp["W_g"], w.E, w.k)
    assert torch.equal(v["topk_idx"], v2["topk_idx"]) and torch.equal(v["gates"], v2["gates"])
    assert torch.equal(counts, counts2) and torch.equal(aux, aux2)
    groups = v["topk_idx"] // 8
    assert max(len(set(r)) for r in groups.tolist()) <= 2
    rel = float((y.double() - y2.double()).norm() / y2.double().norm())
    assert rel <= (2 * 1.28 ** 2 + 4) ** 0.5 * 2.0 ** -4 / 3 ** 0.5

"""Calls with stream=: their buffers must not be memory that another stream still
works on, neither when the call starts nor after it, without any wait between the
streams other than the caller's for inputs and results."""
import pytest
import torch

from sparse_mixture_experts_aux_b200 import (Workspace, balance_loss, balance_loss_backward,
                                             dequantize_fp8, dequantize_fp8_block, dequantize_mxfp4,
                                             forward, matmul_fp8_block, quantize_fp8,
                                             quantize_fp8_block, quantize_mxfp4, swiglu_fp8_block)
from sparse_mixture_experts_aux_b200.inputs import Workload, make_inputs
from tests.test_balance_loss_gpu import draw
from tests.test_fp8_block_gpu import operands

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def busy(n=20):
    """Some ten milliseconds of work on the current stream."""
    a = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    for _ in range(n):
        a @ a


def calls(seed):
    """name -> (inputs, call): call(inputs, stream=...) gives a tuple of tensors."""
    logits, idx = draw(5003, 96, 2, seed=seed)
    loss, counts, tokens = balance_loss(logits, idx)
    one = torch.ones(1, device="cuda")
    a, sa, w, sw = operands(515, 1040, 1296, 0, seed=seed)
    x = torch.randn(777, 1296, generator=torch.Generator().manual_seed(seed)).cuda()
    codes, scales = quantize_fp8_block(x, 1)
    return {
        "loss": ([logits, idx], lambda t, **kw: balance_loss(t[0], t[1], **kw)),
        "gradient": ([one, logits, counts, tokens],
                     lambda t, **kw: (balance_loss_backward(*t, 2, **kw),)),
        "quantize": ([x], lambda t, **kw: quantize_fp8_block(t[0], 1, **kw)),
        "dequantize": ([codes, scales], lambda t, **kw: (dequantize_fp8_block(t[0], t[1], 1, **kw),)),
        "matmul": ([a, sa, w, sw], lambda t, **kw: (matmul_fp8_block(*t, **kw),)),
        "swiglu": ([a, sa, w, sw],
                   lambda t, **kw: swiglu_fp8_block(t[0], t[1], t[2], t[2], t[3], t[3], **kw)),
    }


NAMES = ["loss", "gradient", "quantize", "dequantize", "matmul", "swiglu"]


def same(got, want):
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def results_do_not_take_memory(inputs, call):
    want = call(inputs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of the results' sizes, read and written by work that is queued here
    # and freed before it has run: the next allocations of these sizes
    held = [torch.full_like(t, 1) for t in want]
    kept = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    busy()
    for h, k in zip(held, kept):
        k.copy_(h)
        h.fill_(2)
    del h, held
    got = call(inputs, stream=side)
    torch.cuda.synchronize()
    same(got, want)
    for k in kept:
        assert (k == 1).all()


def inputs_and_results_may_be_dropped(first, second, call):
    side = torch.cuda.Stream()
    want, other = call(first), call(second)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    mine = [t.clone() for t in first]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy()
    got = call(mine, stream=side)
    shapes = [(t.shape, t.dtype) for t in mine]
    del mine                                      # its kernel has not begun
    junk = [torch.zeros(s, dtype=d, device="cuda") for s, d in shapes]
    torch.cuda.current_stream().wait_stream(side)
    busy()                                        # read late, here, and dropped at once
    kept = [torch.empty_like(t) for t in got]
    for k, t in zip(kept, got):
        k.copy_(t)
    del t, got
    again = call(second, stream=side)
    torch.cuda.synchronize()
    same(kept, want)
    same(again, other)
    assert all((j == 0).all() for j in junk)


@pytest.mark.parametrize("name", NAMES)
def test_results_do_not_take_memory_the_current_stream_still_uses(name):
    results_do_not_take_memory(*calls(31)[name])


@pytest.mark.parametrize("name", NAMES)
def test_inputs_and_results_may_be_dropped(name):
    first, call = calls(32)[name]
    inputs_and_results_may_be_dropped(first, calls(33)[name][0], call)


def test_raw_handles_and_the_default_stream():
    for name, (inputs, call) in calls(34).items():
        want = call(inputs)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = [call(inputs, stream=side.cuda_stream), call(inputs, stream=0)]
        with torch.cuda.stream(side):             # the default stream is the other one now
            got += [call(inputs, stream=0), call(inputs, stream=torch.cuda.default_stream()),
                    call(inputs, stream=side)]
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
        torch.cuda.synchronize()
        for g in got:
            same(g, want)


def layer_calls(seed):
    inp = make_inputs(Workload("streams", 300, 256, 8, 256, 2, seed=seed), device="cuda")
    names = ("W_g", "W_u", "W_d")
    plain = [inp["x"], inp["W_r"]] + [inp[n] for n in names]
    block = [quantize_fp8_block(inp[n], 128) for n in names]
    scales = torch.cat([s.reshape(-1) for _, s in block])
    w = inp["W_g"].reshape(-1, 256)
    c8, s8 = quantize_fp8(w)
    mx = quantize_mxfp4(w)
    return {
        "forward": (plain, lambda t, **kw: forward(*t, k=2, **kw)),
        "forward fp8 blocks": (plain[:2] + [c for c, _ in block] + [scales],
                               lambda t, **kw: forward(*t[:5], k=2, weight_scales=t[5], fp8_block=True, **kw)),
        "quantize fp8": ([w], lambda t, **kw: quantize_fp8(t[0], **kw)),
        "dequantize fp8": ([c8, s8], lambda t, **kw: (dequantize_fp8(*t, **kw),)),
        "quantize mxfp4": ([w], lambda t, **kw: quantize_mxfp4(t[0], **kw)),
        "dequantize mxfp4": (list(mx), lambda t, **kw: (dequantize_mxfp4(*t, **kw),)),
    }


LAYER = ["forward", "forward fp8 blocks", "quantize fp8", "dequantize fp8", "quantize mxfp4",
         "dequantize mxfp4"]


@pytest.mark.parametrize("name", LAYER)
def test_layer_results_do_not_take_memory_the_current_stream_still_uses(name):
    results_do_not_take_memory(*layer_calls(35)[name])


@pytest.mark.parametrize("name", LAYER)
def test_layer_inputs_and_results_may_be_dropped(name):
    first, call = layer_calls(36)[name]
    inputs_and_results_may_be_dropped(first, layer_calls(37)[name][0], call)


@pytest.mark.parametrize("name", LAYER)
def test_layer_raw_handles(name):
    inputs, call = layer_calls(38)[name]
    want = call(inputs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [call(inputs, stream=s) for s in (side, side.cuda_stream, 0)]
    torch.cuda.synchronize()
    for g in got:
        same(g, want)


def test_layer_workspace_lent_to_another_stream():
    # a workspace of the caller's, made on the current stream, dropped while the
    # side stream still runs in it
    inp = make_inputs(Workload("streams", 300, 256, 8, 256, 2, seed=39), device="cuda")
    args = [inp[n] for n in ("x", "W_r", "W_g", "W_u", "W_d")]
    want = forward(*args, k=2)
    ws = Workspace()
    forward(*args, k=2, workspace=ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy()
    got = forward(*args, k=2, workspace=ws, stream=side)
    size = ws.buf.numel()
    del ws
    junk = torch.zeros(size, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    same(got, want)
    assert not junk.any()

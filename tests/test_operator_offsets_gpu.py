"""Tensors of more than 2^31 elements or bytes: the rows behind the 32-bit border
are those that the same call makes of them alone."""
import pytest
import torch

from sparse_mixture_experts_aux_b200 import (balance_loss, balance_loss_backward, dequantize_fp8_block,
                                             matmul_fp8_block, moe_get_device_status,
                                             quantize_fp8_block, swiglu_fp8_block)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def test_balance_loss():
    # two sequences; the second one and its gradient lie behind 2^31 logits
    E, first, rest = 600, 3_600_000, 5_003
    T = first + rest
    assert first * E > 2 ** 31
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    logits[first - 500:] = torch.randn(rest + 500, E, generator=gen(1), device="cuda").bfloat16()
    idx = torch.zeros(T, 2, dtype=torch.int32, device="cuda")
    idx[first:] = torch.topk(logits[first:].float(), 2, dim=1).indices.int()
    cu = torch.tensor([0, first, T], dtype=torch.int32, device="cuda")
    loss, counts, tokens = balance_loss(logits, idx, cu_seqlens=cu)
    d = balance_loss_backward(torch.ones(2, device="cuda"), logits, counts, tokens, 2, cu_seqlens=cu)
    part, few = logits[first:].contiguous(), idx[first:].contiguous()
    want, wc, wn = balance_loss(part, few)
    wd = balance_loss_backward(torch.ones(1, device="cuda"), part, wc, wn, 2)
    assert tokens.tolist() == [first, rest] and torch.equal(counts[1:], wc)
    # the two calls cut the rows into other chunks: sums of 64 rows and parts round apart
    assert abs(loss[1].item() - want.item()) <= 2 * 68 * 2.0 ** -24 * want.item()
    assert torch.equal(d[first:], wd)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantizer(block_rows):
    rows, cols = 2_097_152 + 256, 1040
    assert (rows - 256) * cols > 2 ** 31
    w = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    w[-256:] = torch.randn(256, cols, generator=gen(2), device="cuda").bfloat16()
    w[5] = 3.0
    codes, scales = quantize_fp8_block(w, block_rows)
    c, s = quantize_fp8_block(w[-256:].contiguous(), block_rows)
    assert torch.equal(codes[-256:], c) and torch.equal(scales[-s.shape[0]:], s)
    assert not codes[256:-256].any() and (codes[5] == 0x7E).all()
    del w
    back = dequantize_fp8_block(codes, scales, block_rows)
    assert torch.equal(back[-256:], dequantize_fp8_block(c, s, block_rows))
    assert (back[5] == 3.0).all() and not back[256:-256].any()


@pytest.mark.parametrize("K", [128, 16])
def test_products(K):
    # outputs behind 2^31 elements; one K block, so that every form adds in one order
    M, N = 140_000, 16_400
    assert (M - 3000) * N > 2 ** 31
    g = gen(3)
    a, sa = quantize_fp8_block(torch.randn(M, K, generator=g, device="cuda"), 1)
    w, sw = quantize_fp8_block(torch.randn(2, N, K, generator=g, device="cuda"), 128)
    off = torch.tensor([0, M - 3000, M - 1], dtype=torch.int32, device="cuda")
    out = torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")
    matmul_fp8_block(a, sa, w, sw, offsets=off, out=out)
    tail = matmul_fp8_block(a[-3000:-1].contiguous(), sa[-3000:-1].contiguous(), w[1], sw[1])
    assert torch.equal(out[-3000:-1], tail) and (out[-1] == 5.0).all()
    head = matmul_fp8_block(a[:300].contiguous(), sa[:300].contiguous(), w[0], sw[0])
    assert torch.equal(out[:300], head)
    del out
    codes, scales = swiglu_fp8_block(a, sa, w, w, sw, sw, offsets=off)
    tail = swiglu_fp8_block(a[-3000:-1].contiguous(), sa[-3000:-1].contiguous(), w[1], w[1], sw[1], sw[1])
    assert torch.equal(codes[-3000:-1], tail[0]) and torch.equal(scales[-3000:-1], tail[1])
    assert moe_get_device_status() == 0


def test_weights():
    # a stack of experts behind 2^31 codes
    E, N, K = 3, 32_768, 32_768
    assert 2 * N * K >= 2 ** 31
    g = gen(4)
    w = torch.randint(0, 0x7E, (E, N, K), generator=g, device="cuda", dtype=torch.uint8)
    sw = torch.rand(E, N // 128, K // 128, generator=g, device="cuda")
    a, sa = quantize_fp8_block(torch.randn(40, K, generator=g, device="cuda"), 1)
    off = torch.tensor([0, 1, 2, 40], dtype=torch.int32, device="cuda")
    got = matmul_fp8_block(a, sa, w, sw, offsets=off, out_dtype=torch.float32)
    x = dequantize_fp8_block(a, sa, 1)
    y = dequantize_fp8_block(w[2, -512:].contiguous(), sw[2, -4:].contiguous(), 128)
    want = x[2:].double() @ y.double().t()
    mag = x[2:].double().abs() @ y.double().abs().t()
    # a block's 128 additions, the blocks' own, and the values' rounding
    bound = (128 * 2.0 ** -23 + (K // 128 + 4) * 2.0 ** -24) * mag
    assert ((got[2:, -512:].double() - want).abs() <= bound).all()

"""Block-scaled FP8: quantiser, dequantiser, dense and grouped products, SwiGLU half.

References are fp64 on the codes themselves. Tolerances of a product element:
a K block is a sum of 128 products of two E4M3 values, each exact in fp32, added
in fp32 by the tensor core (at most one ulp lost an addition: 128 2^-23 of the
block's sum of magnitudes), the scales' product and the promoted sum round once
a block. With S = sum_b sA sW sum_k |a w|:
    |C - exact| <= (128 2^-23 + (blocks + 4) 2^-24) S + half a step of the output type
"""
import pytest
import torch

from sparse_mixture_experts_aux_b200 import (_lib, dequantize_fp8_block, matmul_fp8_block,
                                             moe_get_device_status, quantize_fp8_block,
                                             swiglu_fp8_block)

pytestmark = pytest.mark.gpu
BLK = 128


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def ceil(n, b):
    return -(-n // b)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def reference_codes(w, block_rows):
    """Codes and scales by fp32 divisions, on the CPU ([stack, rows, cols])."""
    w = w.cpu().float()
    stack, rows, cols = w.shape
    nb, kb = ceil(rows, block_rows), ceil(cols, BLK)
    full = torch.nn.functional.pad(w, (0, kb * BLK - cols, 0, nb * block_rows - rows))
    full = full.view(stack, nb, block_rows, kb, BLK)
    top = full.abs().amax(dim=(2, 4))
    scale = torch.where(top > 0, (top / 448.0).clamp(min=2.0 ** -126), torch.ones_like(top))
    q = full / scale[:, :, None, :, None]
    codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(stack, nb * block_rows, kb * BLK)[:, :rows, :cols], scale


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("stack,rows,cols", [
    (1, 1, 16), (1, 1, 7168), (1, 5, 144), (2, 127, 128), (3, 129, 272), (1, 300, 1040), (2, 256, 512)])
def test_quantizer_bit_exact(stack, rows, cols, block_rows, dtype):
    w = torch.randn(stack, rows, cols, generator=gen(rows + cols), device="cuda")
    w *= torch.exp2(torch.randint(-30, 30, (stack, rows, 1), generator=gen(1), device="cuda").float())
    if rows > 4:
        w[0, 1] = 0.0
        w[0, 2, :16] = 0.0
    w = w.to(dtype)
    codes, scales = quantize_fp8_block(w, block_rows)
    rc, rs = reference_codes(w, block_rows)
    assert scales.shape == (stack, rows if block_rows == 1 else ceil(rows, 128), ceil(cols, BLK))
    assert torch.equal(scales.cpu(), rs)
    assert torch.equal(codes.cpu(), rc)
    back = dequantize_fp8_block(codes, scales, block_rows)
    s = scales.repeat_interleave(BLK, dim=-1)[..., :cols]
    if block_rows > 1:
        s = s.repeat_interleave(BLK, dim=-2)[..., :rows, :]
    assert torch.equal(back, codes.view(torch.float8_e4m3fn).float() * s)


def test_quantizer_agrees_with_division_for_every_bf16_pair():
    # each significand of a block's maximum (128) against each significand of an
    # element at every distance that still makes a code: ties included
    sig = 1.0 + torch.arange(128, dtype=torch.float64) / 128
    for e in range(0, 20):
        tops = sig[:, None] * 2.0
        rows = torch.cat([tops.expand(128, 1), (sig[None, :] * 2.0 ** -e).expand(128, 128)[:, :127]], dim=1)
        more = torch.cat([tops.expand(128, 1), (-sig[None, :] * 2.0 ** -e).expand(128, 128)[:, 1:]], dim=1)
        w = torch.cat([rows, more]).to(torch.bfloat16)
        codes, scales = quantize_fp8_block(w.cuda(), 1)
        rc, rs = reference_codes(w[None], 1)
        assert torch.equal(scales.cpu(), rs[0]) and torch.equal(codes.cpu(), rc[0])


@pytest.mark.parametrize("exp", [-149, -140, -126, -120, -100, -82, -70, 0, 90, 107, 115, 127])
def test_quantizer_range(exp):
    # blocks from the smallest subnormal to the largest finite value
    g = torch.Generator().manual_seed(exp + 200)
    w = torch.ldexp(torch.rand(64, 128, generator=g) + 0.5, torch.tensor(exp)).float()
    w *= torch.where(torch.rand(64, 128, generator=g) < 0.5, -1.0, 1.0)
    w = torch.ldexp(w, torch.randint(-12, 1, (64, 128), generator=g))
    codes, scales = quantize_fp8_block(w.cuda(), 1)
    rc, rs = reference_codes(w[None], 1)
    assert torch.equal(scales.cpu(), rs[0]) and torch.equal(codes.cpu(), rc[0])


def test_quantizer_not_a_number_and_infinity():
    w = torch.ones(4, 256, device="cuda")
    w[1, 5] = float("nan")
    w[2, 200] = float("inf")
    codes, scales = quantize_fp8_block(w, 1)
    v = codes.view(torch.float8_e4m3fn).float()
    assert torch.isnan(scales[1, 0]) and torch.isnan(v[1, :128]).all()
    assert (v[1, 128:] == 448).all() and (v[0] == 448).all() and (v[3] == 448).all()
    assert torch.isinf(scales[2, 1]) and torch.isnan(v[2, 200]) and (v[2, 128:200] == 0).all()
    back = dequantize_fp8_block(codes, scales, 1)
    assert torch.isfinite(back[0]).all() and torch.isnan(back[2, 200])
    codes, scales = quantize_fp8_block(w, 128)
    assert torch.isnan(scales[0, 0]) and torch.isinf(scales[0, 1])


def test_quantizer_strided_rows_and_float8_views():
    wide = torch.randn(100, 512, generator=gen(2), device="cuda")
    for block_rows in (1, 128):
        a = quantize_fp8_block(wide[:, 128:400], block_rows)
        b = quantize_fp8_block(wide[:, 128:400].contiguous(), block_rows)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        x = dequantize_fp8_block(a[0].view(torch.float8_e4m3fn), a[1], block_rows)
        assert torch.equal(x, dequantize_fp8_block(a[0], a[1], block_rows))


# ------------------------------------------------------------------- products
def operands(M, N, K, E, seed=0, tail=0.0):
    """Codes and scales of random rows and weights (a few large columns)."""
    x = torch.randn(M, K, generator=gen(seed), device="cuda")
    x[:, :: max(1, K // 3)] *= 16
    a, sa = quantize_fp8_block(x, 1)
    w = torch.randn(max(1, E), N, K, generator=gen(seed + 1), device="cuda") / K ** 0.5
    w *= torch.exp2(torch.randint(-3, 4, (max(1, E), N, 1), generator=gen(seed + 2), device="cuda").float())
    c, sw = quantize_fp8_block(w, 128)
    return (a, sa, c, sw) if E else (a, sa, c[0], sw[0])


def values(codes, scales, block_rows):
    rows, cols = codes.shape[-2:]
    s = scales.double().repeat_interleave(BLK, dim=-1)[..., :cols]
    if block_rows > 1:
        s = s.repeat_interleave(BLK, dim=-2)[..., :rows, :]
    return codes.view(torch.float8_e4m3fn).double() * s


def product(a, sa, w, sw, offsets=None):
    """The exact product and its sum of magnitudes, fp64; rows without an expert are NaN."""
    x, y = values(a, sa, 1), values(w, sw, 128)
    if offsets is None:
        return x @ y.t(), x.abs() @ y.abs().t()
    c = torch.full((x.shape[0], y.shape[1]), float("nan"), dtype=torch.float64, device="cuda")
    m = c.clone()
    for e, (b, t) in enumerate(zip(offsets[:-1], offsets[1:])):
        if t > b:
            c[b:t] = x[b:t] @ y[e].t()
            m[b:t] = x[b:t].abs() @ y[e].abs().t()
    return c, m


def sum_eps(K):
    return 128 * 2.0 ** -23 + (ceil(K, BLK) + 4) * 2.0 ** -24


def near(got, want, mag, K, rows=slice(None)):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double() - want).abs()[rows]
    bound = (sum_eps(K) * mag * (1 + half) + half * want.abs() + 1e-37)[rows]
    assert torch.isfinite(got[rows].float()).all()
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 128, 128), (1, 4096, 7168), (2, 255, 144), (15, 257, 272), (16, 256, 1024),
    (17, 300, 1040), (33, 129, 400), (64, 512, 4096), (65, 1000, 512), (127, 77, 128), (128, 256, 128),
    (129, 640, 2048), (200, 8, 4096), (1000, 333, 560), (8, 14336, 256),
    (2500, 2100, 272), (6000, 1023, 144)])
def test_dense(M, N, K, out_dtype):
    a, sa, w, sw = operands(M, N, K, 0, seed=M + N)
    c = matmul_fp8_block(a, sa, w, sw, out_dtype=out_dtype)
    assert c.shape == (M, N) and c.dtype == out_dtype
    near(c, *product(a, sa, w, sw), K)
    assert moe_get_device_status() == 0


@pytest.mark.parametrize("lens,behind", [
    ([5], 0), ([0, 3, 0], 2), ([130, 1, 0, 127, 128, 129], 7), ([0, 0, 0], 4), ([1] * 40, 0),
    ([16, 17, 64, 65, 300], 33), ([2, 0, 700, 0, 31], 1),
    # several row tiles an expert, the last of them short
    ([700, 400], 0), ([1, 129, 1900, 130], 9), ([0, 1537, 0], 3), ([640], 0), ([384, 1000, 256], 5)])
@pytest.mark.parametrize("N,K", [(384, 512), (200, 272)])
def test_grouped(lens, behind, N, K):
    E, M = len(lens), sum(lens) + behind
    offsets = [0]
    for n in lens:
        offsets.append(offsets[-1] + n)
    a, sa, w, sw = operands(M, N, K, E, seed=E)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    gates = torch.rand(M, generator=gen(3), device="cuda")
    want, mag = product(a, sa, w, sw, offsets)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    got = matmul_fp8_block(a, sa, w, sw, offsets=off, row_scale=gates, out=out)
    assert got is out
    g = gates.double()[:, None]
    used = slice(0, offsets[-1])
    near(out, want * g, mag * g, K, used)
    assert (out[offsets[-1]:] == 7.0).all()       # rows of no expert stay as they were
    assert moe_get_device_status() == 0


def test_grouped_rows_need_not_start_at_zero():
    a, sa, w, sw = operands(300, 256, 384, 2, seed=5)
    offsets = [40, 100, 290]
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    out = torch.full((300, 256), -3.0, dtype=torch.float32, device="cuda")
    matmul_fp8_block(a, sa, w, sw, offsets=off, out=out)
    want, mag = product(a, sa, w, sw, offsets)
    near(out, want, mag, 384, slice(40, 290))
    assert (out[:40] == -3.0).all() and (out[290:] == -3.0).all()


def test_careless_offsets_stay_inside_the_rows():
    a, sa, w, sw = operands(100, 256, 256, 3, seed=6)
    bad = torch.tensor([-50, 30, 60, 4000], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 30, 60, 100], dtype=torch.int32, device="cuda")
    assert torch.equal(matmul_fp8_block(a, sa, w, sw, offsets=bad),
                       matmul_fp8_block(a, sa, w, sw, offsets=good))


@pytest.mark.parametrize("M", [30, 1000])
def test_overlapping_offsets_write_nowhere_else(M):
    E, N, K = 40, 272, 256
    a, sa, w, sw = operands(M, N, K, E, seed=8)
    off = torch.tensor([0, M] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    store = torch.full((M + 256, N + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    matmul_fp8_block(a, sa, w, sw, offsets=off, out=store[128:128 + M, :N])
    assert (store[:128] == 9.0).all() and (store[128 + M:] == 9.0).all() and (store[:, N:] == 9.0).all()
    off = torch.tensor([0] * E + [M], dtype=torch.int32, device="cuda")   # the last expert has them all
    want = matmul_fp8_block(a, sa, w[-1], sw[-1])
    assert torch.equal(matmul_fp8_block(a, sa, w, sw, offsets=off), want)
    assert moe_get_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(3, 200, 384), (300, 264, 640)])
def test_strides_and_float8_views(M, N, K):
    a, sa, w, sw = operands(M, N, K, 0, seed=7)
    want = matmul_fp8_block(a, sa, w, sw)
    wide = torch.zeros(M, K + 48, dtype=torch.uint8, device="cuda")
    wide[:, 16:16 + K] = a
    store = torch.full((M, N + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    got = matmul_fp8_block(wide[:, 16:16 + K].view(torch.float8_e4m3fn), sa, w.view(torch.float8_e4m3fn),
                           sw, out=store[:, 1:1 + N])
    assert torch.equal(got, want)
    assert (store[:, 0] == 9.0).all() and (store[:, 1 + N:] == 9.0).all()


def test_nan_and_infinity_stay_in_their_rows():
    a, sa, w, sw = operands(140, 256, 512, 0, seed=8)
    clean = matmul_fp8_block(a, sa, w, sw, out_dtype=torch.float32)
    a2, sa2 = a.clone(), sa.clone()
    a2[3, 100] = 0x7F
    sa2[135, 2] = float("inf")
    got = matmul_fp8_block(a2, sa2, w, sw, out_dtype=torch.float32)
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[135]).any()
    keep = [i for i in range(140) if i not in (3, 135)]
    assert torch.equal(got[keep], clean[keep])


def test_large_scales_and_zeros():
    a = torch.zeros(5, 256, dtype=torch.uint8, device="cuda")
    sa = torch.ones(5, 2, device="cuda")
    w = torch.full((130, 256), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    sw = torch.full((2, 2), 1e30, device="cuda")
    assert (matmul_fp8_block(a, sa, w, sw, out_dtype=torch.float32) == 0).all()
    a[:] = 0x38
    sa[:] = 2.0 ** -90
    got = matmul_fp8_block(a, sa, w, sw, out_dtype=torch.float32)
    want, mag = product(a, sa, w, sw)
    near(got, want, mag, 256)


def swiglu_reference(a, sa, g, sg, u, su, offsets=None):
    """H in fp64 and the bound on the kernel's fp32 H."""
    K = a.shape[1]
    (x, mx), (y, my) = product(a, sa, g, sg, offsets), product(a, sa, u, su, offsets)
    sig = torch.sigmoid(x)
    h = x * sig * y
    # |silu'| <= 1.1; silu's own error: the exponent's argument rounds once, the
    # approximate exponential and quotient a few ulp more: (|x| + 8) 2^-22
    dh = (1.1 * sum_eps(K) * mx * (y.abs() + sum_eps(K) * my) + (x * sig).abs() * sum_eps(K) * my
          + (x.abs().clamp(max=128) + 8) * 2.0 ** -22 * h.abs())
    return h, dh


def check_swiglu(codes, scales, h, dh, rows=slice(None)):
    M, N = h.shape
    got = values(codes, scales, 1)
    s = scales.double().repeat_interleave(BLK, dim=1)[:, :N]
    top = torch.nn.functional.pad((h.abs() + dh), (0, ceil(N, BLK) * BLK - N)).view(M, -1, BLK).amax(2)
    low = torch.nn.functional.pad((h.abs() - dh), (0, ceil(N, BLK) * BLK - N)).view(M, -1, BLK).amax(2)
    assert ((scales.double() <= top / 448 * (1 + 2.0 ** -23)) | (top == 0))[rows].all()
    assert (scales.double() >= low / 448 * (1 - 2.0 ** -23))[rows].all()
    # a code is the nearest E4M3 value: half a step is 2^-4 of the value, or 2^-10 among the subnormals
    bound = dh + 2.0 ** -4 * (h.abs() + dh) + 2.0 ** -10 * s * (1 + 2.0 ** -20)
    err = (got - h).abs()
    assert (err <= bound)[rows].all(), float((err / bound)[rows].max())


@pytest.mark.parametrize("M,N,K", [
    (1, 16, 16), (1, 1024, 4096), (2, 144, 272), (16, 128, 128), (31, 400, 1040), (64, 1024, 512),
    (128, 256, 384), (129, 1040, 640), (500, 336, 256), (2500, 1040, 272)])
def test_swiglu_dense(M, N, K):
    a, sa, g, sg = operands(M, N, K, 0, seed=N)
    _, _, u, su = operands(1, N, K, 0, seed=N + 50)
    codes, scales = swiglu_fp8_block(a, sa, g, u, sg, su)
    assert codes.shape == (M, N) and scales.shape == (M, ceil(N, BLK))
    check_swiglu(codes, scales, *swiglu_reference(a, sa, g, sg, u, su))
    assert moe_get_device_status() == 0


@pytest.mark.parametrize("lens,behind", [([0, 3, 0, 130], 2), ([128, 1, 65, 16], 40), ([0, 0], 3),
                                         ([700, 400], 0), ([1, 129, 1900, 130], 9), ([0, 1537, 0], 3)])
def test_swiglu_grouped(lens, behind):
    E, M, N, K = len(lens), sum(lens) + behind, 272, 400
    offsets = [0]
    for n in lens:
        offsets.append(offsets[-1] + n)
    a, sa, g, sg = operands(M, N, K, E, seed=30)
    _, _, u, su = operands(1, N, K, E, seed=31)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    codes = torch.full((M, N), 0x41, dtype=torch.uint8, device="cuda")
    scales = torch.full((M, ceil(N, BLK)), 5.0, device="cuda")
    swiglu_fp8_block(a, sa, g, u, sg, su, offsets=off, codes=codes, scales=scales)
    check_swiglu(codes, scales, *swiglu_reference(a, sa, g, sg, u, su, offsets), rows=slice(0, offsets[-1]))
    assert (codes[offsets[-1]:] == 0x41).all() and (scales[offsets[-1]:] == 5.0).all()


def test_experts_end_to_end():
    """Quantise, gate and up, down, weighted by the gates: an expert stack as it is used."""
    E, M, d, de = 6, 180, 512, 384
    lens = [50, 0, 1, 99, 20, 10]
    offsets = [0]
    for n in lens:
        offsets.append(offsets[-1] + n)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x = torch.randn(M, d, generator=gen(40), device="cuda").to(torch.bfloat16)
    wg, wu = (torch.randn(E, de, d, generator=gen(41 + i), device="cuda") / d ** 0.5 for i in range(2))
    wd = torch.randn(E, d, de, generator=gen(43), device="cuda") / de ** 0.5
    gates = torch.rand(M, generator=gen(44), device="cuda")
    a, sa = quantize_fp8_block(x, 1)
    (g, sg), (u, su), (dn, sd) = (quantize_fp8_block(w, 128) for w in (wg, wu, wd))
    h, sh = swiglu_fp8_block(a, sa, g, u, sg, su, offsets=off)
    y = matmul_fp8_block(h, sh, dn, sd, offsets=off, row_scale=gates)
    want, mag = product(h, sh, dn, sd, offsets)
    near(y, want * gates.double()[:, None], mag * gates.double()[:, None], de)
    ref = torch.empty(M, d, dtype=torch.float64, device="cuda")
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        xe = x[r].double()
        ge = xe @ wg[e].double().t()
        ref[r] = ((ge * torch.sigmoid(ge) * (xe @ wu[e].double().t())) @ wd[e].double().t())
    ref *= gates.double()[:, None]
    # six independent roundings on the way (x and W_g through SiLU, whose relative
    # slope is at most 1.28 for positive gates; x and W_u; H; W_d), each at most
    # 2^-4 of a value, uniform within its step: 2^-4 / sqrt(3) in the mean square
    rel = float((y.double() - ref).norm() / ref.norm())
    assert rel <= (2 * 1.28 ** 2 + 4) ** 0.5 * 2.0 ** -4 / 3 ** 0.5


def test_repeat_streams_and_graph_give_the_same_bits():
    cases = [(1, 1024, 4096, 0), (300, 512, 1024, 0), (90, 384, 512, 5)]
    ops, want = [], []
    for i, (M, N, K, E) in enumerate(cases):
        o = operands(M, N, K, E, seed=60 + i)
        off = torch.arange(0, M + 1, M // 5, dtype=torch.int32, device="cuda")[:6] if E else None
        ops.append((o, off))
        want.append(matmul_fp8_block(*o, offsets=off))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(5):
        for s, (o, off) in zip(streams, ops):
            with torch.cuda.stream(s):
                got.append(matmul_fp8_block(*o, offsets=off))
    torch.cuda.synchronize()
    for i, c in enumerate(got):
        assert torch.equal(c, want[i % 3])
    for (o, off), w in zip(ops, want):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c = matmul_fp8_block(*o, offsets=off)
        c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, w)


def test_two_streams_at_once():
    # a persistent launch beside clusters that share a tile, each on its own stream
    a, sa, w, sw = operands(1500, 1024, 2048, 0, seed=60)
    big = matmul_fp8_block(a, sa, w, sw)
    small = swiglu_fp8_block(a[:3], sa[:3], w, w, sw, sw)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append((matmul_fp8_block(a, sa, w, sw, stream=s1),
                    swiglu_fp8_block(a[:3], sa[:3], w, w, sw, sw, stream=s2)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, big) and torch.equal(y[0], small[0]) and torch.equal(y[1], small[1])
    assert moe_get_device_status() == 0


def test_no_rows():
    a, sa, w, sw = operands(4, 256, 256, 0)
    assert matmul_fp8_block(a[:0], sa[:0], w, sw).shape == (0, 256)
    codes, scales = swiglu_fp8_block(a[:0], sa[:0], w, w, sw, sw)
    assert codes.shape == (0, 256) and scales.shape == (0, 2)
    c, s = quantize_fp8_block(torch.empty(0, 256, device="cuda"), 1)
    assert c.shape == (0, 256) and s.shape == (0, 2)


def test_timeout_is_reported_and_the_context_stays_usable():
    a, sa, w, sw = operands(200, 512, 4096, 0, seed=70)
    want = matmul_fp8_block(a, sa, w, sw)
    torch.cuda.synchronize()
    assert moe_get_device_status() == 0
    # single CTAs (grouped) and clusters that share a tile (dense)
    w2, sw2 = torch.stack([w, w]), torch.stack([sw, sw])
    b, sb = a.repeat(6, 1), sa.repeat(6, 1)
    for n in (200, 1200):
        off = torch.tensor([0, n - 50, n], dtype=torch.int32, device="cuda")
        swiglu_fp8_block(b[:n], sb[:n], w2, w2, sw2, sw2, offsets=off, wait_timeout_ns=1)
        matmul_fp8_block(b[:n], sb[:n], w2, sw2, offsets=off, wait_timeout_ns=1)
        torch.cuda.synchronize()
        assert moe_get_device_status() == _lib.MOE_ERR_DEVICE_TIMEOUT
    for M in (1, 200):
        matmul_fp8_block(a[:M], sa[:M], w, sw, wait_timeout_ns=1)
        swiglu_fp8_block(a[:M], sa[:M], w, w, sw, sw, wait_timeout_ns=1)
        torch.cuda.synchronize()
        assert moe_get_device_status() == _lib.MOE_ERR_DEVICE_TIMEOUT
    assert torch.equal(matmul_fp8_block(a, sa, w, sw), want)
    assert moe_get_device_status() == 0


# One K block a tile and many tiles a CTA, some of which reach into the second
# 32 rows and some not: the epilogue's warps exchange row maxima tile by tile.
ONE_BLOCK_LENS = [3, 40, 1, 128, 20, 70, 33, 0, 5, 256, 31, 64]


@pytest.mark.parametrize("K", [16, 128])
def test_swiglu_of_one_block(K):
    lens, N = ONE_BLOCK_LENS * 2, 4096
    E, M = len(lens), sum(lens)
    offsets = [0]
    for n in lens:
        offsets.append(offsets[-1] + n)
    a, sa, g, sg = operands(M, N, K, E, seed=90)
    _, _, u, su = operands(1, N, K, E, seed=91)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    want = swiglu_fp8_block(a, sa, g, u, sg, su, offsets=off)
    check_swiglu(*want, *swiglu_reference(a, sa, g, sg, u, su, offsets))
    for _ in range(20):
        got = swiglu_fp8_block(a, sa, g, u, sg, su, offsets=off)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert moe_get_device_status() == 0
    # every limit ends in a status, wherever the roles are when it runs out
    for limit in (1, 100, 1000, 3000, 10000):
        for _ in range(4):
            swiglu_fp8_block(a, sa, g, u, sg, su, offsets=off, wait_timeout_ns=limit)
        torch.cuda.synchronize()
        assert moe_get_device_status() in (0, _lib.MOE_ERR_DEVICE_TIMEOUT)
    got = swiglu_fp8_block(a, sa, g, u, sg, su, offsets=off)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert moe_get_device_status() == 0


def test_refusals():
    a, sa, w, sw = operands(20, 256, 256, 2, seed=80)
    off = torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda")
    ok = dict(offsets=off)
    matmul_fp8_block(a, sa, w, sw, **ok)
    with pytest.raises(RuntimeError):
        matmul_fp8_block(a.cpu(), sa, w, sw, **ok)
    with pytest.raises(RuntimeError):
        matmul_fp8_block(a.float(), sa, w, sw, **ok)
    with pytest.raises(RuntimeError):
        matmul_fp8_block(a, sa, w, sw)                       # three dimensions without offsets
    with pytest.raises(RuntimeError):
        matmul_fp8_block(a, sa[:, :1], w, sw, **ok)
    with pytest.raises(RuntimeError):
        matmul_fp8_block(a, sa, w, sw[:, :1], **ok)
    with pytest.raises(TypeError):
        matmul_fp8_block(a, sa.double(), w, sw, **ok)
    with pytest.raises(RuntimeError):
        matmul_fp8_block(a[:, ::2], sa, w, sw, **ok)
    with pytest.raises(TypeError):
        matmul_fp8_block(a, sa, w, sw, offsets=off.long())
    with pytest.raises(RuntimeError):
        matmul_fp8_block(a, sa, w, sw, offsets=off[:2])      # one expert's offsets for two
    with pytest.raises(TypeError):
        matmul_fp8_block(a, sa, w, sw, out_dtype=torch.float16, **ok)
    with pytest.raises(RuntimeError):
        matmul_fp8_block(a, sa, w, sw, out=torch.empty(20, 128, device="cuda"), **ok)
    with pytest.raises(RuntimeError):                        # K not a multiple of 16
        matmul_fp8_block(a[:, :200], sa, w[:, :, :200].contiguous(), sw, **ok)
    with pytest.raises(RuntimeError):                        # rows 8 bytes off
        matmul_fp8_block(torch.zeros(21, 264, dtype=torch.uint8, device="cuda")[:20, 8:], sa, w, sw, **ok)
    with pytest.raises(RuntimeError):                        # N not a multiple of 16
        swiglu_fp8_block(a, sa, *[w[:, :250].contiguous()] * 2, sw, sw, **ok)
    with pytest.raises(RuntimeError):
        quantize_fp8_block(torch.zeros(4, 250, device="cuda"), 1)
    with pytest.raises(RuntimeError):
        quantize_fp8_block(torch.zeros(4, 256, device="cuda"), 64)
    with pytest.raises(RuntimeError):
        quantize_fp8_block(torch.zeros(4, 4, 512, device="cuda")[:, :, :256], 1)
    with pytest.raises(TypeError):
        quantize_fp8_block(torch.zeros(4, 256, device="cuda", dtype=torch.float16), 1)
    with pytest.raises(RuntimeError):
        dequantize_fp8_block(a, sa[:, :1], 1)


def small_codes(shape, top, g):
    """Random nonzero codes of both signs up to `top`."""
    c = torch.randint(1, top + 1, shape, generator=g, device="cuda", dtype=torch.uint8)
    return c | torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7


def scales_near(shape, e, g):
    return torch.ldexp(1 + torch.rand(shape, generator=g, device="cuda"), torch.tensor(e, device="cuda"))


# Powers of two of the scales: products among the subnormals, below them, above the
# largest number, each with sums that bring the result back among the numbers
FAR_SCALES = [(-126, -14), (-14, -126), (-70, -72), (-126, -126), (70, 60), (120, 10), (10, 117),
              (-126, 126)]


@pytest.mark.parametrize("ea,ew", FAR_SCALES)
@pytest.mark.parametrize("M,N,K,E", [(1, 256, 256, 0), (5, 200, 384, 0), (300, 4096, 272, 0),
                                     (140, 272, 512, 3), (3000, 2048, 128, 0)])
def test_scale_products_out_of_range(M, N, K, E, ea, ew):
    # the result of scales whose product no normal fp32 number holds is as exact as
    # any other, and a sum of zero stays zero. Beside the bound above, an addition
    # rounds among the subnormals by 2^-150, and the output by half its own smallest
    g = gen(M + N)
    kb, nb = ceil(K, BLK), ceil(N, BLK)
    top = 3 if ea + ew > 0 else 126               # 3 * 2^-9, or the largest code
    a, w = small_codes((M, K), top, g), small_codes((max(1, E), N, K), top, g)
    sa, sw = scales_near((M, kb), ea, g), scales_near((max(1, E), nb, kb), ew, g)
    a[0] = 0
    sa[1::2, 0] = 1.0                             # beside blocks of ordinary scales
    if kb > 1:
        sw[:, 0, -1] = 1.0
    offsets, cuts = None, None
    if E:
        cuts = [0, 10, 10, M]
        offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    else:
        w, sw = w[0], sw[0]
    want, mag = product(a, sa, w, sw, cuts)
    for dtype in (torch.float32, torch.bfloat16):
        info = torch.finfo(dtype)
        got = matmul_fp8_block(a, sa, w, sw, offsets=offsets, out_dtype=dtype)
        bound = (sum_eps(K) * mag * (1 + info.eps / 2) + info.eps / 2 * want.abs()
                 + kb * 2.0 ** -150 + info.smallest_normal * info.eps / 2)
        fits = mag * (1 + sum_eps(K)) < info.max  # no partial sum overflows
        assert fits.any() and torch.isfinite(got[fits]).all()
        assert ((got.double() - want).abs() <= bound)[fits].all()
        assert (got[0] == 0).all()
    assert moe_get_device_status() == 0


@pytest.mark.parametrize("M", [3, 200, 2500])
@pytest.mark.parametrize("ea,eg,eu,top", [(-100, -44, 110, 126), (90, 40, -92, 3), (-30, 30, 2, 126)])
def test_swiglu_scale_products_out_of_range(ea, eg, eu, top, M):
    N, K = 272, 384
    gn = gen(M)
    a, wg, wu = small_codes((M, K), top, gn), small_codes((N, K), top, gn), small_codes((N, K), top, gn)
    sa, sg, su = (scales_near(s, e, gn) for s, e in (((M, 3), ea), ((3, 3), eg), ((3, 3), eu)))
    codes, scales = swiglu_fp8_block(a, sa, wg, wu, sg, su)
    check_swiglu(codes, scales, *swiglu_reference(a, sa, wg, sg, wu, su))


def test_scales_of_zero_and_infinity():
    # a scale of zero makes its blocks zero; an infinite one makes inf, or NaN of a zero sum
    a, sa, w, sw = operands(70, 256, 512, 0, seed=9)
    sa0 = sa.clone()
    sa0[:, 1] = 0.0
    a0 = a.clone()
    a0[:, 128:256] = 0
    assert torch.equal(matmul_fp8_block(a, sa0, w, sw, out_dtype=torch.float32),
                       matmul_fp8_block(a0, sa, w, sw, out_dtype=torch.float32))
    sa1 = sa.clone()
    sa1[3, 1] = float("inf")
    got = matmul_fp8_block(a, sa1, w, sw, out_dtype=torch.float32)
    clean = matmul_fp8_block(a, sa, w, sw, out_dtype=torch.float32)
    assert torch.isinf(got[3]).all()
    assert torch.isnan(matmul_fp8_block(a0, sa1, w, sw)[3]).all()
    keep = [i for i in range(70) if i != 3]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantizer_keeps_the_sign_of_zero(block_rows, dtype):
    # zeros of both signs, and quotients that round to them, beside ordinary elements
    # and in blocks of nothing else
    w = torch.randn(300, 272, generator=gen(3), device="cuda").to(dtype)
    w[::3, ::2] = -0.0
    w[::3, 1::2] = 0.0
    w[1::3, ::4] *= -2.0 ** -20
    w[5] = -0.0
    w[128:256, 128:256] = -0.0
    codes, scales = quantize_fp8_block(w, block_rows)
    rc, rs = reference_codes(w[None], block_rows)
    assert (rc == 0x80).any() and (rc == 0).any()
    assert torch.equal(scales.cpu(), rs[0]) and torch.equal(codes.cpu(), rc[0])


def test_empty_matrices():
    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    for shape, block_rows, scales in [((0, 256), 1, (0, 2)), ((0, 256), 128, (0, 2)),
                                      ((0, 5, 144), 1, (0, 5, 2)), ((3, 0, 16), 128, (3, 0, 1))]:
        c, s = quantize_fp8_block(empty(*shape), block_rows)
        assert c.shape == shape and s.shape == scales
        assert dequantize_fp8_block(c, s, block_rows).shape == shape
    # refused with and without rows: no columns, and sizes that are refused of any matrix
    for rows in (0, 4):
        for cols, block_rows in ((0, 1), (0, 128), (24, 1)):
            with pytest.raises(RuntimeError):
                quantize_fp8_block(empty(rows, cols), block_rows)
            with pytest.raises(RuntimeError):
                dequantize_fp8_block(empty(rows, cols, dtype=torch.uint8),
                                     empty(rows if block_rows == 1 else ceil(rows, 128), ceil(cols, 128)),
                                     block_rows)


@pytest.mark.parametrize("M,N,K,E", [(3, 1200, 2304, 0), (3000, 2100, 2304, 0), (900, 272, 1296, 5)])
def test_a_few_blocks_of_far_scales(M, N, K, E):
    # two K blocks far apart, each out of range one way, among ordinary ones; some
    # rows and weight blocks are ordinary there too; a zero and a negative scale
    a, sa, w, sw = operands(M, N, K, E, seed=95)
    kb = ceil(K, BLK)
    lo, hi = kb // 2 - 1, kb - 1
    sa[::2, lo] *= 2.0 ** -110
    sw[..., lo] *= 2.0 ** -20
    sa[:, hi] *= 2.0 ** 90
    sw[..., hi] *= 2.0 ** 50
    a[:, hi * BLK:] = 0                           # a product of 2^140, of sums that are zero
    sa[1, 0] = 0.0
    sa[2, 1] *= -1.0
    offsets = cuts = None
    if E:
        cuts = [0, 200, 200, 201, 650, M]
        offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    want, mag = product(a, sa, w, sw, cuts)
    near(matmul_fp8_block(a, sa, w, sw, offsets=offsets, out_dtype=torch.float32), want, mag, K)
    if N % 16 == 0:
        u = w.flip(0).contiguous()
        codes, scales = swiglu_fp8_block(a, sa, w, u, sw, sw, offsets=offsets)
        check_swiglu(codes, scales, *swiglu_reference(a, sa, w, sw, u, sw, cuts))
    assert moe_get_device_status() == 0

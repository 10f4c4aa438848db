"""The balance loss and block-scaled FP8 entry points refuse bad arguments on the
host, before anything is enqueued (no GPU)."""
import ctypes
import shutil
import subprocess

import pytest

from sparse_mixture_experts_aux_b200 import _lib
from sparse_mixture_experts_aux_b200 import build as B

BAD, UNSUPPORTED, WORKSPACE = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
P = 1 << 20  # an aligned address that no case below dereferences


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return _lib.load()


def balance(**kw):
    d = _lib.moe_balance_dims()
    base = dict(T=64, E=8, k=2, dtype=_lib.MOE_F32, gate_mode=0, ld=0, num_seqs=1, cu_seqlens=None,
                token_mask=None, workspace=P, workspace_bytes=1 << 30, stream=None)
    for name, v in dict(base, **kw).items():
        setattr(d, name, v)
    return d


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), BAD), (dict(E=0), BAD), (dict(k=0), BAD), (dict(k=9), BAD), (dict(dtype=2), BAD),
    (dict(gate_mode=3), BAD), (dict(gate_mode=-1), BAD), (dict(ld=7), BAD), (dict(num_seqs=0), BAD),
    (dict(num_seqs=2), BAD), (dict(cu_seqlens=P + 2), BAD), (dict(E=1025), UNSUPPORTED),
    (dict(E=64, k=33), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(T=1 << 30, k=2), UNSUPPORTED),
    (dict(num_seqs=1 << 29, cu_seqlens=P), UNSUPPORTED)])
def test_balance_dims(kw, want):
    d = balance(**kw)
    assert _lib.moe_balance_loss_workspace_size(d) == 0
    assert _lib.moe_balance_loss(d, P, P, P, P, P) == want
    assert _lib.moe_balance_loss_backward(d, P, P, P, P, P) == want


def test_balance_pointers():
    assert _lib.moe_balance_loss(None, P, P, P, P, P) == BAD
    for i in range(5):
        for v in (0, P + 2):
            args = [P] * 5
            args[i] = v
            assert _lib.moe_balance_loss(balance(), *args) == BAD
            assert _lib.moe_balance_loss_backward(balance(), *args) == BAD
    need = _lib.moe_balance_loss_workspace_size(balance())
    assert need > 0
    for kw in (dict(workspace=None), dict(workspace=P + 16), dict(workspace_bytes=need - 1)):
        assert _lib.moe_balance_loss(balance(**kw), P, P, P, P, P) == WORKSPACE
    assert _lib.moe_balance_loss_backward(balance(T=0), 0, 0, 0, 0, 0) == _lib.MOE_OK


def test_balance_token_limit():
    # the kernels count tokens, a block's look-ahead included, in 32 bits
    assert _lib.moe_balance_loss_workspace_size(balance(T=1 << 30, k=1)) > 0
    for T in ((1 << 30) + 1, (1 << 31) - 1):
        assert _lib.moe_balance_loss_workspace_size(balance(T=T, k=1)) == 0
        assert _lib.moe_balance_loss(balance(T=T, k=1), P, P, P, P, P) == UNSUPPORTED
        assert _lib.moe_balance_loss_backward(balance(T=T, k=1), P, P, P, P, P) == UNSUPPORTED


def test_balance_workspace_covers_every_chunk_and_sequence():
    for T, S, E in [(1, 1, 8), (148 * 32, 1, 8), (148 * 32 + 1, 5, 256), (1 << 20, 4096, 64)]:
        chunk = max(32, -(-T // 148))
        slots = -(-T // chunk) + S
        d = balance(T=T, E=E, num_seqs=S, cu_seqlens=P)
        assert _lib.moe_balance_loss_workspace_size(d) >= slots * (8 * E + 4)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(stack=-1), dict(rows=-1), dict(cols=0), dict(cols=24), dict(ld=240),
    dict(ld=258), dict(block_rows=0), dict(block_rows=64), dict(w=0), dict(codes=0), dict(scales=0),
    dict(w=P + 8), dict(codes=P + 8), dict(scales=P + 2)])
def test_quantize(kw):
    a = dict(w=P, dtype=_lib.MOE_F32, stack=1, rows=4, cols=256, ld=0, block_rows=1, codes=P, scales=P)
    a.update(kw)
    assert _lib.moe_quantize_fp8_block(**a) == BAD
    if "ld" not in kw and "dtype" not in kw:
        b = {k: a[k] for k in ("codes", "scales", "stack", "rows", "cols", "block_rows")}
        assert _lib.moe_dequantize_fp8_block(out=a["w"], **b) == BAD


def test_quantize_nothing():
    for kw in (dict(stack=0, rows=4), dict(stack=1, rows=0)):
        assert _lib.moe_quantize_fp8_block(P, 0, kw["stack"], kw["rows"], 256, 0, 1, P, P) == _lib.MOE_OK
        assert _lib.moe_dequantize_fp8_block(P, P, kw["stack"], kw["rows"], 256, 1, P) == _lib.MOE_OK
    # more 128 x 128 blocks than a grid holds
    assert _lib.moe_quantize_fp8_block(P, 0, 1 << 20, 1 << 20, 1 << 20, 0, 128, P, P) == UNSUPPORTED


def product(**kw):
    d = _lib.moe_fp8_block_dims()
    base = dict(M=64, N=256, K=512, E=0, out_dtype=_lib.MOE_BF16, lda=0, ld_out=0, offsets=None,
                row_scale=None, wait_timeout_ns=0, stream=None)
    for name, v in dict(base, **kw).items():
        setattr(d, name, v)
    return d


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), BAD), (dict(N=0), BAD), (dict(K=0), BAD), (dict(K=24), BAD), (dict(E=-1), BAD),
    (dict(E=2), BAD), (dict(offsets=P), BAD), (dict(E=2, offsets=P + 2), BAD), (dict(lda=496), BAD),
    (dict(lda=520), BAD), (dict(ld_out=255), BAD), (dict(out_dtype=2), BAD),
    (dict(E=1025, offsets=P), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED),
    (dict(N=(1 << 30) + 16), UNSUPPORTED), (dict(N=1 << 20, K=1 << 20), UNSUPPORTED)])
def test_product_dims(kw, want):
    assert _lib.moe_matmul_fp8_block(product(**kw), P, P, P, P, P) == want
    assert _lib.moe_swiglu_fp8_block(product(**kw), P, P, P, P, P, P, P, P) == want


def test_product_pointers():
    assert _lib.moe_matmul_fp8_block(None, P, P, P, P, P) == BAD
    assert _lib.moe_swiglu_fp8_block(None, P, P, P, P, P, P, P, P) == BAD
    for i in range(5):
        for off in (0, 1):
            args = [P] * 5
            args[i] = P + off if off else 0
            assert _lib.moe_matmul_fp8_block(product(), *args) == BAD, (i, off)
    for i in range(8):
        for off in (0, 2):
            args = [P] * 8
            args[i] = P + off if off else 0
            assert _lib.moe_swiglu_fp8_block(product(), *args) == BAD, (i, off)
    # the SwiGLU half writes rows of codes for the next product
    for kw in (dict(N=250), dict(ld_out=264), dict(row_scale=P)):
        assert _lib.moe_swiglu_fp8_block(product(**kw), P, P, P, P, P, P, P, P) == BAD
    assert _lib.moe_matmul_fp8_block(product(row_scale=P + 2), P, P, P, P, P) == BAD


def test_product_of_no_rows():
    assert _lib.moe_matmul_fp8_block(product(M=0), 0, 0, 0, 0, 0) == _lib.MOE_OK
    assert _lib.moe_swiglu_fp8_block(product(M=0), 0, 0, 0, 0, 0, 0, 0, 0) == _lib.MOE_OK


def test_layer_format():
    def dims(**kw):
        base = dict(T=128, d=256, d_e=320, dtype=_lib.MOE_BF16,
                    weight_format=_lib.MOE_WEIGHTS_FP8_BLOCK)
        return _lib.make_dims(**dict(base, **kw))

    need = _lib.moe_workspace_size(dims(), 8, 2, 0.0)
    assert 0 < need < _lib.moe_workspace_size(dims(weight_format=0), 8, 2, 0.0)
    L = _lib.moe_workspace_layout(dims(), 8, 2, 0.0)
    assert max(L.xscale, L.hq, L.hscale) < need
    assert L.hq - L.xscale >= L.rows_max * 2 * 4          # ceil(256 / 128) scales a row
    assert need - L.hscale >= L.rows_max * 3 * 4          # ceil(320 / 128)
    for kw in (dict(d_s=128), dict(dtype=_lib.MOE_F32), dict(d=288)):
        st = _lib.moe_forward(dims(**kw), P, P, P, P, P, None, 8, 2, 0.0, P, P, P, check=False)
        assert st == UNSUPPORTED
    st = _lib.moe_forward(dims(workspace=P, workspace_bytes=need), P, P, P, P, P, None, 8, 2, 0.0, P,
                          P, P, check=False)
    assert st == BAD                                      # no weight_scales


SPLIT_PROBE = """
#include "split_clusters.cuh"
extern "C" void clusters(const int* known, const int* counts, int* out) {
  moe::f8b::co_resident_clusters(
      [&](int s, int* n) { *n = counts[s]; return known[s] != 0; }, out);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_cluster_sizes_the_runtime_does_not_know_are_left_out(tmp_path):
    # a size whose occupancy query fails is not used; it refuses no call
    src, so = tmp_path / "probe.cpp", tmp_path / "probe.so"
    src.write_text(SPLIT_PROBE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", B.CSRC, "-x", "c++",
                    str(src), "-o", str(so)], check=True)
    probe = ctypes.CDLL(str(so))
    ints = ctypes.c_int * 9
    counts = ints(0, 0, 74, 48, 36, 28, 22, 20, 15)
    for known, want in [([1] * 9, [74, 48, 36, 28, 22, 20, 15]), ([0] * 9, [0] * 7),
                        ([1, 1, 1, 1, 0, 1, 0, 1, 0], [74, 48, 0, 28, 0, 20, 0])]:
        out = ints(*[7] * 9)
        probe.clusters(ints(*known), counts, out)
        assert list(out)[2:] == want
    out = ints()
    probe.clusters(ints(*[1] * 9), ints(0, 0, -1, 0, 5, 0, 0, 0, 0), out)
    assert list(out)[2:] == [0, 0, 5, 0, 0, 0, 0]


def test_sizes_are_checked_where_there_is_nothing_to_do():
    for stack, rows in ((0, 4), (1, 0)):
        assert _lib.moe_quantize_fp8_block(0, 0, stack, rows, 256, 0, 1, 0, 0) == _lib.MOE_OK
        assert _lib.moe_dequantize_fp8_block(0, 0, stack, rows, 256, 1, 0) == _lib.MOE_OK
        for cols, block_rows in ((0, 1), (24, 1), (256, 64)):
            assert _lib.moe_quantize_fp8_block(0, 0, stack, rows, cols, 0, block_rows, 0, 0) == BAD
            assert _lib.moe_dequantize_fp8_block(0, 0, stack, rows, cols, block_rows, 0) == BAD

"""GPU: the dense products of 1 to 128 rows, whose loads of A are as high as the
rows need (boxes of 32, 64 or 128 rows; none in the odd CTA of a pair), through
several turns of the operand ring (K = 2880) and several rounds of tiles.

The tolerances are those of test_gpu_gemm: 1e-5 * sum|a b| for FP32, one bf16
rounding more for bf16.  A row's sums do not depend on the rows beside it, so
the same rows of a taller product have the same bits.
"""
import numpy as np
import pytest
import torch

import oracle
import quantize_block_scaled_rht_b200 as mx
import synth
import test_gpu_gemm as base
from mxfp4_testutil import assert_gemm_close, dev_bf16, dev_u8, host, to_mma

pytestmark = pytest.mark.gpu

ROWS = [1, 31, 32, 33, 64, 65, 127, 128]
K = 2880


@pytest.mark.parametrize("M", ROWS)
def test_fp32_and_bf16_outputs(M):
    base.test_gemm_shapes(M, 200, K)
    base.test_gemm_bf16_output(M, 200, K)
    assert mx.mxfp4_get_error() == mx.MXFP4_OK


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("mma", [False, True])
def test_mxfp4_output(M, mma):
    base.test_gemm_mxfp4_output(M, 224, K, mma)


@pytest.mark.parametrize("M", ROWS)
def test_nvfp4(M):
    """The first M of 256 quantized rows (the quantizer takes whole blocks of rows)."""
    N = 208
    a, b = synth.normal_bf16((256, K), 40), synth.normal_bf16((N, K), 41, 0.02)
    qa = mx.mxfp4_nvfp4_quantize(dev_bf16(a), scale_layout=mx.SCALES_MMA)
    qb = mx.mxfp4_nvfp4_quantize(dev_bf16(b), scale_layout=mx.SCALES_MMA)
    c = mx.mxfp4_nvfp4_gemm(mx.NvQuantized(qa.codes[:M], qa.scales, qa.amax, M, K, qa.layout, qa.scale_layout), qb)
    assert mx.mxfp4_get_error() == mx.MXFP4_OK and c.shape == (M, N)
    ca, sa, aa = oracle.nvfp4_quantize(a, oracle.LAYOUT_1D_ROW)
    cb, sb, ab = oracle.nvfp4_quantize(b, oracle.LAYOUT_1D_ROW)
    pairs = [(m, n) for m in range(M) for n in range(m % 5, N, 5)]
    ref, s = oracle.nvfp4_gemm_entries(ca, sa, aa, cb, sb, ab, K, pairs)
    at = np.array(pairs)
    assert_gemm_close(host(c)[at[:, 0], at[:, 1]].astype(np.float64), ref, s)


@pytest.mark.parametrize("M", [1, 33, 65, 128])
def test_several_rounds_of_tiles(M):
    """149 column tiles on at most 74 pairs; the rows of a 256-row product, bit for bit."""
    N = 28512
    a, b = synth.normal_bf16((256, K), 1), synth.normal_bf16((N, K), 2, 0.02)
    (ca, sa), (cb, sb) = base._oracle_operand(a), base._oracle_operand(b)
    args = (dev_u8(cb), dev_u8(to_mma(sb, K)), K)
    da, dsa = dev_u8(ca), dev_u8(to_mma(sa, K))
    c32, tall = mx.mxfp4_gemm(da[:M], dsa, *args), mx.mxfp4_gemm(da, dsa, *args)
    assert torch.equal(c32, tall[:M])
    assert torch.equal(mx.mxfp4_gemm_bf16(da[:M], dsa, *args), tall[:M].to(torch.bfloat16))
    q = mx.mxfp4_gemm_mxfp4(da[:M], dsa, *args)
    qt = mx.mxfp4_gemm_mxfp4(da, dsa, *args)
    assert torch.equal(q.codes, qt.codes[:M]) and torch.equal(q.scales, qt.scales[:M])
    assert mx.mxfp4_get_error() == mx.MXFP4_OK
    g = np.random.default_rng(M)
    pairs = list(zip(g.integers(0, M, 400), g.integers(0, N, 400))) + [(0, 0), (M - 1, N - 1)]
    ref, s = oracle.gemm_entries(ca, sa, cb, sb, K, pairs)
    assert_gemm_close(np.array([c32[m, n].item() for m, n in pairs], np.float64), ref, s)


@pytest.mark.parametrize("M", [1, 33, 65, 128])
def test_nvfp4_several_rounds_of_tiles(M):
    N = 28512
    qa = mx.mxfp4_nvfp4_quantize(dev_bf16(synth.normal_bf16((256, K), 3)), scale_layout=mx.SCALES_MMA)
    qb = mx.mxfp4_nvfp4_quantize(dev_bf16(synth.normal_bf16((N, K), 4, 0.02)), scale_layout=mx.SCALES_MMA)
    few = mx.NvQuantized(qa.codes[:M], qa.scales, qa.amax, M, K, qa.layout, qa.scale_layout)
    assert torch.equal(mx.mxfp4_nvfp4_gemm(few, qb), mx.mxfp4_nvfp4_gemm(qa, qb)[:M])
    assert mx.mxfp4_get_error() == mx.MXFP4_OK

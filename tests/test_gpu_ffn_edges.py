"""GPU: calls of the expert feed-forward operators at the edges of what they
document.  Bounds as in test_gpu_ffn, or derived beside the check."""
import numpy as np
import pytest
import torch

import ffn_testutil as ffn
import oracle
import quantize_block_scaled_rht_b200 as mx
import synth
import test_gpu_ffn as base
from mxfp4_testutil import dev_bf16
from test_gpu_ffn import GEMM_REL, assert_within, f64, no_error, operand

pytestmark = pytest.mark.gpu

NO_LIMIT = dict(alpha=1.702, limit=float("inf"), beta=0.5)


# ------------------------------------------------------------------ gated backward: extreme z
@pytest.mark.parametrize("act", [ffn.SWIGLU, ffn.CLAMPED, NO_LIMIT])
@pytest.mark.parametrize("M", [3, 150])
def test_gated_backward_of_gates_near_the_largest_finite_value(M, act):
    """alpha g may leave FP32's range although g does not.  A gate far below zero
    passes nothing.  One far above has s = 1 and 1 - s = 0, so dz = dh (u + beta)
    and dh g (0 beyond the limit)."""
    I, K = 72, 128
    ca, sa, da, dsa = operand(M, K, 3, 1e-2)
    cb, sb, db, dsb = operand(I, K, 4, 0.1)
    z = np.random.default_rng(5).standard_normal((M, 2 * I)).astype(np.float32)
    gates = np.array([-3.3e38, -2.9e38, -2.1e38, 2.1e38, 2.9e38, 3.3e38], np.float32)
    z[:, 0::2] = gates[np.arange(M * I).reshape(M, I) % 6]
    zb = synth.bf16_bits(z)
    dz = f64(mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, dev_bf16(zb), K, **act))
    no_error()
    dh, s = oracle.gemm(ca, sa, cb, sb, K)
    z64 = synth.bf16_to_f32(zb).astype(np.float64)
    below, above = z64[:, 0::2] < 0, z64[:, 0::2] > 0
    assert np.all(dz[:, 0::2][below] == 0) and np.all(dz[:, 1::2][below] == 0)
    g, u = np.minimum(z64[:, 0::2], act["limit"]), np.clip(z64[:, 1::2], -act["limit"], act["limit"])
    if np.isinf(act["limit"]):
        # s = 1 and the derivative 1 exactly; two FP32 roundings, then bf16's
        for k, f in ((0, u + act["beta"]), (1, g)):
            want = dh * f
            slack = GEMM_REL * s * np.abs(f) + 3 * 2.0 ** -24 * np.abs(want)
            assert_within(dz[:, k::2][above], want[above],
                          (ffn.BF16_HALF * (np.abs(want) + slack) + slack + ffn.FLOOR)[above], "dz")
    else:
        assert np.all(dz[:, 0::2][above] == 0)
        want, bound = ffn.gated_backward(dh, np.where(z64 > 1e30, 100.0, np.maximum(z64, -100.0)), **act), \
            ffn.gated_backward_bound(dh, GEMM_REL * s, np.where(z64 > 1e30, 100.0, np.maximum(z64, -100.0)), **act)
        assert_within(dz[:, 1::2][above], want[:, 1::2][above], bound[:, 1::2][above], "dz up")


@pytest.mark.parametrize("act", [ffn.SWIGLU, ffn.CLAMPED])
@pytest.mark.parametrize("M", [3, 150])
def test_gated_backward_nan_pre_activations(M, act):
    """NaN in a gate gives NaN in both gradients of the pair, NaN in an up value in
    its own and, unless the gate is beyond the limit, in the gate's."""
    I, K = 72, 128
    _, _, da, dsa = operand(M, K, 3, 1e-2)
    _, _, db, dsb = operand(I, K, 4, 0.1)
    z = dev_bf16(synth.normal_bf16((M, 2 * I), 5, 1.0))
    clean = f64(mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, z, K, **act))
    z[1, 10] = float("nan")                # gate of pair 5
    z[2, 21] = float("nan")                # up of pair 10
    z[0, 30], z[0, 31] = 8.0, float("nan")
    dz = f64(mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, z, K, **act))
    no_error()
    bad = np.zeros(dz.shape, bool)
    bad[1, 10:12] = bad[2, 20:22] = True
    bad[0, 31], bad[0, 30] = True, np.isinf(act["limit"])
    assert np.array_equal(np.isnan(dz), bad)
    if not np.isinf(act["limit"]):
        assert dz[0, 30] == 0
    bad[0, 30:32] = True
    assert np.array_equal(dz[~bad], clean[~bad])


# ------------------------------------------------------------------ one buffer
def test_outputs_in_other_columns_of_an_operands_buffer():
    """Refused only where bytes are shared: h, z, the int8 product and its codes beside
    the operand they come from, at its row stride."""
    M, I, K = 150, 64, 128
    _, _, da, dsa = operand(M, K, 1, 1.0)
    _, _, db, dsb = operand(2 * I, K, 2, 0.2)
    want = mx.mxfp4_gated_gemm(da, dsa, db, dsb, K, save_z=True)
    buf = torch.zeros((M, K // 2 + 6 * I), dtype=torch.uint8, device="cuda")
    buf[:, :K // 2] = da
    wide = buf.view(torch.bfloat16)
    h, z = wide[:, K // 4:K // 4 + I], wide[:, K // 4 + I:]
    mx.mxfp4_gated_gemm(buf[:, :K // 2], dsa, db, dsb, K, out=h, z_out=z)
    assert torch.equal(h, want[0]) and torch.equal(z, want[1]) and torch.equal(buf[:, :K // 2], da)
    want = mx.mxfp4_int8_quantize(want[0])
    buf = torch.zeros((M, 4 * I), dtype=torch.int8, device="cuda")
    x = buf.view(torch.bfloat16)[:, :I]
    x.copy_(h)
    q = mx.mxfp4_int8_quantize(x, out=mx.Int8Quantized(buf[:, 2 * I:3 * I], torch.empty(M, device="cuda")))
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales) and torch.equal(x, h)
    one = torch.ones(M, device="cuda")
    y = mx.mxfp4_int8_gemm(want.codes, one, want.codes[:I // 4], one[:I // 4])
    out = buf.view(torch.bfloat16)[:, 3 * I // 2:3 * I // 2 + I // 4]
    mx.mxfp4_int8_gemm(q.codes, one, want.codes[:I // 4], one[:I // 4], out=out)
    assert torch.equal(out, y) and torch.equal(q.codes, want.codes)
    no_error()


# ------------------------------------------------------------------ few rows, large products
@pytest.mark.parametrize("M,I,K", [(1, 226_000, 64), (2, 3300, 4096), (3, 2900, 2880), (4, 2900, 2880), (3, 56_600, 64),
                                   (4, 1500, 2880), (2, 2200, 4096)])
@pytest.mark.parametrize("keep", [False, True])
def test_gated_few_rows_on_both_sides_of_the_kernels_limit(M, I, K, keep):
    """One to four rows by the tile kernel and (the last two sizes) the streaming one."""
    base.test_gated_gemm(M, I, K, keep, ffn.CLAMPED)


@pytest.mark.parametrize("M,N,K", [(2, 2_000_000, 64), (3, 209_000, 208), (4, 209_000, 208), (1, 500_000, 208),
                                   (4, 60_000, 208)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_int8_few_rows_on_both_sides_of_the_kernels_limit(M, N, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    a = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    b = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    out = mx.mxfp4_int8_gemm(a, torch.ones(M, device="cuda"), b, torch.ones(N, device="cuda"), out_dtype=dtype)
    no_error()
    # unit scales and sums below 2^24: exact in FP32, bf16 the sum rounded once
    assert torch.equal(out, (a.double() @ b.double().t()).to(torch.float32).to(dtype))

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


@pytest.mark.parametrize("act", [ffn.SWIGLU, NO_LIMIT])
@pytest.mark.parametrize("M", [3, 150])
def test_gated_backward_where_the_up_gradient_overflows(M, act):
    """dh g beyond the largest finite value is an infinity in the up value's gradient
    and nothing else: the gate's is dh (u + beta), or 0 where s is."""
    I, K = 72, 128
    ca, sa, da, dsa = operand(M, K, 3, 1e3)
    cb, sb, db, dsb = operand(I, K, 4, 10.0)
    z = np.random.default_rng(5).standard_normal((M, 2 * I)).astype(np.float32)
    z[:, 0::2] = np.array([-3.3e38, -2.9e38, 2.9e38, 3.3e38], np.float32)[np.arange(M * I).reshape(M, I) % 4]
    zb = synth.bf16_bits(z)
    dz = f64(mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, dev_bf16(zb), K, **act))
    no_error()
    dh, s = oracle.gemm(ca, sa, cb, sb, K)
    z64 = synth.bf16_to_f32(zb).astype(np.float64)
    below, above = z64[:, 0::2] < 0, z64[:, 0::2] > 0
    assert np.all(dz[:, 0::2][below] == 0) and np.all(dz[:, 1::2][below] == 0)
    far = above & (np.abs(dh) > 10 + GEMM_REL * s)
    assert far.sum() > 0.4 * far.size and np.array_equal(dz[:, 1::2][far], np.copysign(np.inf, dh[far]))
    u = z64[:, 1::2] + act["beta"]
    want = dh * u
    slack = GEMM_REL * s * np.abs(u) + 3 * 2.0 ** -24 * np.abs(want)
    assert_within(dz[:, 0::2][above], want[above], (ffn.BF16_HALF * (np.abs(want) + slack) + slack + ffn.FLOOR)[above], "dz gate")


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


# ------------------------------------------------------------------ columns that end inside 16 bytes
def padded(t):
    """t as the first columns of rows that start on 16 bytes, as the operators take them."""
    rows, cols = t.shape
    wide = torch.full((rows, (cols + 15) // 8 * 8), 11.0, dtype=t.dtype, device="cuda")
    wide[:, :cols] = t
    return wide[:, :cols]


def check_backward(M, I, K, act):
    ca, sa, da, dsa = operand(M, K, M + 1, 1e-2)
    cb, sb, db, dsb = operand(I, K, I + 1, 1.0 / K ** 0.5)
    zb = base.z_values(M, I, M + I)
    z = padded(dev_bf16(zb))
    dz = mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, z, K, **act)
    no_error()
    dh, s = oracle.gemm(ca, sa, cb, sb, K)
    z64 = synth.bf16_to_f32(zb).astype(np.float64)
    assert dz.shape == (M, 2 * I)
    assert_within(f64(dz), ffn.gated_backward(dh, z64, **act), ffn.gated_backward_bound(dh, GEMM_REL * s, z64, **act), "dz")
    mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, z, K, **act, out=z)       # in place
    assert torch.equal(z, dz) and torch.all(z._base[:, 2 * I:] == 11)


ODD = [(1, 1, 64), (3, 7, 128), (5, 33, 64), (40, 2, 64), (130, 101, 320), (128, 98, 512), (300, 31, 2880), (257, 501, 576),
       (64, 1606, 64), (1000, 263, 192), (1300, 2182, 128)]


@pytest.mark.parametrize("act", base.ACTS)
@pytest.mark.parametrize("M,I,K", ODD)
def test_gated_odd_columns(M, I, K, act):
    ca, sa, da, dsa = operand(M, K, M + K, 1.5)
    cb, sb, db, dsb = operand(2 * I, K, I, 2.0 / K ** 0.5)
    h, z = mx.mxfp4_gated_gemm(da, dsa, db, dsb, K, **act, save_z=True)
    no_error()
    ref, s = oracle.gemm(ca, sa, cb, sb, K)
    assert h.shape == (M, I) and z.shape == (M, 2 * I)
    assert_within(f64(h), ffn.gated(ref, **act), ffn.gated_bound(ref, GEMM_REL * s, **act), "h")
    assert_within(f64(z), ref, ffn.BF16_HALF * (np.abs(ref) + GEMM_REL * s) + GEMM_REL * s + ffn.FLOOR, "z")
    check_backward(M, I, K, act)


@pytest.mark.parametrize("M,I,K", [(3500, 1343, 64), (23000, 99, 64), (4000, 13, 576), (20, 29998, 64), (100, 29999, 320)])
def test_gated_backward_odd_columns_last_round_in_pieces(M, I, K):
    check_backward(M, I, K, ffn.CLAMPED)


@pytest.mark.parametrize("I", [55, 57, 58])
@pytest.mark.parametrize("M", [4, 150])
def test_gated_odd_columns_leave_what_stands_behind_them(M, I):
    K = 128
    ca, sa, da, dsa = operand(M, K, 41, 1e-2)
    cb, sb, db, dsb = operand(I, K, 42, 0.1)
    zb = base.z_values(M, I, 43)
    ldz = (2 * I + 37) // 8 * 8
    z = torch.full((M + 1, ldz), 11.0, dtype=torch.bfloat16, device="cuda")
    z[:M, :2 * I] = dev_bf16(zb)
    out = torch.full((M + 1, ldz + 8), 13.0, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, z[:M, :2 * I], K, **ffn.CLAMPED, out=out[:M, :2 * I])
    no_error()
    dh, s = oracle.gemm(ca, sa, cb, sb, K)
    z64 = synth.bf16_to_f32(zb).astype(np.float64)
    assert_within(f64(out[:M, :2 * I]), ffn.gated_backward(dh, z64, **ffn.CLAMPED),
                  ffn.gated_backward_bound(dh, GEMM_REL * s, z64, **ffn.CLAMPED), "dz")
    assert torch.all(out[:, 2 * I:] == 13) and torch.all(out[M] == 13)
    mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, z[:M, :2 * I], K, **ffn.CLAMPED, out=z[:M, :2 * I])
    assert torch.equal(z[:M, :2 * I], out[:M, :2 * I])
    assert torch.all(z[:, 2 * I:] == 11) and torch.all(z[M] == 11)
    # forward: h and z in wider buffers
    _, _, dw, dsw = operand(2 * I, K, 44, 0.1)
    want_h, want_z = mx.mxfp4_gated_gemm(da, dsa, dw, dsw, K, **ffn.CLAMPED, save_z=True)
    h = torch.full((M + 1, ldz), 7.0, dtype=torch.bfloat16, device="cuda")
    zo = torch.full((M + 1, ldz), 9.0, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_gated_gemm(da, dsa, dw, dsw, K, **ffn.CLAMPED, out=h[:M, :I], z_out=zo[:M, :2 * I])
    assert torch.equal(h[:M, :I], want_h) and torch.equal(zo[:M, :2 * I], want_z)
    assert torch.all(h[:, I:] == 7) and torch.all(h[M] == 7) and torch.all(zo[:, 2 * I:] == 9) and torch.all(zo[M] == 9)


@pytest.mark.parametrize("sizes,I,K", [([1, 130, 0, 257, 128], 95, 256), ([300, 5, 64], 202, 576), ([0, 17], 1, 64),
                                       ([33] * 40, 54, 128), ([700, 900, 0, 100], 2879, 64)])
def test_grouped_gated_odd_columns(sizes, I, K):
    """Rows of 2I columns in a wider buffer; the columns behind them and the rows
    between the groups stay, in place too."""
    act = ffn.CLAMPED
    c = base.grouped_operands(sizes, I, K, 51, 1e-2, 0.1, slack=1)
    w = base.grouped_operands(sizes, 2 * I, K, 61, 1.0, 0.2, slack=1)
    ld = (2 * I + 15) // 8 * 8
    z = torch.full((c["rows"], ld), 5.0, dtype=torch.bfloat16, device="cuda")
    zb = base.z_values(c["rows"], I, 52)
    z[:, :2 * I] = dev_bf16(zb)
    out = torch.full((c["rows"], ld), 9.0, dtype=torch.bfloat16, device="cuda")
    args = (c["a"][2], c["a"][3], c["d_off"], c["d_sizes"], c["b"], c["sb"], z[:, :2 * I], K)
    mx.mxfp4_grouped_gated_gemm_backward(*args, **act, out=out[:, :2 * I])
    h = torch.full((w["rows"], ld), 9.0, dtype=torch.bfloat16, device="cuda")
    zo = torch.full((w["rows"], ld), 9.0, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_grouped_gated_gemm(w["a"][2], w["a"][3], w["d_off"], w["d_sizes"], w["b"], w["sb"], K, **act, out=h[:, :I],
                                z_out=zo[:, :2 * I])
    no_error()
    z64 = synth.bf16_to_f32(zb).astype(np.float64)
    written = torch.zeros(c["rows"], dtype=torch.bool)
    for g, n in enumerate(sizes):
        o = int(c["offsets"][g])
        written[o:o + n] = True
        if n:
            dh, s = oracle.gemm(c["a"][0][o:o + n], c["a"][1][o:o + n], c["ws"][g][0], c["ws"][g][1], K)
            zz = z64[o:o + n]
            assert_within(f64(out[o:o + n, :2 * I]), ffn.gated_backward(dh, zz, **act),
                          ffn.gated_backward_bound(dh, GEMM_REL * s, zz, **act), "dz")
            ref, s = oracle.gemm(w["a"][0][o:o + n], w["a"][1][o:o + n], w["ws"][g][0], w["ws"][g][1], K)
            assert_within(f64(h[o:o + n, :I]), ffn.gated(ref, **act), ffn.gated_bound(ref, GEMM_REL * s, **act), "h")
            assert_within(f64(zo[o:o + n, :2 * I]), ref, ffn.BF16_HALF * (np.abs(ref) + GEMM_REL * s) + GEMM_REL * s + ffn.FLOOR, "z")
    for t, n in ((out, 2 * I), (h, I), (zo, 2 * I)):
        assert torch.all(t[~written] == 9) and torch.all(t[:, n:] == 9)
    before = z.clone()
    mx.mxfp4_grouped_gated_gemm_backward(*args, **act, out=z[:, :2 * I])
    assert torch.equal(z[written, :2 * I], out[written, :2 * I])
    assert torch.equal(z[~written], before[~written]) and torch.equal(z[:, 2 * I:], before[:, 2 * I:])


# ------------------------------------------------------------------ dropout's counter
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("first", [2 ** 32 - 1000, 2 ** 32 - 100_000_000, 2 ** 32, 3 * 2 ** 32 + 12345])
def test_dropout_block_numbers_past_32_bits(first, dtype):
    """A large tensor whose Philox blocks (four elements each) start before 2^32 and
    run past it inside the launch, and ones that lie behind it: rows on both sides
    draw the words of their 64-bit number."""
    rows, cols = 150_000, 4096                                  # 153.6 M blocks
    x = torch.ones((rows, cols), dtype=dtype, device="cuda")
    y = mx.mxfp4_dropout(x, 0.5, 5, 4 * first)
    cross = (2 ** 32 - first) * 4 // cols
    at = {0, 1, 2, 3, rows // 2, rows - 1} | {r for r in range(cross - 2, cross + 3) if 0 <= r < rows}
    for r in sorted(at):
        want = ffn.dropout_words(cols, 5, 4 * first + r * cols) >= (1 << 31)
        assert np.array_equal(y[r].float().cpu().numpy() == 2, want), r

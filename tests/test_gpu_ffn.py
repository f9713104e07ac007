"""GPU: the expert feed-forward operators (gated product forward and backward,
int8 quantizer and product, dropout) against plain 64-bit forms.

The pre-activations and dh come from the fp64 oracle product with its bound
1e-5 * sum|a b|; ffn_testutil derives what the activation and the one rounding
to bf16 add.  int8 sums are exact, so with unit scales the FP32 product is the
correctly rounded integer.  Codes and dropout are bit-exact.
"""
import numpy as np
import pytest
import torch

import ffn_testutil as ffn
import oracle
import quantize_block_scaled_rht_b200 as mx
import synth
from mxfp4_testutil import dev_bf16, dev_u8, host, to_mma

pytestmark = pytest.mark.gpu

ACTS = [ffn.SWIGLU, ffn.CLAMPED]
GEMM_REL = 1e-5


def f64(t):
    return t.detach().double().cpu().numpy()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def operand(rows, k, seed, std):
    """MXFP4 of N(0, std^2): host codes and scales, device codes and GEMM-ready scales."""
    c, s = oracle.quantize(synth.normal_bf16((rows, k), seed, std), oracle.LAYOUT_1D_ROW)[:2]
    return c, s, dev_u8(c), dev_u8(to_mma(s, k))


def grouped_operands(sizes, N, K, seed, std_a, std_b, slack=0):
    """Routed rows (each group from a multiple of 128, `slack` extra row tiles at the end) and G weights."""
    offsets = np.zeros(len(sizes) + 1, np.int32)
    offsets[1:] = np.cumsum([(s + 127) // 128 * 128 for s in sizes])
    rows = max(int(offsets[-1]), 128) + 128 * slack
    a = operand(rows, K, seed, std_a)
    ws = [operand(N, K, seed + 1 + g, std_b) for g in range(len(sizes))]
    return dict(sizes=sizes, offsets=offsets, rows=rows, a=a, ws=ws, d_off=dev(offsets), d_sizes=dev(np.asarray(sizes, np.int32)),
                b=torch.stack([w[2] for w in ws]), sb=torch.cat([w[3] for w in ws]))


def assert_within(got, want, bound, what):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside; worst {np.max(np.abs(got - want) / bound)}"


def no_error():
    assert mx.mxfp4_get_error() == mx.MXFP4_OK


# ------------------------------------------------------------------ gated product
FWD = [(1, 8, 64), (2, 96, 128), (3, 1000, 64), (7, 40, 2880), (8, 96, 4160), (9, 96, 128), (37, 48, 192), (128, 96, 512), (130, 104, 320),
       (300, 200, 2880), (257, 500, 576), (513, 64, 64),
       (4, 16, 12032), (3, 16, 4096),
       (1100, 2500, 128), (2600, 700, 320)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("M,I,K", FWD)
def test_gated_gemm(M, I, K, keep, act):
    ca, sa, da, dsa = operand(M, K, M + K, 1.5)
    cb, sb, db, dsb = operand(2 * I, K, I, 2.0 / K ** 0.5)
    h, z = mx.mxfp4_gated_gemm(da, dsa, db, dsb, K, **act, save_z=keep)
    no_error()
    ref, s = oracle.gemm(ca, sa, cb, sb, K)
    assert h.shape == (M, I) and h.dtype == torch.bfloat16
    assert_within(f64(h), ffn.gated(ref, **act), ffn.gated_bound(ref, GEMM_REL * s, **act), "h")
    if keep:
        assert_within(f64(z), ref, ffn.BF16_HALF * (np.abs(ref) + GEMM_REL * s) + GEMM_REL * s + ffn.FLOOR, "z")
        if M > 64:     # the same accumulators as the bf16 product's
            assert torch.equal(z, mx.mxfp4_gemm_bf16(da, dsa, db, dsb, K))
    else:
        assert z is None


@pytest.mark.parametrize("M", [1, 5, 200])
def test_gated_gemm_strided_outputs_and_rows(M):
    I, K = 72, 256
    ca, sa, _, dsa = operand(M, K, 3, 1.0)
    cb, sb, _, dsb = operand(2 * I, K, 4, 0.2)
    a = torch.zeros((M, K), dtype=torch.uint8, device="cuda")
    b = torch.zeros((2 * I, K), dtype=torch.uint8, device="cuda")
    a[:, :K // 2], b[:, :K // 2] = dev_u8(ca), dev_u8(cb)
    out = torch.full((M + 2, I + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    zo = torch.full((M + 2, 2 * I + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_gated_gemm(a[:, :K // 2], dsa, b[:, :K // 2], dsb, K, out=out[1:M + 1, :I], z_out=zo[1:M + 1, :2 * I])
    no_error()
    ref, s = oracle.gemm(ca, sa, cb, sb, K)
    assert_within(f64(out[1:M + 1, :I]), ffn.gated(ref, **ffn.SWIGLU), ffn.gated_bound(ref, GEMM_REL * s, **ffn.SWIGLU), "h")
    assert torch.all(out[:, I:] == 3) and torch.all(out[0] == 3) and torch.all(out[M + 1] == 3)
    assert torch.all(zo[:, 2 * I:] == 5) and torch.all(zo[0] == 5) and torch.all(zo[M + 1] == 5)


@pytest.mark.parametrize("M", [3, 140])
def test_gated_gemm_nan_scales_stay_in_their_rows(M):
    I, K = 96, 256
    ca, sa, da, _ = operand(M, K, 5, 1.0)
    cb, sb, db, _ = operand(2 * I, K, 6, 0.2)
    sa, sb = sa.copy(), sb.copy()
    sa[1, 3] = 0xFF
    sb[2 * 7 + 1, 0] = 0xFF           # up row of column 7
    h, z = mx.mxfp4_gated_gemm(da, dev_u8(to_mma(sa, K)), db, dev_u8(to_mma(sb, K)), K, **ffn.CLAMPED, save_z=True)
    no_error()
    bad = np.zeros((M, I), bool)
    bad[1] = bad[:, 7] = True
    assert np.array_equal(np.isnan(f64(h)), bad)
    badz = np.zeros((M, 2 * I), bool)
    badz[1] = badz[:, 15] = True
    assert np.array_equal(np.isnan(f64(z)), badz)


@pytest.mark.parametrize("M", [2, 150])
def test_gated_gemm_large_and_tiny_values(M):
    """Pre-activations of thousands (the exponential over- and underflows) and of 1e-30."""
    I, K = 64, 128
    for std in (1e3, 1e-30):
        ca, sa, da, dsa = operand(M, K, 8, std)
        cb, sb, db, dsb = operand(2 * I, K, 9, 1.0)
        ref, s = oracle.gemm(ca, sa, cb, sb, K)
        for act in ACTS:
            h, _ = mx.mxfp4_gated_gemm(da, dsa, db, dsb, K, **act)
            with np.errstate(over="ignore"):
                want, bound = ffn.gated(ref, **act), ffn.gated_bound(ref, GEMM_REL * s, **act)
            # s at an exponent x beyond -60: below 1e-26 of the row's values either way
            bound = bound + 1e-20 * np.abs(ref).max()
            assert_within(f64(h), want, bound, f"h at {std}")


@pytest.mark.parametrize("sizes,I,K", [([1, 130, 0, 257, 128], 96, 256), ([300, 5, 64], 200, 576), ([0, 0, 17], 8, 64),
                                       ([33] * 40, 48, 128), ([700, 900, 0, 100], 2880, 64)])
@pytest.mark.parametrize("keep", [False, True])
def test_grouped_gated_gemm(sizes, I, K, keep):
    c = grouped_operands(sizes, 2 * I, K, 11, 1.0, 0.2, slack=1)
    out = torch.full((c["rows"], I), 9.0, dtype=torch.bfloat16, device="cuda")
    zo = torch.full((c["rows"], 2 * I), 9.0, dtype=torch.bfloat16, device="cuda") if keep else None
    mx.mxfp4_grouped_gated_gemm(c["a"][2], c["a"][3], c["d_off"], c["d_sizes"], c["b"], c["sb"], K, **ffn.CLAMPED, out=out,
                                z_out=zo)
    no_error()
    written = np.zeros(c["rows"], bool)
    for g, n in enumerate(sizes):
        o = int(c["offsets"][g])
        written[o:o + n] = True
        if n:
            ref, s = oracle.gemm(c["a"][0][o:o + n], c["a"][1][o:o + n], c["ws"][g][0], c["ws"][g][1], K)
            assert_within(f64(out[o:o + n]), ffn.gated(ref, **ffn.CLAMPED), ffn.gated_bound(ref, GEMM_REL * s, **ffn.CLAMPED), "h")
            if keep:
                assert_within(f64(zo[o:o + n]), ref, ffn.BF16_HALF * (np.abs(ref) + GEMM_REL * s) + GEMM_REL * s + ffn.FLOOR, "z")
    assert torch.all(out[~torch.from_numpy(written)] == 9)
    if keep:
        assert torch.all(zo[~torch.from_numpy(written)] == 9)


@pytest.mark.parametrize("offsets,sizes,kept", [([0, 100, 256], [10, 20], 100), ([-128, 0, 256], [10, 20], 20),
                                                 ([0, 128, 512], [10, 300], 10), ([128, 0, 256], [10, 20], 20),
                                                 ([0, 128, 256], [-5, 129], 0)])
def test_grouped_gated_bad_groups_are_reported_and_skipped(offsets, sizes, kept):
    """Groups off a 128-row boundary, before the first row, past the end, backwards,
    of a negative or too large size: reported, and nothing of them is written."""
    c = grouped_operands([10, 20], 64, 64, 3, 1.0, 0.2)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full((c["rows"], 32), 9.0, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_grouped_gated_gemm(c["a"][2], c["a"][3], i32(offsets), i32(sizes), c["b"], c["sb"], 64, out=out)
    assert mx.mxfp4_get_error() == mx.MXFP4_ERR_INVALID_ARG
    assert torch.all(out[kept:] == 9)
    no_error()


# ------------------------------------------------------------------ gated backward
def z_values(rows, I, seed):
    """Pre-activations of both signs with values on, next to and beyond the clamps."""
    g = np.random.default_rng(seed)
    z = (g.standard_normal((rows, 2 * I)) * 4).astype(np.float32)
    edge = np.array([0.0, -0.0, 7.0, -7.0, 7.03125, -7.03125, 6.96875, 30.0, -40.0, 1e-20], np.float32)
    at = g.random(z.shape) < 0.2
    z[at] = edge[g.integers(0, len(edge), int(at.sum()))]
    return synth.bf16_bits(z)


BWD = [(1, 8, 64), (5, 40, 128), (128, 96, 512), (130, 104, 320), (300, 200, 2880), (257, 500, 576), (64, 1600, 64),
       (1000, 260, 192), (1300, 2180, 128), (2600, 1004, 576)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,I,K", BWD)
def test_gated_backward(M, I, K, act):
    ca, sa, da, dsa = operand(M, K, M + 1, 1e-2)
    cb, sb, db, dsb = operand(I, K, I + 1, 1.0 / K ** 0.5)
    zb = z_values(M, I, M + I)
    z = dev_bf16(zb)
    dz = mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, z, K, **act)
    no_error()
    dh, s = oracle.gemm(ca, sa, cb, sb, K)
    z64 = synth.bf16_to_f32(zb).astype(np.float64)
    assert_within(f64(dz), ffn.gated_backward(dh, z64, **act), ffn.gated_backward_bound(dh, GEMM_REL * s, z64, **act), "dz")
    # in place: the same bits, z overwritten
    again = mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, z, K, **act, out=z)
    no_error()
    assert again is z and torch.equal(z, dz)


@pytest.mark.parametrize("M,I,K", [(3500, 1344, 64), (3400, 1332, 192), (23000, 100, 64), (4000, 12, 576), (300, 1152, 320),
                                   (20, 30000, 64), (100, 30000, 320)])
def test_gated_backward_last_round_in_pieces(M, I, K):
    """Tiles of one or several rounds whose last is cut: both tile widths, pieces
    that end inside their columns and ones past the last column."""
    test_gated_backward(M, I, K, ffn.CLAMPED)


@pytest.mark.parametrize("act", ACTS)
def test_gated_backward_against_differences_of_the_forward(act):
    """dz against central differences of the 64-bit forward form, not its derivative."""
    M, I, K = 140, 72, 192
    ca, sa, da, dsa = operand(M, K, 31, 1.0)
    cb, sb, db, dsb = operand(I, K, 32, 0.3)
    zb = synth.normal_bf16((M, 2 * I), 33, 3.0)
    z = synth.bf16_to_f32(zb).astype(np.float64)
    dz = f64(mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, dev_bf16(zb), K, **act))
    dh, s = oracle.gemm(ca, sa, cb, sb, K)
    step = 1e-5
    num = np.empty_like(z)
    for k in (0, 1):
        d = np.zeros_like(z)
        d[:, k::2] = step
        num[:, k::2] = (ffn.gated(z + d, **act) - ffn.gated(z - d, **act)) / (2 * step) * dh
    away = np.abs(np.abs(z) - act["limit"]) > 2 * step
    bound = ffn.gated_backward_bound(dh, GEMM_REL * s, z, **act) + 1e-7 * np.abs(dh).max()
    assert np.all((np.abs(num - dz) <= bound)[away]) and away.mean() > 0.9


def test_gated_backward_strided_and_nan():
    M, I, K = 150, 56, 128
    ca, sa, da, _ = operand(M, K, 41, 1e-2)
    cb, sb, db, dsb = operand(I, K, 42, 0.1)
    sa = sa.copy()
    sa[3, 0] = 0xFF
    zb = z_values(M, I, 43)
    z = torch.full((M + 1, 2 * I + 16), 11.0, dtype=torch.bfloat16, device="cuda")
    z[:M, :2 * I] = dev_bf16(zb)
    z[9, 20] = float("nan")
    out = torch.full((M + 1, 2 * I + 8), 13.0, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_gated_gemm_backward(da, dev_u8(to_mma(sa, K)), db, dsb, z[:M, :2 * I], K, **ffn.CLAMPED, out=out[:M, :2 * I])
    no_error()
    dh, s = oracle.gemm(ca, sa, cb, sb, K)
    z64 = f64(z[:M, :2 * I])
    got = f64(out[:M, :2 * I])
    want, bound = ffn.gated_backward(dh, z64, **ffn.CLAMPED), ffn.gated_backward_bound(dh, GEMM_REL * s, z64, **ffn.CLAMPED)
    ok = np.ones((M, 2 * I), bool)
    ok[3] = False
    ok[9, 20:22] = False
    assert np.all((np.abs(got - want) <= bound)[ok])
    assert np.all(np.isnan(got[9, 20:22]))
    past = (z64[3, 0::2] > 7) | False
    assert np.all(got[3, 0::2][past] == 0) and np.all(np.isnan(got[3, 0::2][~past]))
    assert torch.all(out[:, 2 * I:] == 13) and torch.all(out[M] == 13)


@pytest.mark.parametrize("sizes,I,K", [([1, 130, 0, 257, 128], 96, 256), ([300, 5, 64], 200, 576), ([0, 17], 8, 64),
                                       ([33] * 40, 52, 128), ([700, 400], 1000, 64), ([700, 900, 0, 100], 2880, 64)])
def test_grouped_gated_backward(sizes, I, K):
    c = grouped_operands(sizes, I, K, 51, 1e-2, 0.1, slack=1)
    zb = z_values(c["rows"], I, 52)
    out = torch.full((c["rows"], 2 * I), 9.0, dtype=torch.bfloat16, device="cuda")
    z = dev_bf16(zb)
    args = (c["a"][2], c["a"][3], c["d_off"], c["d_sizes"], c["b"], c["sb"], z, K)
    mx.mxfp4_grouped_gated_gemm_backward(*args, **ffn.CLAMPED, out=out)
    no_error()
    z64 = synth.bf16_to_f32(zb).astype(np.float64)
    written = torch.zeros(c["rows"], dtype=torch.bool)
    for g, n in enumerate(sizes):
        o = int(c["offsets"][g])
        written[o:o + n] = True
        if n:
            dh, s = oracle.gemm(c["a"][0][o:o + n], c["a"][1][o:o + n], c["ws"][g][0], c["ws"][g][1], K)
            zz = z64[o:o + n]
            assert_within(f64(out[o:o + n]), ffn.gated_backward(dh, zz, **ffn.CLAMPED),
                          ffn.gated_backward_bound(dh, GEMM_REL * s, zz, **ffn.CLAMPED), "dz")
    assert torch.all(out[~written] == 9)
    before = z.clone()
    mx.mxfp4_grouped_gated_gemm_backward(*args, **ffn.CLAMPED, out=z)      # in place
    assert torch.equal(z[written], out[written]) and torch.equal(z[~written], before[~written])


# ------------------------------------------------------------------ int8 quantizer
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (33, 256), (5, 272), (64, 512), (9, 1040), (130, 2880), (7, 4112),
                                       (31, 5760), (4, 8208), (5, 11520), (3, 16400), (2, 33040), (2, 70000)])
def test_int8_quantize_bit_exact(rows, cols):
    x = synth.student_t_bf16((rows, cols), seed=rows + cols)
    q = mx.mxfp4_int8_quantize(dev_bf16(x))
    codes, scales = ffn.int8_quantize(synth.bf16_to_f32(x))
    assert np.array_equal(host(q.codes), codes)
    assert np.array_equal(host(q.scales).view(np.uint32), scales.view(np.uint32))
    assert np.abs(codes).max() == 127


def test_int8_quantize_special_rows():
    cols = 96
    g = np.random.default_rng(2)
    x = g.standard_normal((14, cols)).astype(np.float32)
    x[0] = 0.0
    x[1] = -0.0
    x[2, 5] = np.inf
    x[3, 95] = -np.inf
    x[4, 0] = np.nan
    x[5] *= 1e-38                     # subnormal and least normal values
    x[6] *= 2.0 ** -100               # around the floor
    x[7] *= 1e38
    x[8, :] = 127.0                   # ties: x * (127 / 127) = 0.5, 1.5, ...
    x[8, :64] = np.arange(64) + 0.5
    x[9] = -x[8]
    x[10, :] = 3.3895e38
    x[11, :] = 0; x[11, 17] = 1e-40   # noqa: E702
    x[12, 1] = 3.3895e38
    x[13, :] = np.float32(2.0 ** -100)
    bits = synth.bf16_bits(np.nan_to_num(x, nan=0, posinf=0, neginf=0))
    bits[2, 5], bits[3, 95], bits[4, 0] = 0x7F80, 0xFF80, 0xFFC1
    q = mx.mxfp4_int8_quantize(dev_bf16(bits))
    codes, scales = ffn.int8_quantize(synth.bf16_to_f32(bits))
    assert np.array_equal(host(q.codes), codes)
    got = host(q.scales)
    assert np.array_equal(np.isnan(got), np.isnan(scales)) and np.isnan(got[[2, 3, 4]]).all()
    ok = ~np.isnan(scales)
    assert np.array_equal(got[ok].view(np.uint32), scales[ok].view(np.uint32))
    assert not host(q.codes)[[0, 1, 2, 3, 4]].any()


def test_int8_quantize_every_bf16_value_and_strides():
    every = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    fin = every[(every & 0x7F80) != 0x7F80]
    x = np.concatenate([fin, fin[:(-len(fin)) % 1024]]).reshape(-1, 1024)
    wide = torch.zeros((x.shape[0], 1024 + 64), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:1032] = dev_bf16(x)
    out = mx.Int8Quantized(torch.full((x.shape[0], 2048), 99, dtype=torch.int8, device="cuda")[:, 16:1040],
                           torch.empty(x.shape[0], device="cuda"))
    mx.mxfp4_int8_quantize(wide[:, 8:1032], out=out)
    codes, scales = ffn.int8_quantize(synth.bf16_to_f32(x))
    assert np.array_equal(host(out.codes), codes) and np.array_equal(host(out.scales), scales)
    base = out.codes._base if out.codes._base is not None else out.codes
    assert torch.all(base[:, :16] == 99) and torch.all(base[:, 1040:] == 99)


# ------------------------------------------------------------------ int8 product
I8_SHAPES = [(1, 8, 16), (1, 200, 2880), (2, 13, 48), (4, 64, 5760), (5, 260, 144), (8, 512, 1040), (9, 40, 272), (16, 300, 512),
             (17, 256, 256), (64, 96, 2880), (129, 257, 528), (256, 256, 256), (300, 1000, 208), (513, 72, 4112),
             (40, 48, 240), (2, 72, 112), (100, 24, 496), (1100, 2700, 208), (5000, 600, 272)]


def int8_operands(M, N, K, seed, G=None):
    g = np.random.default_rng(seed)
    a = g.integers(-128, 128, (M, K), dtype=np.int8)
    b = g.integers(-128, 128, (N, K) if G is None else (G, N, K), dtype=np.int8)
    return a, b


def exact_sums(a, b):
    return (a.astype(np.float64) @ b.astype(np.float64).T)     # integers below 2^53: exact


def pad_cols(N, dtype):
    e = 16 // (2 if dtype == torch.bfloat16 else 4)
    return (N + e - 1) // e * e


@pytest.mark.parametrize("M,N,K", I8_SHAPES)
def test_int8_gemm_sums_are_exact(M, N, K):
    """Unit scales: the FP32 product is the nearest FP32 to the integer sum, the bf16 one that rounded again."""
    a, b = int8_operands(M, N, K, M * 7 + N)
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((M + 1, pad_cols(N, dtype)), 7.0, dtype=dtype, device="cuda")
        mx.mxfp4_int8_gemm(dev(a), one(M), dev(b), one(N), out=out[:M, :N])
        no_error()
        want = torch.from_numpy(exact_sums(a, b).astype(np.float32)).to(dtype)
        assert torch.equal(out[:M, :N].cpu(), want)
        assert torch.all(out[M] == 7) and torch.all(out[:, N:] == 7)


@pytest.mark.parametrize("M,N,K", [(2048, 2880, 64), (1900, 2850, 272), (4000, 2880, 48), (1024, 5700, 32), (19000, 250, 32),
                                   (40, 19500, 48), (100, 19500, 272), (200, 19000, 128)])
def test_int8_gemm_last_round_in_pieces(M, N, K):
    """Several rounds of tiles whose last is cut, the last columns in one piece or two."""
    test_int8_gemm_sums_are_exact(M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 96, 2880), (7, 136, 272), (16, 72, 96), (130, 200, 528)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_int8_gemm_scales(M, N, K, dtype):
    a, b = int8_operands(M, N, K, 5)
    g = np.random.default_rng(6)
    sa = (10.0 ** g.uniform(-6, 3, M)).astype(np.float32)
    sb = (10.0 ** g.uniform(-6, 3, N)).astype(np.float32)
    got = f64(mx.mxfp4_int8_gemm(dev(a), dev(sa), dev(b), dev(sb), out_dtype=dtype))
    no_error()
    want = exact_sums(a, b) * sa.astype(np.float64)[:, None] * sb.astype(np.float64)[None]
    # the sum, and each factor: three roundings of 2^-24, and bf16's
    rel = (1 + 2.0 ** -24) ** 3 - 1
    rel = rel if dtype == torch.float32 else rel + ffn.BF16_HALF * (1 + rel)
    assert np.all(np.abs(got - want) <= rel * np.abs(want))


@pytest.mark.parametrize("M", [1, 3, 20])
def test_int8_gemm_largest_sums(M):
    """K just below the limit, every product 2^14 or -2^14 + 128: the 32-bit sums neither wrap nor saturate."""
    K, N = 131056, 24
    a = np.full((M, K), -128, np.int8)
    b = np.full((N, K), -128, np.int8)
    b[1::2] = 127
    b[2, :K // 2] = 127
    got = mx.mxfp4_int8_gemm(dev(a), torch.ones(M, device="cuda"), dev(b), torch.ones(N, device="cuda"), out_dtype=torch.float32)
    no_error()
    assert np.array_equal(host(got), exact_sums(a, b).astype(np.float32))


def test_int8_gemm_nan_scales_and_strides():
    for M in (3, 70):
        N, K = 40, 64
        a, b = int8_operands(M, N, K, 9)
        wa = torch.zeros((M, K + 32), dtype=torch.int8, device="cuda")
        wb = torch.zeros((N, K + 16), dtype=torch.int8, device="cuda")
        wa[:, 16:16 + K], wb[:, :K] = dev(a), dev(b)
        sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
        sa[2], sb[5] = float("nan"), float("nan")
        out = f64(mx.mxfp4_int8_gemm(wa[:, 16:16 + K], sa, wb[:, :K], sb, out_dtype=torch.float32))
        bad = np.zeros((M, N), bool)
        bad[2] = bad[:, 5] = True
        assert np.array_equal(np.isnan(out), bad)
        assert np.array_equal(out[~bad], exact_sums(a, b)[~bad])


@pytest.mark.parametrize("sizes,N,K", [([1, 130, 0, 257, 128], 192, 256), ([300, 5, 64], 260, 528), ([0, 17], 8, 16),
                                       ([33] * 40, 72, 144), ([2, 0, 1, 1], 2880, 1440), ([700, 900, 0, 100], 2880, 80)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_int8_grouped_gemm(sizes, N, K, dtype):
    G = len(sizes)
    offsets = np.zeros(G + 1, np.int32)
    offsets[1:] = np.cumsum([(s + 127) // 128 * 128 for s in sizes])
    rows = int(offsets[-1]) + 128
    a, b = int8_operands(rows, N, K, 12, G)
    g = np.random.default_rng(13)
    sa, sb = g.uniform(0.5, 2, rows).astype(np.float32), g.uniform(0.5, 2, (G, N)).astype(np.float32)
    wide = torch.full((rows, pad_cols(N, dtype)), 9.0, dtype=dtype, device="cuda")
    out = wide[:, :N]
    mx.mxfp4_int8_grouped_gemm(dev(a), dev(sa), dev(offsets), dev(np.asarray(sizes, np.int32)), dev(b), dev(sb), out=out)
    no_error()
    rel = (1 + 2.0 ** -24) ** 3 - 1
    rel = rel if dtype == torch.float32 else rel + ffn.BF16_HALF * (1 + rel)
    got, written = f64(out), np.zeros(rows, bool)
    for i, n in enumerate(sizes):
        o = int(offsets[i])
        written[o:o + n] = True
        want = exact_sums(a[o:o + n], b[i]) * sa[o:o + n].astype(np.float64)[:, None] * sb[i].astype(np.float64)[None]
        assert np.all(np.abs(got[o:o + n] - want) <= rel * np.abs(want))
    assert np.all(got[~written] == 9) and torch.all(wide[:, N:] == 9)


# ------------------------------------------------------------------ dropout
def drop_want(x, p, seed, off=0, residual=None):
    y = ffn.dropout_f32(x.float().cpu().numpy(), p, seed, off, None if residual is None else residual.float().cpu().numpy())
    return torch.from_numpy(y).to(x.dtype)


def same_bits(a, b):
    t = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.cpu().contiguous().view(t), b.cpu().contiguous().view(t))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 3), (1, 8), (1, 1001), (7, 13), (64, 40), (5, 2880), (33, 36), (301, 4099)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("res", [False, True])
def test_dropout_bit_exact(rows, cols, dtype, res):
    g = torch.Generator().manual_seed(rows * 10007 + cols)
    x = torch.randn((rows, cols), generator=g).to(dtype).cuda()
    r = torch.randn((rows, cols), generator=g).to(dtype).cuda() if res else None
    for p, seed, off in ((0.1, 42, 0), (0.5, 0xFEDCBA9876543210, 4 * ((1 << 34) - 3)), (0.0, 1, 8), (1.0, 1, 0), (1e-3, 3, 0)):
        y = mx.mxfp4_dropout(x, p, seed, off, residual=r)
        assert same_bits(y, drop_want(x, p, seed, off, r)), (p, seed, off)
    assert torch.equal(mx.mxfp4_dropout(x, 0.0, 7), x)
    z = mx.mxfp4_dropout(x, 1.0, 7, residual=r)
    assert torch.equal(z, r if res else torch.zeros_like(x))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dropout_strides_alignment_and_in_place(dtype):
    big = torch.randn((50, 200), generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    for sl in ((slice(1, 31), slice(8, 88)), (slice(0, 30), slice(1, 82)), (slice(2, 5), slice(3, 4)), (slice(4, 5), slice(5, 150))):
        x, r = big[sl], big.flip(0)[sl]
        out = torch.full((50, 256), 5.0, dtype=dtype, device="cuda")
        o = out[1:1 + x.shape[0], 8:8 + x.shape[1]]
        mx.mxfp4_dropout(x, 0.3, 9, residual=r, out=o)
        want = drop_want(x, 0.3, 9, 0, r)
        assert same_bits(o, want)
        o.fill_(5.0)
        assert torch.all(out == 5)
        y = big.clone()
        mx.mxfp4_dropout(y[sl], 0.3, 9, residual=r, out=y[sl])
        assert same_bits(y[sl], want)
        y2 = big.flip(0).contiguous()
        mx.mxfp4_dropout(x, 0.3, 9, residual=y2[sl], out=y2[sl])
        assert same_bits(y2[sl], want)
        rest = torch.ones_like(big, dtype=torch.bool)
        rest[sl] = False
        assert torch.equal(y[rest], big[rest])


def test_dropout_masks_nan_and_inf_and_slices_draw_the_whole_mask():
    rows, cols, seed = 96, 352, 11
    x = torch.randn((rows, cols), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    whole = mx.mxfp4_dropout(x, 0.4, seed)
    dropped = ffn.dropout_words(rows * cols, seed).reshape(rows, cols) < round(0.4 * 2 ** 32)
    bad = x.clone()
    bad[:, ::2], bad[:, 1::2] = float("nan"), float("-inf")
    y = mx.mxfp4_dropout(bad, 0.4, seed).float().cpu().numpy()
    assert np.all(y[dropped] == 0) and not np.isfinite(y[~dropped]).any()
    parts = [mx.mxfp4_dropout(x[o:o + n], 0.4, seed, o * cols) for o, n in ((0, 32), (32, 1), (33, 63))]
    assert torch.equal(torch.cat(parts), whole)
    # the backward pass draws the same mask
    dy = torch.ones_like(x)
    assert torch.equal(mx.mxfp4_dropout(dy, 0.4, seed) != 0, torch.from_numpy(~dropped).cuda())


def test_dropout_index_past_32_bits():
    """More than 2^32 / 8 groups: the last rows of a 2.4 GB tensor draw the words of their 64-bit index."""
    rows, cols = 300_000, 4096
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda")
    base = (1 << 33) - 4 * 1000
    y = mx.mxfp4_dropout(x, 0.5, 5, base)
    for r in (0, 1, 200_000, rows - 1):
        want = ffn.dropout_words(cols, 5, base + r * cols) >= (1 << 31)
        assert np.array_equal(y[r].float().cpu().numpy() == 2, want)


# ------------------------------------------------------------------ together
def test_expert_block_forward_and_backward_together():
    """One step of the block: quantize X -> gated product (h, z) -> int8 tokens ->
    down product -> dropout onto the residual; back: dropout of dY -> quantize ->
    gated backward.  Each stage is held to its plain form on the stage's own inputs."""
    T, H, I, act = 333, 320, 192, ffn.CLAMPED
    x = synth.activations_with_outliers(T, H, seed=2)
    wgu = synth.normal_bf16((2 * I, H), 3, 0.05)
    wd = synth.normal_bf16((H, I), 4, 0.05)
    qx = mx.mxfp4_quantize(dev_bf16(x), scale_layout=mx.SCALES_MMA)
    qw = mx.mxfp4_quantize(dev_bf16(wgu), mx.LAYOUT_2D, scale_layout=mx.SCALES_MMA)
    qwd = mx.mxfp4_quantize(dev_bf16(wd), mx.LAYOUT_2D, scale_layout=mx.SCALES_MMA, transposed_copy=True)
    h, z = mx.mxfp4_gated_gemm(qx.codes, qx.scales, qw.codes, qw.scales, H, **act, save_z=True)
    qh, q8 = mx.mxfp4_int8_quantize(h), mx.mxfp4_int8_quantize(dev_bf16(wd))
    y = mx.mxfp4_int8_gemm(qh.codes, qh.scales, q8.codes, q8.scales)
    out = mx.mxfp4_dropout(y, 0.1, 42, residual=dev_bf16(x))
    no_error()
    cx, sx = oracle.quantize(x, oracle.LAYOUT_1D_ROW)[:2]
    cw, sw, _ = oracle.quantize(wgu, oracle.LAYOUT_2D, transposed_copy=True)
    ref, s = oracle.gemm(cx, sx, cw, sw, H, 0, 1)
    assert_within(f64(h), ffn.gated(ref, **act), ffn.gated_bound(ref, GEMM_REL * s, **act), "h")
    codes, scales = ffn.int8_quantize(h.float().cpu().numpy())
    assert np.array_equal(host(qh.codes), codes) and np.array_equal(host(qh.scales), scales)
    want = exact_sums(codes, host(q8.codes)) * scales.astype(np.float64)[:, None] * f64(q8.scales)[None]
    assert np.all(np.abs(f64(y) - want) <= (ffn.BF16_HALF + 1e-6) * np.abs(want))
    assert same_bits(out, drop_want(y, 0.1, 42, 0, dev_bf16(x)))
    # h in int8 and back stands for h to half a step of its token
    assert np.all(np.abs(codes * scales[:, None] - f64(h)) <= (0.5 + 1e-4) * scales[:, None])
    dy = dev_bf16(synth.normal_bf16((T, H), 7, 1e-2))
    dyd = mx.mxfp4_dropout(dy, 0.1, 42)
    qdy = mx.mxfp4_quantize(dyd, scale_layout=mx.SCALES_MMA)
    dz = mx.mxfp4_gated_gemm_backward(qdy.codes, qdy.scales, qwd.codes_t, qwd.scales_t, z, H, **act)
    no_error()
    cdy, sdy = oracle.quantize(host(dyd), oracle.LAYOUT_1D_ROW)[:2]
    _, swd, cwt = oracle.quantize(wd, oracle.LAYOUT_2D, transposed_copy=True)
    dh, s = oracle.gemm(cdy, sdy, cwt, swd, H, 0, 2)
    assert_within(f64(dz), ffn.gated_backward(dh, f64(z), **act), ffn.gated_backward_bound(dh, GEMM_REL * s, f64(z), **act), "dz")


def test_graph_capture_replay_and_side_streams():
    """The block captured in a CUDA graph and replayed on new inputs equals eager
    calls, and so do calls on another stream than the tensors'."""
    K, I, act = 256, 96, ffn.CLAMPED
    for M in (3, 200):
        ops = [operand(M, K, 60 + i, 1.0) for i in range(2)]
        _, _, db, dsb = operand(2 * I, K, 70, 0.2)
        _, _, dt, dst = operand(I, K, 71, 0.2)
        w8 = mx.mxfp4_int8_quantize(dev_bf16(synth.normal_bf16((64, I), 5, 0.1)))
        a, sa = ops[0][2].clone(), ops[0][3].clone()

        def step(stream=None):
            h, z = mx.mxfp4_gated_gemm(a, sa, db, dsb, K, **act, save_z=True, stream=stream)
            dz = mx.mxfp4_gated_gemm_backward(a, sa, dt, dst, z, K, **act, stream=stream)
            q = mx.mxfp4_int8_quantize(h, stream=stream)
            y = mx.mxfp4_int8_gemm(q.codes, q.scales, w8.codes, w8.scales, stream=stream)
            return h, z, dz, q.codes, q.scales, mx.mxfp4_dropout(y, 0.2, 3, residual=y, stream=stream)

        eager = [t.clone() for t in step()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = step(stream=side)
        raw = step(stream=side.cuda_stream)
        torch.cuda.synchronize()
        for e, o, r in zip(eager, other, raw):
            assert torch.equal(e, o) and torch.equal(e, r)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step()
        for k in (1, 0, 1):
            a.copy_(ops[k][2])
            sa.copy_(ops[k][3])
            graph.replay()
            torch.cuda.synchronize()
            for c, e in zip(captured, step()):
                assert torch.equal(c, e)
        no_error()


def test_outputs_in_other_columns_of_the_inputs_buffer():
    M, I, K = 150, 40, 128
    _, _, da, dsa = operand(M, K, 1, 1e-2)
    _, _, db, dsb = operand(I, K, 2, 0.1)
    buf = torch.zeros((M, 4 * I), dtype=torch.bfloat16, device="cuda")
    buf[:, :2 * I] = dev_bf16(z_values(M, I, 3))
    want = mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, buf[:, :2 * I].clone(), K)
    mx.mxfp4_gated_gemm_backward(da, dsa, db, dsb, buf[:, :2 * I], K, out=buf[:, 2 * I:])
    assert torch.equal(buf[:, 2 * I:], want)
    x = torch.randn((30, 64), generator=torch.Generator().manual_seed(1)).cuda()
    want = mx.mxfp4_dropout(x[:, :32].clone(), 0.3, 4)
    mx.mxfp4_dropout(x[:, :32], 0.3, 4, out=x[:, 32:])
    assert torch.equal(x[:, 32:], want)


def test_calls_at_once_on_two_streams():
    """The operators keep no state between calls: two streams at once give what one gives."""
    M, I, K = 520, 384, 512
    ops = [(operand(M, K, 10 + i, 1.0)[2:], operand(2 * I, K, 20 + i, 0.1)[2:], operand(I, K, 30 + i, 0.1)[2:]) for i in range(2)]
    w8 = mx.mxfp4_int8_quantize(dev_bf16(synth.normal_bf16((200, I), 5, 0.1)))

    def step(i, stream=None):
        (a, sa), (b, sb), (t, st) = ops[i]
        h, z = mx.mxfp4_gated_gemm(a, sa, b, sb, K, **ffn.CLAMPED, save_z=True, stream=stream)
        dz = mx.mxfp4_gated_gemm_backward(a, sa, t, st, z, K, **ffn.CLAMPED, stream=stream)
        q = mx.mxfp4_int8_quantize(h, stream=stream)
        y = mx.mxfp4_int8_gemm(q.codes, q.scales, w8.codes, w8.scales, stream=stream)
        return h, z, dz, q.codes, q.scales, mx.mxfp4_dropout(y, 0.2, i, stream=stream)

    want = [[t.clone() for t in step(i)] for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[step(i, streams[i]) for i in range(2)] for _ in range(20)]
    torch.cuda.synchronize()
    no_error()
    for pair in got:
        for w, g in zip(want, pair):
            assert all(torch.equal(x, y) for x, y in zip(w, g))


FIRST_CALL = """
import sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import torch
import quantize_block_scaled_rht_b200 as mx
g = torch.Generator(device="cuda").manual_seed(1)
u8 = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=g)
M, I, K = int(sys.argv[2]), 96, 256
a, b, t = u8(M, K // 2), u8(2 * I, K // 2), u8(I, K // 2)
sc = lambda n: torch.full((mx.mma_scales_bytes(n, K),), 124, dtype=torch.uint8, device="cuda")
sa, sb, st = sc(M), sc(2 * I), sc(I)
w, ws = torch.randint(-127, 128, (64, I), dtype=torch.int8, device="cuda", generator=g), torch.rand(64, device="cuda", generator=g)
def step():
    h, z = mx.mxfp4_gated_gemm(a, sa, b, sb, K, save_z=True)
    dz = mx.mxfp4_gated_gemm_backward(a, sa, t, st, z, K)
    q = mx.mxfp4_int8_quantize(h)
    y = mx.mxfp4_int8_gemm(q.codes, q.scales, w, ws)
    return h, z, dz, q.codes, y, mx.mxfp4_dropout(y, 0.2, 3)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, step())) and mx.mxfp4_get_error() == 0
print("ok")
"""


@pytest.mark.parametrize("M", [2, 300])
def test_first_call_of_a_process_inside_a_capture(M):
    import subprocess
    import sys
    from conftest import ROOT
    r = subprocess.run([sys.executable, "-c", FIRST_CALL, ROOT, str(M)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


def test_repeated_calls_give_the_same_bits():
    """No atomics: every operator is deterministic."""
    M, I, K = 700, 400, 704
    _, _, da, dsa = operand(M, K, 1, 1.0)
    _, _, db, dsb = operand(2 * I, K, 2, 0.1)
    first = mx.mxfp4_gated_gemm(da, dsa, db, dsb, K, save_z=True)
    for _ in range(5):
        again = mx.mxfp4_gated_gemm(da, dsa, db, dsb, K, save_z=True)
        assert all(torch.equal(x, y) for x, y in zip(first, again))

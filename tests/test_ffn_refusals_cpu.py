"""Refusals of the expert feed-forward operators that need no GPU: outputs over
operands.  Every call here is refused before anything is launched, so the
pointers are never dereferenced."""
import ctypes

import pytest

import quantize_block_scaled_rht_b200 as mx

INF = float("inf")
BAD = mx.MXFP4_ERR_INVALID_ARG


def at(base, off=0):
    return ctypes.c_void_p(base + off)


# operands far from each other and from the outputs; 4 rows of A, 128 of B, K = 64
A, SA, B, SB, OFF, SIZES, OUT, Z = (0x10000000 * (i + 1) for i in range(8))
M, N, K = 300, 128, 64
A_BYTES, SA_BYTES, B_BYTES, SB_BYTES = M * 32, 3 * 512, N * 32, 512
OPERANDS = {"a": (A, A_BYTES), "a_scales": (SA, SA_BYTES), "b": (B, B_BYTES), "b_scales": (SB, SB_BYTES)}
GROUP_TABLE = {"offsets": (OFF, 12), "sizes": (SIZES, 8)}


def spots(base, size, out_bytes):
    """Places of an output of out_bytes that shares the operand's first or last 16 bytes, or holds it all."""
    last = (base + size - 1) // 16 * 16
    return [base, last, (base - out_bytes + 16) // 16 * 16]


def gated(out, z):
    return mx.lib().mxfp4_gated_gemm(at(A), 32, at(SA), at(B), 32, at(SB), M, N, K, 1.0, INF, 0.0, at(out), 64, at(z), 128, None)


def gated_bwd(out, z=Z):
    return mx.lib().mxfp4_gated_gemm_backward(at(A), 32, at(SA), at(B), 32, at(SB), M, N, K, 1.0, INF, 0.0, at(z), 256, at(out),
                                              256, None)


@pytest.mark.parametrize("name", OPERANDS)
def test_gated_outputs_over_operands(name):
    base, size = OPERANDS[name]
    for out in spots(base, size, M * 128):
        assert gated(out, Z) == BAD
    for z in spots(base, size, M * 256):
        assert gated(OUT, z) == BAD
    for out in spots(base, size, M * 512):
        assert gated_bwd(out) == BAD


@pytest.mark.parametrize("name", [*OPERANDS, *GROUP_TABLE])
def test_grouped_gated_outputs_over_operands(name):
    L, G = mx.lib(), 2
    base, size = {**OPERANDS, **GROUP_TABLE}[name]
    size *= G if name in ("b", "b_scales") else 1

    def fwd(out, z):
        return L.mxfp4_grouped_gated_gemm(at(A), 32, at(SA), M, at(OFF), at(SIZES), G, at(B), 32, at(SB), N, K, 1.0, INF, 0.0,
                                          at(out), 64, at(z), 128, None)

    def bwd(out):
        return L.mxfp4_grouped_gated_gemm_backward(at(A), 32, at(SA), M, at(OFF), at(SIZES), G, at(B), 32, at(SB), N, K, 1.0,
                                                   INF, 0.0, at(Z), 256, at(out), 256, None)

    for out in spots(base, size, M * 128):
        assert fwd(out, Z) == BAD
    for z in spots(base, size, M * 256):
        assert fwd(OUT, z) == BAD
    for out in spots(base, size, M * 512):
        assert bwd(out) == BAD


@pytest.mark.parametrize("dtype,size", [(mx.OUT_F32, 4), (mx.OUT_BF16, 2)])
@pytest.mark.parametrize("grouped", [False, True])
def test_int8_product_over_operands(grouped, dtype, size):
    L, G = mx.lib(), 2 if grouped else 1
    operands = {"a": (A, M * K), "b": (B, G * N * K), "a_scales": (SA, 4 * M), "b_scales": (SB, 4 * G * N)}
    if grouped:
        operands.update(GROUP_TABLE)
    for base, n in operands.values():
        for c in spots(base, n, M * N * size):
            if grouped:
                rc = L.mxfp4_int8_grouped_gemm(at(A), K, at(SA), M, at(OFF), at(SIZES), G, at(B), K, at(SB), N, K, at(c), N,
                                               dtype, None)
            else:
                rc = L.mxfp4_int8_gemm(at(A), K, at(SA), at(B), K, at(SB), M, N, K, at(c), N, dtype, None)
            assert rc == BAD


def test_int8_quantizer_over_its_input():
    L = mx.lib()

    def quantize(codes, scales, ldc=64):
        return L.mxfp4_int8_quantize(at(A), M, 64, 64, at(codes), ldc, at(scales), None)

    for codes in spots(A, M * 128, M * 64):
        assert quantize(codes, SA) == BAD
    assert quantize(A, SA, 128) == BAD                       # each row's codes over the row itself
    for scales in (A, A + 128 * M - 4, A - 4 * M + 4):
        assert quantize(OUT, scales) == BAD
    for scales in (OUT, OUT + 64 * M - 4, OUT - 4 * M + 4):
        assert quantize(OUT, scales) == BAD


@pytest.mark.parametrize("alpha", [3e38, -3e38, 2.4e38])
def test_alpha_whose_exponent_factor_overflows(alpha):
    """alpha * log2(e) has to be finite: times a gate of 0 an infinity would give NaN."""
    L = mx.lib()
    assert L.mxfp4_gated_gemm(at(A), 32, at(SA), at(B), 32, at(SB), M, N, K, alpha, INF, 0.0, at(OUT), 64, None, 0, None) == BAD
    assert L.mxfp4_gated_gemm_backward(at(A), 32, at(SA), at(B), 32, at(SB), M, N, K, alpha, INF, 0.0, at(Z), 256, at(OUT), 256,
                                       None) == BAD

"""Expert feed-forward operators, what needs no GPU: the plain forms against
independent checks (differences, the oracle's generator), and the refusals of
the C ABI and of the binding before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import ffn_testutil as ffn
import oracle
import quantize_block_scaled_rht_b200 as mx

INF = float("inf")


@pytest.mark.parametrize("act", [ffn.SWIGLU, ffn.CLAMPED])
def test_gated_backward_formula_equals_differences(act):
    g = np.random.default_rng(1)
    z = g.uniform(-9, 9, (64, 10))
    z[0] = 0.0
    dh = g.standard_normal((64, 5))
    dz = ffn.gated_backward(dh, z, **act)
    step = 1e-5
    for j in range(10):
        d = np.zeros_like(z)
        d[:, j] = step
        num = ((ffn.gated(z + d, **act) - ffn.gated(z - d, **act)) * dh).sum(axis=1) / (2 * step)
        far = np.abs(np.abs(z[:, j]) - act["limit"]) > 2 * step      # not across the clamp's corner
        # central differences: step^2 / 6 times the third derivative (below 20 here), and
        # roundings of 2^-53 * |h| / step
        assert np.all(np.abs(num - dz[:, j])[far] <= 1e-8)


def test_gated_at_the_clamp():
    a = ffn.CLAMPED
    z = np.array([[7.0, 7.0, 7.03125, -7.03125, -50.0, -7.0]])
    dz = ffn.gated_backward(np.ones((1, 3)), z, **a)
    assert dz[0, 0] != 0 and dz[0, 1] != 0          # on the border the gradient passes
    assert dz[0, 2] == 0 and dz[0, 3] == 0          # beyond it nothing does
    assert dz[0, 4] != 0                            # the gate has no lower clamp


def test_philox_of_the_tests_equals_the_oracles():
    ctr = np.array([[0, 0, 0, 0], [1, 2, 3, 4], [0xFFFFFFFF] * 4, [7, 0, 0, ffn.DROPOUT_TAG]], np.uint64)
    got = ffn.philox(ctr, (0xDEADBEEF, 0x12345678))
    L = oracle.lib()
    for row, want in zip(ctr, got):
        c = (ctypes.c_uint32 * 4)(*[int(v) for v in row])
        k = (ctypes.c_uint32 * 2)(0xDEADBEEF, 0x12345678)
        o = (ctypes.c_uint32 * 4)()
        L.orc_philox4x32_10(c, k, o)
        assert list(o) == [int(v) for v in want]


def test_dropout_words_of_a_slice_are_the_wholes():
    whole = ffn.dropout_words(4000, 77)
    assert np.array_equal(ffn.dropout_words(1000, 77, 1200), whole[1200:2200])
    share = np.mean(ffn.dropout_words(1 << 20, 5) < round(0.1 * 2 ** 32))
    assert abs(share - 0.1) < 6 * (0.09 / 2 ** 20) ** 0.5


FAKE, OFF = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
FAR = ctypes.c_void_p(0x10000000)


def _gated(alpha=1.0, limit=INF, beta=0.0, N=128, K=64, M=4, h=FAKE, ldh=64, z=FAR, ldz=128, a=FAKE, lda=32):
    return mx.lib().mxfp4_gated_gemm(a, lda, FAKE, FAKE, 32, FAKE, M, N, K, alpha, limit, beta, h, ldh, z, ldz, None)


@pytest.mark.parametrize("kw,want", [
    (dict(a=None), 1), (dict(h=None), 1), (dict(M=0), 1), (dict(N=0), 1), (dict(N=127), 1), (dict(K=80), 1),
    (dict(K=96, lda=48), 3), (dict(ldh=56), 1), (dict(ldz=120), 1), (dict(ldh=68), 2), (dict(ldz=132), 2),
    (dict(h=OFF), 2), (dict(z=OFF), 2), (dict(limit=0.0), 1), (dict(limit=-1.0), 1), (dict(limit=float("nan")), 1),
    (dict(alpha=INF), 1), (dict(alpha=float("nan")), 1), (dict(beta=INF), 1), (dict(z=FAKE), 1),
    (dict(z=ctypes.c_void_p(0x10000 + 3 * 128)), 1), (dict(M=1 << 32, z=None), 3)])
def test_gated_gemm_refusals(kw, want):
    assert _gated(**kw) == want


def _bwd(z=FAR, ldz=128, dz=FAKE, lddz=128, M=4, N=64, alpha=1.0, limit=INF):
    return mx.lib().mxfp4_gated_gemm_backward(FAKE, 32, FAKE, FAKE, 32, FAKE, M, N, 64, alpha, limit, 0.0, z, ldz, dz, lddz,
                                              None)


@pytest.mark.parametrize("kw,want", [
    (dict(z=None), 1), (dict(dz=None), 1), (dict(ldz=120), 1), (dict(lddz=120), 1), (dict(ldz=132), 2),
    (dict(z=OFF), 2), (dict(z=FAKE, ldz=136), 1), (dict(z=ctypes.c_void_p(0x10000 + 256)), 1), (dict(limit=0.0), 1)])
def test_gated_backward_refusals(kw, want):
    assert _bwd(**kw) == want


def test_columns_of_one_buffer_are_not_an_overlap():
    """Refused only where elements are shared: the calls below pass the overlap check
    and fail at a later one (a row count, an offset), so nothing is launched."""
    L = mx.lib()
    at = lambda off: ctypes.c_void_p(0x10000 + off)  # noqa: E731
    # bf16 rows of 64 elements: x in columns 0-31, y in 32-63 (apart) or 16-47 (shared)
    drop = lambda y, ld_y: L.mxfp4_dropout(at(0), 64, None, 0, 1 << 40, 32, mx.OUT_BF16, 0.5, 1, 0, at(y), ld_y, None)  # noqa: E731
    assert drop(32, 64) == mx.MXFP4_ERR_INVALID_ARG and drop(2 * 64 * 3 + 32, 64) == mx.MXFP4_ERR_INVALID_ARG
    assert drop(64, 72) == mx.MXFP4_ERR_INVALID_ARG
    big = 1 << 32                      # rows: unsupported, checked after the overlap
    bwd = lambda dz, ld: L.mxfp4_gated_gemm_backward(  # noqa: E731
        FAKE, 32, FAKE, FAKE, 32, FAKE, big, 16, 64, 1.0, INF, 0.0, at(0), 64, at(dz), ld, None)
    assert bwd(64, 64) == mx.MXFP4_ERR_UNSUPPORTED and bwd(0, 64) == mx.MXFP4_ERR_UNSUPPORTED
    assert bwd(32, 64) == mx.MXFP4_ERR_INVALID_ARG and bwd(64, 72) == mx.MXFP4_ERR_INVALID_ARG
    assert bwd(128 * 5 + 64, 64) == mx.MXFP4_ERR_UNSUPPORTED and bwd(128 * 5 + 96, 64) == mx.MXFP4_ERR_INVALID_ARG


def test_grouped_gated_refusals():
    L = mx.lib()
    f = lambda off=FAKE, sizes=FAKE, G=2, N=128: L.mxfp4_grouped_gated_gemm(  # noqa: E731
        FAKE, 32, FAKE, 256, off, sizes, G, FAKE, 32, FAKE, N, 64, 1.0, INF, 0.0, FAKE, 64, None, 0, None)
    assert f(off=None) == 1 and f(sizes=None) == 1 and f(G=0) == 1 and f(G=1025) == 3 and f(N=127) == 1
    assert f(G=1000, N=1 << 22) == 3


@pytest.mark.parametrize("args,want", [
    ((None, 4, 32, 32, FAKE, 32, FAKE), 1), ((FAKE, 4, 32, 32, None, 32, FAKE), 1), ((FAKE, 4, 32, 32, FAKE, 32, None), 1),
    ((FAKE, 0, 32, 32, FAKE, 32, FAKE), 1), ((FAKE, 4, 24, 32, FAKE, 32, FAKE), 1), ((FAKE, 4, 32, 24, FAKE, 32, FAKE), 1),
    ((FAKE, 4, 32, 32, FAKE, 16, FAKE), 1), ((FAKE, 4, 32, 36, FAKE, 32, FAKE), 2), ((FAKE, 4, 32, 32, FAKE, 40, FAKE), 2),
    ((OFF, 4, 32, 32, FAKE, 32, FAKE), 2), ((FAKE, 4, 32, 32, OFF, 32, FAKE), 2),
    ((FAKE, 4, 32, 32, FAKE, 32, ctypes.c_void_p(0x10002)), 2), ((FAKE, 1 << 31, 32, 32, FAKE, 32, FAKE), 3)])
def test_int8_quantize_refusals(args, want):
    assert mx.lib().mxfp4_int8_quantize(*args, None) == want


def _i8(a=FAKE, lda=64, sa=FAKE, b=FAKE, ldb=64, sb=FAKE, M=4, N=16, K=64, c=FAKE, ldc=16, dt=mx.OUT_F32):
    return mx.lib().mxfp4_int8_gemm(a, lda, sa, b, ldb, sb, M, N, K, c, ldc, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(a=None), 1), (dict(b=None), 1), (dict(sa=None), 1), (dict(sb=None), 1), (dict(c=None), 1), (dict(M=0), 1),
    (dict(N=0), 1), (dict(K=0), 1), (dict(K=40), 1), (dict(lda=48), 1), (dict(ldb=48), 1), (dict(ldc=12), 1),
    (dict(lda=72), 2), (dict(ldb=72), 2), (dict(ldc=18), 2), (dict(ldc=20, dt=mx.OUT_BF16), 2), (dict(a=OFF), 2),
    (dict(c=OFF), 2), (dict(sa=ctypes.c_void_p(0x10001)), 2), (dict(dt=7), 1),
    (dict(K=131072, lda=131072, ldb=131072), 3), (dict(M=1 << 32), 3)])
def test_int8_gemm_refusals(kw, want):
    assert _i8(**kw) == want


def _drop(x=FAR, ld_x=32, r=None, ld_r=0, rows=4, cols=32, dt=mx.OUT_BF16, p=0.5, off=0, y=FAKE, ld_y=32):
    return mx.lib().mxfp4_dropout(x, ld_x, r, ld_r, rows, cols, dt, p, 1, off, y, ld_y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(rows=0), 1), (dict(cols=-1), 1), (dict(dt=2), 1), (dict(p=-0.1), 1),
    (dict(p=1.01), 1), (dict(p=float("nan")), 1), (dict(off=2), 1), (dict(ld_x=31), 1), (dict(ld_y=31), 1),
    (dict(r=FAR, ld_r=16), 1), (dict(x=ctypes.c_void_p(0x10001)), 2),
    (dict(x=ctypes.c_void_p(0x20002), y=FAR, dt=mx.OUT_F32), 2),
    (dict(x=FAKE, ld_x=40), 1), (dict(x=ctypes.c_void_p(0x10002)), 1),
    (dict(r=ctypes.c_void_p(0x10000 + 64), ld_r=32), 1)])
def test_dropout_refusals(kw, want):
    assert _drop(**kw) == want


def test_bindings_refuse_before_the_abi():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    M, N, K = 256, 192, 512
    a, b = u8(M, K // 2), u8(N, K // 2)
    sa, sb = u8(mx.mma_scales_bytes(M, K)), u8(mx.mma_scales_bytes(N, K))
    with pytest.raises(ValueError, match="SCALES_MMA"):
        mx.mxfp4_gated_gemm(a, u8(M, K // 32), b, sb, K)
    with pytest.raises(ValueError, match="odd"):
        mx.mxfp4_gated_gemm(a, sa, b[:191], sb, K)
    with pytest.raises(ValueError, match="row-major"):
        mx.mxfp4_gated_gemm(a.t().contiguous().t(), sa, b, sb, K)
    with pytest.raises(ValueError, match="out must be"):
        mx.mxfp4_gated_gemm(a, sa, b, sb, K, out=bf(M, N))
    with pytest.raises(ValueError, match="z must be"):
        mx.mxfp4_gated_gemm(a, sa, b, sb, K, z_out=torch.zeros(M, N))
    with pytest.raises(ValueError, match="z must be"):
        mx.mxfp4_gated_gemm_backward(a, sa, b, sb, bf(M, N), K)
    with pytest.raises(ValueError, match="CUDA tensors"):
        mx.mxfp4_gated_gemm(a, sa, b, sb, K)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    bg, sbg = u8(2, N, K // 2), u8(2 * mx.mma_scales_bytes(N, K))
    for off, sizes in ((i32(0, 128), i32(1, 1)), (i32(0, 128, 256).long(), i32(1, 1)), (i32(0, 128, 256), i32(1))):
        with pytest.raises(ValueError):
            mx.mxfp4_grouped_gated_gemm(a, sa, off, sizes, bg, sbg, K)
    with pytest.raises(ValueError, match="contiguous groups"):
        mx.mxfp4_grouped_gated_gemm(a, sa, i32(0, 128, 256), i32(1, 1), u8(2, 2 * N, K // 2)[:, :N], sbg, K)
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8)  # noqa: E731
    f = lambda *s: torch.zeros(s)  # noqa: E731
    with pytest.raises(ValueError, match="int8"):
        mx.mxfp4_int8_gemm(a, f(M), i8(N, K // 2), f(N))
    with pytest.raises(ValueError, match="K = "):
        mx.mxfp4_int8_gemm(i8(M, K), f(M), i8(N, K // 2), f(N))
    with pytest.raises(ValueError, match="a_scales"):
        mx.mxfp4_int8_gemm(i8(M, K), f(M, 1), i8(N, K), f(N))
    with pytest.raises(ValueError, match="b_scales"):
        mx.mxfp4_int8_grouped_gemm(i8(M, K), f(M), i32(0, 128, 256), i32(1, 1), i8(2, N, K), f(N))
    with pytest.raises(ValueError, match="out_dtype"):
        mx.mxfp4_int8_gemm(i8(M, K), f(M), i8(N, K), f(N), out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out must be"):
        mx.mxfp4_int8_gemm(i8(M, K), f(M), i8(N, K), f(N), out=f(M, N + 1))
    with pytest.raises(ValueError, match="x must be"):
        mx.mxfp4_int8_quantize(f(4, 32))
    with pytest.raises(ValueError, match="x must be"):
        mx.mxfp4_int8_quantize(bf(32, 4).t())
    with pytest.raises(ValueError, match="CUDA tensors"):
        mx.mxfp4_int8_quantize(bf(4, 32))
    with pytest.raises(ValueError, match="x must be"):
        mx.mxfp4_dropout(f(4, 4).half(), 0.1, 1)
    with pytest.raises(ValueError, match="residual must be"):
        mx.mxfp4_dropout(f(4, 4), 0.1, 1, residual=bf(4, 4))
    with pytest.raises(ValueError, match="elem_offset"):
        mx.mxfp4_dropout(f(4, 4), 0.1, 1, elem_offset=-4)
    for p in (-0.5, 1.5, float("nan")):
        with pytest.raises(ValueError, match="p must be"):
            mx.mxfp4_dropout(f(4, 4), p, 1)
    with pytest.raises(ValueError, match="CUDA tensors"):
        mx.mxfp4_dropout(f(4, 4), 0.1, 1)

"""GPU: products whose columns end inside 16 bytes, into rows of a wider buffer:
the columns behind them are the caller's and stay."""
import numpy as np
import pytest
import torch

import oracle
import quantize_block_scaled_rht_b200 as mx
import synth
import test_gpu_gemm as base
from mxfp4_testutil import dev_bf16, dev_u8, host, to_mma

pytestmark = pytest.mark.gpu


def _wide(rows, N, dtype):
    """(buffer of 5s, its first N columns); its row stride is a multiple of 16 bytes."""
    buf = torch.full((rows, (N + 23) // 8 * 8), 5.0, dtype=dtype, device="cuda")
    return buf, buf[:, :N]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(1, 1, 64), (40, 3, 128), (128, 197, 320), (300, 210, 576), (130, 4095, 192)])
def test_dense(M, N, K, dtype):
    ca, sa = base._oracle_operand(synth.normal_bf16((M, K), 1))
    cb, sb = base._oracle_operand(synth.normal_bf16((N, K), 2, 0.1))
    buf, out = _wide(M, N, dtype)
    fn = mx.mxfp4_gemm if dtype == torch.float32 else mx.mxfp4_gemm_bf16
    fn(dev_u8(ca), dev_u8(to_mma(sa, K)), dev_u8(cb), dev_u8(to_mma(sb, K)), K, out=out)
    assert mx.mxfp4_get_error() == mx.MXFP4_OK
    ref, s = oracle.gemm(ca, sa, cb, sb, K)
    got = out.float().cpu().numpy()
    base.assert_gemm_close(got, ref, s) if dtype == torch.float32 else base._assert_bf16_close(got, ref, s)
    assert torch.all(buf[:, N:] == 5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [30, 300])
def test_every_remainder(M, dtype):
    """Last columns at every place of a box and of 16 bytes: the columns of a wider product, bit for bit."""
    N, K = 216, 128
    ca, sa = base._oracle_operand(synth.normal_bf16((M, K), 1))
    cb, sb = base._oracle_operand(synth.normal_bf16((N, K), 2, 0.1))
    a, b, s = (dev_u8(ca), dev_u8(to_mma(sa, K))), dev_u8(cb), dev_u8(to_mma(sb, K))
    fn = mx.mxfp4_gemm if dtype == torch.float32 else mx.mxfp4_gemm_bf16
    whole = fn(*a, b, s, K)
    for n in [*range(1, 74), *range(121, 138), *range(185, 217)]:
        buf, out = _wide(M, n, dtype)
        fn(*a, b[:n], s, K, out=out)
        assert torch.equal(out, whole[:, :n]) and torch.all(buf[:, n:] == 5), n
    assert mx.mxfp4_get_error() == mx.MXFP4_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,N,K", [([1, 130, 0, 257, 128], 195, 256), ([300, 5, 64], 390, 576)])
def test_grouped(sizes, N, K, dtype):
    sizes, offsets, rows, a, _ = base._grouped_case(sizes, N, K)
    G = len(sizes)
    w = [base._oracle_operand(synth.normal_bf16((N, K), 7 + g, 0.1)) for g in range(G)]
    ca, sa = base._oracle_operand(a)
    buf, out = _wide(rows, N, dtype)
    fn = mx.mxfp4_grouped_gemm if dtype == torch.float32 else mx.mxfp4_grouped_gemm_bf16
    fn(dev_u8(ca), dev_u8(to_mma(sa, K)), torch.from_numpy(offsets).cuda(), torch.from_numpy(sizes).cuda(),
       torch.stack([dev_u8(c) for c, _ in w]), torch.cat([dev_u8(to_mma(s, K)) for _, s in w]), N, K, out=out)
    assert mx.mxfp4_get_error() == mx.MXFP4_OK
    c = out.float().cpu().numpy()
    for g in range(G):
        o, n = int(offsets[g]), int(sizes[g])
        if n:
            ref, s = oracle.gemm(ca[o:o + n], sa[o:o + n], *w[g], K)
            base.assert_gemm_close(c[o:o + n], ref, s) if dtype == torch.float32 else base._assert_bf16_close(c[o:o + n], ref, s)
        assert np.all(c[o + n:int(offsets[g + 1])] == 5)
    assert torch.all(buf[:, N:] == 5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped_wgrad(dtype):
    M, N = 130, 197
    dy, x, offsets, K = base._routed_wgrad_case([200, 0, 300], M + 30, N + 27, seed=5)
    ca, sa = oracle.quantize(dy, oracle.LAYOUT_1D_COL)[:2]
    cb, sb = oracle.quantize(x, oracle.LAYOUT_1D_COL)[:2]
    ca, sa, cb, sb = ca[:M], sa[:M], cb[:N], sb[:N]
    G = len(offsets) - 1
    buf, out = _wide(G * M, N, dtype)
    fn = mx.mxfp4_grouped_gemm_wgrad if dtype == torch.float32 else mx.mxfp4_grouped_gemm_wgrad_bf16
    fn(dev_u8(ca), dev_u8(to_mma(sa, K)), dev_u8(cb), dev_u8(to_mma(sb, K)), torch.from_numpy(offsets).cuda(), K, out=out)
    assert mx.mxfp4_get_error() == mx.MXFP4_OK
    c = out.float().cpu().numpy()
    for g in range(G):
        o0, o1 = int(offsets[g]), int(offsets[g + 1])
        ce = c[g * M:(g + 1) * M]
        if o1 == o0:
            assert np.all(ce == 0)
            continue
        ref, s = oracle.gemm(ca[:, o0 // 2:o1 // 2], sa[:, o0 // 32:o1 // 32], cb[:, o0 // 2:o1 // 2], sb[:, o0 // 32:o1 // 32],
                             o1 - o0)
        base.assert_gemm_close(ce, ref, s) if dtype == torch.float32 else base._assert_bf16_close(ce, ref, s)
    assert torch.all(buf[:, N:] == 5)


def test_nvfp4():
    M, N, K = 130, 197, 320
    qa = mx.mxfp4_nvfp4_quantize(dev_bf16(synth.normal_bf16((144, K), 3)), scale_layout=mx.SCALES_MMA)
    qb = mx.mxfp4_nvfp4_quantize(dev_bf16(synth.normal_bf16((208, K), 4, 0.1)), scale_layout=mx.SCALES_MMA)
    want = host(mx.mxfp4_nvfp4_gemm(qa, qb))
    few = lambda q, n: mx.NvQuantized(q.codes[:n], q.scales, q.amax, n, K, q.layout, q.scale_layout)  # noqa: E731
    buf, out = _wide(M, N, torch.float32)
    mx.mxfp4_nvfp4_gemm(few(qa, M), few(qb, N), out=out)
    assert mx.mxfp4_get_error() == mx.MXFP4_OK
    assert np.array_equal(host(out), want[:M, :N]) and torch.all(buf[:, N:] == 5)

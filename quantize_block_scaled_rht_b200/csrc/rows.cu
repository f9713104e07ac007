// rows.cu -- the gated product and the int8 product for few rows of A (one to
// four tokens of decoding), where the time is reading B once.
//
// A tile of the tensor-core kernel would be almost empty there, and its 30 to 45
// tiles would leave most SMs without a load in flight: 5760 x 2880, 1 / 2 / 4 rows,
// gated 5.0 / 6.3 / 8.1 us against 7.4 there, int8 3.9 / 4.2 / 5.1 against 9.9
// (weights in L2; from HBM 5.7 / 6.8 / 9.8 against 8.0, and 5.5 / 6.0 / 6.8 against
// 11.0).  The integer work grows with the rows, so the tile kernel takes over where
// rows * N * K outgrows it (gated_by_rows, int8_by_rows), and at 5 rows: an
// 8-row gated form takes 11.8 us at that size, and an int8 one 12.3 (and 11.5
// against 14.5 at 2880 x 5760, 4.8 against 7.2 at 2880 x 1472: it was not kept).
// Here a CTA takes 8 rows of B: two groups of four rows, each walked by four
// warps that take the steps of K in turn, eight lanes to a row with 16 bytes each
// (128 consecutive bytes of a row per step).  Products are integer: four at a time by dp4a, an E2M1
// value doubled to one of 0, +-1, +-2, +-3, +-4, +-6, +-8, +-12.
#include <cstdint>

#include "common.cuh"
#include "ffn.cuh"

namespace mxfp4 {

namespace {

constexpr int KSPLIT = 4, GROUPS = 2, ROWS_PER_CTA = 4 * GROUPS, THREADS = 32 * KSPLIT * GROUPS;

__device__ __forceinline__ uint4 ld_nc_v4(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Four bytes of (a, b) chosen by the four low nibbles of sel: bits 0-2 the byte,
// bit 3 set: eight copies of its top bit instead.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// Eight E2M1 codes (one 32-bit word) to eight signed bytes 2 * value, in order.
// A code is a byte-permute selector: bits 0-2 pick the magnitude from the table
// and the sign bit replaces it by copies of its (clear) top bit, so the first
// permute keeps the positive elements and the second, on flipped signs, the
// negative ones; the difference is taken without borrows between bytes.
__device__ __forceinline__ void e2m1x8_doubled(uint32_t w, uint32_t &lo, uint32_t &hi) {
    constexpr uint32_t T0 = 0x03020100u, T1 = 0x0C080604u, TOP = 0x80808080u;
    const uint32_t n = w ^ 0x88888888u;
    lo = ((prmt(T0, T1, w) | TOP) - prmt(T0, T1, n)) ^ TOP;
    hi = ((prmt(T0, T1, w >> 16) | TOP) - prmt(T0, T1, n >> 16)) ^ TOP;
}

// 2^e as a product of two halves, each in range wherever the product is not zero
// or infinite by itself.
__device__ __forceinline__ float scale_pow2(float v, int e) {
    const int h = e >> 1;
    const float a = __uint_as_float((uint32_t)(max(h, -126) + 127) << 23);
    const float b = __uint_as_float((uint32_t)(max(e - h, -126) + 127) << 23);
    return __fmul_rn(__fmul_rn(v, a), b);
}

__device__ __forceinline__ float sum8(float v) {
    v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
    v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
    return __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
}
__device__ __forceinline__ int sum8(int v) {
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
    return v + __shfl_xor_sync(0xFFFFFFFFu, v, 1);
}

struct GatedRowsParams {
    const uint8_t *a, *sa, *b, *sb;
    int64_t lda, ldb, N;
    int M, K;
    GatedAct act;
    uint16_t *h, *z;
    int64_t ldh, ldz;
};

// MT: rows of A handled (M <= MT; rows past M repeat the last one).  Shared
// memory: the doubled bytes of A as two planes of 16 bytes per block (first and
// second half of every block, so that eight lanes' reads hit all banks), then
// the scale codes.
template <int MT>
__global__ void __launch_bounds__(THREADS) gated_rows_kernel(const GatedRowsParams p) {
    extern __shared__ __align__(16) uint8_t xs[];
    __shared__ float red[KSPLIT][ROWS_PER_CTA][MT];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nblk = p.K / 32, plane = nblk * 16;
    const int64_t katoms = mma_katoms(p.K);
    uint8_t *sc = xs + (int64_t)MT * p.K;
    for (int i = threadIdx.x; i < MT * nblk; i += THREADS) {
        const int m = i / nblk, kb = i - m * nblk, row = min(m, p.M - 1);
        const uint4 u = ld_nc_v4(p.a + row * p.lda + kb * 16);
        uint4 lo, hi;
        e2m1x8_doubled(u.x, lo.x, lo.y);
        e2m1x8_doubled(u.y, lo.z, lo.w);
        e2m1x8_doubled(u.z, hi.x, hi.y);
        e2m1x8_doubled(u.w, hi.z, hi.w);
        uint8_t *dst = xs + (int64_t)m * p.K + kb * 16;
        *reinterpret_cast<uint4 *>(dst) = lo;
        *reinterpret_cast<uint4 *>(dst + plane) = hi;
        sc[i] = p.sa[mma_scale_off(row, kb, katoms)];
    }
    __syncthreads();
    const int group = warp / KSPLIT, part = warp % KSPLIT, sub = lane >> 3, l8 = lane & 7;
    const int64_t row0 = (int64_t)blockIdx.x * ROWS_PER_CTA + 4 * group;
    const int64_t row = min(row0 + sub, p.N - 1);
    const uint8_t *b = p.b + row * p.ldb;
    float acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = 0.0f;
#pragma unroll 4
    for (int kb = part * 8 + l8; kb < nblk; kb += 8 * KSPLIT) {
        const uint4 u = ld_nc_v4(b + kb * 16);
        const int eb = p.sb[mma_scale_off(row, kb, katoms)];
        uint4 lo, hi;
        e2m1x8_doubled(u.x, lo.x, lo.y);
        e2m1x8_doubled(u.y, lo.z, lo.w);
        e2m1x8_doubled(u.z, hi.x, hi.y);
        e2m1x8_doubled(u.w, hi.z, hi.w);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint8_t *x = xs + m * p.K + kb * 16;
            const uint4 xl = *reinterpret_cast<const uint4 *>(x), xh = *reinterpret_cast<const uint4 *>(x + plane);
            const int ea = sc[m * nblk + kb];
            int s = __dp4a((int)lo.x, (int)xl.x, 0);
            s = __dp4a((int)lo.y, (int)xl.y, s);
            s = __dp4a((int)lo.z, (int)xl.z, s);
            s = __dp4a((int)lo.w, (int)xl.w, s);
            s = __dp4a((int)hi.x, (int)xh.x, s);
            s = __dp4a((int)hi.y, (int)xh.y, s);
            s = __dp4a((int)hi.z, (int)xh.z, s);
            s = __dp4a((int)hi.w, (int)xh.w, s);
            // both factors were doubled: 2^-2; scale code 255 is NaN
            float v = scale_pow2(__int2float_rn(s), ea + eb - 256);
            if (max(ea, eb) == 255) v = __uint_as_float(0x7FC00000u);
            acc[m] = __fadd_rn(acc[m], v);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const float v = sum8(acc[m]);
        if (l8 == 0) red[part][4 * group + sub][m] = v;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS_PER_CTA / 2 * MT; i += THREADS) {
        const int m = i / (ROWS_PER_CTA / 2), pr = i % (ROWS_PER_CTA / 2);
        const int64_t n = (int64_t)blockIdx.x * ROWS_PER_CTA + 2 * pr;
        if (m >= p.M || n >= p.N) continue;
        float z[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            z[e] = 0.0f;
#pragma unroll
            for (int k = 0; k < KSPLIT; ++k) z[e] = __fadd_rn(z[e], red[k][2 * pr + e][m]);
        }
        const uint32_t v[4] = {__float_as_uint(z[0]), __float_as_uint(z[1]), 0u, 0u};
        float2 h;
        p.act.forward<1>(v, &h);
        p.h[m * p.ldh + n / 2] = (uint16_t)pack_bf16x2(h.x, 0.0f);
        if (p.z) *reinterpret_cast<uint32_t *>(p.z + m * p.ldz + n) = pack_bf16x2(z[0], z[1]);
    }
}

struct Int8RowsParams {
    const int8_t *a, *b;
    const float *sa, *sb;
    int64_t lda, ldb, N;
    int M, K;
    void *c;
    int64_t ldc;
    int bf16;
};

template <int MT>
__global__ void __launch_bounds__(THREADS) int8_rows_kernel(const Int8RowsParams p) {
    __shared__ int red[KSPLIT][ROWS_PER_CTA][MT];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / KSPLIT, part = warp % KSPLIT, sub = lane >> 3, l8 = lane & 7;
    const int64_t row0 = (int64_t)blockIdx.x * ROWS_PER_CTA + 4 * group;
    const int8_t *b = p.b + min(row0 + sub, p.N - 1) * p.ldb;
    const int nchunk = p.K / 16;
    int acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = 0;
#pragma unroll 4
    for (int c = part * 8 + l8; c < nchunk; c += 8 * KSPLIT) {
        const uint4 u = ld_nc_v4(b + c * 16);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint4 x = ld_nc_v4(p.a + min(m, p.M - 1) * p.lda + c * 16);
            acc[m] = __dp4a((int)u.x, (int)x.x, acc[m]);
            acc[m] = __dp4a((int)u.y, (int)x.y, acc[m]);
            acc[m] = __dp4a((int)u.z, (int)x.z, acc[m]);
            acc[m] = __dp4a((int)u.w, (int)x.w, acc[m]);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int v = sum8(acc[m]);
        if (l8 == 0) red[part][4 * group + sub][m] = v;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS_PER_CTA * MT; i += THREADS) {
        const int m = i / ROWS_PER_CTA, r = i % ROWS_PER_CTA;
        const int64_t n = (int64_t)blockIdx.x * ROWS_PER_CTA + r;
        if (m >= p.M || n >= p.N) continue;
        int s = 0;
#pragma unroll
        for (int k = 0; k < KSPLIT; ++k) s += red[k][r][m];
        const float v = __fmul_rn(__fmul_rn(__int2float_rn(s), p.sa[m]), p.sb[n]);
        if (p.bf16) static_cast<uint16_t *>(p.c)[m * p.ldc + n] = (uint16_t)pack_bf16x2(v, 0.0f);
        else static_cast<float *>(p.c)[m * p.ldc + n] = v;
    }
}

dim3 rows_grid(int64_t N) { return dim3((unsigned)((N + ROWS_PER_CTA - 1) / ROWS_PER_CTA)); }

template <int MT>
cudaError_t run_gated_rows(const GatedRowsParams &p, cudaStream_t s) {
    return launch_pdl(gated_rows_kernel<MT>, rows_grid(p.N), dim3(THREADS), (size_t)MT * (p.K + p.K / 32), s, p);
}
template <int MT>
cudaError_t run_int8_rows(const Int8RowsParams &p, cudaStream_t s) {
    return launch_pdl(int8_rows_kernel<MT>, rows_grid(p.N), dim3(THREADS), 0, s, p);
}

}  // namespace

int launch_gated_rows(const GatedArgs &a, cudaStream_t s) {
    const GatedRowsParams p{a.a_codes, a.a_scales, a.b_codes, a.b_scales, a.lda, a.ldb, a.N, (int)a.M, (int)a.K,
                            GatedAct{a.alpha, a.limit, a.beta}, static_cast<uint16_t *>(a.out),
                            static_cast<uint16_t *>(a.z), a.ld_out, a.ldz};
    const cudaError_t e = a.M == 1   ? run_gated_rows<1>(p, s)
                          : a.M == 2 ? run_gated_rows<2>(p, s)
                                     : run_gated_rows<4>(p, s);
    return e == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA;
}

int launch_int8_rows(const Int8Args &a, cudaStream_t s) {
    const Int8RowsParams p{a.a, a.b, a.a_scales, a.b_scales, a.lda, a.ldb, a.N, (int)a.M, (int)a.K, a.c, a.ldc, a.bf16};
    const cudaError_t e = a.M == 1   ? run_int8_rows<1>(p, s)
                          : a.M == 2 ? run_int8_rows<2>(p, s)
                                     : run_int8_rows<4>(p, s);
    return e == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA;
}

}  // namespace mxfp4

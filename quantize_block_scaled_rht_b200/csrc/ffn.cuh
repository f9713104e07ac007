// ffn.cuh -- what the expert feed-forward operators share: the gated
// activation and its derivative, and the arguments of their launches.
//
// Activation of a pre-activation pair (zg, zu), "GPT-OSS" expert layers and
// plain SwiGLU alike:
//   g = min(zg, L), u = clamp(zu, -L, L), s = 1 / (1 + exp(-alpha g))
//   h = g s (u + beta)
// and, given dh,
//   dzg = dh (u + beta) s (1 + alpha g (1 - s))   where zg <= L, else 0
//   dzu = dh g s                                  where |zu| <= L, else 0
// SwiGLU is alpha = 1, L = inf, beta = 0; GPT-OSS alpha = 1.702, L = 7, beta = 1.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace mxfp4 {

struct GatedAct {
    float alpha, limit, beta;

    // s = 1 / (1 + 2^(-alpha log2(e) g)) of N values with the hardware's base-2
    // exponential and reciprocal: the roundings of log2(e), of its product with
    // alpha and of that with g move the exponent by at most 1.1 x 2^-23 |alpha g|,
    // which leaves a relative error under 1e-5 for |alpha g| < 60 and under 2e-5 up
    // to where s is 0 or 1, a two-hundredth of bf16's half-step.  Both flush
    // subnormals (an exponential below 2^-126 leaves s = 1, a sum above 2^126
    // s = 0); the forms that keep them cost a branch each.  One step for all N
    // values at a time: a warp of the GEMM's epilogue has a scheduler to itself,
    // so only independent values hide the latency of a step.
    template <int N>
    __device__ __forceinline__ void sigmoid(const float2 *g, float2 *s) const {
        const float k = __fmul_rn(alpha, -1.44269504f);
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = mul2(g[i], make_float2(k, k));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(s[i].x));
            asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(s[i].y));
        }
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = add2(s[i], make_float2(1.0f, 1.0f));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            asm volatile("rcp.approx.ftz.f32 %0, %0;" : "+f"(s[i].x));
            asm volatile("rcp.approx.ftz.f32 %0, %0;" : "+f"(s[i].y));
        }
    }
    // One instruction per bound; a NaN goes through.
    __device__ __forceinline__ float clamp_gate(float z) const {
        float r;
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(limit));
        return r;
    }
    __device__ __forceinline__ float clamp_up(float z) const {
        float r;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(clamp_gate(z)), "f"(-limit));
        return r;
    }
    // 2N pairs (zg, zu) in v, FP32 bits, to 2N values h, two at a time in packed
    // FP32 (each lane rounded as the scalar operation, half the issue slots).
    template <int N>
    __device__ __forceinline__ void forward(const uint32_t *v, float2 *h) const {
        float2 s[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            h[i] = make_float2(clamp_gate(__uint_as_float(v[4 * i])), clamp_gate(__uint_as_float(v[4 * i + 2])));
        sigmoid<N>(h, s);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 u = make_float2(clamp_up(__uint_as_float(v[4 * i + 1])), clamp_up(__uint_as_float(v[4 * i + 3])));
            h[i] = mul2(mul2(h[i], s[i]), add2(u, make_float2(beta, beta)));
        }
    }
    // 2N values dh (FP32 bits) and packed bf16 pairs z (zg low, zu high), the
    // pairs replaced by (dzg, dzu).
    template <int N>
    __device__ __forceinline__ void backward(const uint32_t *dh, uint32_t *z) const {
        float2 g[N], s[N];
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = make_float2(clamp_gate(bf16lo(z[2 * i])), clamp_gate(bf16lo(z[2 * i + 1])));
        sigmoid<N>(g, s);
        const float2 a = make_float2(alpha, alpha), b = make_float2(beta, beta), one = make_float2(1.0f, 1.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t z0 = z[2 * i], z1 = z[2 * i + 1];
            const float2 u = make_float2(clamp_up(bf16hi(z0)), clamp_up(bf16hi(z1)));
            const float2 d = make_float2(__uint_as_float(dh[2 * i]), __uint_as_float(dh[2 * i + 1]));
            // dh s (1 + alpha g (1 - s)) as hs + alpha (hs (g (1 - s))), hs = dh s: alpha g
            // and du = dh g s may leave FP32's range for finite g, and as infinities would
            // meet a zero s or 1 - s.  (With du (1 - s) in the middle, one product less, du's
            // overflow made dg NaN.)
            const float2 hs = mul2(d, s[i]), du = mul2(hs, g[i]);
            const float2 dg = mul2(fma2(a, mul2(hs, mul2(g[i], sub2(one, s[i]))), hs), add2(u, b));
            // beyond the limit 0, and NaN where zu is
            const float2 o = sub2(u, u);
            z[2 * i] = pack_bf16x2(bf16lo(z0) > limit ? 0.0f : dg.x, fabsf(bf16hi(z0)) <= limit ? du.x : o.x);
            z[2 * i + 1] = pack_bf16x2(bf16lo(z1) > limit ? 0.0f : dg.y, fabsf(bf16hi(z1)) <= limit ? du.y : o.y);
        }
    }
};

struct GatedArgs {
    const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
    int64_t lda, ldb, M, N, K;      // backward: N = columns of dh
    float alpha, limit, beta;
    void *out;                      // h [M, N/2], or dz [M, 2N]
    int64_t ld_out;
    void *z;                        // forward: z out (may be null); backward: z in
    int64_t ldz;
    const int32_t *offsets, *sizes;
    int G;
    bool backward;
};

struct Int8Args {
    const int8_t *a, *b;
    const float *a_scales, *b_scales;
    int64_t lda, ldb, M, N, K;
    void *c;
    int64_t ldc;
    bool bf16;
    const int32_t *offsets, *sizes;
    int G;
};

// Products of few rows (rows.cu): at most ROWS_MAX, handled 1, 2 or 4 at a time.
// Their integer work goes with rows * N * K, while the tile kernel's time goes
// with K (a first round of tiles: about (5000 + K) * 0.9 ns) until N fills the
// device, and hardly with the rows.  The limits are where the two times meet (41
// sizes, N 256 to 178560, K 256 to 8192, weights in L2 and from HBM): by these
// rules no size is more than 7% (gated) or 3% (int8) off the faster kernel, where
// all calls of up to four rows by the streaming kernel were up to 2.9 and 1.7
// times slower (4 rows of 178560 x 2880: gated 199 us against 68, int8 156
// against 94).  One int8 row streams B as fast as the tile kernel at any size
// (178560 x 2880: 91 us, 94 there).
constexpr int64_t ROWS_MAX = 4;
inline int64_t rows_handled(int64_t M) { return M <= 2 ? M : 4; }
// The gated kernel also needs the rows of A, one byte per element and scale, in 48
// KB of shared memory (less what it has besides).
inline bool gated_by_rows(int64_t M, int64_t N, int64_t K) {
    return M <= ROWS_MAX && rows_handled(M) * (K + K / 32) <= 47 * 1024 && rows_handled(M) * N * K <= 5700 * (5000 + K);
}
inline bool int8_by_rows(int64_t M, int64_t N, int64_t K) {
    return M <= ROWS_MAX && (rows_handled(M) - 1) * N * K <= 25000 * (5000 + K);
}
int launch_gated_rows(const GatedArgs &a, cudaStream_t s);
int launch_int8_rows(const Int8Args &a, cudaStream_t s);

int launch_gated(const GatedArgs &a, cudaStream_t s);
int launch_int8_gemm(const Int8Args &a, cudaStream_t s);
cudaError_t launch_int8_quantize(const void *x, int64_t rows, int64_t cols, int64_t ld_x, int8_t *codes,
                                 int64_t ld_codes, float *scales, cudaStream_t s);
cudaError_t launch_dropout(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual, int64_t rows,
                           int64_t cols, int dtype, double p, uint64_t seed, uint64_t elem_offset, void *y,
                           int64_t ld_y, cudaStream_t s);

}  // namespace mxfp4

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

    // 1 / (1 + 2^(-alpha log2(e) g)) with the hardware's base-2 exponential and
    // reciprocal: the product's rounding moves the exponent by at most
    // |alpha g| 2^-23, which for the |g| where s is not yet 0 or 1 leaves a
    // relative error under 1e-5, a hundredth of bf16's half-step.
    __device__ __forceinline__ float sigmoid(float g) const {
        float e, s;
        const float x = __fmul_rn(g, __fmul_rn(alpha, -1.44269504f));
        asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(x));
        const float d = __fadd_rn(1.0f, e);
        asm("rcp.approx.f32 %0, %1;" : "=f"(s) : "f"(d));
        return s;
    }
    // Comparisons, not fmin / fmax, so that a NaN goes through.
    __device__ __forceinline__ float clamp_gate(float z) const { return z > limit ? limit : z; }
    __device__ __forceinline__ float clamp_up(float z) const {
        return z > limit ? limit : (z < -limit ? -limit : z);
    }
    __device__ __forceinline__ float forward(float zg, float zu) const {
        const float g = clamp_gate(zg);
        return __fmul_rn(__fmul_rn(g, sigmoid(g)), __fadd_rn(clamp_up(zu), beta));
    }
    // dh and the packed bf16 pair (zg low, zu high) to the packed pair (dzg, dzu).
    __device__ __forceinline__ uint32_t backward(float dh, uint32_t z) const {
        const float zg = bf16lo(z), zu = bf16hi(z);
        const float g = clamp_gate(zg), u = clamp_up(zu), s = sigmoid(g);
        const float t = __fmaf_rn(__fmul_rn(alpha, g), __fsub_rn(1.0f, s), 1.0f);
        const float hs = __fmul_rn(dh, s);
        const float dg = __fmul_rn(__fmul_rn(hs, __fadd_rn(u, beta)), t);
        const float du = __fmul_rn(hs, g);
        return pack_bf16x2(zg > limit ? 0.0f : dg, fabsf(zu) > limit ? 0.0f : du);
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

int launch_gated(const GatedArgs &a, cudaStream_t s);
int launch_int8_gemm(const Int8Args &a, cudaStream_t s);
cudaError_t launch_int8_quantize(const void *x, int64_t rows, int64_t cols, int64_t ld_x, int8_t *codes,
                                 int64_t ld_codes, float *scales, cudaStream_t s);
cudaError_t launch_dropout(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual, int64_t rows,
                           int64_t cols, int dtype, double p, uint64_t seed, uint64_t elem_offset, void *y,
                           int64_t ld_y, cudaStream_t s);

}  // namespace mxfp4

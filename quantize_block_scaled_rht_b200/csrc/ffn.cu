// ffn.cu -- streaming kernels of the expert feed-forward operators: the int8
// token quantizer and dropout from the counter-based generator.
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "ffn.cuh"

namespace mxfp4 {

namespace {

__device__ __forceinline__ uint4 ld_v4(const void *p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_v4(void *p, const uint4 &v) {
    asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void st_v2(void *p, uint32_t a, uint32_t b) {
    asm volatile("st.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(a), "r"(b) : "memory");
}

// ---------------------------------------------------------------------------
// int8 token quantizer: per row a = max(amax, 2^-100), scale = a / 127, codes
// RNE(x * i) with i = 127 * (1 / a), each step rounded to FP32 (i is within 1.5 x
// 2^-24 of 127 / a, relative, and for a > 2^126, where 1 / a is subnormal, within
// 4.1 x 2^-24: |x i| stays below 127.001).  The floor keeps 1 / a finite; a NaN or
// Inf anywhere in the row gives the scale NaN and codes 0.
//
// Bound by HBM (2 B read, 1 B written per element; 16384 x 11520: 81 us, 7.0 TB/s
// with part of the writes still in L2).  T threads hold one row in registers (V
// 16-byte vectors each), so it is read once; a row that does not fit takes V = 0,
// which reads it twice (the second time mostly from L2).  T grows with the row so
// that a thread has no more than eight loads in flight and short rows still fill
// the SMs.
// ---------------------------------------------------------------------------

// Largest magnitude of 8 bf16 as two 16-bit halves (NaN where there is one).
__device__ __forceinline__ uint32_t absmax8(const uint4 &u) {
    return bf16x2_absmax(bf16x2_absmax(u.x, u.y), bf16x2_absmax(u.z, u.w));
}

// Four values, already scaled, to four signed bytes by nearest-even: adding
// 1.5 * 2^23 leaves the integer, rounded to nearest even, in the low mantissa
// bits, whose low byte is its two's complement.
__device__ __forceinline__ uint32_t pack4_s8(float a, float b, float c, float d) {
    constexpr float MAGIC = 12582912.0f;
    const uint32_t ua = __float_as_uint(__fadd_rn(a, MAGIC)), ub = __float_as_uint(__fadd_rn(b, MAGIC));
    const uint32_t uc = __float_as_uint(__fadd_rn(c, MAGIC)), ud = __float_as_uint(__fadd_rn(d, MAGIC));
    return __byte_perm(__byte_perm(ua, ub, 0x0040), __byte_perm(uc, ud, 0x0040), 0x5410);
}

__device__ __forceinline__ void quantize8(const uint4 &u, float inv, int8_t *dst) {
    float f[8];
    unpack_bf16x8(u, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(f[i], inv);
    st_v2(dst, pack4_s8(f[0], f[1], f[2], f[3]), pack4_s8(f[4], f[5], f[6], f[7]));
}

template <int T, int V>
__global__ void __launch_bounds__(T < 256 ? 256 / T * T : T)
    int8_quantize_kernel(const uint16_t *__restrict__ x, int64_t rows, int64_t cols, int64_t ld_x,
                         int8_t *__restrict__ codes, int64_t ld_codes, float *__restrict__ scales) {
    pdl_wait();
    pdl_trigger();
    constexpr int R = T < 256 ? 256 / T : 1;          // rows per CTA
    __shared__ uint32_t part[R][T / 32 > 0 ? T / 32 : 1];
    const int sub = threadIdx.x / T, tid = threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * R + sub;
    const bool live = row < rows;
    const uint16_t *src = x + (live ? row : 0) * ld_x;
    const int64_t nvec = live ? cols / 8 : 0;
    uint4 u[V > 0 ? V : 1];
    uint32_t m = 0;
    if constexpr (V > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t c = tid + (int64_t)T * i;
            u[i] = make_uint4(0, 0, 0, 0);
            if (c < nvec) u[i] = ld_v4(src + 8 * c);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) m = bf16x2_absmax(m, absmax8(u[i]));
    } else {
        for (int64_t c = tid; c < nvec; c += T) m = bf16x2_absmax(m, absmax8(ld_v4(src + 8 * c)));
    }
    m &= 0x7FFF7FFFu;
    // as unsigned integers magnitudes order like their values, Inf above every
    // finite one and NaN above Inf
    uint32_t a = max(m << 16, m & 0xFFFF0000u);
    a = __reduce_max_sync(0xFFFFFFFFu, a);
    if constexpr (T > 32) {
        if ((tid & 31) == 0) part[sub][tid >> 5] = a;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < T / 32; ++i) a = max(a, part[sub][i]);
    }
    if (!live) return;
    int8_t *dst = codes + row * ld_codes;
    const bool finite = a < 0x7F800000u;
    const float amax = fmaxf(__uint_as_float(a), __uint_as_float(0x0D800000u));   // 2^-100
    const float inv = finite ? __fmul_rn(__fdiv_rn(1.0f, amax), 127.0f) : 0.0f;
    if (tid == 0) scales[row] = finite ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7FC00000u);
    if constexpr (V > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t c = tid + (int64_t)T * i;
            if (c >= nvec) break;
            if (finite) quantize8(u[i], inv, dst + 8 * c);
            else st_v2(dst + 8 * c, 0u, 0u);
        }
    } else {
        for (int64_t c = tid; c < nvec; c += T) {
            if (finite) quantize8(ld_v4(src + 8 * c), inv, dst + 8 * c);
            else st_v2(dst + 8 * c, 0u, 0u);
        }
    }
}

template <int T, int V>
cudaError_t run_int8_quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ld_x, int8_t *codes,
                              int64_t ld_codes, float *scales, cudaStream_t s) {
    constexpr int R = T < 256 ? 256 / T : 1;
    return launch_pdl(int8_quantize_kernel<T, V>, dim3((unsigned)((rows + R - 1) / R)), dim3(R * T), 0, s, x, rows,
                      cols, ld_x, codes, ld_codes, scales);
}

}  // namespace

cudaError_t launch_int8_quantize(const void *xv, int64_t rows, int64_t cols, int64_t ld_x, int8_t *codes,
                                 int64_t ld_codes, float *scales, cudaStream_t s) {
    const uint16_t *x = static_cast<const uint16_t *>(xv);
    const int64_t nvec = cols / 8;
#define RUN(T, V) return run_int8_quantize<T, V>(x, rows, cols, ld_x, codes, ld_codes, scales, s)
    if (nvec <= 32) RUN(32, 1);
    if (nvec <= 64) RUN(32, 2);
    if (nvec <= 128) RUN(32, 4);
    if (nvec <= 256) RUN(128, 2);
    if (nvec <= 512) RUN(128, 4);
    if (nvec <= 1024) RUN(256, 4);
    if (nvec <= 2048) RUN(256, 8);
    if (nvec <= 4096) RUN(512, 8);
    RUN(512, 0);
#undef RUN
}

// ---------------------------------------------------------------------------
// Dropout: y = [residual +] (keep ? x / (1 - p) : 0), keep iff the element's
// Philox word is at least round(p 2^32).  Word g mod 4 of the block with
// counter (g / 4, 0, tag), g = row * cols + col + elem_offset: the stream of
// stochastic rounding under another tag, so that a slice of the rows draws the
// words of the whole tensor and the backward pass draws the forward's mask
// again, without it ever being stored.
//
// A dropped element is 0 (or the residual) whatever x holds there, NaN and Inf
// included.  Bound by HBM: 4 B per bf16 element, 6 B with the residual.
// ---------------------------------------------------------------------------
constexpr uint32_t DROPOUT_TAG = 0x44524F50u;

namespace {

struct DropParams {
    const void *x, *residual;
    void *y;
    int64_t rows, cols, ld_x, ld_r, ld_y;
    uint64_t block0;               // elem_offset / 4
    uint32_t k0, k1, last;         // dropped: words up to `last` = round(p 2^32) - 1
    float scale;
    uint32_t key0[10], key1[10];   // the rounds' keys, operands straight from the constant bank
};

// ALL: round(p 2^32) is 0, every element is kept and no word is drawn.
template <bool ALL>
__device__ __forceinline__ float drop1(float x, uint32_t word, const DropParams &p) {
    return ALL || word > p.last ? __fmul_rn(x, p.scale) : 0.0f;
}
template <bool ALL>
__device__ __forceinline__ U4 drop_words(uint64_t b, const DropParams &p) {
    if constexpr (ALL) return U4{0, 0, 0, 0};
    return philox4x32_10((uint32_t)b, (uint32_t)(b >> 32), 0u, DROPOUT_TAG, p.k0, p.k1);
}

// The same words with what depends on the counter's high half alone taken out of
// the loop over blocks.  Counter words 2 and 3 are constant, so the first round
// turns (lo, hi, 0, tag) into (hi ^ k0, 0, f(lo), g(lo)), and one of the second
// round's two products is that of hi ^ k0.
struct DropCounter {
    uint32_t x, c3;                // of the second round: x = high half of M0 (hi ^ k0) ^ key, c3 = its low half

    __device__ __forceinline__ void set(uint32_t hi, const DropParams &p) {
        const uint64_t q = (uint64_t)0xD2511F53u * (hi ^ p.k0);
        x = (uint32_t)(q >> 32) ^ (p.k1 + 0xBB67AE85u);
        c3 = (uint32_t)q;
    }
    __device__ __forceinline__ U4 words(uint32_t lo, const DropParams &p) const {
        const uint64_t a = (uint64_t)0xD2511F53u * lo;
        const uint64_t b = (uint64_t)0xCD9E8D57u * ((uint32_t)(a >> 32) ^ (DROPOUT_TAG ^ p.key1[0]));
        uint32_t c0 = (uint32_t)(b >> 32) ^ p.key0[1], c1 = (uint32_t)b, c2 = (uint32_t)a ^ x, w3 = c3;
#pragma unroll
        for (int r = 2; r < 10; ++r) {
            const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
            c0 = (uint32_t)(p1 >> 32) ^ c1 ^ p.key0[r];
            c2 = (uint32_t)(p0 >> 32) ^ w3 ^ p.key1[r];
            c1 = (uint32_t)p1;
            w3 = (uint32_t)p0;
        }
        return U4{c0, c1, c2, w3};
    }
};

// A thread takes 16 bytes of a row (8 bf16 or 4 fp32) per step; cols is a
// multiple of that, or there is one row with a tail.  FLAT: one row (contiguous
// tensors), where a step's address is its index, whose blocks all have the same
// high counter half (any tensor below 2^34 elements, but for an offset that
// happens to cross a multiple of that).
//
// Bound by HBM with the residual (65536 x 2880: 174 us, the measured copy
// bandwidth) or in FP32; plain bf16 by the issue of its instructions, 130 per 8
// elements, of which Philox is about 80 (61% of the issue slots, the integer
// multiply pipe 74% busy): 150 us, 0.77 of HBM.  With addresses from row and
// column and every word from scratch 180, with the rounds' keys added up in the
// kernel 154, with the shift of the low bf16 moved off the multiply pipe 155;
// without drawing 118.
template <bool BF16, bool RES, bool ALL, bool FLAT>
__global__ void __launch_bounds__(256) dropout_kernel(const DropParams p) {
    pdl_wait();
    pdl_trigger();
    constexpr int E = BF16 ? 8 : 4, SZ = BF16 ? 2 : 4;
    const int64_t per_row = p.cols / E, n = FLAT ? per_row : p.rows * per_row;
    const char *x = static_cast<const char *>(p.x), *res = static_cast<const char *>(p.residual);
    char *y = static_cast<char *>(p.y);
    DropCounter ctr;
    if constexpr (FLAT && !ALL) ctr.set((uint32_t)(p.block0 >> 32), p);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        int64_t ox = 16 * i, orr = ox, oy = ox;
        if constexpr (!FLAT) {
            const int64_t row = i / per_row, c = (i - row * per_row) * E;
            ox = (row * p.ld_x + c) * SZ;
            oy = (row * p.ld_y + c) * SZ;
            if constexpr (RES) orr = (row * p.ld_r + c) * SZ;
        }
        const uint4 u = ld_v4(x + ox);
        uint4 r = make_uint4(0, 0, 0, 0);
        if constexpr (RES) r = ld_v4(res + orr);
        const uint64_t b = p.block0 + (uint64_t)i * (E / 4);
        U4 w0{}, w1{};
        if constexpr (FLAT && !ALL) {
            w0 = ctr.words((uint32_t)b, p);
            if constexpr (BF16) w1 = ctr.words((uint32_t)b + 1u, p);
        } else {
            w0 = drop_words<ALL>(b, p);
            if constexpr (BF16) w1 = drop_words<ALL>(b + 1, p);
        }
        uint4 o;
        if constexpr (BF16) {
            const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            float f[8], g[8];
            unpack_bf16x8(u, f);
            if constexpr (RES) unpack_bf16x8(r, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = drop1<ALL>(f[e], w[e], p);
                if constexpr (RES) f[e] = __fadd_rn(f[e], g[e]);
            }
            o = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                           pack_bf16x2(f[6], f[7]));
        } else {
            float f[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
            const float g[4] = {__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w)};
            const uint32_t w[4] = {w0.x, w0.y, w0.z, w0.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[e] = drop1<ALL>(f[e], w[e], p);
                if constexpr (RES) f[e] = __fadd_rn(f[e], g[e]);
            }
            o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        }
        st_v4(y + oy, o);
    }
}

// Any size, stride and alignment: a thread takes one Philox block, four
// consecutive elements of the [rows, cols] order, from element `first` on.
template <bool BF16, bool RES, bool ALL>
__global__ void __launch_bounds__(256) dropout_any_kernel(const DropParams p, int64_t first) {
    pdl_wait();
    pdl_trigger();
    const int64_t total = p.rows * p.cols, n = (total - first + 3) / 4;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t e0 = first + 4 * i;
        const uint64_t b = p.block0 + (uint64_t)(e0 / 4);
        const U4 w0 = drop_words<ALL>(b, p);
        const uint32_t w[4] = {w0.x, w0.y, w0.z, w0.w};
        int64_t row = e0 / p.cols, c = e0 - row * p.cols;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (e0 + e < total) {
                if constexpr (BF16) {
                    const uint32_t v = static_cast<const uint16_t *>(p.x)[row * p.ld_x + c];
                    float f = drop1<ALL>(__uint_as_float(v << 16), w[e], p);
                    if constexpr (RES)
                        f = __fadd_rn(f, __uint_as_float((uint32_t)static_cast<const uint16_t *>(p.residual)[row * p.ld_r + c] << 16));
                    static_cast<uint16_t *>(p.y)[row * p.ld_y + c] = (uint16_t)pack_bf16x2(f, 0.0f);
                } else {
                    float f = drop1<ALL>(static_cast<const float *>(p.x)[row * p.ld_x + c], w[e], p);
                    if constexpr (RES) f = __fadd_rn(f, static_cast<const float *>(p.residual)[row * p.ld_r + c]);
                    static_cast<float *>(p.y)[row * p.ld_y + c] = f;
                }
                if (++c == p.cols) { c = 0; ++row; }
            }
        }
    }
}

template <bool BF16, bool RES, bool ALL>
cudaError_t run_dropout(DropParams p, cudaStream_t s) {
    constexpr int E = BF16 ? 8 : 4;
    auto al = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
    auto grid = [](int64_t threads) {
        const int64_t b = (threads + 255) / 256;
        return dim3((unsigned)(b < 148 * 32 ? b : 148 * 32));
    };
    const bool flat = p.rows == 1 || (p.ld_x == p.cols && p.ld_y == p.cols && (!RES || p.ld_r == p.cols));
    const bool aligned = al(p.x) && al(p.y) && (!RES || al(p.residual));
    const bool strided = p.cols % E == 0 && p.ld_x % E == 0 && p.ld_y % E == 0 && (!RES || p.ld_r % E == 0);
    int64_t done = 0;
    if (flat) {
        p.cols *= p.rows;
        p.rows = 1;
        p.ld_x = p.ld_r = p.ld_y = p.cols;
    }
    if (aligned && (flat || strided)) {
        done = flat ? p.cols / E * E : p.rows * p.cols;
        if (done) {
            const bool one_hi = (p.block0 >> 32) == ((p.block0 + (uint64_t)(done / 4) - 1) >> 32);
            const cudaError_t e = launch_pdl(flat && one_hi ? dropout_kernel<BF16, RES, ALL, true>
                                                  : dropout_kernel<BF16, RES, ALL, false>,
                                             grid(done / E), dim3(256), 0, s, p);
            if (e != cudaSuccess) return e;
        }
    }
    if (done == p.rows * p.cols) return cudaSuccess;
    return launch_pdl(dropout_any_kernel<BF16, RES, ALL>, grid((p.rows * p.cols - done + 3) / 4), dim3(256), 0, s, p, done);
}

}  // namespace

cudaError_t launch_dropout(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual, int64_t rows,
                           int64_t cols, int dtype, double prob, uint64_t seed, uint64_t elem_offset, void *y,
                           int64_t ld_y, cudaStream_t s) {
    const double t = std::nearbyint(prob * 4294967296.0);   // 0 .. 2^32
    DropParams p{x, residual, y, rows, cols, ld_x, ld_residual, ld_y, elem_offset / 4, (uint32_t)seed,
                       (uint32_t)(seed >> 32), t > 0.0 ? (uint32_t)(t - 1.0) : 0u, prob < 1.0 ? (float)(1.0 / (1.0 - prob)) : 0.0f, {}, {}};
    for (uint32_t r = 0; r < 10; ++r) {
        p.key0[r] = p.k0 + r * 0x9E3779B9u;
        p.key1[r] = p.k1 + r * 0xBB67AE85u;
    }
    const bool bf16 = dtype == MXFP4_OUT_BF16, res = residual != nullptr;
    if (t == 0.0)
        return bf16 ? (res ? run_dropout<true, true, true>(p, s) : run_dropout<true, false, true>(p, s))
                    : (res ? run_dropout<false, true, true>(p, s) : run_dropout<false, false, true>(p, s));
    return bf16 ? (res ? run_dropout<true, true, false>(p, s) : run_dropout<true, false, false>(p, s))
                : (res ? run_dropout<false, true, false>(p, s) : run_dropout<false, false, false>(p, s));
}

}  // namespace mxfp4

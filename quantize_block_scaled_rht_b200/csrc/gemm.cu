// gemm.cu -- MXFP4 block-scaled GEMM (dense and grouped) for sm_100a, with the
// gated epilogues of the expert feed-forward block and the int8 product.
//
// "MXFP4" (aiwiki.ai), "Conversion rules": the block dot product
// C = X(A) X(B) sum_i Pi(A) Pi(B), block products summed, FP32 result; the
// order of operations is the implementation's.  "Hardware support": Blackwell
// tensor cores apply MXFP4 block scales in hardware.  Here that is
// tcgen05.mma kind::mxf4.block_scale: E2M1 operands from shared memory, one
// UE8M0 scale per 32 K-elements from tensor memory, FP32 accumulators in
// tensor memory (TMEM), 64 K-elements per instruction.
//
// Kernel structure: persistent, clusters of two CTAs (one per SM) that share
// one 256 x BN output tile with the pair MMA (cta_group::2): each CTA holds 128
// rows of A and BN/2 rows of B, so every SM streams 128 + BN/2 operand rows per
// K step instead of 128 + BN.  Per CTA, 6 warps:
//   warp 0      TMA producer: its A rows, its half of B and the scale atoms
//               (A: its own 128 rows; B: all BN rows) into a STAGES-deep ring
//               (MXFP4: 3 stages of 512 K-elements); every load completes on
//               the even CTA's stage barrier;
//   warp 1      TMEM owner; in the even CTA also the MMA issuer: scale atoms
//               to TMEM (tcgen05.cp, both CTAs), 4 * KCH pair MMAs of K = 64
//               per stage into one of two accumulators, stage release by a
//               commit to both CTAs;
//   warps 2..5  epilogue: TMEM -> registers -> swizzled smem -> TMA store of
//               this CTA's 128 rows (FP32, or bf16 rounded to nearest even),
//               overlapping the next tile's MMAs, then an arrive on the even
//               CTA's accumulator-empty barrier (warps 2..9 with the gated
//               activation or its derivative in the epilogue).
// Every barrier wait is bounded by the GPU global timer; a wait that runs out
// records MXFP4_ERR_TIMEOUT, raises the CTA's abort flag, and each role drains
// what it has in flight before both CTAs meet at the final cluster barrier.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "ffn.cuh"
#include "ptx.cuh"

namespace mxfp4 {

constexpr int BM = 128;                               // rows per CTA
constexpr int CHUNK = 128;                            // K bytes per swizzled chunk (256 E2M1 = 8 scale blocks)
constexpr int EPI_BUF = 32 * 32 * 4;                  // 32 rows x 32 FP32
constexpr int BAR_BYTES = 256;
constexpr uint32_t TMEM_COLS = 512;
constexpr int MAX_GROUPS = 1024;
constexpr int MAX_STAGES = 8;

// Tile configuration: a pair tile is 256 x BN; each stage of the STAGES-deep
// smem ring holds KCH chunks of K (KCH * 256 E2M1 elements, 4 * KCH MMAs).
// KIND_NV: NVFP4 operands (UE4M3 scales per 16 elements, kind::mxf4nvf4) instead
// of MXFP4 (UE8M0 per 32, kind::mxf4).  A scale atom holds 4 blocks of every row
// of a 128-row tile: 128 K-elements for MXFP4, 64 for NVFP4.  KIND_I8: signed
// 8-bit integers (kind::i8, exact 32-bit integer sums), one element per byte and
// no scale atoms; the token and channel scales go in with the epilogue.
// EPI_BUFS: 4 KB staging buffers per epilogue warp.  EPI_WARPS: 4, or 8 for the
// epilogues with real arithmetic: a warp may read only the quarter of the tensor
// memory lanes that its index selects, so two warps share a quarter and take
// its column steps in turn.
// SUB: if not 0, the tiles of the last, partial round are cut into pieces of SUB
// columns (get_item).
// RAGGED: dense FP32 and bf16 outputs whose columns end inside 16 bytes
// (ragged_box).  The output's tensor map ends at the last whole 16 bytes, and the
// columns behind go out with plain stores (4096 x 190 x 2880 bf16 8.8 us; the whole
// last box that way 9.6, the whole last tile 10.1).  A form of its own: the test,
// even once per tile, cost the bf16 product of 4096 x 5760 x 2880 2% (35.9 -> 36.6
// us; grouped forms, which have both ways of storing anyway, nothing: they store the
// last column of tiles plainly).
constexpr int KIND_MX = 0, KIND_NV = 1, KIND_I8 = 2;
template <int BN_, int STAGES_, int KCH_, int KIND_ = KIND_MX, int EPI_BUFS_ = 2, int EPI_WARPS_ = 4, int SUB_ = 0,
          bool RAGGED_ = false>
struct TileCfg {
    static constexpr int BN = BN_;
    static constexpr int STAGES = STAGES_;
    static constexpr int KCH = KCH_;
    static constexpr bool NV = KIND_ == KIND_NV, I8 = KIND_ == KIND_I8;
    static constexpr int EPI_BUFS = EPI_BUFS_;
    static constexpr int EPI_WARPS = EPI_WARPS_;
    static constexpr int SPLIT = EPI_WARPS / 4;       // warps per lane quarter
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
    static constexpr int SUB = SUB_;
    static constexpr bool RAGGED = RAGGED_;
    static constexpr int PIECES = SUB ? BN / SUB : 1;
    static constexpr int EPI_BYTES = EPI_WARPS * EPI_BUFS * EPI_BUF;
    static constexpr int KPB = I8 ? 1 : 2;            // K-elements per byte
    static constexpr int KMMA = 32 * KPB;             // K-elements per instruction (32 bytes)
    static constexpr int KSTEP = 128 * KPB * KCH;     // K-elements per stage
    static constexpr int KATOM = NV ? 64 : 128;       // K-elements per scale atom
    static constexpr int NATOM = I8 ? 0 : KSTEP / KATOM;   // scale atoms per row tile per stage
    // B scale atoms span one 128-row tile when BN = 128, two when BN = 192
    // (a 192-column tile starts at 0 or 64 within a 128-row scale tile).
    static constexpr int NRT = BN == 128 ? 1 : 2;
    static constexpr int A_CHUNK = BM * CHUNK;               // 16 KB per chunk
    static constexpr int B_CHUNK = (BN / 2) * CHUNK;         // this CTA's half of the B tile
    static constexpr int A_BYTES = KCH * A_CHUNK;
    static constexpr int B_BYTES = KCH * B_CHUNK;
    static constexpr int SFA_BYTES = NATOM * 512;
    static constexpr int SFB_BYTES = NRT * NATOM * 512;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr uint32_t STAGE_TX = 2u * STAGE_BYTES;   // both CTAs complete on the even CTA's barrier
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_BYTES + BAR_BYTES + 1024;   // + alignment
    // TMEM columns (per CTA): accumulator 0 at [0, BN), the scale factors of
    // two consecutive stages after it, accumulator 1 at the top.
    static constexpr uint32_t SF_COL = BN;
    static constexpr uint32_t SF_STAGE_COLS = 4 * NATOM * (1 + NRT);
    static constexpr uint32_t ACC1_COL = TMEM_COLS - BN;
    // Instruction descriptor, kind::mxf4 block-scaled: A/B E2M1 (1), K-major,
    // N >> 3 at bit 17, UE8M0 scales (bit 23), M >> 4 at bit 24 (M = 256 for
    // the pair), scale-factor byte selectors at bits 4 (B) and 29 (A).
    // kind::i8: signed A and B (1), 32-bit integer accumulators (2 at bit 4).
    static constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) |
                                      (I8 ? 2u << 4 : (NV ? 0u : 1u) << 23) | ((uint32_t)(256 >> 4) << 24);
    static_assert(BN == 128 || BN == 192 || (I8 && BN == 256), "tile width");
    static_assert(KCH == 1 || KCH == 2, "chunks per stage");
    static_assert(EPI_WARPS == 4 || EPI_WARPS == 8, "epilogue warps");
    static_assert(SUB == 0 || (BN % SUB == 0 && (SUB == 64 || (I8 && SUB == 128))), "pieces of a tile (E2M1: that start on an even 32-column scale group)");
    static_assert(STAGES <= MAX_STAGES, "stages");
    static_assert(SF_COL + 2 * SF_STAGE_COLS <= ACC1_COL, "TMEM layout");
    static_assert(A_CHUNK % 1024 == 0 && B_CHUNK % 1024 == 0 && STAGE_BYTES % 1024 == 0, "swizzle alignment");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// Output of the epilogue: FP32, bf16 (nearest even), or MXFP4 (each 1D row
// block of 32 FP32 results requantized: amax, E8M0 scale, E2M1 RNE codes).
// OUT_GATED: the gated activation of column pairs (2j gate, 2j + 1 up) to bf16 h
// [.., N/2], with the pre-activations z optionally kept in bf16.  OUT_GATED_BWD:
// the accumulators are dh; with z they give dz (bf16 [.., 2N]).
constexpr int OUT_F32 = 0, OUT_BF16 = 1, OUT_MX = 2, OUT_GATED = 3, OUT_GATED_BWD = 4;

using DefaultCfg = TileCfg<192, 3, 2>;
using NvCfg = TileCfg<192, 5, 1, KIND_NV>;
using RaggedCfg = TileCfg<192, 3, 2, KIND_MX, 2, 4, 0, true>;
using RaggedNvCfg = TileCfg<192, 5, 1, KIND_NV, 2, 4, 0, true>;
// The gated epilogues take eight warps.  Forward: one staging buffer each, which
// keeps the 3 x 512 ring (4096 x 5760 x 2880, h alone: 35.1 us, the bf16
// product's time; 4 warps and two buffers 48.8, 8 warps and two buffers on a
// ring of 5 x 256 40.2).  Backward: two buffers carry z in and dz out, beside a
// ring of 5 x 256 (when chosen, with whole last rounds, 4096 x 2880 x 2880 37.0 us,
// K = 5760 50.8; three buffers and a ring of 4 x 256 37.0 and 54.2, four of 3 x 256
// 41.7 and 61.6, 4 warps 43.3, 12 warps 41.2).
using GatedCfg = TileCfg<192, 3, 2, KIND_MX, 1, 8>;
using BwdCfg = TileCfg<192, 5, 1, KIND_MX, 2, 8>;
// Calls take 128-column tiles where those finish in clearly fewer rounds of
// tiles (launch_tiles): 256 x 5760 x 2880 8.0 against 9.1 us, 768 rows 11.5
// against 13.0; backward, 768 x 2880 x 2880, 12.4 against 14.1.
using GatedNarrowCfg = TileCfg<128, 3, 2, KIND_MX, 2, 8>;
using BwdNarrowCfg = TileCfg<128, 6, 1, KIND_MX, 2, 8>;
// The backward epilogue outlasts the MMAs, so a last round that only a few pairs
// take part in costs a whole tile's epilogue.  A dense call whose last round
// still fits one round in 64-column pieces takes the form that cuts it (launch_cut):
// 4096 x 2880 x 2880 34.1 against 38.4 us (K = 64: 25.7 against 30.4), 16 rows
// 9.6 against 10.9, 1024 x 1024 x 1024 7.6 against 9.1.  The counting costs calls
// that cut nothing 1 to 3%, so they, and the grouped calls, whose number of tiles
// the host does not know, have the plain form.
using BwdCutCfg = TileCfg<192, 5, 1, KIND_MX, 2, 8, 64>;
using BwdNarrowCutCfg = TileCfg<128, 6, 1, KIND_MX, 2, 8, 64>;
// int8: without scale factors in tensor memory two 256-column accumulators fit,
// and a 256 x 256 tile reads 1/8 fewer operand bytes per product than 256 x 192
// (4096 x 2880 x 2880 with a whole last round: 27.3 us, 256 x 192 30.4, and 28.8
// with the ring as 3 x 256 instead of 6 x 128 K-elements).
// Narrow: 128 x 2880 x 2880 10.2 against 12.6 us, 64 x 8192 x 8192 19.8 against
// 24.4; where it would take two rounds to the wide tile's one, the fewer operand
// bytes win (1024 x 2880 x 2880: 13.8 against 16.4).
using I8Cfg = TileCfg<256, 6, 1, KIND_I8>;
using I8NarrowCfg = TileCfg<128, 8, 1, KIND_I8>;
// The last round of a dense call in 128-column pieces, with B boxes of their
// size, where those fit one round: 2048 x 2880 x 2880 18.5 against 20.1 us (96
// tiles: a round of 74, then 14 tiles in two pieces and 8 of the last 64 columns in
// one), 1024 x 5760 x 2880 18.6 against 20.2, 4096 x 2880 x 2880 26.1 against 27.3.
// Narrow tiles in 64-column pieces: 512 x 1024 x 1024 6.3 against 6.6, but 16 x
// 2880 x 2880 9.85 against 9.5; not kept.
using I8CutCfg = TileCfg<256, 6, 1, KIND_I8, 2, 4, 128>;
using I8GroupedCfg = TileCfg<256, 5, 1, KIND_I8>;   // the group table takes 4 KB of shared memory
using I8GroupedNarrowCfg = TileCfg<128, 7, 1, KIND_I8>;

__device__ unsigned int g_error_code;

__device__ __forceinline__ void record_error(unsigned int code) { atomicCAS(&g_error_code, 0u, code); }

struct GemmParams {
    int64_t M, N, K;
    int64_t katoms;            // ceil(K / 128): scale atoms per 128-row tile
    int64_t b_rowtiles;        // ceil(N / 128): 128-row scale tiles of one B operand
    void *c;                   // FP32, bf16 [.., ldc elements] or MXFP4 codes [.., ldc bytes]
    int64_t ldc;
    uint8_t *c_scales;         // MXFP4 output: scales, row-major [.., ld_c_scales] or GEMM-ready
    int64_t ld_c_scales, c_katoms;
    int c_scale_mma;
    const int32_t *group_offsets;
    const int32_t *group_sizes;
    const float *a_amax, *b_amax;   // NVFP4 tensor amaxes (second-level scales amax / 2688)
    const float *a_tok, *b_chan;    // int8: one scale per row of A, one per row of B (all groups')
    int64_t box_n0;                 // grouped FP32, bf16: last first column of a tile without a ragged box
    int64_t box_cols;               // RAGGED: columns up to the last whole 16 bytes
    void *z;                        // gated: pre-activations out (may be null); backward: in
    int64_t ldz;
    float act_alpha, act_limit, act_beta;
    int num_groups;
    uint32_t stage_tx;         // bytes of both CTAs' loads of one stage
    // with TileCfg::SUB: tiles of the full rounds, then tiles in PIECES pieces each,
    // then (int8) tiles of the last columns in as many as N needs; work items in all
    int cut_whole, cut_tiles, cut_last, cut_items;
    uint64_t wait_limit_ns;
};

struct Shared {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];
    uint64_t tmem_full[2], tmem_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    volatile int abort;
    int drain_failed;    // set in both CTAs by the leader when a bounded drain wait ran out
    int ntiles;
};

// Mark the pair's drain as failed, in this CTA and in its peer (rank ^ 1).
__device__ __forceinline__ void mark_drain_failed(Shared *sh, uint32_t rank) {
    sh->drain_failed = 1;
    const uint32_t peer = mapa_shared(smem_u32(&sh->drain_failed), rank ^ 1u);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer), "r"(1u) : "memory");
}

// Bounded wait: true once the phase of `parity` has completed; false if the
// CTA aborted or the wait ran past the limit (which records the timeout and
// aborts the CTA).  `hard` waits ignore the abort flag (used while draining).
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, Shared *sh, uint64_t limit,
                                           bool hard = false) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 31u) == 0u) {
            if (!hard && sh->abort) return false;
            if (globaltimer_ns() - t0 > limit) {
                if (!hard) {
                    record_error(MXFP4_ERR_TIMEOUT);
                    sh->abort = 1;
                }
                return false;
            }
        }
    }
}

__device__ __forceinline__ void spin_ns(uint64_t ns) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < ns) {
    }
}

struct TileInfo {
    int64_t row0;       // first A row of this CTA's half
    int64_t c_row0;     // first C row of this CTA's half
    int rows_valid;     // rows of this CTA's half that belong to the problem (grouped: to the group)
    int64_t n0;         // first C column
    int64_t b_row;      // TMA row coordinate of the first B row of the pair tile
    int64_t sfb_rt_base;  // first 128-row scale tile of this B operand (expert)
    int64_t k0;         // first K element of the tile's reduction (grouped K: the group's offset)
    int64_t kg;         // K elements of the reduction
    int width;          // columns (get_item)
};

// Kernel modes: dense; grouped rows (per-expert row ranges of A, one B per
// expert); grouped K (per-expert K ranges of both operands, one C per expert).
constexpr int MODE_DENSE = 0, MODE_GROUPED_M = 1, MODE_GROUPED_K = 2;

// Pair tile t -> coordinates.  Dense: M in steps of 256 (fastest), then N.
// Grouped rows: group g owns cum[g+1] - cum[g] pair tiles.  Grouped K: group
// g owns tiles_m x tiles_n tiles of its [M, N] output over K range
// [cum[g], cum[g+1]) (cum holds the validated K offsets).  g_at: a group at or
// before the tile's, from which the search goes on (a role's tiles only grow);
// with 32 groups a search from the first one cost each role 700 cycles a tile.
template <int BN, int MODE>
__device__ __forceinline__ TileInfo get_tile(int t, uint32_t rank, const GemmParams &p, const int *cum,
                                             int tiles_n, int &g_at) {
    TileInfo ti;
    ti.k0 = 0;
    ti.kg = p.K;
    if constexpr (MODE == MODE_GROUPED_K) {
        const int tiles_m = (int)((p.M + 255) / 256);
        const int g = t / (tiles_m * tiles_n), local = t - g * (tiles_m * tiles_n);
        const int tm = local % tiles_m, tn = local / tiles_m;
        ti.row0 = (int64_t)tm * 256 + 128 * rank;
        ti.c_row0 = (int64_t)g * p.M + ti.row0;
        const int64_t left = p.M - ti.row0;
        ti.rows_valid = left <= 0 ? 0 : (left < BM ? (int)left : BM);
        ti.n0 = (int64_t)tn * BN;
        ti.b_row = ti.n0;
        ti.sfb_rt_base = 0;
        ti.k0 = cum[g];
        ti.kg = (int64_t)cum[g + 1] - cum[g];
    } else if constexpr (MODE == MODE_DENSE) {
        const int tiles_m = (int)((p.M + 255) / 256);
        const int tm = t % tiles_m, tn = t / tiles_m;
        ti.row0 = (int64_t)tm * 256 + 128 * rank;
        const int64_t left = p.M - ti.row0;
        ti.rows_valid = left <= 0 ? 0 : (left < BM ? (int)left : BM);
        ti.n0 = (int64_t)tn * BN;
        ti.b_row = ti.n0;
        ti.sfb_rt_base = 0;
        ti.c_row0 = ti.row0;
    } else {
        int g = g_at;
        while (g + 1 < p.num_groups && cum[g + 1] <= t) ++g;
        g_at = g;
        const int local = t - cum[g];
        const int tiles_g = (cum[g + 1] - cum[g]) / tiles_n;
        const int tm = local % tiles_g, tn = local / tiles_g;
        const int64_t size = p.group_sizes[g];
        const int64_t r_in = (int64_t)tm * 256 + 128 * rank;
        ti.row0 = (int64_t)p.group_offsets[g] + r_in;
        const int64_t left = size - r_in;
        ti.rows_valid = left <= 0 ? 0 : (left < BM ? (int)left : BM);
        ti.n0 = (int64_t)tn * BN;
        ti.b_row = (int64_t)g * p.N + ti.n0;
        ti.sfb_rt_base = (int64_t)g * p.b_rowtiles;
        ti.c_row0 = ti.row0;
    }
    return ti;
}

// Work item t: pair tile t in the full rounds; with SUB, the tiles of the last
// round in pieces of SUB columns.  int8: tiles of the last columns have only the
// pieces that N reaches.  The backward product, whose small pieces notice the
// arithmetic (K = 64: 26.2 against 27.0 us), counts all and finds some empty.
template <class Cfg, int MODE>
__device__ __forceinline__ TileInfo get_item(int t, uint32_t rank, const GemmParams &p, const int *cum, int tiles_n,
                                             int &g_at) {
    if constexpr (Cfg::SUB == 0) {
        return get_tile<Cfg::BN, MODE>(t, rank, p, cum, tiles_n, g_at);
    } else {
        int tile = t, piece = 0;
        if (t >= p.cut_whole) {
            const int u = t - p.cut_whole;
            if (!Cfg::I8 || u < p.cut_tiles * Cfg::PIECES) {
                tile = p.cut_whole + u / Cfg::PIECES;
                piece = u % Cfg::PIECES;
            } else {                            // first pieces of all, second pieces of all, ..
                tile = t - p.cut_tiles * (Cfg::PIECES - 1);
                while (tile >= p.cut_whole + p.cut_tiles + p.cut_last) {
                    tile -= p.cut_last;
                    ++piece;
                }
            }
        }
        TileInfo ti = get_tile<Cfg::BN, MODE>(tile, rank, p, cum, tiles_n, g_at);
        ti.n0 += Cfg::SUB * piece;
        ti.b_row += Cfg::SUB * piece;
        ti.width = t < p.cut_whole ? Cfg::BN : Cfg::SUB;
        return ti;
    }
}

// int8 epilogue: 32 integer sums of one row to (sum * token scale) * channel
// scale.  A sum up to 2^31 is rounded once to FP32 (24 bits) and each factor
// once: three half-steps of 2^-24, far below bf16's and within 2e-7 for FP32.
// Lane i holds the channel scale of column i of the step.
__device__ __forceinline__ void scale_i8(uint32_t *v, float tok, float chan) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float c = __shfl_sync(0xFFFFFFFFu, chan, i);
        v[i] = __float_as_uint(__fmul_rn(__fmul_rn(__int2float_rn((int)v[i]), tok), c));
    }
}

// 64-byte swizzled staging row (32 bf16) and 128-byte one (64 bf16): the
// 16-byte unit index is xored with address bits 7-8 or 7-9, as the tensor maps
// of the stores expect, which also spreads a warp's rows over all banks.
__device__ __forceinline__ void stage_row64(uint32_t buf, int lane, const uint32_t *w) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(buf + (uint32_t)lane * 64u +
                                                                      (((uint32_t)c ^ ((lane >> 1) & 3)) << 4)),
                     "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                     : "memory");
}
__device__ __forceinline__ void stage_row128(uint32_t buf, int lane, const uint32_t *w) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(buf + (uint32_t)lane * 128u +
                                                                      (((uint32_t)c ^ (lane & 7)) << 4)),
                     "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                     : "memory");
}
__device__ __forceinline__ void unstage_row128(uint32_t buf, int lane, uint32_t *w) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * c]), "=r"(w[4 * c + 1]), "=r"(w[4 * c + 2]), "=r"(w[4 * c + 3])
                     : "r"(buf + (uint32_t)lane * 128u + (((uint32_t)c ^ (lane & 7)) << 4))
                     : "memory");
}

// 8 * NV bf16 of one row straight to or from global memory, columns at or past
// `left` untouched (16-byte pieces; the rows are 16-byte aligned).
template <int NV>
__device__ __forceinline__ void store_row_bf16(uint16_t *dst, const uint32_t *w, int64_t left) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        if (8 * c + 8 <= left) {
            asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(dst + 8 * c), "r"(w[4 * c]),
                         "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                         : "memory");
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (8 * c + e < left) dst[8 * c + e] = (uint16_t)(w[4 * c + e / 2] >> (16 * (e & 1)));
        }
    }
}
template <int NV>
__device__ __forceinline__ void load_row_bf16(const uint16_t *src, uint32_t *w, int64_t left) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        if (8 * c + 8 <= left) {
            asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[4 * c]), "=r"(w[4 * c + 1]), "=r"(w[4 * c + 2]), "=r"(w[4 * c + 3])
                         : "l"(src + 8 * c)
                         : "memory");
        } else {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const uint32_t lo = 8 * c + e < left ? src[8 * c + e] : 0, hi = 8 * c + e + 1 < left ? src[8 * c + e + 1] : 0;
                w[4 * c + e / 2] = lo | (hi << 16);
            }
        }
    }
}

// A tensor-map store whose box reaches past the last column still writes whole
// 16-byte units: where the columns do not end on one (ncols elements of `esize`
// bytes) it would put zeros into the columns behind them, which belong to the
// caller, so the box of `width` columns at `col` goes out with plain stores.
__device__ __forceinline__ bool ragged_box(int64_t col, int width, int64_t ncols, int esize) {
    return col + width > ncols && (ncols * esize) % 16 != 0;
}

// Backward epilogue, per warp: z boxes (32 rows x 64 columns, 4 KB) stream into
// two staging buffers by TMA, one box ahead of the one computed; each box is
// replaced in place by dz and stored.  Load n goes into buffer n % 2 once the
// store of box n - 2, the newest one committed, has read it.  Boxes that reach
// past their group's rows, and ragged ones, do not go through the ring.
template <class Cfg, int MODE>
struct ZRing {
    int t, j, g_at;          // next box to look at: pair tile, 32-column step; its group
    uint32_t issued, used;
    TileInfo ti;

    __device__ __forceinline__ void start(int t0, int part) { t = t0; j = part; g_at = 0; issued = used = 0; }
    // Issue loads up to the box after the current one.
    __device__ __forceinline__ void fill(const CUtensorMap *map, uint8_t *bufs, uint64_t *bars, const GemmParams &p,
                                         const int *cum, int tiles_n, int ntiles, int npairs, uint32_t rank,
                                         int row_lo, int lane, int part) {
        while (issued < used + 2 && t < ntiles) {
            if (j == part) ti = get_item<Cfg, MODE>(t, rank, p, cum, tiles_n, g_at);
            const bool boxes = row_lo < ti.rows_valid && (MODE == MODE_DENSE || row_lo + 32 <= ti.rows_valid);
            const int64_t col0 = ti.n0 + 32 * j;
            if (boxes && col0 < p.N && !ragged_box(2 * col0, 64, 2 * p.N, 2)) {
                if (lane == 0) {
                    const uint32_t b = issued & 1u;
                    if (issued >= 2) bulk_wait_group_read<0>();
                    mbar_arrive_expect_tx(&bars[b], EPI_BUF);
                    tma_load_2d(bufs + b * EPI_BUF, map, (int32_t)(2 * col0), (int32_t)(ti.c_row0 + row_lo), &bars[b]);
                }
                ++issued;
            }
            j += Cfg::SPLIT;
            if (!boxes || j >= (Cfg::SUB ? ti.width : Cfg::BN) / 32) { j = part; t += npairs; }
        }
        __syncwarp();
    }
};

// One K stage of the pair tile, issued by the converged MMA warp: the stage's
// scale atoms go to tensor memory (A: NATOMS atoms of this pair's rows; B: NRT
// 128-row tiles x NATOMS atoms), then NK MMAs of K = 64 walk the 128-byte
// swizzled chunk rows 32 bytes at a time (4 MMAs per chunk).  The scale
// selector k & 1 picks bytes 0-1 or 2-3 of each 32-bit scale word (two
// 32-element blocks per MMA); k >> 1 steps to the next 4-block atom.
template <class Cfg, int NATOMS, int NK>
__device__ __forceinline__ void issue_stage(uint32_t d_tmem, uint32_t st, uint32_t sfa_col, uint32_t b_shift,
                                            bool first, uint32_t desc = Cfg::IDESC) {
    constexpr int NRT = Cfg::NRT, NATOM = Cfg::NATOM;
    if constexpr (Cfg::I8) {
        const uint64_t adesc = smem_desc(st, 16, 1024, 2);
        const uint64_t bdesc = smem_desc(st + Cfg::A_BYTES, 16, 1024, 2);
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            const uint64_t a_off = (uint64_t)(((k >> 2) * Cfg::A_CHUNK + (k & 3) * 32) >> 4);
            const uint64_t b_off = (uint64_t)(((k >> 2) * Cfg::B_CHUNK + (k & 3) * 32) >> 4);
            mma_i8_pair_elect(d_tmem, adesc + a_off, bdesc + b_off, desc, (k == 0 && first) ? 0u : 1u);
        }
        return;
    }
    const uint32_t sfb_col = sfa_col + 4u * NATOM;
    const uint64_t sf_desc = smem_desc(st + Cfg::A_BYTES + Cfg::B_BYTES, 0, 128, 0);
#pragma unroll
    for (int a = 0; a < NATOMS; ++a) {
        tc_cp_32x128_warpx4_pair_elect(sfa_col + 4u * a, sf_desc + (uint64_t)((512 * a) >> 4));
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt)
            tc_cp_32x128_warpx4_pair_elect(sfb_col + 4u * NRT * a + 4u * rt,
                                           sf_desc + (uint64_t)((Cfg::SFA_BYTES + NATOM * 512 * rt + 512 * a) >> 4));
    }
    const uint64_t adesc = smem_desc(st, 16, 1024, 2);
    const uint64_t bdesc = smem_desc(st + Cfg::A_BYTES, 16, 1024, 2);
#pragma unroll
    for (int k = 0; k < NK; ++k) {
        const uint64_t a_off = (uint64_t)(((k >> 2) * Cfg::A_CHUNK + (k & 3) * 32) >> 4);
        const uint64_t b_off = (uint64_t)(((k >> 2) * Cfg::B_CHUNK + (k & 3) * 32) >> 4);
        if constexpr (Cfg::NV) {
            // one atom (4 scales of 16) per K = 64 instruction
            mma_nvf4_pair_elect(d_tmem, adesc + a_off, bdesc + b_off, Cfg::IDESC, sfa_col + 4u * (uint32_t)k,
                                sfb_col + 4u * NRT * (uint32_t)k + b_shift, (k == 0 && first) ? 0u : 1u);
        } else {
            const uint32_t idesc = (k & 1) ? (desc | (2u << 29) | (2u << 4)) : desc;
            mma_mxf4_pair_elect(d_tmem, adesc + a_off, bdesc + b_off, idesc, sfa_col + 4u * (uint32_t)(k >> 1),
                                sfb_col + 4u * NRT * (uint32_t)(k >> 1) + b_shift, (k == 0 && first) ? 0u : 1u);
        }
    }
}

// Partial last K stage (K not a multiple of the stage depth): NK = ceil(kleft /
// KMMA) MMAs (kleft / 64 for E2M1) and ceil(NK / 2) scale atoms.
template <class Cfg>
__device__ __noinline__ void issue_stage_tail(uint32_t d_tmem, uint32_t st, uint32_t sfa_col, uint32_t b_shift,
                                              bool first, int nk, uint32_t desc) {
    if constexpr (Cfg::NV) {                  // one atom per MMA; a stage holds 4 * KCH MMAs
        switch (nk) {
            case 1: issue_stage<Cfg, 1, 1>(d_tmem, st, sfa_col, b_shift, first); break;
            case 2: issue_stage<Cfg, 2, 2>(d_tmem, st, sfa_col, b_shift, first); break;
            case 3: issue_stage<Cfg, 3, 3>(d_tmem, st, sfa_col, b_shift, first); break;
            default: break;
        }
        return;
    }
    switch (nk) {
        case 1: issue_stage<Cfg, 1, 1>(d_tmem, st, sfa_col, b_shift, first, desc); break;
        case 2: issue_stage<Cfg, 1, 2>(d_tmem, st, sfa_col, b_shift, first, desc); break;
        case 3: issue_stage<Cfg, 2, 3>(d_tmem, st, sfa_col, b_shift, first, desc); break;
        case 4: issue_stage<Cfg, 2, 4>(d_tmem, st, sfa_col, b_shift, first, desc); break;
        case 5: issue_stage<Cfg, 3, 5>(d_tmem, st, sfa_col, b_shift, first, desc); break;
        case 6: issue_stage<Cfg, 3, 6>(d_tmem, st, sfa_col, b_shift, first, desc); break;
        case 7: issue_stage<Cfg, 4, 7>(d_tmem, st, sfa_col, b_shift, first, desc); break;
        default: break;   // a full stage never takes this path
    }
}

template <class Cfg, int MODE, int OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg::THREADS, 1)
    mxfp4_gemm_kernel(const __grid_constant__ CUtensorMap tma_a, const __grid_constant__ CUtensorMap tma_b,
                      const __grid_constant__ CUtensorMap tma_c, const __grid_constant__ CUtensorMap tma_sfa,
                      const __grid_constant__ CUtensorMap tma_sfb, const __grid_constant__ CUtensorMap tma_z,
                      const GemmParams p) {
    constexpr int BN = Cfg::BN, STAGES = Cfg::STAGES;
    constexpr int A_BYTES = Cfg::A_BYTES, B_BYTES = Cfg::B_BYTES, SFA_BYTES = Cfg::SFA_BYTES;
    constexpr int STAGE_BYTES = Cfg::STAGE_BYTES, KCH = Cfg::KCH, NATOM = Cfg::NATOM;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *stage_base = smem;
    uint8_t *epi_base = smem + STAGES * STAGE_BYTES;
    Shared *sh = reinterpret_cast<Shared *>(epi_base + Cfg::EPI_BYTES);
    constexpr bool GROUPED = MODE == MODE_GROUPED_M;
    __shared__ int cum[MODE != MODE_DENSE ? MAX_GROUPS + 1 : 1];
    __shared__ uint64_t zbar[OUT == OUT_GATED_BWD ? Cfg::EPI_WARPS * Cfg::EPI_BUFS : 1];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();               // 0 = MMA issuer of the pair
    const int pair = (int)cluster_id_x(), npairs = (int)nclusters_x();
    const int tiles_n = (int)((p.N + BN - 1) / BN);
    auto ktiles_of = [](const TileInfo &ti) { return (int)((ti.kg + Cfg::KSTEP - 1) / Cfg::KSTEP); };
    const uint64_t limit = p.wait_limit_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(&sh->full[s], 1); mbar_init(&sh->empty[s], 1); }
        for (int b = 0; b < 2; ++b) { mbar_init(&sh->tmem_full[b], 1); mbar_init(&sh->tmem_empty[b], 2 * Cfg::EPI_WARPS); }
        mbar_init(&sh->drain, 1);
        if constexpr (OUT == OUT_GATED_BWD)
            for (int b = 0; b < Cfg::EPI_WARPS * Cfg::EPI_BUFS; ++b) mbar_init(&zbar[b], 1);
        sh->abort = 0;
        sh->drain_failed = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
        prefetch_tmap(&tma_a);
        prefetch_tmap(&tma_b);
        prefetch_tmap(&tma_c);
        if constexpr (!Cfg::I8) {
            prefetch_tmap(&tma_sfa);
            prefetch_tmap(&tma_sfb);
        }
        if constexpr (OUT == OUT_GATED || OUT == OUT_GATED_BWD) prefetch_tmap(&tma_z);
    }
    if (warp == 1) {
        tmem_alloc_pair(&sh->tmem_base, TMEM_COLS);
        tmem_relinquish_pair();
    }
    // the prologue above touches no global memory; from here on the previous
    // kernel's outputs are read (operands, group offsets) and C is written
    pdl_wait();
    pdl_trigger();
    if constexpr (GROUPED) {
        if (warp == 2) {
            // 32 groups at a time: their loads together, their tile counts summed
            // by a warp scan
            int acc = 0;
            for (int g0 = 0; g0 < p.num_groups; g0 += 32) {
                const int g = g0 + lane;
                int tiles = 0;
                if (g < p.num_groups) {
                    const int64_t off = p.group_offsets[g], nxt = p.group_offsets[g + 1];
                    const int64_t size = p.group_sizes[g];
                    if (off < 0 || (off % BM) != 0 || size < 0 || off + size > nxt || nxt > p.M) {
                        if (rank == 0) record_error(MXFP4_ERR_INVALID_ARG);
                    } else {
                        tiles = (int)((size + 255) / 256) * tiles_n;
                    }
                }
                int sum = tiles;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int below = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                    if (lane >= d) sum += below;
                }
                if (g < p.num_groups) cum[g] = acc + sum - tiles;
                acc += __shfl_sync(0xFFFFFFFFu, sum, 31);
            }
            if (lane == 0) {
                cum[p.num_groups] = acc;
                sh->ntiles = acc;
            }
        }
    } else if constexpr (MODE == MODE_GROUPED_K) {
        if (threadIdx.x == 32 * 2) {
            // K offsets: multiples of 128, non-decreasing, within K; a bad
            // entry records INVALID_ARG and empties the group
            int prev = 0;
            bool bad = false;
            for (int g = 0; g <= p.num_groups; ++g) {
                int o = p.group_offsets[g];
                if (o % 128 != 0 || o < prev || o > p.K) { bad = true; o = prev; }
                cum[g] = o;
                prev = o;
            }
            if (bad && rank == 0) record_error(MXFP4_ERR_INVALID_ARG);
            sh->ntiles = p.num_groups * (int)((p.M + 255) / 256) * tiles_n;
        }
    } else {
        if (threadIdx.x == 0) sh->ntiles = (int)((p.M + 255) / 256) * tiles_n;
    }
    // barriers of both CTAs initialized before any cross-CTA traffic
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sh->tmem_base;
    const int ntiles = Cfg::SUB ? p.cut_items : sh->ntiles;
    bool aborted_any = false;

    if (warp == 0) {
        // ------------------------------------------------------------ producer (both CTAs)
        // The whole warp runs the loop; one elected lane issues the copies.
        const bool issuer = elect_one();
        {
            uint32_t armed = 0, armed_par = 0;   // even CTA: stages armed, parity of the last arm
            int s = 0, g_at = 0;
            uint32_t ph = 0;
            for (int t = pair; t < ntiles && !sh->abort; t += npairs) {
                const TileInfo ti = get_item<Cfg, MODE>(t, rank, p, cum, tiles_n, g_at);
                const int half_b = (Cfg::SUB ? ti.width : BN) / 2;   // rows of B of this CTA
                const bool small_b = Cfg::SUB && Cfg::I8 && ti.width < BN;   // (other types load BN / 2 all the same)
                const int32_t sfa_rt = (int32_t)(ti.row0 / 128);
                const int32_t sfb_rt = (int32_t)(ti.sfb_rt_base + ti.n0 / 128);
                const int ktiles = ktiles_of(ti);
                const int32_t katom0 = (int32_t)(ti.k0 / Cfg::KATOM);   // grouped K: the group's first scale atom
                bool ok = true;
                for (int kt = 0; kt < ktiles; ++kt) {
                    if (!wait_phase(&sh->empty[s], ph ^ 1u, sh, limit)) { ok = false; break; }
                    uint8_t *st = stage_base + s * STAGE_BYTES;
                    const uint32_t full_leader = mapa_shared(smem_u32(&sh->full[s]), 0);
                    if (rank == 0) {
                        armed |= 1u << s;
                        armed_par = (armed_par & ~(1u << s)) | (ph << s);
                    }
                    if (issuer) {
                        if (rank == 0)
                            mbar_arrive_expect_tx(&sh->full[s], p.stage_tx - (small_b ? (BN - Cfg::SUB) * CHUNK * KCH : 0));
#pragma unroll
                        for (int c = 0; c < KCH; ++c) {
                            const int32_t kx = (int32_t)(ti.k0 / Cfg::KPB) + (kt * KCH + c) * CHUNK;
                            // (dense, one row tile: the odd CTA has no rows of A)
                            if (MODE != MODE_DENSE || rank == 0 || p.M > BM)
                                tma_load_2d_pair(st + c * Cfg::A_CHUNK, &tma_a, kx, (int32_t)ti.row0, full_leader);
                            tma_load_2d_pair(st + A_BYTES + c * Cfg::B_CHUNK, small_b ? &tma_z : &tma_b, kx,
                                             (int32_t)(ti.b_row + rank * half_b), full_leader);
                        }
                        // scale atoms: NATOM consecutive K atoms of one (A) or NRT (B) 128-row tiles
                        if constexpr (!Cfg::I8) {
                            tma_load_3d_pair(st + A_BYTES + B_BYTES, &tma_sfa, 0, katom0 + kt * NATOM, sfa_rt,
                                             full_leader);
                            tma_load_3d_pair(st + A_BYTES + B_BYTES + SFA_BYTES, &tma_sfb, 0, katom0 + kt * NATOM,
                                             sfb_rt, full_leader);
                        }
                    }
                    __syncwarp();
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                }
                if (!ok) break;
            }
            if (rank == 0) {
                // drain: the last load of every armed stage (both CTAs' bytes) has landed
                bool drained = true;
                for (int i = 0; i < STAGES; ++i)
                    if (armed & (1u << i))
                        drained &= wait_phase(&sh->full[i], (armed_par >> i) & 1u, sh, limit, true);
                if (!drained && issuer) mark_drain_failed(sh, rank);
            }
            if (sh->abort) aborted_any = true;
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (even CTA)
        // The whole warp runs the loop (warp-uniform operands); one elected
        // lane issues each tcgen05 instruction.
        if (rank == 0) {
            bool issued = false;
            int s = 0;
            uint32_t ph = 0, kglobal = 0;
            int acc = 0, g_at = 0;
            uint32_t acc_ph = 0;
            for (int t = pair; t < ntiles && !sh->abort; t += npairs) {
                const TileInfo ti = get_item<Cfg, MODE>(t, 0, p, cum, tiles_n, g_at);
                uint32_t desc = Cfg::IDESC;
                if constexpr (Cfg::SUB != 0) desc = (desc & ~(63u << 17)) | ((uint32_t)(ti.width >> 3) << 17);
                const int64_t rt0 = ti.n0 / 128;
                const uint32_t b_shift = (uint32_t)((ti.n0 - rt0 * 128) / 32);
                if (!wait_phase(&sh->tmem_empty[acc], acc_ph ^ 1u, sh, limit)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem + (acc ? Cfg::ACC1_COL : 0u);
                const int ktiles = ktiles_of(ti);
                bool ok = true;
                for (int kt = 0; kt < ktiles; ++kt) {
                    if (!wait_phase(&sh->full[s], ph, sh, limit)) { ok = false; break; }
                    tc_fence_after();
                    const int64_t kleft = ti.kg - (int64_t)kt * Cfg::KSTEP;
                    const uint32_t sfa_col = tmem + Cfg::SF_COL + Cfg::SF_STAGE_COLS * (kglobal & 1u);
                    const uint32_t st = smem_u32(stage_base + s * STAGE_BYTES);
                    // a stage whose last instruction is partial (int8, K not a
                    // multiple of 32) is full too: TMA filled it up with zeros
                    if (kleft > Cfg::KSTEP - Cfg::KMMA)
                        issue_stage<Cfg, NATOM, 4 * KCH>(d_tmem, st, sfa_col, b_shift, kt == 0, desc);
                    else
                        issue_stage_tail<Cfg>(d_tmem, st, sfa_col, b_shift, kt == 0,
                                              (int)((kleft + Cfg::KMMA - 1) / Cfg::KMMA), desc);
                    issued = true;
                    tc_commit_pair_elect(&sh->empty[s]);
                    ++kglobal;
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                }
                if (!ok) break;
                tc_commit_pair_elect(&sh->tmem_full[acc]);
                if (++acc == 2) { acc = 0; acc_ph ^= 1u; }
            }
            if (issued) {
                // drain: all MMAs / copies of this thread complete before TMEM or smem go away
                tc_commit_pair_elect(&sh->drain);
                if (!wait_phase(&sh->drain, 0, sh, limit, true) && lane == 0) mark_drain_failed(sh, rank);
            }
            if (sh->abort) aborted_any = true;
        }
    } else {
        // ------------------------------------------------------------ epilogue (both CTAs)
        const int q = warp & 3;                 // TMEM lane quarter of this warp
        const int ew = warp - 2;                // epilogue warp index
        const int part = ew >> 2;               // which of the SPLIT warps of the quarter
        int tile_i = 0;                         // tiles done by this CTA
        const uint32_t empty_leader0 = mapa_shared(smem_u32(&sh->tmem_empty[0]), 0);
        const uint32_t empty_leader1 = mapa_shared(smem_u32(&sh->tmem_empty[1]), 0);
        int acc = 0;
        uint32_t acc_ph = 0;
        uint32_t buf_i = 0;
        // NVFP4: the product of the two second-level scales (amax / 2688 each)
        float nv_scale = 1.0f;
        if constexpr (Cfg::NV) nv_scale = __fmul_rn(__fdiv_rn(*p.a_amax, 2688.0f), __fdiv_rn(*p.b_amax, 2688.0f));
        ZRing<Cfg, MODE> ring;
        uint8_t *ring_bufs = epi_base + ew * Cfg::EPI_BUFS * EPI_BUF;
        uint64_t *ring_bars = zbar + (OUT == OUT_GATED_BWD ? ew * Cfg::EPI_BUFS : 0);
        ring.start(pair, part);
        int g_at = 0;
        for (int t = pair; t < ntiles; t += npairs) {
            const TileInfo ti = get_item<Cfg, MODE>(t, rank, p, cum, tiles_n, g_at);
            const int row_lo = 32 * q;
            // int8: this lane's token scale, and the channel scale of column
            // 32 j + lane of the tile, one 32-column step ahead
            auto load_chan = [&](int j) {
                const int64_t col = ti.n0 + 32 * j + lane;
                return j < BN / 32 && col < p.N ? __ldg(p.b_chan + (ti.b_row - ti.n0) + col) : 0.0f;
            };
            float tok = 0.0f, chan = 0.0f;
            if constexpr (Cfg::I8) {
                if (row_lo + lane < ti.rows_valid) tok = __ldg(p.a_tok + ti.c_row0 + row_lo + lane);
                chan = load_chan(0);
            }
            if constexpr (OUT == OUT_GATED_BWD)
                ring.fill(&tma_z, ring_bufs, ring_bars, p, cum, tiles_n, ntiles, npairs, rank, row_lo, lane, part);
            // one answer for the warp: what follows needs it whole
            if (!__all_sync(0xFFFFFFFFu, wait_phase(&sh->tmem_full[acc], acc_ph, sh, limit))) break;
            tc_fence_after();
            bool full_box = MODE == MODE_DENSE || (row_lo + 32 <= ti.rows_valid);
            if constexpr (!Cfg::I8 && (OUT == OUT_F32 || OUT == OUT_BF16) && MODE != MODE_DENSE)
                full_box = full_box && ti.n0 <= p.box_n0;
            const bool any_row = row_lo < ti.rows_valid;
            const bool empty_k = ti.kg <= 0;              // grouped K: an empty group's output is zero
            if constexpr (OUT == OUT_MX) {
                // fused requantization: after each 32-column TMEM load a lane
                // holds 32 consecutive results of one row, i.e. one 1D row
                // block of C: amax, E8M0 scale and RNE E2M1 codes as in
                // mxfp4_quantize, stored straight from registers
                static_assert(MODE == MODE_DENSE, "MXFP4 output: dense GEMM only");
                const uint32_t tm = tmem + ((uint32_t)(32 * q) << 16) + (acc ? Cfg::ACC1_COL : 0u);
                const int64_t row = ti.c_row0 + row_lo + lane;
                const bool row_ok = row < p.M;
                for (int j = 0; j < BN / 32; ++j) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tm + 32u * j, v);
                    tmem_ld_wait();
                    if (j == BN / 32 - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(acc ? empty_leader1 : empty_leader0);
                    }
                    const int64_t col0 = ti.n0 + 32 * j;
                    if (!row_ok || col0 >= p.N) continue;
                    float f[32];
                    float amax = 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        f[i] = __uint_as_float(v[i]);
                        if constexpr (Cfg::NV) f[i] = __fmul_rn(f[i], nv_scale);
                        amax = amax_nan(amax, f[i]);
                    }
                    const uint32_t code = scale_code_from_amax(amax);
                    uint4 qv = make_uint4(0, 0, 0, 0);
                    if (code != 0xFFu) {
                        const float inv = inv_scale_from_code(code);
#pragma unroll
                        for (int i = 0; i < 32; ++i) f[i] = __fmul_rn(f[i], inv);
                        qv = make_uint4(e2m1x8_rn(f), e2m1x8_rn(f + 8), e2m1x8_rn(f + 16), e2m1x8_rn(f + 24));
                    }
                    asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(static_cast<uint8_t *>(p.c) +
                                                                                 row * p.ldc + (col0 >> 1)),
                                 "r"(qv.x), "r"(qv.y), "r"(qv.z), "r"(qv.w)
                                 : "memory");
                    const int64_t kb = col0 >> 5;
                    if (p.c_scale_mma) p.c_scales[mma_scale_off(row, kb, p.c_katoms)] = (uint8_t)code;
                    else p.c_scales[row * p.ld_c_scales + kb] = (uint8_t)code;
                }
            } else if constexpr (OUT == OUT_GATED) {
                // 64 columns of z per step: a lane holds 32 (gate, up) pairs of
                // one row, so the activation needs no exchange between lanes;
                // 32 h (and the 64 z, if kept) leave as one box each
                const GatedAct act{p.act_alpha, p.act_limit, p.act_beta};
                const uint32_t tm = tmem + ((uint32_t)(32 * q) << 16) + (acc ? Cfg::ACC1_COL : 0u);
                // with two warps to a quarter, steps alternate over all tiles
                // (three per tile: 2 and 1, then 1 and 2)
                constexpr int NS = BN / 64;
                const int first = Cfg::SPLIT == 1 ? 0 : ((tile_i * NS) & 1) ^ part;
                const int last = Cfg::SPLIT == 1 ? NS - 1 : NS - 1 - ((NS - 1 - first) & 1);
                for (int j = first; j < NS; j += Cfg::SPLIT) {
                    uint32_t w[32], hw[16];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(tm + 64u * j + 32u * h, v);
                        tmem_ld_wait();
                        float2 hv[8];
                        act.forward<8>(v, hv);
#pragma unroll
                        for (int i = 0; i < 8; ++i) hw[8 * h + i] = pack_bf16x2(hv[i].x, hv[i].y);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[16 * h + i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    }
                    if (j == last) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(acc ? empty_leader1 : empty_leader0);
                    }
                    const int64_t col0 = ti.n0 + 64 * j;
                    if (!any_row || col0 >= p.N) continue;
                    if (full_box && !ragged_box(col0 >> 1, 32, p.N >> 1, 2)) {
                        for (int o = p.z ? 0 : 1; o < 2; ++o) {
                            uint8_t *buf = epi_base + (ew * Cfg::EPI_BUFS + buf_i % Cfg::EPI_BUFS) * EPI_BUF;
                            if (lane == 0) bulk_wait_group_read<Cfg::EPI_BUFS - 1>();
                            __syncwarp();
                            if (o == 0) stage_row128(smem_u32(buf), lane, w);
                            else stage_row64(smem_u32(buf), lane, hw);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                if (o == 0) tma_store_2d(&tma_z, (int32_t)col0, (int32_t)(ti.c_row0 + row_lo), buf);
                                else tma_store_2d(&tma_c, (int32_t)(col0 >> 1), (int32_t)(ti.c_row0 + row_lo), buf);
                                bulk_commit_group();
                            }
                            ++buf_i;
                        }
                    } else if (row_lo + lane < ti.rows_valid) {
                        const int64_t row = ti.c_row0 + row_lo + lane;
                        store_row_bf16<4>(static_cast<uint16_t *>(p.c) + row * p.ldc + (col0 >> 1), hw, (p.N - col0) >> 1);
                        if (p.z) store_row_bf16<8>(static_cast<uint16_t *>(p.z) + row * p.ldz + col0, w, p.N - col0);
                    }
                }
            } else if constexpr (OUT == OUT_GATED_BWD) {
                // 32 columns of dh per step with the 64 columns of z they belong to
                static_assert(Cfg::EPI_BUFS == 2, "the ring has two buffers a warp");
                const GatedAct act{p.act_alpha, p.act_limit, p.act_beta};
                const uint32_t tm = tmem + ((uint32_t)(32 * q) << 16) + (acc ? Cfg::ACC1_COL : 0u);
                bool ok = true;
                const int steps = (Cfg::SUB ? ti.width : BN) / 32;
                for (int j = part; j < steps; j += Cfg::SPLIT) {
                    uint32_t v[32], w[32];
                    tmem_ld_32x32b_x32(tm + 32u * j, v);
                    // z arrives while the accumulators do
                    const int64_t col0 = ti.n0 + 32 * j;
                    const bool used = any_row && col0 < p.N;
                    const int64_t row = ti.c_row0 + row_lo + lane, zleft = 2 * (p.N - col0);
                    const bool lane_row = used && row_lo + lane < ti.rows_valid;
                    const bool in_ring = used && full_box && !ragged_box(2 * col0, 64, 2 * p.N, 2);
                    const uint32_t b = ring.used & 1u;
                    uint8_t *buf = ring_bufs + b * EPI_BUF;
                    if (in_ring) {
                        ring.fill(&tma_z, ring_bufs, ring_bars, p, cum, tiles_n, ntiles, npairs, rank, row_lo, lane, part);
                        // one answer for the warp: the tensor memory instructions need it whole
                        ok = __all_sync(0xFFFFFFFFu, wait_phase(&ring_bars[b], (ring.used >> 1) & 1u, sh, limit));
                        if (ok) unstage_row128(smem_u32(buf), lane, w);
                    } else if (lane_row) {
                        load_row_bf16<8>(static_cast<const uint16_t *>(p.z) + row * p.ldz + 2 * col0, w, zleft);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = 0u;
                    }
                    __syncwarp();
                    tmem_ld_wait_x32(v);
                    if (j + Cfg::SPLIT >= steps) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(acc ? empty_leader1 : empty_leader0);
                    }
                    if (!ok) break;
                    if (!used) continue;
                    act.backward<8>(v, w);
                    act.backward<8>(v + 16, w + 16);
                    if (in_ring) {
                        stage_row128(smem_u32(buf), lane, w);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(&tma_c, (int32_t)(2 * col0), (int32_t)(ti.c_row0 + row_lo), buf);
                            bulk_commit_group();
                        }
                        ++ring.used;
                    } else if (lane_row) {
                        store_row_bf16<8>(static_cast<uint16_t *>(p.c) + row * p.ldc + 2 * col0, w, zleft);
                    }
                }
                if (!ok) break;
            } else if constexpr (OUT == OUT_BF16) {
                // 64 columns per step: two 32-column TMEM loads rounded to
                // bf16 pairs (RNE), one 128-byte row segment per lane
                const uint32_t tm = tmem + ((uint32_t)(32 * q) << 16) + (acc ? Cfg::ACC1_COL : 0u);
                const int steps = (Cfg::SUB ? ti.width : BN) / 64;
                for (int j = 0; j < steps; ++j) {
                    uint32_t w[32];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(tm + 64u * j + 32u * h, v);
                        tmem_ld_wait();
                        if (empty_k) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = 0u;
                        }
                        if constexpr (Cfg::NV) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] = __float_as_uint(__fmul_rn(__uint_as_float(v[i]), nv_scale));
                        }
                        if constexpr (Cfg::I8) scale_i8(v, tok, chan);
                        if constexpr (Cfg::I8) chan = load_chan(2 * j + h + 1);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[16 * h + i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    }
                    if (j == steps - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(acc ? empty_leader1 : empty_leader0);
                    }
                    if (!any_row) continue;
                    const int64_t col0 = ti.n0 + 64 * j;
                    if (col0 >= p.N) continue;
                    if (full_box && !(Cfg::I8 && ragged_box(col0, 64, p.N, 2))) {
                        uint8_t *buf = epi_base + (ew * Cfg::EPI_BUFS + (buf_i & 1u)) * EPI_BUF;
                        if (lane == 0) bulk_wait_group_read<1>();
                        __syncwarp();
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const uint32_t off = (uint32_t)lane * 128u + (((uint32_t)c ^ (uint32_t)(lane & 7)) << 4);
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(smem_u32(buf) + off),
                                         "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                                         : "memory");
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && (!Cfg::RAGGED || col0 < p.box_cols)) {
                            tma_store_2d(&tma_c, (int32_t)col0, (int32_t)(ti.c_row0 + row_lo), buf);
                            bulk_commit_group();
                        }
                        ++buf_i;
                        if (Cfg::RAGGED && col0 + 64 > p.box_cols && row_lo + lane < ti.rows_valid) {
                            uint16_t *dst = static_cast<uint16_t *>(p.c) + (ti.c_row0 + row_lo + lane) * p.ldc + p.box_cols;
                            const int left = (int)(p.N - p.box_cols);
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                if (col0 + 8 * c != p.box_cols) continue;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    if (2 * e + 2 <= left) *reinterpret_cast<uint32_t *>(dst + 2 * e) = w[4 * c + e];
                                    else if (2 * e < left) dst[2 * e] = (uint16_t)w[4 * c + e];
                                }
                            }
                        }
                    } else if (row_lo + lane < ti.rows_valid) {
                        uint16_t *dst = static_cast<uint16_t *>(p.c) + (ti.c_row0 + row_lo + lane) * p.ldc + col0;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const int64_t cc = col0 + 8 * c;
                            if (cc + 8 <= p.N) {
                                asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(dst + 8 * c),
                                             "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                                             : "memory");
                            } else {
                                for (int e = 0; e < 8; ++e)
                                    if (cc + e < p.N) dst[8 * c + e] = (uint16_t)(w[4 * c + e / 2] >> (16 * (e & 1)));
                            }
                        }
                    }
                }
            } else {
                const int steps = (Cfg::SUB ? ti.width : BN) / 32;
                for (int j = 0; j < steps; ++j) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * q) << 16) + (acc ? Cfg::ACC1_COL : 0u) + 32u * j, v);
                    tmem_ld_wait();
                    if (empty_k) {
    #pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0u;
                    }
                    if constexpr (Cfg::NV) {
    #pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__fmul_rn(__uint_as_float(v[i]), nv_scale));
                    }
                    if constexpr (Cfg::I8) scale_i8(v, tok, chan);
                    if constexpr (Cfg::I8) chan = load_chan(j + 1);
                    if (j == steps - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(acc ? empty_leader1 : empty_leader0);
                    }
                    if (!any_row) continue;
                    const int64_t col0 = ti.n0 + 32 * j;
                    if (col0 >= p.N) continue;
                    if (full_box && !(Cfg::I8 && ragged_box(col0, 32, p.N, 4))) {
                        uint8_t *buf = epi_base + (ew * Cfg::EPI_BUFS + (buf_i & 1u)) * EPI_BUF;
                        if (lane == 0) bulk_wait_group_read<1>();
                        __syncwarp();
    #pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const uint32_t off = (uint32_t)lane * 128u + (((uint32_t)c ^ (uint32_t)(lane & 7)) << 4);
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(smem_u32(buf) + off),
                                         "r"(v[4 * c]), "r"(v[4 * c + 1]), "r"(v[4 * c + 2]), "r"(v[4 * c + 3])
                                         : "memory");
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && (!Cfg::RAGGED || col0 < p.box_cols)) {
                            tma_store_2d(&tma_c, (int32_t)col0, (int32_t)(ti.c_row0 + row_lo), buf);
                            bulk_commit_group();
                        }
                        ++buf_i;
                        if (Cfg::RAGGED && col0 + 32 > p.box_cols && row_lo + lane < ti.rows_valid) {
                            float *dst = static_cast<float *>(p.c) + (ti.c_row0 + row_lo + lane) * p.ldc + p.box_cols;
                            const int left = (int)(p.N - p.box_cols);
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                if (col0 + 4 * c != p.box_cols) continue;
#pragma unroll
                                for (int e = 0; e < 3; ++e)
                                    if (e < left) dst[e] = __uint_as_float(v[4 * c + e]);
                            }
                        }
                    } else if (row_lo + lane < ti.rows_valid) {
                        float *dst = static_cast<float *>(p.c) + (ti.c_row0 + row_lo + lane) * p.ldc + col0;
    #pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const int64_t cc = col0 + 4 * c;
                            if (cc + 4 <= p.N) {
                                asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(dst + 4 * c), "r"(v[4 * c]),
                                             "r"(v[4 * c + 1]), "r"(v[4 * c + 2]), "r"(v[4 * c + 3])
                                             : "memory");
                            } else {
                                for (int e = 0; e < 4; ++e)
                                    if (cc + e < p.N) dst[4 * c + e] = __uint_as_float(v[4 * c + e]);
                            }
                        }
                    }
                }
            }
            if (++acc == 2) { acc = 0; acc_ph ^= 1u; }
            ++tile_i;
        }
        if constexpr (OUT == OUT_GATED_BWD) {
            // after an abort: loads in flight land before the shared memory goes away
            bool landed = true;
            for (; ring.used < ring.issued; ++ring.used)
                landed &= wait_phase(&ring_bars[ring.used & 1u], (ring.used >> 1) & 1u, sh, limit, true);
            if (!landed && lane == 0) mark_drain_failed(sh, rank);
        }
        if (lane == 0) bulk_wait_group_all();
        __syncwarp();
        if (sh->abort) aborted_any = true;
    }
    (void)aborted_any;
    __syncthreads();
    cluster_sync();   // neither CTA leaves while the pair may still touch its smem or TMEM
    // The leader's drain waited (bounded) for every load of both CTAs and for
    // its MMAs; only if such a wait ran out can a copy or an MMA still be in
    // flight: then give it time before the shared and tensor memory go away.
    if (sh->drain_failed) spin_ns(200000);
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

// Bounded-wait probe: one barrier that only `arrive` can complete.
__global__ void wait_probe_kernel(int arrive, uint64_t limit) {
    __shared__ uint64_t bar;
    __shared__ Shared sh;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        if (arrive) mbar_arrive(&bar);
        wait_phase(&bar, 0, &sh, limit);
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static uint64_t g_wait_limit_ns = 2000000000ull;

uint64_t set_wait_limit(uint64_t ns) {
    const uint64_t old = g_wait_limit_ns;
    g_wait_limit_ns = ns ? ns : 2000000000ull;
    return old;
}

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

static bool make_map(CUtensorMap *m, CUtensorMapDataType dt, const void *base, uint64_t inner, uint64_t outer,
                     uint64_t stride_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {stride_bytes};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, dt, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale atoms of the GEMM-ready layout: 512-byte atoms, katoms per 128-row
// tile, `tiles` row tiles; boxes of `box_k` atoms x `box_t` tiles.
static bool make_map_3d(CUtensorMap *m, const void *base, uint64_t katoms, uint64_t tiles, uint32_t box_k,
                        uint32_t box_t) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {128, katoms, tiles};
    const cuuint64_t strides[2] = {512, 512 * katoms};
    const cuuint32_t box[3] = {128, box_k, box_t};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int sm_count() {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

template <class Cfg, int MODE, int OUT>
static cudaError_t set_smem_attr() {
    // once per device and instantiation: keep cudaFuncSetAttribute off the hot path
    static int done[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(mxfp4_gemm_kernel<Cfg, MODE, OUT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = 1;
    return e;
}

struct GemmArgs {
    const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
    int64_t lda, ldb, M, N, K, ldc;
    void *c;
    const int32_t *offsets, *sizes;
    int G;
    const float *a_amax = nullptr, *b_amax = nullptr;
    uint8_t *c_scales = nullptr;
    int64_t ld_c_scales = 0;
    int c_scale_mma = 0;
    const float *a_tok = nullptr, *b_chan = nullptr;
    void *z = nullptr;
    int64_t ldz = 0;
    float alpha = 1.0f, limit = 0.0f, beta = 0.0f;
    int cut_whole = 0, cut_tiles = 0, cut_last = 0, cut_items = 0;
};

// Returns 0 on success, MXFP4_ERR_CUDA when a map or launch fails.
// Grouped K: a and b are [M, K/2] and [N, K/2] over all groups' K ranges, c is
// [G * M, N]; the B operand and C map cover G groups only in grouped-rows mode.
// OUT_BF16: C is bf16 (RNE of the FP32 accumulators), stored in 64-column
// boxes; OUT_MX: C is MXFP4 codes + scales written without the C tensor map
// (a map over the codes is still passed, never used).  OUT_GATED: C is h
// [.., N/2] in 32-column boxes and z [.., N], if kept, in 64-column ones;
// OUT_GATED_BWD: z in and C = dz out, both [.., 2N], in 64-column boxes.
template <class Cfg, int MODE, int OUT = OUT_F32>
static int launch_cfg(const GemmArgs &g, cudaStream_t s) {
    constexpr int BN = Cfg::BN;
    const int G = MODE == MODE_GROUPED_M ? g.G : 1;
    const int64_t c_rows = MODE == MODE_GROUPED_K ? (int64_t)g.G * g.M : g.M;
    const int64_t katoms = (g.K + Cfg::KATOM - 1) / Cfg::KATOM;
    const int64_t a_tiles = (g.M + 127) / 128, b_tiles = (g.N + 127) / 128;
    // Few rows: filling the box's rows past M is slower than loading rows, so the
    // box is as high as it has to be and the odd CTA loads none (what stands in
    // shared memory there only reaches rows that are not stored).  16 rows of
    // 178560 x 2880: 88 -> 60 us.
    const uint32_t a_box = MODE == MODE_DENSE && g.M <= 64 ? (g.M <= 32 ? 32 : 64) : BM;
    CUtensorMap ta, tb, tc, tz, tsa, tsb;
    constexpr CUtensorMapDataType BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    constexpr CUtensorMapSwizzle SW128 = CU_TENSOR_MAP_SWIZZLE_128B;
    const uint64_t kbytes = (uint64_t)(g.K / Cfg::KPB), N = (uint64_t)g.N, ldc = (uint64_t)g.ldc;
    constexpr int64_t per16 = OUT == OUT_F32 ? 4 : 8;
    // (a map has at least one column; where there are none to store it is not used)
    const uint64_t c_cols = !Cfg::RAGGED ? N : (uint64_t)(g.N < per16 ? per16 : g.N / per16 * per16);
    bool ok = make_map(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.a_codes, kbytes, (uint64_t)g.M, (uint64_t)g.lda, CHUNK, a_box,
                       SW128) &&
              make_map(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.b_codes, kbytes, (uint64_t)G * N, (uint64_t)g.ldb, CHUNK,
                       BN / 2, SW128);
    if constexpr (OUT == OUT_MX)
        ok = ok && make_map(&tc, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.c, N / 2, (uint64_t)c_rows, ldc, 16, 32,
                            CU_TENSOR_MAP_SWIZZLE_NONE);
    else if constexpr (OUT == OUT_GATED)
        ok = ok && make_map(&tc, BF, g.c, N / 2, (uint64_t)c_rows, ldc * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    else if constexpr (OUT == OUT_GATED_BWD)
        ok = ok && make_map(&tc, BF, g.c, 2 * N, (uint64_t)c_rows, ldc * 2, 64, 32, SW128);
    else if constexpr (OUT == OUT_BF16)
        ok = ok && make_map(&tc, BF, g.c, c_cols, (uint64_t)c_rows, ldc * 2, 64, 32, SW128);
    else
        ok = ok && make_map(&tc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, g.c, c_cols, (uint64_t)c_rows, ldc * 4, 32, 32, SW128);
    if (!ok) return MXFP4_ERR_CUDA;
    tz = tsa = tsb = tc;                       // never used where an operand below does not exist
    if ((OUT == OUT_GATED || OUT == OUT_GATED_BWD) && g.z &&
        !make_map(&tz, BF, g.z, OUT == OUT_GATED ? N : 2 * N, (uint64_t)c_rows, (uint64_t)g.ldz * 2, 64, 32, SW128))
        return MXFP4_ERR_CUDA;
    if constexpr (Cfg::I8 && Cfg::SUB)         // B's boxes of a piece
        if (!make_map(&tz, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.b_codes, kbytes, (uint64_t)G * N, (uint64_t)g.ldb, CHUNK,
                      Cfg::SUB / 2, SW128))
            return MXFP4_ERR_CUDA;
    // scale atoms as a 3D tensor [128-row tile][K atom][512 bytes = 128 x 32-bit]:
    // one box holds NATOM consecutive atoms of one (A) or NRT (B) row tiles
    if constexpr (!Cfg::I8)
        if (!make_map_3d(&tsa, g.a_scales, (uint64_t)katoms, (uint64_t)a_tiles, Cfg::NATOM, 1) ||
            !make_map_3d(&tsb, g.b_scales, (uint64_t)katoms, (uint64_t)(G * b_tiles), Cfg::NATOM, Cfg::NRT))
            return MXFP4_ERR_CUDA;
    if (set_smem_attr<Cfg, MODE, OUT>() != cudaSuccess) return MXFP4_ERR_CUDA;
    GemmParams p{};
    p.M = g.M; p.N = g.N; p.K = g.K;
    p.katoms = katoms;
    p.b_rowtiles = b_tiles;
    p.c = g.c; p.ldc = g.ldc;
    p.c_scales = g.c_scales; p.ld_c_scales = g.ld_c_scales; p.c_scale_mma = g.c_scale_mma;
    p.c_katoms = (g.N / 32 + 3) / 4;
    p.group_offsets = g.offsets; p.group_sizes = g.sizes; p.num_groups = g.G;
    p.a_amax = g.a_amax; p.b_amax = g.b_amax;
    p.a_tok = g.a_tok; p.b_chan = g.b_chan;
    p.box_n0 = g.N % per16 ? g.N - BN : g.N;
    p.box_cols = g.N / per16 * per16;
    p.z = g.z; p.ldz = g.ldz;
    p.act_alpha = g.alpha; p.act_limit = g.limit; p.act_beta = g.beta;
    p.cut_whole = g.cut_whole; p.cut_tiles = g.cut_tiles; p.cut_last = g.cut_last; p.cut_items = g.cut_items;
    p.wait_limit_ns = g_wait_limit_ns;
    p.stage_tx = Cfg::STAGE_TX - (uint32_t)(Cfg::KCH * (BM - a_box) * CHUNK) -
                 (MODE == MODE_DENSE && g.M <= BM ? (uint32_t)Cfg::A_BYTES : 0u);
    const int pairs_max = sm_count() / 2;
    int pairs = pairs_max;
    if (MODE != MODE_GROUPED_M) {
        const int64_t tiles = (MODE == MODE_GROUPED_K ? g.G : 1) * ((g.M + 255) / 256) * ((g.N + BN - 1) / BN);
        const int64_t items = Cfg::SUB ? g.cut_items : tiles;
        pairs = (int)(items < pairs_max ? items : pairs_max);
    }
    const cudaError_t e = launch_pdl(mxfp4_gemm_kernel<Cfg, MODE, OUT>, dim3((unsigned)(2 * pairs)), dim3(Cfg::THREADS),
                                     (size_t)Cfg::SMEM_BYTES, s, ta, tb, tc, tsa, tsb, tz, p);
    return e == cudaSuccess ? 0 : MXFP4_ERR_CUDA;
}

int launch_gemm(const uint8_t *a_codes, int64_t lda, const uint8_t *a_scales, const uint8_t *b_codes, int64_t ldb,
                const uint8_t *b_scales, int64_t M, int64_t N, int64_t K, float *c, int64_t ldc, cudaStream_t s) {
    GemmArgs g{a_codes, a_scales, b_codes, b_scales, lda, ldb, M, N, K, ldc, c, nullptr, nullptr, 1};
    return N % 4 ? launch_cfg<RaggedCfg, MODE_DENSE>(g, s) : launch_cfg<DefaultCfg, MODE_DENSE>(g, s);
}

int launch_grouped_gemm(const uint8_t *a_codes, int64_t lda, const uint8_t *a_scales, int64_t a_rows,
                        const int32_t *offsets, const int32_t *sizes, int G, const uint8_t *b_codes, int64_t ldb,
                        const uint8_t *b_scales, int64_t N, int64_t K, float *c, int64_t ldc, cudaStream_t s) {
    GemmArgs g{a_codes, a_scales, b_codes, b_scales, lda, ldb, a_rows, N, K, ldc, c, offsets, sizes, G};
    return launch_cfg<DefaultCfg, MODE_GROUPED_M>(g, s);
}

int launch_gemm_bf16(const uint8_t *a_codes, int64_t lda, const uint8_t *a_scales, const uint8_t *b_codes,
                     int64_t ldb, const uint8_t *b_scales, int64_t M, int64_t N, int64_t K, uint16_t *c, int64_t ldc,
                     cudaStream_t s) {
    GemmArgs g{a_codes, a_scales, b_codes, b_scales, lda, ldb, M, N, K, ldc, c, nullptr, nullptr, 1};
    return N % 8 ? launch_cfg<RaggedCfg, MODE_DENSE, OUT_BF16>(g, s) : launch_cfg<DefaultCfg, MODE_DENSE, OUT_BF16>(g, s);
}

int launch_grouped_gemm_bf16(const uint8_t *a_codes, int64_t lda, const uint8_t *a_scales, int64_t a_rows,
                             const int32_t *offsets, const int32_t *sizes, int G, const uint8_t *b_codes,
                             int64_t ldb, const uint8_t *b_scales, int64_t N, int64_t K, uint16_t *c, int64_t ldc,
                             cudaStream_t s) {
    GemmArgs g{a_codes, a_scales, b_codes, b_scales, lda, ldb, a_rows, N, K, ldc, c, offsets, sizes, G};
    return launch_cfg<DefaultCfg, MODE_GROUPED_M, OUT_BF16>(g, s);
}

int launch_gemm_mx(const uint8_t *a_codes, int64_t lda, const uint8_t *a_scales, const uint8_t *b_codes,
                   int64_t ldb, const uint8_t *b_scales, int64_t M, int64_t N, int64_t K, uint8_t *c_codes,
                   int64_t ld_c_codes, uint8_t *c_scales, int64_t ld_c_scales, int c_scale_mma, cudaStream_t s) {
    GemmArgs g{a_codes, a_scales, b_codes, b_scales, lda, ldb, M, N, K, ld_c_codes, c_codes, nullptr, nullptr, 1};
    g.c_scales = c_scales;
    g.ld_c_scales = ld_c_scales;
    g.c_scale_mma = c_scale_mma;
    return launch_cfg<DefaultCfg, MODE_DENSE, OUT_MX>(g, s);
}

int launch_grouped_wgrad(const uint8_t *a_codes, int64_t lda, const uint8_t *a_scales, const uint8_t *b_codes,
                         int64_t ldb, const uint8_t *b_scales, const int32_t *offsets, int G, int64_t M, int64_t N,
                         int64_t K, float *c, int64_t ldc, cudaStream_t s) {
    GemmArgs g{a_codes, a_scales, b_codes, b_scales, lda, ldb, M, N, K, ldc, c, offsets, nullptr, G};
    return launch_cfg<DefaultCfg, MODE_GROUPED_K>(g, s);
}

int launch_grouped_wgrad_bf16(const uint8_t *a_codes, int64_t lda, const uint8_t *a_scales, const uint8_t *b_codes,
                              int64_t ldb, const uint8_t *b_scales, const int32_t *offsets, int G, int64_t M,
                              int64_t N, int64_t K, uint16_t *c, int64_t ldc, cudaStream_t s) {
    GemmArgs g{a_codes, a_scales, b_codes, b_scales, lda, ldb, M, N, K, ldc, c, offsets, nullptr, G};
    return launch_cfg<DefaultCfg, MODE_GROUPED_K, OUT_BF16>(g, s);
}

int launch_nvfp4_gemm(const uint8_t *a_codes, int64_t lda, const uint8_t *a_scales, const float *a_amax,
                      const uint8_t *b_codes, int64_t ldb, const uint8_t *b_scales, const float *b_amax, int64_t M,
                      int64_t N, int64_t K, float *c, int64_t ldc, cudaStream_t s) {
    GemmArgs g{a_codes, a_scales, b_codes, b_scales, lda, ldb, M, N, K, ldc, c, nullptr, nullptr, 1, a_amax, b_amax};
    return N % 4 ? launch_cfg<RaggedNvCfg, MODE_DENSE>(g, s) : launch_cfg<NvCfg, MODE_DENSE>(g, s);
}

// Launch with the last round of tiles cut into pieces where those fit one round.
template <class Cfg, class Cut, int MODE, int OUT>
static int launch_cut(const GemmArgs &g, cudaStream_t s) {
    if constexpr (Cut::SUB != 0) {
        static_assert(MODE == MODE_DENSE && Cut::BN == Cfg::BN, "the same tiles, counted on the host");
        const int64_t pairs = sm_count() / 2, tiles_m = (g.M + 255) / 256, tiles_n = (g.N + Cfg::BN - 1) / Cfg::BN;
        const int64_t rest = tiles_m * tiles_n % pairs;
        const int64_t last = !Cut::I8 ? 0 : rest < tiles_m ? rest : tiles_m;      // (M is the fast axis)
        const int64_t tail = (g.N - (tiles_n - 1) * Cfg::BN + Cut::SUB - 1) / Cut::SUB;
        const int64_t pieces = (rest - last) * Cut::PIECES + last * tail;
        if (rest && pieces <= pairs) {
            GemmArgs c = g;
            c.cut_whole = (int)(tiles_m * tiles_n - rest);
            c.cut_tiles = (int)(rest - last);
            c.cut_last = (int)last;
            c.cut_items = c.cut_whole + (int)pieces;
            return launch_cfg<Cut, MODE, OUT>(c, s);
        }
    }
    return launch_cfg<Cfg, MODE, OUT>(g, s);
}

// Launch with the wide or the narrow tile: a narrow tile costs 0.65 to 0.8 of a
// wide one (its instructions are shorter, its operand bytes per product more),
// so it has to save that much in rounds of the resident pairs.  The row tiles of
// groups are on the device: their number is taken as that of all rows and a
// quarter per group (half a tile for every other group, whose rows end in the
// first half of one).
// WideCut, NarrowCut: the same tiles with the last round cut into pieces.
template <class Wide, class Narrow, int MODE, int OUT, class WideCut = Wide, class NarrowCut = Narrow>
static int launch_tiles(const GemmArgs &g, cudaStream_t s) {
    const int64_t pairs = sm_count() / 2, tiles_m = (g.M + 255) / 256 + (MODE == MODE_GROUPED_M ? g.G / 4 : 0);
    auto rounds = [&](int64_t bn) { return (tiles_m * ((g.N + bn - 1) / bn) + pairs - 1) / pairs; };
    if (4 * rounds(Narrow::BN) < 5 * rounds(Wide::BN)) return launch_cut<Narrow, NarrowCut, MODE, OUT>(g, s);
    return launch_cut<Wide, WideCut, MODE, OUT>(g, s);
}

// Gated products: the activation of column pairs of A B^T (forward), or dz from
// dh = A B^T and z (backward); offsets null for the dense forms.
int launch_gated(const GatedArgs &a, cudaStream_t s) {
    if (!a.offsets && !a.backward && gated_by_rows(a.M, a.N, a.K)) return launch_gated_rows(a, s);
    GemmArgs g{a.a_codes, a.a_scales, a.b_codes, a.b_scales, a.lda, a.ldb, a.M, a.N, a.K, a.ld_out, a.out, a.offsets,
               a.sizes, a.offsets ? a.G : 1};
    g.z = a.z;
    g.ldz = a.ldz;
    g.alpha = a.alpha;
    g.limit = a.limit;
    g.beta = a.beta;
    if (a.backward)
        return a.offsets ? launch_tiles<BwdCfg, BwdNarrowCfg, MODE_GROUPED_M, OUT_GATED_BWD>(g, s)
                         : launch_tiles<BwdCfg, BwdNarrowCfg, MODE_DENSE, OUT_GATED_BWD, BwdCutCfg, BwdNarrowCutCfg>(g, s);
    return a.offsets ? launch_tiles<GatedCfg, GatedNarrowCfg, MODE_GROUPED_M, OUT_GATED>(g, s)
                     : launch_tiles<GatedCfg, GatedNarrowCfg, MODE_DENSE, OUT_GATED>(g, s);
}

int launch_int8_gemm(const Int8Args &a, cudaStream_t s) {
    if (!a.offsets && int8_by_rows(a.M, a.N, a.K)) return launch_int8_rows(a, s);
    GemmArgs g{reinterpret_cast<const uint8_t *>(a.a), nullptr, reinterpret_cast<const uint8_t *>(a.b), nullptr, a.lda,
               a.ldb, a.M, a.N, a.K, a.ldc, a.c, a.offsets, a.sizes, a.offsets ? a.G : 1};
    g.a_tok = a.a_scales;
    g.b_chan = a.b_scales;
    if (a.offsets)
        return a.bf16 ? launch_tiles<I8GroupedCfg, I8GroupedNarrowCfg, MODE_GROUPED_M, OUT_BF16>(g, s)
                      : launch_tiles<I8GroupedCfg, I8GroupedNarrowCfg, MODE_GROUPED_M, OUT_F32>(g, s);
    return a.bf16 ? launch_tiles<I8Cfg, I8NarrowCfg, MODE_DENSE, OUT_BF16, I8CutCfg>(g, s)
                  : launch_tiles<I8Cfg, I8NarrowCfg, MODE_DENSE, OUT_F32, I8CutCfg>(g, s);
}

int get_error(cudaStream_t s) {
    if (cudaStreamSynchronize(s) != cudaSuccess) return MXFP4_ERR_CUDA;
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_error_code, sizeof(v)) != cudaSuccess) return MXFP4_ERR_CUDA;
    const unsigned int zero = 0;
    if (v && cudaMemcpyToSymbol(g_error_code, &zero, sizeof(zero)) != cudaSuccess) return MXFP4_ERR_CUDA;
    return (int)v;
}

int launch_wait_probe(int arrive, cudaStream_t s) {
    wait_probe_kernel<<<1, 32, 0, s>>>(arrive, g_wait_limit_ns);
    return cudaGetLastError() == cudaSuccess ? 0 : MXFP4_ERR_CUDA;
}

}  // namespace mxfp4

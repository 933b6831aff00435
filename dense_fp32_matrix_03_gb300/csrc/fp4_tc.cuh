// fp4_tc.cuh -- products in microscaled 4-bit floating point on the tensor
// cores (include/fp4_gemm.h): C[m][n] = scaleA[m] scaleB[n] sum_k A[m][k] B[n][k]
// with the block scales inside the sum.
//
// tcgen05.mma kind::mxf4nvf4 takes 64 values of k an instruction, codes from
// shared memory (rows of 128 bytes = 256 values, 128-byte swizzle, as TMA
// writes them) and block scales from tensor memory: four bytes per row and 64
// values (NV, 16 values a scale) or two (MX, 32 values a scale).  The scales'
// layout in memory is the one tcgen05.cp wants: a tile of 128 rows by four
// blocks is 512 bytes that one copy spreads over four columns.
//
// The weights are the MMA's M side (128 channels per CTA) and the tokens its N
// side, so that few tokens cost MMAs of their own size.
//   narrow  one CTA, 128 channels x up to 128 tokens; a cluster of up to 8 CTAs
//           may share a tile, each a part of k, whose partial sums meet in
//           distributed shared memory, in CTA order
//   slim    the same for up to 32 tokens in all, with a deeper ring
//   wide    a CTA pair (cta_group::2), 256 channels x 256 tokens
//
// Tensor memory, wide: two accumulators of 256 columns do not fit beside the
// scales, so they overlap: the second starts 208 columns after the first, and
// the epilogue reads the 64 columns that hold the overlap before all others; the
// next tile's MMAs wait for that, not for the whole accumulator.
//
// Warps: 0 TMA producer, 1 tensor memory and MMA issuer, 2 idle, 3 asks L2 for the
// first weights (one CTA), then the epilogue (tensor memory -> scales -> result type -> staging -> C).  Every wait
// is bounded.
//
// Measured on GB300, bf16 results: 8192 x 8192 x 4096 101 to 104 us (NV, 5300 to 5400
// TFLOP/s, by box; in 32 bits 115), x 8192 183 to 188 (MX 180 to 184), 4096^3 30, 1024 x
// 4096 x 4096 11.5; narrow 128 x 4096 x 4096 8.2; slim 1 to 32 tokens x 4096 x 4096 5.8
// to 6.4.  What bounds the wide form: at 8192^3 the multiplies alone take 135 us and
// the loads alone as long (19 TB/s out of L2, all five stages on their way; 134 us
// with a pair's token scales loaded once); together they share the multiprocessor's
// memory.  Four stages cost 5%, three 20%.  What bounds the others: latency; a stage of k is
// 0.3 us, and a tile without any takes 2.5.
#pragma once

#include "fp4.cuh"
#include "i8_tc.cuh"
#include "tc_ss.cuh"

namespace sg {
namespace fp4 {

using tc::Ring;
using tcp::cta_rank;
using tcp::drain_cl;

struct Args {
    int M, N, K;
    const unsigned char *A, *sfA, *B, *sfB;
    long long lda, ldb;  // bytes
    long long tiles;     // of block scales, per row
    const float *scaleA, *scaleB;  // null: ones
    void *C;
    long long ldc;
    unsigned int *status;
    int num_sms;
};

constexpr int kCh = 128;       // channels per CTA
constexpr int kStageK = 256;   // k per stage: 128 bytes
constexpr int kMmaK = 64;
constexpr int kSteps = kStageK / kMmaK;
constexpr int kEWarp0 = 4;

// TCOLS: columns of tensor memory to allocate.
template <int CG_, int NT_, int STAGES_, int EWARPS_, uint32_t TCOLS_>
struct Cfg {
    static constexpr int CG = CG_, NT = NT_, STAGES = STAGES_, EWARPS = EWARPS_;
    static constexpr uint32_t TCOLS = TCOLS_;
    static constexpr int NTC = NT / CG;         // tokens per CTA's half
    static constexpr int RB = (NT + 127) / 128; // row blocks of the tokens' scales
    static constexpr int W_BYTES = kCh * 128, T_BYTES = NTC * 128;
    static constexpr int SF_BYTES = kSteps * kTileBytes;  // of one row block, at most (NV)
    static constexpr int OFF_T = W_BYTES, OFF_SW = OFF_T + T_BYTES, OFF_ST = OFF_SW + SF_BYTES;
    static constexpr int STAGE = OFF_ST + RB * SF_BYTES;
    static constexpr int ECOLS = NT / (EWARPS / 4);  // tokens per epilogue warp
    static constexpr int THREADS = (kEWarp0 + EWARPS) * 32;
    static constexpr int STAGING = 32 * 32 * 2;      // per epilogue warp, 16-bit results
    static constexpr int NBAR = 2 * STAGES + 4 + 1;
    static constexpr int OFF_STAGING = STAGES * STAGE;
    static constexpr int OFF_SCALE = OFF_STAGING + EWARPS * STAGING;
    static constexpr int OFF_BAR = OFF_SCALE + EWARPS * ECOLS * 4;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
    // columns of tensor memory: accumulators, then the scales of a stage
    static constexpr uint32_t ACC_STEP = NT == 256 ? 208 : NT;
    static constexpr uint32_t SW_COL = ACC_STEP + NT, ST_COL = SW_COL + 4 * kSteps;
    static_assert(ST_COL + 4 * kSteps * RB <= TCOLS && TCOLS <= 512, "tensor-memory columns");
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
    static_assert(STAGE % 1024 == 0, "swizzled boxes on 1024 bytes");
    static_assert(CG == 2 || NT * kCh * 4 <= STAGES * STAGE, "partial sums fit the stages");
};
using Slim = Cfg<1, 32, 8, 4, 128>;
using Narrow = Cfg<1, 128, 5, 4, 512>;
using Wide = Cfg<2, 256, 5, 8, 512>;

// A copy's source: 32 rows of 16 bytes without swizzle, eight rows 128 bytes
// apart from the next eight.
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem_addr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(128 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}
// One tile of block scales into four columns of all four lane quarters (of both
// CTAs of a pair, each from its own shared memory).
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc, uint32_t one)
{
    if constexpr (CG == 2)
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                     "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(tmem),
                     "l"(desc), "r"(one)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                     "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(tmem),
                     "l"(desc), "r"(one)
                     : "memory");
}
// Whether this thread is the one of its (converged) warp that issues.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(one));
    return one;
}
// d (+)= 64 values of k of weights times tokens; it overwrites d unless acc.
template <int CG, int FORMAT>
__device__ __forceinline__ void mma(uint32_t d, uint64_t w, uint64_t t, uint32_t idesc,
                                    uint32_t sw, uint32_t st, uint32_t acc, uint32_t one)
{
#define SG_FP4_MMA(GROUP, VEC)                                                                   \
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\t"                            \
                 "setp.ne.b32 q, %7, 0;\n\t"                                                     \
                 "@q tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC   \
                 " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                              \
                 "l"(w), "l"(t), "r"(idesc), "r"(sw), "r"(st), "r"(acc), "r"(one)                \
                 : "memory")
    if constexpr (CG == 2 && FORMAT == SGEMM_FP4_NV)
        SG_FP4_MMA("2", "4X");
    else if constexpr (CG == 2)
        SG_FP4_MMA("2", "2X");
    else if constexpr (FORMAT == SGEMM_FP4_NV)
        SG_FP4_MMA("1", "4X");
    else
        SG_FP4_MMA("1", "2X");
#undef SG_FP4_MMA
}
// Instruction descriptor: both operands e2m1, block scales e4m3 (NV) or powers
// of two (MX), tokens n, channels m; id: which bytes of the scales' columns
// (MX: 0 or 2).
template <int FORMAT>
__device__ __forceinline__ uint32_t inst_desc(int m, int n, uint32_t id)
{
    return (id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (FORMAT == SGEMM_FP4_MX ? 1u << 23 : 0u) | (static_cast<uint32_t>(m >> 4) << 24) |
           (id << 29);
}

// One output tile: tokens row0 .. row0 + n - 1, channels from ch0 on (this
// CTA's 128); neff: the MMA's N.
struct Job {
    int n, neff, ch0;
    long long row0;
};
// Tile u: groups of eight token tiles by all channel tiles, so that CTAs at work
// together share tokens and weights in L2.
template <class C>
__device__ __forceinline__ Job job(const Args &a, long long u, uint32_t half)
{
    const long long mt = (a.M + C::NT - 1LL) / C::NT, ct = (a.N + kCh * C::CG - 1LL) / (kCh * C::CG);
    const long long g = u / (8 * ct), in = u - g * 8 * ct;
    const long long rows_ = min(8LL, mt - 8 * g);
    const long long c = in / rows_, m = 8 * g + in - c * rows_;
    Job j;
    j.row0 = m * C::NT;
    j.n = static_cast<int>(min(static_cast<long long>(C::NT), a.M - j.row0));
    constexpr int STEP = 16 * C::CG;
    j.neff = (j.n + STEP - 1) / STEP * STEP;
    j.ch0 = static_cast<int>((c * C::CG + half) * kCh);
    return j;
}

// tmW, tmT: codes as bytes (K / 2, rows) in boxes of 128 bytes by 128 rows,
// 128-byte swizzle; tmSW, tmST: block scales in boxes of a stage's tiles of one
// row block.  What a box holds past the last row, value or scale is
// zeros.  split: CTAs of the cluster that share a tile's k (narrow only); then
// each cluster has one tile.  c_bytes: accesses that C's rows allow.
template <class C, class T, int FORMAT>
__global__ void __launch_bounds__(C::THREADS, 1)
    fp4_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT,
               const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmST,
               const Args a, int split, int c_bytes)
{
    constexpr int CG = C::CG;
    constexpr int TILES = FORMAT == SGEMM_FP4_NV ? 4 : 2;  // of scales a stage
    constexpr uint32_t BYTES =
        C::W_BYTES + C::T_BYTES + (1 + C::RB) * TILES * kTileBytes;  // a stage's, one CTA
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(base + C::OFF_BAR);  // issuing CTA's
    uint64_t *empty = full + C::STAGES;        // per CTA: commits
    uint64_t *acc_full = empty + C::STAGES;    // per CTA: commits
    uint64_t *acc_free = acc_full + 2;         // issuing CTA's: epilogues
    uint64_t *mma_done = acc_free + 2;
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_base + 1);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    const uint32_t half = CG == 2 ? rank : 0u, krank = CG == 2 ? 0u : rank;
    const int cluster = CG == 2 ? 2 : split;
    const long long cid = static_cast<int>(blockIdx.x) / cluster;
    const long long ncl = static_cast<int>(gridDim.x) / cluster;
    const bool issuer = CG == 1 || rank == 0;
    const int stages = (a.K + kStageK - 1) / kStageK;
    const int ks_lo = static_cast<int>(static_cast<long long>(stages) * krank / split);
    const int ks_hi = static_cast<int>(static_cast<long long>(stages) * (krank + 1) / split);
    const long long tiles = ((a.M + C::NT - 1LL) / C::NT) * ((a.N + kCh * CG - 1LL) / (kCh * CG));


    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1u);
            mbar_init(&empty[s], 1u);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&acc_full[s], 1u);
            mbar_init(&acc_free[s], static_cast<uint32_t>(CG * C::EWARPS));
        }
        mbar_init(mma_done, 1u);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmT);
        tma_prefetch_desc(&tmSW);
        tma_prefetch_desc(&tmST);
    }
    if (warp == 1) {
        if constexpr (CG == 2)
            tcp::tmem_alloc_pair(tmem_base, C::TCOLS);
        else
            tc::tmem_alloc(tmem_base, C::TCOLS);
    }
    dependent_release();
    // few tokens: the weights start on their way into L2 while the kernel before
    // (the quantiser, as a rule) runs; nothing is read yet
    if (CG == 1 && warp == 3 && lane == 0 && cid < tiles) {
        const int ch0 = job<C>(a, cid, 0).ch0;
        for (int ks = ks_lo; ks < ks_hi && ks < ks_lo + 16; ++ks) {
            i8::tma_prefetch_3d(&tmW, ks * 128, ch0, 0);
            i8::tma_prefetch_3d(&tmSW, 0, ks * TILES, ch0 / kTileRows);
        }
    }
    dependent_wait();
    tc::tc_fence_before();
    if constexpr (CG == 2)
        tcp::cluster_sync();
    else
        __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_base, 0);
    const Abort ab{abort_flag, a.status, kWaitLimitCycles};
    float *part = reinterpret_cast<float *>(base);  // split: [token][channel]

    if (warp == 0) {
        // -------------------------------------------------------- producer
        if (lane == 0) {
            Ring<C::STAGES> rr;
            long long issued = 0;
            bool ok = true;
            for (long long u = cid; ok && u < tiles; u += ncl) {
                const Job j = job<C>(a, u, half);
                const int first = static_cast<int>(j.row0) + static_cast<int>(half) * (j.neff / CG);
                for (int ks = ks_lo; ks < ks_hi; ++ks) {
                    if (!i8::wait_pair<CG>(&empty[rr.s], rr.ph ^ 1u, ab, kStatusWaitEmpty)) {
                        ok = false;
                        break;
                    }
                    uint8_t *st = base + rr.s * C::STAGE;
                    if constexpr (CG == 2) {
                        if (rank == 0) mbar_arrive_expect_tx(&full[rr.s], 2 * BYTES);
                        const uint32_t fb = tcs::cluster_addr(&full[rr.s], 0);
                        tcs::tma_load_pair(st, &tmW, fb, ks * 128, j.ch0, 0);
                        tcs::tma_load_pair(st + C::OFF_T, &tmT, fb, ks * 128, first, 0);
                        tcs::tma_load_pair(st + C::OFF_SW, &tmSW, fb, 0, ks * TILES, j.ch0 / kTileRows);
                        // both CTAs need all tokens' scales
#pragma unroll
                        for (int b = 0; b < C::RB; ++b)
                            tcs::tma_load_pair(st + C::OFF_ST + b * TILES * kTileBytes, &tmST, fb, 0,
                                               ks * TILES, static_cast<int>(j.row0 / kTileRows) + b);
                    } else {
                        mbar_arrive_expect_tx(&full[rr.s], BYTES);
                        tma_load_3d(st, &tmW, &full[rr.s], ks * 128, j.ch0, 0);
                        tma_load_3d(st + C::OFF_T, &tmT, &full[rr.s], ks * 128, first, 0);
                        tma_load_3d(st + C::OFF_SW, &tmSW, &full[rr.s], 0, ks * TILES,
                                    j.ch0 / kTileRows);
                        tma_load_3d(st + C::OFF_ST, &tmST, &full[rr.s], 0, ks * TILES,
                                    static_cast<int>(j.row0 / kTileRows));
                    }
                    ++issued;
                    rr.next();
                }
            }
            // stopping early: no load is in flight when the CTA leaves (of a pair,
            // the even CTA's barrier counts both CTAs' loads)
            if (issuer && (!ok || *abort_flag)) {
                Ring<C::STAGES> d;
                for (long long i = 0; i < issued; ++i) {
                    if (i + C::STAGES >= issued) drain_cl(&full[d.s], d.ph, ab.limit);
                    d.next();
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------------- MMA issuer
        // The whole warp walks the loop, so that descriptors and addresses live in
        // uniform registers, and one elected thread issues: issued by a lane of its
        // own, each instruction costs some 50 clocks of moves to uniform registers.
        if (issuer) {
            const uint32_t one = elect_one();
            Ring<C::STAGES> sr;
            bool ok = true, any = false;
            const uint32_t s0 = smem_u32(base);
            const uint64_t wd = tc::kmajor_sw128_desc(s0), td = tc::kmajor_sw128_desc(s0 + C::OFF_T);
            const uint64_t swd = scale_desc(s0 + C::OFF_SW), std_ = scale_desc(s0 + C::OFF_ST);
            int n = 0;  // tiles done
            for (long long u = cid; ok && u < tiles; u += ncl, ++n) {
                const Job j = job<C>(a, u, half);
                // the accumulator of two tiles ago is read (and, of a pair, the
                // columns that the last tile's shares with it)
                const int buf = n & 1;
                if (CG == 2 ? n > 0 : n > 1) {
                    const int w = CG == 2 ? n - 1 : n - 2;  // the tile waited for
                    if (!i8::warp_wait_pair<CG>(&acc_free[w & 1], static_cast<uint32_t>(w >> 1) & 1u,
                                                ab, kStatusWaitAcc)) {
                        ok = false;
                        break;
                    }
                }
                tc::tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(buf) * C::ACC_STEP;
                const uint32_t idesc = inst_desc<FORMAT>(kCh * CG, j.neff, 0);
                for (int ks = ks_lo; ks < ks_hi; ++ks) {
                    if (!i8::warp_wait_pair<CG>(&full[sr.s], sr.ph, ab, kStatusWaitFull)) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    const uint64_t off = static_cast<uint64_t>(sr.s) * (C::STAGE >> 4);
#pragma unroll
                    for (int i = 0; i < TILES; ++i) {
                        copy_scales<CG>(tmem + C::SW_COL + 4 * i, swd + off + i * (kTileBytes >> 4),
                                        one);
#pragma unroll
                        for (int b = 0; b < C::RB; ++b)
                            copy_scales<CG>(tmem + C::ST_COL + 4 * (i * C::RB + b),
                                            std_ + off + (b * TILES + i) * (kTileBytes >> 4), one);
                    }
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        const int t = FORMAT == SGEMM_FP4_NV ? i : i / 2;
                        const uint32_t id = FORMAT == SGEMM_FP4_NV ? 0u : 2u * (i & 1);
                        mma<CG, FORMAT>(d, wd + off + 2 * i, td + off + 2 * i,
                                        idesc | (id << 4) | (id << 29), tmem + C::SW_COL + 4 * t,
                                        tmem + C::ST_COL + 4 * t * C::RB,
                                        ks > ks_lo || i > 0 ? 1u : 0u, one);
                    }
                    any = true;
                    if (one) i8::commit<CG>(&empty[sr.s]);
                    sr.next();
                }
                if (!ok) break;
                if (one) i8::commit<CG>(&acc_full[buf]);
            }
            if (any) {
                if (one) i8::commit<CG>(mma_done);
                drain_cl(mma_done, 0, ab.limit);
            }
        }
        __syncwarp();
    } else if (warp >= kEWarp0) {
        // -------------------------------------------------------- epilogue
        // Lanes of tensor memory are channels, columns tokens; C wants a token's
        // channels side by side.  fp32: 32 lanes store 128 bytes of a token's row
        // as they are.  16 bits: chunks of 32 x 32 go through a transposing matrix
        // store into 64-byte token rows (16-byte pieces XORed with token / 2
        // against bank conflicts) and out in pieces as C's rows allow.
        const int q = warp & 3, w = warp - kEWarp0;
        const int col0 = (w >> 2) * C::ECOLS;  // this warp's first token of the tile
        const uint32_t stage = smem_u32(base + C::OFF_STAGING + w * C::STAGING);
        const uint32_t st_row = stage + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
        float *sa = reinterpret_cast<float *>(base + C::OFF_SCALE) + w * C::ECOLS;
        constexpr bool PACK = sizeof(T) == 2;
        constexpr int NV_ = PACK ? 16 : 32;  // registers of a chunk
        long long tile = 0;
        for (long long u = cid; u < tiles; u += ncl, ++tile) {
            const Job j = job<C>(a, u, half);
            const int chq = j.ch0 + q * 32;  // this warp's first channel
            const int n = min(j.n - col0, C::ECOLS);
            float sb[4] = {};  // 16 bits: channels lane / 4 + 8 i; else channel lane
            if (split == 1) {
                __syncwarp();  // the last tile's readers of sa are done (its stores may diverge)
                for (int i = lane; i < C::ECOLS; i += 32)
                    sa[i] = i < n ? (a.scaleA != nullptr ? a.scaleA[j.row0 + col0 + i] : 1.f) : 0.f;
#pragma unroll
                for (int i = 0; i < (PACK ? 4 : 1); ++i) {
                    const int c = chq + (PACK ? 8 * i + (lane >> 2) : lane);
                    if (c < a.N) sb[i] = a.scaleB != nullptr ? a.scaleB[c] : 1.f;
                }
                __syncwarp();
            }
            const int buf = static_cast<int>(tile & 1);
            const uint32_t ph = static_cast<uint32_t>(tile >> 1) & 1u;
            int got = 1;
            if (lane == 0) got = i8::wait_pair<CG>(&acc_full[buf], ph, ab, kStatusWaitAcc, true);
            if (!__shfl_sync(0xffffffffu, got, 0)) break;
            if constexpr (CG == 2)  // (every lane acquires)
                drain_cl(&acc_full[buf], ph, ab.limit);
            else
                mbar_drain(&acc_full[buf], ph, ab.limit);
            tc::tc_fence_after();
            const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) +
                                static_cast<uint32_t>(buf) * C::ACC_STEP + static_cast<uint32_t>(col0);
            T *crow = static_cast<T *>(a.C) + (j.row0 + col0) * a.ldc + chq;
            // a chunk of 32 tokens; 16 bits: scaled and packed, m[4 t + i] is channels
            // 8 i + lane / 4, tokens 8 t + 2 (lane % 4), + 1; fp32: as it is
            auto read_chunk = [&](int c0, uint32_t (&m)[NV_]) {
                if constexpr (PACK) {
                    uint32_t v[2][16];
                    i8::tmem_ld_16x32(tb + c0, v[0]);
                    i8::tmem_ld_16x32(tb + (16u << 16) + c0, v[1]);
                    i8::tmem_wait_ld();
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const float2 s =
                            *reinterpret_cast<const float2 *>(sa + c0 + 8 * t + 2 * (lane & 3));
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            m[4 * t + i] = i8::pack2<T>(i8::mul2(
                                i8::mul2(make_float2(
                                             __uint_as_float(v[i >> 1][4 * t + 2 * (i & 1)]),
                                             __uint_as_float(v[i >> 1][4 * t + 2 * (i & 1) + 1])),
                                         s),
                                make_float2(sb[i], sb[i])));
                    }
                } else {
                    float v[32];
                    tc::tmem_ld32(tb + c0, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) m[i] = __float_as_uint(v[i]);
                }
            };
            auto store_chunk = [&](int c0, const uint32_t (&m)[NV_]) {
                T *out = crow + static_cast<long long>(c0) * a.ldc;
                const int rows_left = n - c0;
                if constexpr (!PACK) {
                    if (chq + lane < a.N) {
                        T *row = out + lane;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (i < rows_left)
                                *row = rows::from_f<T>(__uint_as_float(m[i]) * sa[c0 + i] * sb[0]);
                            row += a.ldc;
                        }
                    }
                } else {
                    __syncwarp();  // the staging's last readers are done
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const uint32_t x[4] = {m[4 * t], m[4 * t + 1], m[4 * t + 2], m[4 * t + 3]};
                        i8::store_transposed(st_row + t * 512, x);
                    }
                    __syncwarp();
                    if (c_bytes == 16 && chq + 32 <= a.N) {
                        const int r = lane >> 2, p = lane & 3;
                        const uint32_t at = stage + r * 64 + ((p ^ ((r >> 1) & 3)) << 4);
                        T *to = out + r * a.ldc + 8 * p;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 x = i8::lds128(at + i * 512);
                            if (8 * i + r < rows_left) *reinterpret_cast<uint4 *>(to) = x;
                            to += 8 * a.ldc;
                        }
                    } else if (c_bytes >= 8 && chq + 32 <= a.N) {
                        const int r = lane >> 3, p = lane & 7;
                        T *to = out + r * a.ldc + 4 * p;
                        uint32_t at[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            at[i] = stage + r * 64 +
                                    (((p >> 1) ^ ((2 * i + (r >> 1)) & 3)) << 4) + 8 * (p & 1);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            uint2 x;
                            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                         : "=r"(x.x), "=r"(x.y)
                                         : "r"(at[i & 1] + i * 256));
                            if (4 * i + r < rows_left) *reinterpret_cast<uint2 *>(to) = x;
                            to += 4 * a.ldc;
                        }
                    } else {
                        // off 8-byte boundaries, or past the last channel: a value a
                        // lane, a token's row at a time
                        uint32_t at[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            at[i] = stage + (((lane >> 3) ^ i) << 4) + 2 * (lane & 7);
                        const bool mine = chq + lane < a.N;
                        T *row = out + lane;
#pragma unroll
                        for (int r0 = 0; r0 < 32; r0 += 8) {
                            uint16_t x[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                asm volatile("ld.shared.u16 %0, [%1];"
                                             : "=h"(x[i])
                                             : "r"(at[((r0 + i) >> 1) & 3] + (r0 + i) * 64));
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                if (mine && r0 + i < rows_left)
                                    *reinterpret_cast<uint16_t *>(row) = x[i];
                                row += a.ldc;
                            }
                        }
                    }
                }
            };
            auto release = [&]() {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) i8::arrive_issuer<CG>(&acc_free[buf]);
            };
            if (CG == 1 && split > 1) {
#pragma unroll 1
                for (int c0 = 0; c0 < n; c0 += 32) {
                    float v[32];
                    tc::tmem_ld32(tb + c0, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        part[(col0 + c0 + i) * kCh + q * 32 + lane] = v[i];
                }
                release();
            } else if constexpr (CG == 2) {
                // the two chunks that the accumulators share columns in, first
                const int c1 = col0 == 0 ? 0 : C::ECOLS - 64;
                uint32_t m0[NV_], m1[NV_];
                if (c1 < n) read_chunk(c1, m0);
                if (c1 + 32 < n) read_chunk(c1 + 32, m1);
                release();
                if (c1 < n) store_chunk(c1, m0);
                if (c1 + 32 < n) store_chunk(c1 + 32, m1);
                const int c2 = col0 == 0 ? 64 : 0;
#pragma unroll 1
                for (int c0 = c2; c0 < c2 + 64 && c0 < n; c0 += 32) {
                    read_chunk(c0, m0);
                    store_chunk(c0, m0);
                }
            } else {
#pragma unroll 1
                for (int c0 = 0; c0 < n; c0 += 32) {
                    uint32_t m[NV_];
                    read_chunk(c0, m);
                    store_chunk(c0, m);
                }
                release();
            }
        }
    }

    if (CG == 1 && split > 1) {
        // ---- partial sums of the cluster's CTAs, added in CTA order; CTA r takes
        // tokens r, r + split, ...: a warp a token, four channels a lane
        __syncwarp();
        const bool some = cid < tiles;
        Job j{};
        float sb[4] = {};
        if (some) {
            j = job<C>(a, cid, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (j.ch0 + 4 * lane + i < a.N)
                    sb[i] = a.scaleB != nullptr ? a.scaleB[j.ch0 + 4 * lane + i] : 1.f;
        }
        tcp::cluster_sync();
        if (some && *abort_flag == 0) {
            const int ch = j.ch0 + 4 * lane;
            for (int t = static_cast<int>(krank) + warp * split; t < j.n;
                 t += split * (C::THREADS / 32)) {
                const float sc = a.scaleA != nullptr ? a.scaleA[j.row0 + t] : 1.f;
                const uint32_t at = smem_u32(part + t * kCh + 4 * lane);
                const float4 s = split == 8 ? i8::cluster_sum<8>(at)
                                            : split == 4 ? i8::cluster_sum<4>(at)
                                                         : i8::cluster_sum<2>(at);
                const float o[4] = {s.x * sc * sb[0], s.y * sc * sb[1], s.z * sc * sb[2],
                                    s.w * sc * sb[3]};
                T *cp = static_cast<T *>(a.C) + (j.row0 + t) * a.ldc + ch;
                if (c_bytes >= 4 * static_cast<int>(sizeof(T)) && ch + 4 <= a.N) {
                    rows::Vec<T, 4 * static_cast<int>(sizeof(T))> x;
#pragma unroll
                    for (int i = 0; i < 4; ++i) x.set(i, o[i]);
                    x.store(cp);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (ch + i < a.N) cp[i] = rows::from_f<T>(o[i]);
                }
            }
        }
    }

    // ---- teardown: no CTA leaves while another may touch its shared memory
    tc::tc_fence_before();
    __syncwarp();
    if (CG == 2 || split > 1) {
        tcp::cluster_sync();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc::tc_fence_after();
        if constexpr (CG == 2)
            tcp::tmem_dealloc_pair(tmem, C::TCOLS);
        else
            tc::tmem_dealloc(tmem, C::TCOLS);
    }
}

// Enqueues the kernel on `clusters` clusters of CG (or split) CTAs.
template <class C, class T, int FORMAT>
int launch_tc(const Args &a, long long clusters, int split, int c_bytes, cudaStream_t st)
{
    constexpr int TILES = FORMAT == SGEMM_FP4_NV ? 4 : 2;
    alignas(64) CUtensorMap tmW, tmT, tmSW, tmST;
    const long long bytes = (a.K + 1LL) / 2;
    if (!encode_operand8(&tmW, reinterpret_cast<const signed char *>(a.B), a.N, bytes, a.ldb, 1, 0,
                         kCh) ||
        !encode_operand8(&tmT, reinterpret_cast<const signed char *>(a.A), a.M, bytes, a.lda, 1, 0,
                         C::NTC) ||
        !encode_block_scales(&tmSW, a.sfB, a.tiles, (a.N + kTileRows - 1LL) / kTileRows, TILES, 1) ||
        !encode_block_scales(&tmST, a.sfA, a.tiles, (a.M + kTileRows - 1LL) / kTileRows, TILES, 1))
        return SGEMM_ERR_LAUNCH;
    auto kern = fp4_kernel<C, T, FORMAT>;
    if (!smem_attr_once(reinterpret_cast<const void *>(kern), C::SMEM)) return SGEMM_ERR_LAUNCH;
    const unsigned size = C::CG == 2 ? 2u : static_cast<unsigned>(split);
    return launch_dependent(kern, dim3(static_cast<unsigned>(clusters) * size), dim3(C::THREADS),
                            C::SMEM, size, st, tmW, tmT, tmSW, tmST, a, split, c_bytes);
}

}  // namespace fp4
}  // namespace sg

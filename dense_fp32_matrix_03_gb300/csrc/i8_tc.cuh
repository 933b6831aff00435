// i8_tc.cuh -- products of 8-bit integers with a scale for each token and
// channel on the tensor cores:
//   C[m][n] = scaleA[m] * scaleB[n] * sum_k A[m][k] * B[n][k].
//
// Arithmetic.  An 8-bit integer is exact in fp16 and the product of two has
// magnitude at most 2^14, so kind::f16 with fp32 accumulation gives the exact
// integer sum while the sum of magnitudes stays within 2^24.  Beyond, an MMA
// (16 values of k) cuts its products two bits below fp32's last place of the
// largest number in the addition, and the new sum at that place: at most
// 16 * 2^-25 + 2^-23 = 5 * 2^-23 of the partial sum.  (Measured with equal
// codes 127 times 97, whose products are 31 modulo 32: exact to 2^26, then
// lost, of the sum, 2.7e-5 at K = 8192, 1.1e-4 at 16384, 6e-4 at 65536, 1.4e-3 at
// 131056; 1.1e-4 there where eight CTAs share k.)  On this GPU the
// 8-bit integer rate of the tensor cores is far below the 16-bit one, so the
// integers are widened in the kernel: HBM and L2 carry one byte a value, the
// tensor cores run at their 16-bit rate.  Widening four bytes takes five
// instructions: x ^ 0x80 is x + 128 as an unsigned byte u, two byte permutes
// put 0x64 above each u (the fp16 value 1024 + u), and two packed
// subtractions of 1152 leave x.
//
// Roles of the operands.  The weights are the MMA's M side (128 channels per
// CTA, always full) and the tokens its N side (16 to 256, in steps of 16 or
// 32), so that few tokens, or an expert's short last tile, cost MMAs of their
// own size.  Widened weights go to tensor memory (a thread holds a row, as
// tensor memory wants it) and never to shared memory, whose bandwidth the
// widened tokens need: per CTA and 128 k at 256 tokens, in units of 128 bytes
// a clock, 128 (weights in) + 128 (weights read) + 128 (tokens in) + 256
// (tokens widened) + 256 (MMA reads) of the MMA's 1024 clocks.
//
// Data flow, per step of 128 k (a "slot"):
//   producers  weights, 128 rows of 128 bytes, and tokens, in boxes of 32
//              rows, by TMA into a ring each (128-byte swizzle)
//   A warps    a row per thread: 8 x 16 bytes -> 64 columns of packed fp16 in
//              tensor memory
//   B warps    16 bytes at a time -> 32 bytes of fp16 in shared memory
//   MMA        one thread: 8 MMAs of k = 16
//   epilogue   tensor memory -> scales -> result type -> staging -> C
// A and B warps come in two sets that take alternate slots: widening a slot
// takes a set 550 (A) to 1000 (B, 128 tokens) clocks besides its waits.
// The order of k inside a slot is permuted (the first eight values of every
// 16-byte piece, then the second eight), the same way for both operands: a
// token's 16-byte piece then becomes one 16-byte piece of each of the slot's
// two 64-k boxes, at the byte offset it had itself: rows of 128 bytes and
// their swizzle are the same before and after, so widening is a walk over
// offsets, free of bank conflicts.
//
// Two configurations.
//   narrow  one CTA, 128 channels x up to 128 tokens, two accumulators.  For
//           few tokens the weights are what is read, and a cluster of up to
//           8 CTAs may share a tile, each a part of k: the partial sums meet
//           in distributed shared memory, in CTA order, without a workspace
//           or a second launch.
//   wide    a CTA pair (cta_group::2), 256 channels x up to 256 tokens, each
//           CTA widening its 128 channels and half the tokens.
// Every wait is bounded.
//
// Measured on GB300, bf16 results: 8192 x 8192 x 8192 612 us (1796 TFLOP/s,
// 0.94 of the measured 16-bit peak, above its sustained rate), x 4096 317 us,
// x 1024 104 us; 32 experts of 4096 x 2048 over 32768 rows, unevenly, 366 us.
// fp32 results: 8192 x 8192 x 4096 347 us, 8192 x 4096 x 2048 107 us (bf16 91): the
// accumulator is released after the stores, since a tile of them does not fit
// the registers.
// What bounds the wide form: the MMAs' 1024 clocks a slot stretch to about 1220
// beside the converters (without them: 1000 to 1050), and a tile's end leaves
// the tensor pipe idle for about 1850 clocks, while the accumulator is read.
// What bounds the narrow form for few tokens: a slot takes one thread about
// 1100 clocks to issue (eight MMAs cost at least 45 clocks each whatever their
// N), so weights pass at 2.4 (8192 x 8192, 20 to 64 tokens: 27 us) to 3.2 TB/s;
// i8_few.cuh takes over where it is faster.
#pragma once

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/sgemm.h"
#include "dependent.cuh"
#include "i8_gemm.h"
#include "rows.cuh"
#include "tc_pair.cuh"

namespace sg {
namespace i8 {

using tc::Ring;
using tcp::arrive_on;
using tcp::cta_rank;
using tcp::drain_cl;
using tcp::wait_cl;

constexpr int kCh = 128;     // channels per CTA
constexpr int kSlotK = 128;  // k per slot
constexpr int kWStage = kCh * kSlotK;
constexpr int kBoxRows = 32;                      // tokens per TMA box
constexpr int kSets = 2;                          // of A and of B warps
constexpr int kAWarp0 = 4, kBWarp0 = kAWarp0 + 4 * kSets, kEWarp0 = kBWarp0 + 4 * kSets;
constexpr uint32_t kACols = 256;  // first column of the weights' slots
constexpr uint32_t kSlotCols = kSlotK / 2;

// SLOTS: widened slots; WRING / TRING: stages of weights / tokens as bytes.
template <int CG_, int NT_, int SLOTS_, int WRING_, int TRING_, int EWARPS_>
struct Cfg {
    static constexpr int CG = CG_, NT = NT_, SLOTS = SLOTS_, WRING = WRING_, TRING = TRING_,
                         EWARPS = EWARPS_;
    static constexpr int NTC = NT / CG;              // tokens per CTA's half
    static constexpr int TSTAGE = NTC * kSlotK;
    static constexpr int BBOX = NTC * 128;           // 64 k of them, widened
    static constexpr int BSLOT = 2 * BBOX;
    static constexpr int ACCS = NT <= 128 ? 2 : 1;
    static constexpr int ECOLS = NT / (EWARPS / 4);  // tokens per epilogue warp
    static constexpr int THREADS = (kEWarp0 + EWARPS) * 32;
    // One accumulator: the epilogue holds the whole tile, packed to 16 bits,
    // in registers, so that the next tile's MMAs wait for reads of tensor
    // memory only, not for stores.  Registers move from the other roles to the
    // epilogue (kReg*, within the 72 per thread of the launch).
    static constexpr bool HOLD = ACCS == 1;
    static constexpr int STAGING = 32 * 32 * 2;      // per epilogue warp, 16-bit results
    static constexpr int NBAR = 2 * WRING + 2 * TRING + 2 * SLOTS + 2 * ACCS + 1;
    static constexpr int OFF_T = WRING * kWStage;
    static constexpr int OFF_B = OFF_T + TRING * TSTAGE;
    static constexpr int OFF_STAGE = OFF_B + SLOTS * BSLOT;
    static constexpr int OFF_SCALE = OFF_STAGE + EWARPS * STAGING;
    static constexpr int OFF_BAR = OFF_SCALE + EWARPS * ECOLS * 4;
    static constexpr int OFF_TABLE = OFF_BAR + NBAR * 8 + 16;
    static constexpr int SMEM = OFF_TABLE + (kMaxExperts + 1) * 4 + 1024;
    static_assert(NTC == 128, "eight token groups of 16 per converter thread");
    // A converter set waits at its own steps only, every other one, and a wait
    // on a phase's parity is sound only if the phase before has completed.
    // Step n's slot: the set saw the MMAs of step n - 2 - SLOTS done, so those
    // of n - 2 * SLOTS, the phase before, are.  Step n's stage of a ring of R:
    // with R even, step n - R was the set's own; else the slot's wait, taken
    // first, says that the MMAs of step n - SLOTS are done, so step n - R has
    // been loaded and used if R >= SLOTS.
    static_assert(kSets == 2 && SLOTS >= 2 && (WRING % 2 == 0 || WRING >= SLOTS) &&
                      (TRING % 2 == 0 || TRING >= SLOTS),
                  "no parity wait may be two phases ahead");
    static_assert(ACCS * NT <= static_cast<int>(kACols), "accumulator columns");
    static_assert(SLOTS * kSlotCols + kACols <= 512, "tensor-memory columns");
    static_assert(NT * kCh * 4 <= SLOTS * BSLOT || CG == 2, "partial sums fit the token slots");
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};
using Narrow = Cfg<1, 128, 3, 4, 3, 4>;
using Wide = Cfg<2, 256, 3, 3, 3, 8>;

// Registers per thread after a warpgroup's give or take (HOLD, below).
constexpr int kRegMisc = 56, kRegConv = 56, kRegEpi = 112;
template <int N>
__device__ __forceinline__ void give_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void take_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *m, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// Four bytes (8-bit integers) as four fp16 values.
__device__ __forceinline__ void widen4(uint32_t x, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = x ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140);
    uint32_t b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 ha = __hsub2(*reinterpret_cast<__half2 *>(&a), bias);
    __half2 hb = __hsub2(*reinterpret_cast<__half2 *>(&b), bias);
    lo = *reinterpret_cast<uint32_t *>(&ha);
    hi = *reinterpret_cast<uint32_t *>(&hb);
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z),
                 "r"(w)
                 : "memory");
}
// 16 consecutive columns of this warp's 32 tensor-memory lanes.
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
}
// Rows 0-15 (lane field of taddr) of 32 columns in the layout of an 8 x 8
// matrix's registers: v[4 * i + 2 * b + c] is row 8 b + lane / 4, column
// 8 i + 2 (lane % 4) + c.  Completion: tmem_wait_ld.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Two values rounded to 16 bits, the first in the low half.
template <class T>
__device__ __forceinline__ uint32_t pack2(float2 v)
{
    if constexpr (sizeof(T) == 4) {
        return 0u;  // fp32 results are never packed
    } else if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
// Both products at once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// Four 8 x 8 matrices of 16-bit values, each transposed into rows of 16
// bytes: lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void store_transposed(uint32_t addr, const uint32_t (&m)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                     addr),
                 "r"(m[0]), "r"(m[1]), "r"(m[2]), "r"(m[3])
                 : "memory");
}
// One slot's MMAs (kind::f16): d (+)= A[tensor memory] * B[shared memory]^T,
// eight steps of k = 16: A's columns a + 8 i; B's descriptors {b0 + 2 i, hi} in
// the slot's first box, {b1 + 2 i, hi} in its second.  In two parts: the tensor
// pipe's queue holds little more than the MMA in flight, so whatever the
// issuing thread has to work out for the next slot belongs between the parts,
// not after them.  The first MMA overwrites d unless acc.
template <int CG>
__device__ __forceinline__ void issue_first(uint32_t d, uint32_t a, uint32_t b0, uint32_t b1,
                                            uint32_t hi, uint32_t idesc, uint32_t acc)
{
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p0, p1;\n\t.reg .b64 b;\n\t.reg .b32 a, l;\n\t"
            "setp.ne.b32 p0, %5, 0;\n\tsetp.eq.b32 p1, %5, %5;\n\t"
            "add.u32 a, %1, 0;\n\tadd.u32 l, %2, 0;\n\tmov.b64 b, {l, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %4, p0;\n\t"
            "add.u32 a, %1, 8;\n\tadd.u32 l, %2, 2;\n\tmov.b64 b, {l, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %4, p1;\n\t"
            "add.u32 a, %1, 16;\n\tadd.u32 l, %2, 4;\n\tmov.b64 b, {l, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %4, p1;\n\t"
            "add.u32 a, %1, 24;\n\tadd.u32 l, %2, 6;\n\tmov.b64 b, {l, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %4, p1;\n\t"
            "add.u32 a, %1, 32;\n\tadd.u32 l, %6, 0;\n\tmov.b64 b, {l, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %4, p1;\n\t"
            "add.u32 a, %1, 40;\n\tadd.u32 l, %6, 2;\n\tmov.b64 b, {l, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %4, p1;\n\t"
            "}" ::"r"(d), "r"(a), "r"(b0), "r"(hi), "r"(idesc), "r"(acc), "r"(b1)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p0, p1;\n\t.reg .b64 b;\n\t.reg .b32 a, l;\n\t"
            "setp.ne.b32 p0, %5, 0;\n\tsetp.eq.b32 p1, %5, %5;\n\t"
            "add.u32 a, %1, 0;\n\tadd.u32 l, %2, 0;\n\tmov.b64 b, {l, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, p0;\n\t"
            "add.u32 a, %1, 8;\n\tadd.u32 l, %2, 2;\n\tmov.b64 b, {l, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, p1;\n\t"
            "add.u32 a, %1, 16;\n\tadd.u32 l, %2, 4;\n\tmov.b64 b, {l, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, p1;\n\t"
            "add.u32 a, %1, 24;\n\tadd.u32 l, %2, 6;\n\tmov.b64 b, {l, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, p1;\n\t"
            "add.u32 a, %1, 32;\n\tadd.u32 l, %6, 0;\n\tmov.b64 b, {l, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, p1;\n\t"
            "add.u32 a, %1, 40;\n\tadd.u32 l, %6, 2;\n\tmov.b64 b, {l, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, p1;\n\t"
            "}" ::"r"(d), "r"(a), "r"(b0), "r"(hi), "r"(idesc), "r"(acc), "r"(b1)
            : "memory");
}
// The last two, after a test, without blocking, of whether the barrier at
// shared address nbar (the next slot's) has completed the phase of parity
// npar; returns that.
template <int CG>
__device__ __forceinline__ uint32_t issue_last(uint32_t d, uint32_t a, uint32_t b1, uint32_t hi,
                                               uint32_t idesc, uint32_t nbar, uint32_t npar)
{
    uint32_t ready;
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred q, p1;\n\t.reg .b64 b;\n\t.reg .b32 a, l;\n\t"
            "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 q, [%6], %7;\n\t"
            "setp.eq.b32 p1, %5, %5;\n\t"
            "add.u32 a, %2, 48;\n\tadd.u32 l, %3, 4;\n\tmov.b64 b, {l, %4};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%1], [a], b, %5, p1;\n\t"
            "add.u32 a, %2, 56;\n\tadd.u32 l, %3, 6;\n\tmov.b64 b, {l, %4};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%1], [a], b, %5, p1;\n\t"
            "selp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(ready)
            : "r"(d), "r"(a), "r"(b1), "r"(hi), "r"(idesc), "r"(nbar), "r"(npar)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q, p1;\n\t.reg .b64 b;\n\t.reg .b32 a, l;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 q, [%6], %7;\n\t"
            "setp.eq.b32 p1, %5, %5;\n\t"
            "add.u32 a, %2, 48;\n\tadd.u32 l, %3, 4;\n\tmov.b64 b, {l, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%1], [a], b, %5, p1;\n\t"
            "add.u32 a, %2, 56;\n\tadd.u32 l, %3, 6;\n\tmov.b64 b, {l, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%1], [a], b, %5, p1;\n\t"
            "selp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(ready)
            : "r"(d), "r"(a), "r"(b1), "r"(hi), "r"(idesc), "r"(nbar), "r"(npar)
            : "memory");
    return ready;
}
template <int CG>
__device__ __forceinline__ void commit(uint64_t *bar)
{
    if constexpr (CG == 2)
        tcp::umma_commit_both(bar);
    else
        tc::umma_commit(bar);
}
// An arrive on the issuing CTA's barrier.
template <int CG>
__device__ __forceinline__ void arrive_issuer(uint64_t *bar)
{
    if constexpr (CG == 2)
        arrive_on(bar, 0);
    else
        mbar_arrive(bar);
}
// The sum of four floats at this CTA's shared address `addr` over the cluster's
// CTAs, in their order.
template <int CTAS>
__device__ __forceinline__ float4 cluster_sum(uint32_t addr)
{
    float4 v[CTAS];
#pragma unroll
    for (int r = 0; r < CTAS; ++r) {
        uint32_t a;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(r));
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                     : "r"(a)
                     : "memory");
    }
#pragma unroll
    for (int r = 1; r < CTAS; ++r) {
        v[0].x += v[r].x;
        v[0].y += v[r].y;
        v[0].z += v[r].z;
        v[0].w += v[r].w;
    }
    return v[0];
}

// Bounded waits on barriers that the CTA pair shares (wide) acquire at cluster
// scope; the narrow configuration's are its own, and acquire at CTA scope.
template <int CG>
__device__ __forceinline__ bool wait_pair(uint64_t *bar, uint32_t parity, const Abort &ab,
                                          unsigned int code, bool sleep = false)
{
    if constexpr (CG == 2)
        return wait_cl(bar, parity, ab, code, sleep);
    else
        return mbar_wait(bar, parity, ab, code, sleep);
}
template <int CG>
__device__ __forceinline__ bool warp_wait_pair(uint64_t *bar, uint32_t parity, const Abort &ab,
                                               unsigned int code)
{
    const bool ok = wait_pair<CG>(bar, parity, ab, code);
    return __all_sync(0xffffffffu, ok) != 0;
}

// Waits (bounded) for the last loads of a ring that stops early, so that none
// is in flight when the CTA exits.
template <int STAGES>
__device__ __forceinline__ void drain_ring(uint64_t *full, long long issued, const Abort &ab)
{
    Ring<STAGES> d;
    for (long long i = 0; i < issued; ++i) {
        if (i + STAGES >= issued) mbar_drain(&full[d.s], d.ph, ab.limit);
        d.next();
    }
}

// One output tile: tokens row0 .. row0 + n - 1 of expert e, channels from
// ch0 on (this CTA's 128); neff: the MMA's N.
struct Job {
    int e, n, neff, ch0;
    long long row0;
};

// Tile u of the table (first tile of each expert): within an expert, token
// tiles run fastest, so that CTAs at work together share weights in L2.
template <class C>
__device__ __forceinline__ Job job(const Args &a, const int *table, int u, uint32_t half)
{
    int lo = 0, hi = a.E;  // largest e with table[e] <= u
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (table[mid] <= u)
            lo = mid;
        else
            hi = mid;
    }
    int r0, r1;
    expert_rows(a, lo, r0, r1);
    const int mt = (r1 - r0 + C::NT - 1) / C::NT;
    const int v = u - table[lo];
    const int ct = v / mt, m = v - ct * mt;
    Job j;
    j.e = lo;
    j.row0 = r0 + static_cast<long long>(m) * C::NT;
    j.n = min(C::NT, static_cast<int>(r1 - j.row0));
    constexpr int STEP = 16 * C::CG;
    j.neff = (j.n + STEP - 1) / STEP * STEP;
    j.ch0 = (ct * C::CG + static_cast<int>(half)) * kCh;
    return j;
}

// tmW: the weights (K, N, E) in boxes of 128 k by 128 channels, tmT: the
// tokens (K, M) in boxes of 128 k by 32 rows, both in the 128-byte swizzle.
// (A box past an expert's last token holds the next expert's or, past the last
// expert, rows that are no one's -- at most 47, where a pair's second half of
// 16 tokens takes a box of 32: their columns of the result are not stored.)  split: CTAs of the cluster that share a tile's k (narrow only);
// then each cluster has one tile.  c_bytes: accesses that C's rows allow
// (16, 8 or fewer).
template <class C, class T>
__global__ void __launch_bounds__(C::THREADS, 1)
    i8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT,
              const Args a, int split, int c_bytes)
{
    constexpr int CG = C::CG;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + C::OFF_BAR);
    uint64_t *w_full = bars, *w_empty = w_full + C::WRING;
    uint64_t *t_full = w_empty + C::WRING, *t_empty = t_full + C::TRING;
    uint64_t *ready = t_empty + C::TRING;        // issuing CTA's: widened slots
    uint64_t *slot_empty = ready + C::SLOTS;     // per CTA: commits
    uint64_t *acc_full = slot_empty + C::SLOTS;  // per CTA: commits
    uint64_t *acc_empty = acc_full + C::ACCS;    // issuing CTA's: epilogues
    uint64_t *mma_done = acc_empty + C::ACCS;
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_base + 1);
    int *table = reinterpret_cast<int *>(base + C::OFF_TABLE);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    const uint32_t half = CG == 2 ? rank : 0u, krank = CG == 2 ? 0u : rank;
    const int cluster = CG == 2 ? 2 : split;
    const int cid = static_cast<int>(blockIdx.x) / cluster;
    const int ncl = static_cast<int>(gridDim.x) / cluster;
    const bool issuer = CG == 1 || rank == 0;
    const int k_slots = (a.K + kSlotK - 1) / kSlotK;
    const int ks_lo = static_cast<int>(static_cast<long long>(k_slots) * krank / split);
    const int ks_hi = static_cast<int>(static_cast<long long>(k_slots) * (krank + 1) / split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::WRING; ++s) {
            mbar_init(&w_full[s], 1u);
            mbar_init(&w_empty[s], 4u);
        }
        for (int s = 0; s < C::TRING; ++s) {
            mbar_init(&t_full[s], 1u);
            mbar_init(&t_empty[s], 4u);
        }
        for (int s = 0; s < C::SLOTS; ++s) {
            mbar_init(&ready[s], static_cast<uint32_t>(CG * (4 + 4)));
            mbar_init(&slot_empty[s], 1u);
        }
        for (int s = 0; s < C::ACCS; ++s) {
            mbar_init(&acc_full[s], 1u);
            mbar_init(&acc_empty[s], static_cast<uint32_t>(CG * C::EWARPS));
        }
        mbar_init(mma_done, 1u);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmT);
    }
    if (warp == 1) {
        if constexpr (CG == 2)
            tcp::tmem_alloc_pair(tmem_base, 512);
        else
            tc::tmem_alloc(tmem_base, 512);
    }
    // dense: the first tile's weights start on their way into L2 while the
    // kernel before (the quantiser, as a rule) runs; nothing is read yet
    dependent_release();
    if (a.offsets == nullptr && warp == 3 && lane == 0) {
        const int ch0 = (cid / ((a.M + C::NT - 1) / C::NT) * CG + static_cast<int>(half)) * kCh;
        for (int ks = ks_lo; ch0 < a.N && ks < ks_hi && ks < ks_lo + 16; ++ks)
            tma_prefetch_3d(&tmW, ks * kSlotK, ch0, 0);
    }
    dependent_wait();
    if (warp == 2) {  // the tile table
        // (cut at the most that ascending offsets have: what descending ones add
        // up to need not fit an int, and a cluster that shares k has one tile;
        // C bounds `most` and 32 experts' tiles far below 2^31)
        const int cts = (a.N + kCh * CG - 1) / (kCh * CG);
        const int most = static_cast<int>(max_tiles(a, C::NT) * cts);
        int sum = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            int lo = 0, hi = 0;
            if (e0 + lane < a.E) expert_rows(a, e0 + lane, lo, hi);
            const int n = (hi - lo + C::NT - 1) / C::NT * cts;
            int inc = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int x = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += x;
            }
            if (e0 + lane < a.E) table[e0 + lane] = min(sum + inc - n, most);
            sum = min(sum + __shfl_sync(0xffffffffu, inc, 31), most);
        }
        if (lane == 0) table[a.E] = sum;
    }
    tc::tc_fence_before();
    tcp::cluster_sync();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_base;
    const Abort ab{abort_flag, a.status, kWaitLimitCycles};
    const int tiles = table[a.E];
    float *part = reinterpret_cast<float *>(base + C::OFF_B);  // split: [token][channel]
    static_assert(!C::HOLD || (C::EWARPS == 8 && 4 * kRegMisc + 16 * kRegConv + 8 * kRegEpi <=
                                                     28 * 72 && kSets == 2),
                  "the register shares stay within the launch's");

    if (warp < kAWarp0) {
        if constexpr (C::HOLD) give_registers<kRegMisc>();
        if (warp == 0) {
            // ---------------------------------------------------- weights' producer
            if (lane == 0) {
                Ring<C::WRING> rr;
                long long issued = 0;
                bool ok = true;
                for (int u = cid; ok && u < tiles; u += ncl) {
                    const Job j = job<C>(a, table, u, half);
                    for (int ks = ks_lo; ks < ks_hi; ++ks) {
                        if (!mbar_wait(&w_empty[rr.s], rr.ph ^ 1u, ab, kStatusWaitEmpty)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&w_full[rr.s], kWStage);
                        tma_load_3d(base + rr.s * kWStage, &tmW, &w_full[rr.s], ks * kSlotK, j.ch0,
                                    j.e);
                        ++issued;
                        rr.next();
                    }
                }
                if (!ok || *abort_flag) drain_ring<C::WRING>(w_full, issued, ab);
            }
            __syncwarp();
        } else if (warp == 2) {
            // ---------------------------------------------------- tokens' producer
            if (lane == 0) {
                Ring<C::TRING> rr;
                long long issued = 0;
                bool ok = true;
                for (int u = cid; ok && u < tiles; u += ncl) {
                    const Job j = job<C>(a, table, u, half);
                    const int per = j.neff / CG, boxes = (per + kBoxRows - 1) / kBoxRows;
                    const int first = static_cast<int>(j.row0) + static_cast<int>(half) * per;
                    for (int ks = ks_lo; ks < ks_hi; ++ks) {
                        if (!mbar_wait(&t_empty[rr.s], rr.ph ^ 1u, ab, kStatusWaitEmpty)) {
                            ok = false;
                            break;
                        }
                        uint8_t *dst = base + C::OFF_T + rr.s * C::TSTAGE;
                        mbar_arrive_expect_tx(&t_full[rr.s],
                                              static_cast<uint32_t>(boxes * kBoxRows * kSlotK));
                        for (int x = 0; x < boxes; ++x)
                            tma_load_3d(dst + x * kBoxRows * kSlotK, &tmT, &t_full[rr.s], ks * kSlotK,
                                        first + x * kBoxRows, 0);
                        ++issued;
                        rr.next();
                    }
                }
                if (!ok || *abort_flag) drain_ring<C::TRING>(t_full, issued, ab);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ---------------------------------------------------- MMA issuer
            if (issuer && lane == 0) {
                Ring<C::SLOTS> sr;
                Ring<C::ACCS> acc;
                bool ok = true, any = false;
                const uint64_t bdesc = tc::kmajor_sw128_desc(smem_u32(base + C::OFF_B));
                const uint32_t blo = static_cast<uint32_t>(bdesc),
                               bhi = static_cast<uint32_t>(bdesc >> 32);
                for (int u = cid; ok && u < tiles; u += ncl) {
                    const Job j = job<C>(a, table, u, half);
                    const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(j.neff >> 3) << 17) |
                                           (static_cast<uint32_t>((kCh * CG) >> 4) << 24);
                    if (!wait_pair<CG>(&acc_empty[acc.s], acc.ph ^ 1u, ab, kStatusWaitAcc)) break;
                    tc::tc_fence_after();
                    const uint32_t d = tmem + static_cast<uint32_t>(acc.s * C::NT);
                    uint32_t seen = 0;  // this slot is already known to be ready
                    for (int ks = ks_lo; ks < ks_hi; ++ks) {
                        if (!seen && !wait_pair<CG>(&ready[sr.s], sr.ph, ab, kStatusWaitConv)) {
                            ok = false;
                            break;
                        }
                        tc::tc_fence_after();
                        const uint32_t at = tmem + kACols + static_cast<uint32_t>(sr.s) * kSlotCols;
                        const uint32_t b0 =
                            blo + static_cast<uint32_t>(sr.s) * (C::BSLOT >> 4);
                        issue_first<CG>(d, at, b0, b0 + (C::BBOX >> 4), bhi, idesc,
                                        ks > ks_lo ? 1u : 0u);
                        Ring<C::SLOTS> nx = sr;
                        nx.next();
                        seen = issue_last<CG>(d, at, b0 + (C::BBOX >> 4), bhi, idesc,
                                              smem_u32(&ready[nx.s]), nx.ph);
                        if (ks + 1 == ks_hi) seen = 0;
                        any = true;
                        commit<CG>(&slot_empty[sr.s]);
                        sr = nx;
                    }
                    if (!ok) break;
                    commit<CG>(&acc_full[acc.s]);
                    acc.next();
                }
                if (any) {
                    commit<CG>(mma_done);
                    drain_cl(mma_done, 0, ab.limit);
                }
            }
            __syncwarp();
        }
    } else if (warp < kBWarp0) {
        if constexpr (C::HOLD) give_registers<kRegConv>();
        // ---------------------------------------------------- weights: widen into tensor memory
        const int row = (warp & 3) * 32 + lane;
        const uint32_t tl = tmem + kACols + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t src0 = smem_u32(base) + row * 128 + ((row & 7) << 4);
        int turn = (warp - kAWarp0) >> 2;  // 0: this set's slot
        Ring<C::WRING> rr;
        Ring<C::SLOTS> sr;
        bool ok = true;
        for (int u = cid; ok && u < tiles; u += ncl) {
            for (int ks = ks_lo; ks < ks_hi; ++ks) {
                if (turn == 0) {
                    turn = kSets;
                    // the slot before the load (Cfg: the order matters)
                    if (!warp_wait_pair<CG>(&slot_empty[sr.s], sr.ph ^ 1u, ab, kStatusWaitMma) ||
                        !warp_wait(&w_full[rr.s], rr.ph, ab, kStatusWaitFull, lane)) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    const uint32_t src = src0 + static_cast<uint32_t>(rr.s * kWStage);
                    const uint32_t dst = tl + static_cast<uint32_t>(sr.s) * kSlotCols;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t x[16], y[16];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint4 v = lds128(src ^ static_cast<uint32_t>((4 * h + c) << 4));
                            widen4(v.x, x[4 * c], x[4 * c + 1]);
                            widen4(v.y, x[4 * c + 2], x[4 * c + 3]);
                            widen4(v.z, y[4 * c], y[4 * c + 1]);
                            widen4(v.w, y[4 * c + 2], y[4 * c + 3]);
                        }
                        tmem_put16(dst + 16 * h, x);
                        tmem_put16(dst + 32 + 16 * h, y);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&w_empty[rr.s]);
                    tc::tmem_wait_st();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_issuer<CG>(&ready[sr.s]);
                }
                --turn;
                rr.next();
                sr.next();
            }
        }
    } else if (warp < kEWarp0) {
        if constexpr (C::HOLD) give_registers<kRegConv>();
        // ---------------------------------------------------- tokens: widen into shared memory
        const int t = static_cast<int>(threadIdx.x) & 127;
        int turn = (warp - kBWarp0) >> 2;
        Ring<C::TRING> rr;
        Ring<C::SLOTS> sr;
        bool ok = true;
        for (int u = cid; ok && u < tiles; u += ncl) {
            const Job j = job<C>(a, table, u, half);
            const int groups = j.neff / CG / 16;  // this CTA's tokens, 16 at a time
            for (int ks = ks_lo; ks < ks_hi; ++ks) {
                if (turn == 0) {
                    turn = kSets;
                    // the slot before the load (Cfg: the order matters)
                    if (!warp_wait_pair<CG>(&slot_empty[sr.s], sr.ph ^ 1u, ab, kStatusWaitMma) ||
                        !warp_wait(&t_full[rr.s], rr.ph, ab, kStatusWaitFull, lane)) {
                        ok = false;
                        break;
                    }
                    const uint32_t src =
                        smem_u32(base + C::OFF_T + rr.s * C::TSTAGE) + 16u * static_cast<uint32_t>(t);
                    const uint32_t dst =
                        smem_u32(base + C::OFF_B + sr.s * C::BSLOT) + 16u * static_cast<uint32_t>(t);
#pragma unroll
                    for (int g = 0; g < 8; g += 4) {
                        if (g >= groups) break;
                        uint4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (g + i < groups) v[i] = lds128(src + (g + i) * 2048);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (g + i < groups) {
                                uint32_t w[8];
                                widen4(v[i].x, w[0], w[1]);
                                widen4(v[i].y, w[2], w[3]);
                                widen4(v[i].z, w[4], w[5]);
                                widen4(v[i].w, w[6], w[7]);
                                sts128(dst + (g + i) * 2048, w[0], w[1], w[2], w[3]);
                                sts128(dst + (g + i) * 2048 + C::BBOX, w[4], w[5], w[6], w[7]);
                            }
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&t_empty[rr.s]);
                        arrive_issuer<CG>(&ready[sr.s]);
                    }
                }
                --turn;
                rr.next();
                sr.next();
            }
        }
    } else {
        if constexpr (C::HOLD) take_registers<kRegEpi>();
        // ---------------------------------------------------- epilogue
        // Lanes of tensor memory are channels, columns tokens; C wants a
        // token's channels side by side.  fp32: 32 lanes store 128 bytes of a
        // token's row as they are.  16 bits: chunks of 32 x 32 go through a
        // transposing matrix store into 64-byte token rows (16-byte pieces
        // XORed with token / 2 against bank conflicts) and out in 16-byte
        // pieces.
        const int q = warp & 3, w = warp - kEWarp0;
        const int col0 = (w >> 2) * C::ECOLS;  // this warp's first token of the tile
        const uint32_t stage = smem_u32(base + C::OFF_STAGE + w * C::STAGING);
        const uint32_t st_row = stage + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
        float *sa = reinterpret_cast<float *>(base + C::OFF_SCALE) + w * C::ECOLS;
        Ring<C::ACCS> acc;
        constexpr bool PACK = sizeof(T) == 2;
        // Narrow: a tile's place and scales are asked for before the stores of
        // the tile before, since the waits for them would open every tile
        // (19000 x 1088 x 128 29 us; so 25).  Wide holds a tile's results in the
        // registers that would take (8192 x 8192 x 4096 316 us, with it 321).
        constexpr bool AHEAD = !C::HOLD;
        constexpr int NSA = C::ECOLS / 32;
        float nsa[NSA], nsb[4] = {};  // 16 bits: channels lane / 4 + 8 i; else channel lane
        Job nj{};
        auto ask_next = [&](int u) {
            if (u >= tiles) return;
            const Job j = nj = job<C>(a, table, u, half);
            if (split > 1) return;
            const int chq = j.ch0 + q * 32, n = j.n - col0;
            const float *sp = a.scaleB + static_cast<long long>(j.e) * a.N + chq;
#pragma unroll
            for (int i = 0; i < NSA; ++i)
                nsa[i] = lane + 32 * i < n ? a.scaleA[j.row0 + col0 + lane + 32 * i] : 0.f;
#pragma unroll
            for (int i = 0; i < (PACK ? 4 : 1); ++i) {
                const int c = PACK ? 8 * i + (lane >> 2) : lane;
                nsb[i] = chq + c < a.N ? sp[c] : 0.f;
            }
        };
        if (AHEAD) ask_next(cid);
        for (int u = cid; u < tiles; u += ncl) {
            const Job j = AHEAD ? nj : job<C>(a, table, u, half);
            const int chq = j.ch0 + q * 32;        // this warp's first channel
            const int n = min(j.n - col0, C::ECOLS);
            float sb[4] = {};
            if (AHEAD && split == 1) {
#pragma unroll
                for (int i = 0; i < NSA; ++i) sa[lane + 32 * i] = nsa[i];
#pragma unroll
                for (int i = 0; i < 4; ++i) sb[i] = nsb[i];
                __syncwarp();
            } else if (split == 1) {
                const float *sp = a.scaleB + static_cast<long long>(j.e) * a.N;
                for (int i = lane; i < C::ECOLS; i += 32)
                    sa[i] = i < n ? a.scaleA[j.row0 + col0 + i] : 0.f;
                if (PACK) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (chq + 8 * i + (lane >> 2) < a.N) sb[i] = sp[chq + 8 * i + (lane >> 2)];
                } else if (chq + lane < a.N) {
                    sb[0] = sp[chq + lane];
                }
                __syncwarp();
            }
            int got = 1;
            if (lane == 0) got = wait_pair<CG>(&acc_full[acc.s], acc.ph, ab, kStatusWaitAcc, true);
            if (!__shfl_sync(0xffffffffu, got, 0)) break;
            if constexpr (CG == 2)  // (every lane acquires)
                drain_cl(&acc_full[acc.s], acc.ph, ab.limit);
            else
                mbar_drain(&acc_full[acc.s], acc.ph, ab.limit);
            tc::tc_fence_after();
            const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) +
                                static_cast<uint32_t>(acc.s * C::NT + col0);
            T *crow = static_cast<T *>(a.C) + (j.row0 + col0) * a.ldc + chq;
            // a chunk of 32 tokens, scaled and packed: m[4 t + i] is channels
            // 8 i + lane / 4, tokens 8 t + 2 (lane % 4), + 1
            auto pack_chunk = [&](int c0, uint32_t (&m)[16]) {
                uint32_t v[2][16];
                tmem_ld_16x32(tb + c0, v[0]);
                tmem_ld_16x32(tb + (16u << 16) + c0, v[1]);
                tmem_wait_ld();
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float2 s =
                        *reinterpret_cast<const float2 *>(sa + c0 + 8 * t + 2 * (lane & 3));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        m[4 * t + i] = pack2<T>(
                            mul2(mul2(make_float2(
                                          __uint_as_float(v[i >> 1][4 * t + 2 * (i & 1)]),
                                          __uint_as_float(v[i >> 1][4 * t + 2 * (i & 1) + 1])),
                                      s),
                                 make_float2(sb[i], sb[i])));
                }
            };
            auto store_chunk = [&](int c0, const uint32_t (&m)[16]) {
                __syncwarp();  // the staging's last readers are done
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t x[4] = {m[4 * t], m[4 * t + 1], m[4 * t + 2], m[4 * t + 3]};
                    store_transposed(st_row + t * 512, x);
                }
                __syncwarp();
                T *out = crow + static_cast<long long>(c0) * a.ldc;
                // (addresses by additions: computed for each row they cost more
                // than the stores)
                const int rows_left = n - c0;
                if (c_bytes == 16 && chq + 32 <= a.N) {
                    const int r = lane >> 2, p = lane & 3;
                    const uint32_t at = stage + r * 64 + ((p ^ ((r >> 1) & 3)) << 4);
                    T *to = out + r * a.ldc + 8 * p;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 x = lds128(at + i * 512);
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
                    // lane, a token's row at a time; addresses by additions, eight
                    // rows' loads together (a computed address per row made a
                    // chunk 2000 clocks)
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
            };
            if (PACK && C::HOLD) {
                constexpr int NCH = PACK && C::HOLD ? C::ECOLS / 32 : 1;
                uint32_t m[NCH][16];
#pragma unroll
                for (int c = 0; c < NCH; ++c)
                    if (32 * c < n) pack_chunk(32 * c, m[c]);
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_issuer<CG>(&acc_empty[acc.s]);
#pragma unroll
                for (int c = 0; c < NCH; ++c)
                    if (32 * c < n) store_chunk(32 * c, m[c]);
                acc.next();
                continue;
            }
            if (AHEAD) ask_next(u + ncl);
#pragma unroll 1
            for (int c0 = 0; c0 < n; c0 += 32) {
                if (PACK && split == 1) {
                    uint32_t m[16];
                    pack_chunk(c0, m);
                    store_chunk(c0, m);
                    continue;
                }
                float v[32];
                tc::tmem_ld32(tb + c0, v);
                if (split > 1) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        part[(col0 + c0 + i) * kCh + q * 32 + lane] = v[i];
                } else if (chq + lane < a.N) {
                    T *row = crow + static_cast<long long>(c0) * a.ldc + lane;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (c0 + i < n) *row = rows::from_f<T>(v[i] * sa[c0 + i] * sb[0]);
                        row += a.ldc;
                    }
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_issuer<CG>(&acc_empty[acc.s]);
            acc.next();
        }
    }

    if (CG == 1 && split > 1) {
        // ---- partial sums of the cluster's CTAs, added in CTA order; CTA r
        // takes tokens r, r + split, ...: a warp a token, four channels a lane.
        // The scales, and then every CTA's part, are asked for together.
        __syncwarp();
        const bool some = cid < tiles;
        Job j{};
        float sb[4] = {}, sc = 0.f;
        const int t0 = static_cast<int>(krank) + warp * split;
        if (some) {
            j = job<C>(a, table, cid, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (j.ch0 + 4 * lane + i < a.N)
                    sb[i] = a.scaleB[static_cast<long long>(j.e) * a.N + j.ch0 + 4 * lane + i];
            if (t0 < j.n) sc = a.scaleA[j.row0 + t0];
        }
        tcp::cluster_sync();
        if (some && *abort_flag == 0) {
            const int ch = j.ch0 + 4 * lane;
            for (int t = t0; t < j.n; t += split * (C::THREADS / 32)) {
                const uint32_t at = smem_u32(part + t * kCh + 4 * lane);
                const float4 s = split == 8 ? cluster_sum<8>(at)
                                            : split == 4 ? cluster_sum<4>(at) : cluster_sum<2>(at);
                if (t != t0) sc = a.scaleA[j.row0 + t];
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
    tcp::cluster_sync();
    if (warp == 1) {
        tc::tc_fence_after();
        if constexpr (CG == 2)
            tcp::tmem_dealloc_pair(tmem, 512);
        else
            tc::tmem_dealloc(tmem, 512);
    }
}

// Enqueues the kernel on `clusters` clusters of CG (or split) CTAs.
template <class C, class T>
int launch_tc_i8(const Args &a, const CUtensorMap &tmW, const CUtensorMap &tmT, long long clusters,
                 int split, int c_bytes, cudaStream_t st)
{
    auto kern = i8_kernel<C, T>;
    if (!smem_attr_once(reinterpret_cast<const void *>(kern), C::SMEM)) return SGEMM_ERR_LAUNCH;
    const unsigned size = C::CG == 2 ? 2u : static_cast<unsigned>(split);
    return launch_dependent(kern, dim3(static_cast<unsigned>(clusters) * size), dim3(C::THREADS),
                            C::SMEM, size, st, tmW, tmT, a, split, c_bytes);
}

}  // namespace i8
}  // namespace sg

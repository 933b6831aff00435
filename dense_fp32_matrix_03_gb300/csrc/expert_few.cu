// expert_few.cu -- a whole expert layer for a few tokens in two kernels
// (include/expert_layer.h):
//   up    h[t,j] = silu(x G_e^T) * (x U_e^T), in units of a chosen expert and 16
//         of its rows of G and of U
//   down  out[t] = sum_e w D_e h[t,e], a block for 16 channels of out and ALL
//         chosen experts, so that nothing is added across blocks
// Both find the chosen experts and their tokens from the ids themselves (at
// most 512): no sort, no rows in expert order, no counts on the host.
//
// What counts is to read the chosen experts' weights once.  The products run
// on the matrix units (mma.sync m16n8k16, fp32 sums), the weights its 16 rows,
// the tokens its 8 columns; 8-bit weights are widened in registers, exactly, to
// the row type.  Lane (g, t) = (lane / 4, lane % 4) holds rows g and g + 8 of
// the weights and token g; which k it holds is ours to choose as long as both
// operands agree, so a lane takes 16 consecutive bytes of a weight row at a
// time and the same k of the token: every load is 16 bytes, a quad reads 64
// bytes of a row together.  The weights come by asynchronous copies into a ring
// that each lane fills and reads for itself, so that many are on their way
// without registers or barriers.
//
// Measured on GB300, both kernels: one token, 4 of 32 experts of 2048 x 2048, 8 bits
// (fp16 rows) 18.8 us (their 50 MB take 7.4), 16 bits 24.6; 16 tokens, 4 of 32 experts of
// 2048 x 1024 (21 of them chosen), 16 bits 63 (4.2 TB/s), 8 bits 53; 32 tokens, 4 of 64
// (40 chosen), 16 bits 114, 8 bits 94; 64 tokens, 2 of 8 of 4096 x 2048, 16 bits 249,
// 8 bits 152.  Few tokens are bound by latency: ids, weights and sums in sequence,
// twice; more by the loads in flight, those of the tokens among them, and, in 8 bits,
// by widening: both recur for each eight tokens of an expert (down: four, in two
// columns each).
#include <type_traits>

#include "../../include/expert_layer.h"
#include "common.cuh"
#include "dependent.cuh"
#include "rows.cuh"

namespace sg {
namespace few {

constexpr int kMaxRows = 512;   // T * k
constexpr int kMaxTokens = 64;  // T
constexpr int kMaxSide = 65536; // H, F
constexpr int kCh = 16;         // channels of a fragment

struct Args {
    int T, k, E, H, F;
    const void *x;
    long long ldx;
    const int *ids;
    const float *weights;
    const void *W1, *W2;  // addresses in bytes from here on: pitches, strides
    long long p1, stride1, p2, stride2;
    const float *scale1, *scale2;
    void *out;
    long long ldo;
    void *h;       // T * k pairs of rows of ldh values: h rounded, and what that left, kRestUp times
    long long ldh;
};

// What h's rounding to T leaves is kept times this.  In fp16 the rest of an h near
// 2^-14 would be below the least number; 2^11 times it is at most h itself.
template <class T>
constexpr float kRestUp = std::is_same<T, __half>::value ? 2048.f : 1.f;

// The chosen experts in ascending order and, for each, its tokens in ascending
// order.  A token that chose an expert more than once is one row, whose weight
// is the sum.
struct Choices {
    int ids[kMaxRows];
    float w[kMaxRows];
    unsigned map[kMaxExperts / 32];  // chosen experts
    short first[kMaxRows + 1];       // first row of used expert u
    short expert[kMaxRows];          // its id
    short token[kMaxRows];           // of a row
    short choice[kMaxRows];          // t * k + the first j
    float weight[kMaxRows];
    int used;
};

// Fills `c` (all threads of the block call; WARPS: of them).  The loads pass L1
// by: the down kernel may be here while blocks of the up kernel still run.
template <int WARPS>
__device__ __forceinline__ void find_choices(const Args &a, Choices &c)
{
    const int S = a.T * a.k, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (S <= 32) {  // one warp, a lane a choice
        if (warp == 0) {
            constexpr unsigned all = 0xffffffffu;
            int e = -1;
            float w = 1.f;
            if (lane < S) {
                e = __ldcg(a.ids + lane);
                if (a.weights != nullptr) w = __ldcg(a.weights + lane);
            }
            const bool kept = e >= 0 && e < a.E;
            const unsigned none = 0x80000000u | lane;  // like no other lane's
            const int t = lane / a.k;
            const unsigned same = __match_any_sync(all, kept ? static_cast<unsigned>(t << 16 | e) : none);
            const bool row = kept && __ffs(same) - 1 == lane;
            float sum = w;
            if (__any_sync(all, kept && (same & (same - 1u)) != 0u)) {
                sum = 0.f;
                for (int o = 0; o < S; ++o) {
                    const float v = __shfl_sync(all, w, o);
                    if (same >> o & 1u) sum += v;
                }
            }
            const unsigned of_e = __match_any_sync(all, row ? static_cast<unsigned>(e) : none);
            const bool begins = row && __ffs(of_e) - 1 == lane;
            const unsigned rows_ = __ballot_sync(all, row), starts = __ballot_sync(all, begins);
            int pos = 0, u = 0;
            for (unsigned m = rows_; m != 0u; m &= m - 1u) {
                const int o = __ffs(m) - 1, eo = __shfl_sync(all, e, o);
                pos += eo < e || (eo == e && o < lane);
                u += eo < e && (starts >> o & 1u);
            }
            if (row) {
                c.token[pos] = static_cast<short>(t);
                c.choice[pos] = static_cast<short>(lane);
                c.weight[pos] = sum;
            }
            if (begins) {
                c.expert[u] = static_cast<short>(e);
                c.first[u] = static_cast<short>(pos);
            }
            if (lane == 0) {
                c.used = __popc(starts);
                c.first[__popc(starts)] = static_cast<short>(__popc(rows_));
            }
        }
        __syncthreads();
        return;
    }
    if (tid < kMaxExperts / 32) c.map[tid] = 0u;
    __syncthreads();
    for (int s = tid; s < S; s += WARPS * 32) {
        const int e = __ldcg(a.ids + s);
        const bool kept = e >= 0 && e < a.E;
        c.ids[s] = kept ? e : -1;
        c.w[s] = a.weights != nullptr ? __ldcg(a.weights + s) : 1.f;
        if (kept) atomicOr(&c.map[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    // lane l: the experts of word l, and how many there are before them
    unsigned word = c.map[lane];
    const int mine = __popc(word);
    int before = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += o;
    }
    const int used = __shfl_sync(0xffffffffu, before, 31);
    before -= mine;
    if (warp == 0) {
        if (lane == 0) c.used = used;
        while (word != 0u) {
            c.expert[before++] = static_cast<short>(lane * 32 + __ffs(word) - 1);
            word &= word - 1u;
        }
    }
    __syncthreads();
    // this token's first choice of expert e, or -1
    auto choice_of = [&](int t, int e) {
        if (t < a.T)
            for (int j = 0; j < a.k; ++j)
                if (c.ids[t * a.k + j] == e) return t * a.k + j;
        return -1;
    };
    // a warp an expert, a lane a token: count the rows, then place them
    for (int u = warp; u < used; u += WARPS) {
        const int e = c.expert[u];
        int n = 0;
        for (int t0 = 0; t0 < a.T; t0 += 32)
            n += __popc(__ballot_sync(0xffffffffu, choice_of(t0 + lane, e) >= 0));
        if (lane == 0) c.first[u + 1] = static_cast<short>(n);
    }
    if (tid == 0) c.first[0] = 0;
    __syncthreads();
    if (warp == 0) {  // counts to first rows
        int sum = 0;
        for (int u0 = 0; u0 < used; u0 += 32) {
            int n = u0 + lane < used ? c.first[u0 + lane + 1] : 0;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(0xffffffffu, n, d);
                if (lane >= d) n += o;
            }
            if (u0 + lane < used) c.first[u0 + lane + 1] = static_cast<short>(sum + n);
            sum += __shfl_sync(0xffffffffu, n, 31);
        }
    }
    __syncthreads();
    for (int u = warp; u < used; u += WARPS) {
        const int e = c.expert[u];
        int at = c.first[u];
        for (int t0 = 0; t0 < a.T; t0 += 32) {
            const int t = t0 + lane, s = choice_of(t, e);
            const unsigned has = __ballot_sync(0xffffffffu, s >= 0);
            if (s >= 0) {
                float sum = 0.f;
                for (int j = s; j < (t + 1) * a.k; ++j)
                    if (c.ids[j] == e) sum += c.w[j];
                const int p = at + __popc(has & ((1u << lane) - 1u));
                c.token[p] = static_cast<short>(t);
                c.choice[p] = static_cast<short>(s);
                c.weight[p] = sum;
            }
            at += __popc(has);
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------- the operands

// Four 8-bit integers as four values of T: pairs lo, hi.
template <class T>
__device__ __forceinline__ void widen4(uint32_t x, uint32_t &lo, uint32_t &hi)
{
    if constexpr (std::is_same<T, __half>::value) {
        // x ^ 0x80 = x + 128 as an unsigned byte u; 0x64uu is fp16's 1024 + u
        const uint32_t u = x ^ 0x80808080u;
        const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140);
        const uint32_t b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 ha = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias);
        const __half2 hb = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
        lo = *reinterpret_cast<const uint32_t *>(&ha);
        hi = *reinterpret_cast<const uint32_t *>(&hb);
    } else {
        // 0x43uu is bf16's 128 + u below u = 128 and 2 u from there on: less 256, that
        // is x where x is negative and 2 x where it is not, from which max(0, x) is
        // taken.  (Every step is exact.  Logic on the bits instead, which runs at half
        // the rate of packed arithmetic: 128 + low seven bits, plus -128 or -256.)
        const uint32_t u = x ^ 0x80808080u;
        const __nv_bfloat162 half = __float2bfloat162_rn(0.5f), minus = __float2bfloat162_rn(-1.f);
        auto pair = [&](uint32_t w) {
            const __nv_bfloat162 f = *reinterpret_cast<const __nv_bfloat162 *>(&w);
            const __nv_bfloat162 r = __hadd2(f, __float2bfloat162_rn(-256.f));
            const __nv_bfloat162 p = __hfma2_relu(f, half, __float2bfloat162_rn(-128.f));
            const __nv_bfloat162 s = __hfma2(p, minus, r);
            return *reinterpret_cast<const uint32_t *>(&s);
        };
        lo = pair(__byte_perm(u, 0x43434343u, 0x4140));
        hi = pair(__byte_perm(u, 0x43434343u, 0x4342));
    }
}

// d (+)= the 16 x 16 weights times 16 x 8 tokens.
template <class T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<T, __half>::value)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight 16-bit values of a row from value k on, one by one; zeros past K, nothing
// past K is read.  (A call of its own: inlined, its comparisons are made at every
// whole step as well.)
__device__ __noinline__ uint4 load_token(const char *row, int k, int K)
{
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K)
            w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[k + i])
                        << (16 * (i % 2));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// What differs between 8-bit weights and weights of the row type T: the values
// in 16 bytes.
template <class T, bool I8>
struct Weights {
    static constexpr int ES = I8 ? 1 : 2;
    static constexpr int N = 16 / ES;         // values of a lane's piece
    static constexpr int TOK = N / 8;         // 16-byte pieces of a token's values
    static constexpr int STEP = 8 * N;        // k of a warp's step: two pieces a lane
    // pairs of T from a piece
    static __device__ __forceinline__ void pairs(const uint4 &v, uint32_t (&p)[N / 2])
    {
        if constexpr (I8) {
            widen4<T>(v.x, p[0], p[1]);
            widen4<T>(v.y, p[2], p[3]);
            widen4<T>(v.z, p[4], p[5]);
            widen4<T>(v.w, p[6], p[7]);
        } else {
            p[0] = v.x;
            p[1] = v.y;
            p[2] = v.z;
            p[3] = v.w;
        }
    }
};

// The lane's ring of weight pieces: DEPTH steps of 2 CF rows (g and g + 8 of each
// fragment) times two pieces of 16 bytes.
template <class T, bool I8, int CF, int DEPTH>
struct Pieces {
    using W = Weights<T, I8>;
    static constexpr int PER = 4 * CF;                       // pieces a step
    static constexpr int BYTES = DEPTH * PER * 32 * 16;      // a warp's ring
    uint32_t base;  // of this lane
    int t;
    __device__ __forceinline__ Pieces(void *smem, int warp, int lane)
        : base(smem_u32(smem) + static_cast<uint32_t>(warp * BYTES + lane * 16)), t(lane & 3)
    {
    }
    // Copies the step from k0 on of the rows, given from this lane's first piece
    // on; zeros past K, nothing past K is read.
    __device__ __forceinline__ void ask(int slot, const char *const (&row)[CF][2], int k0, int K)
    {
        const uint32_t to = base + static_cast<uint32_t>(slot * PER * 512);
        if (k0 + W::STEP <= K) {
#pragma unroll
            for (int c = 0; c < CF; ++c)
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        cp_async_16(to + static_cast<uint32_t>(((c * 2 + r) * 2 + i) * 512),
                                    row[c][r] + k0 * W::ES + 64 * i, 16u);
        } else {
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const int left = min(max((K - k0 - W::N * t - 4 * W::N * i) * W::ES, 0), 16);
#pragma unroll
                for (int c = 0; c < CF; ++c)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        cp_async_16(to + static_cast<uint32_t>(((c * 2 + r) * 2 + i) * 512),
                                    left > 0 ? row[c][r] + k0 * W::ES + 64 * i
                                             : row[c][r] - W::N * W::ES * t,
                                    static_cast<uint32_t>(left));
            }
        }
    }
    static __device__ __forceinline__ void commit()
    {
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // All but the last DEPTH - 1 committed steps have arrived.
    static __device__ __forceinline__ void arrived()
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    }
    __device__ __forceinline__ void take(int slot, uint4 (&w)[CF][2][2]) const
    {
#pragma unroll
        for (int c = 0; c < CF; ++c)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint4 &v = w[c][r][i];
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(base + static_cast<uint32_t>(
                                                  (slot * PER + (c * 2 + r) * 2 + i) * 512))
                                 : "memory");
                }
    }
};

// A token's values for the step from k0 on: row from lane t's first value on.
template <class T, bool I8, bool XV>
__device__ __forceinline__ void load_step(uint4 (&x)[2][Weights<T, I8>::TOK], const char *row,
                                          int k0, int K, int t)
{
    using W = Weights<T, I8>;
    const bool whole = XV && k0 + W::STEP <= K;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < W::TOK; ++j) {
            const int k = k0 + 4 * W::N * i + 8 * j;
            if (whole)
                x[i][j] = *reinterpret_cast<const uint4 *>(row + 2 * k);
            else
                x[i][j] = load_token(row, k, K - W::N * t);
        }
}

// acc += weights * tokens over the step from k0 on: CF fragments of weights, the
// groups of eight tokens that there are, the first one's values in x.
template <class T, bool I8, int CF, int NF, bool XV>
__device__ __forceinline__ void multiply(float (&acc)[CF][NF][4], const uint4 (&w)[CF][2][2],
                                         uint4 (&x)[2][Weights<T, I8>::TOK],
                                         const char *const (&trow)[NF], int k0, int K, int t,
                                         int tokens)
{
    using W = Weights<T, I8>;
#pragma unroll
    for (int n = 0; n < NF; ++n) {
        if (n > 0) {
            if (8 * n >= tokens) break;
            load_step<T, I8, XV>(x, trow[n], k0, K, t);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < CF; ++c) {
                uint32_t lo[W::N / 2], hi[W::N / 2];
                W::pairs(w[c][0][i], lo);
                W::pairs(w[c][1][i], hi);
#pragma unroll
                for (int j = 0; j < W::N / 4; ++j) {
                    const uint4 &v = x[i][j / 2];
                    mma<T>(acc[c][n], lo[2 * j], hi[2 * j], lo[2 * j + 1], hi[2 * j + 1],
                           j % 2 ? v.z : v.x, j % 2 ? v.w : v.y);
                }
            }
    }
}

// ---------------------------------------------------------------------- up

// Two steps of 4 KB a warp on their way (three leave room for one block of eight
// warps: one token 20.0 us instead of 18.8).
constexpr int kUpWarps = 8, kUpDepth = 2;
template <class T, bool I8, int NF>
struct Up {
    using P = Pieces<T, I8, 2, kUpDepth>;
    static constexpr int TK = 8 * NF, RING = kUpWarps * P::BYTES;
    static constexpr int SMEM = RING + kUpWarps * TK * (2 * kCh + 4) * 4;
    // Blocks of a multiprocessor: one where the sums and the widened weights do not fit
    // in half the registers (8 bits, 17 to 32 tokens: 94 us against 116 with two, which
    // spill, for 32 tokens, 4 of 64 experts of 2048 x 1024).
    static constexpr int BLOCKS = NF <= (I8 ? 2 : 4) ? 2 : 1;
};

// A unit is 16 rows of G and of U of one used expert; a block takes every
// gridDim.x-th.  The warps share a unit's steps of k, and the next unit's weights
// are on their way before this one's sums meet in shared memory, in the warps'
// order.
template <class T, bool I8, int NF, bool XV>
__global__ void __launch_bounds__(kUpWarps * 32, Up<T, I8, NF>::BLOCKS) up_kernel(const Args a)
{
    using W = Weights<T, I8>;
    using U = Up<T, I8, NF>;
    using P = typename U::P;
    __shared__ Choices c;
    extern __shared__ __align__(16) unsigned char dyn[];  // the rings, then the sums
    float(*part)[U::TK][2 * kCh + 4] =
        reinterpret_cast<float(*)[U::TK][2 * kCh + 4]>(dyn + U::RING);
    dependent_wait();
    dependent_release();  // (after the wait: the next kernel reads ids and weights early)
    find_choices<kUpWarps>(a, c);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int slices = (a.F + kCh - 1) / kCh, units = c.used * slices;
    constexpr int k_step = kUpWarps * W::STEP;
    P ring(dyn, warp, lane);
    // the step asked for next: of unit au, from ak on
    int au = blockIdx.x, ak = warp * W::STEP;
    const char *arow[2][2];
    auto ask_rows = [&]() {
        const int u = au / slices, f0 = (au - u * slices) * kCh;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                arow[i][r] = static_cast<const char *>(a.W1) + c.expert[u] * a.stride1 +
                             (static_cast<long long>(i) * a.F + min(f0 + g + 8 * r, a.F - 1)) * a.p1 +
                             W::N * W::ES * t;
    };
    auto ask_next = [&](int slot) {
        if (au < units && warp * W::STEP < a.H) {
            ring.ask(slot, arow, ak, a.H);
            ak += k_step;
            if (ak >= a.H) {
                ak = warp * W::STEP;
                au += gridDim.x;
                if (au < units) ask_rows();
            }
        }
        P::commit();
    };
    if (au < units) ask_rows();
    for (int d = 0; d < kUpDepth; ++d) ask_next(d);
    int slot = 0;
    for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int u = unit / slices, f0 = (unit - u * slices) * kCh;
        const int e = c.expert[u], r0 = c.first[u], n = c.first[u + 1] - r0;
        const char *trow[NF];
#pragma unroll
        for (int i = 0; i < NF; ++i)
            trow[i] = static_cast<const char *>(a.x) +
                      c.token[r0 + min(8 * i + g, n - 1)] * a.ldx * 2 + 2 * W::N * t;
        // the scales of the results that this thread will make, all of one row of
        // G and U
        const int f = threadIdx.x % kCh;
        const bool live = f0 + f < a.F;
        float sg = 1.f, su = 1.f;
        if (I8 && live && threadIdx.x < n * kCh) {
            const float *s = a.scale1 + static_cast<long long>(e) * 2 * a.F + f0 + f;
            sg = s[0];
            su = s[a.F];
        }
        float acc[2][NF][4] = {};
        uint4 x[2][W::TOK];
        if (warp * W::STEP < a.H) load_step<T, I8, XV>(x, trow[0], warp * W::STEP, a.H, t);
        for (int k = warp * W::STEP; k < a.H; k += k_step) {
            uint4 w[2][2][2], nx[2][W::TOK];
            if (k + k_step < a.H) load_step<T, I8, XV>(nx, trow[0], k + k_step, a.H, t);
            P::arrived();
            ring.take(slot, w);
            ask_next(slot);
            multiply<T, I8, 2, NF, XV>(acc, w, x, trow, k, a.H, t, n);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < W::TOK; ++j) x[i][j] = nx[i][j];
            slot = slot + 1 == kUpDepth ? 0 : slot + 1;
        }
        __syncthreads();  // the last unit's sums are read
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int m = 0; m < NF; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    part[warp][8 * m + 2 * t + (j & 1)][kCh * i + 8 * (j >> 1) + g] = acc[i][m][j];
        __syncthreads();
        for (int i = threadIdx.x; i < n * kCh; i += kUpWarps * 32) {
            const int m = i / kCh;
            float gate = 0.f, up = 0.f;
            if (live) {
#pragma unroll
                for (int w = 0; w < kUpWarps; ++w) {
                    gate += part[w][m][f];
                    up += part[w][m][kCh + f];
                }
                gate *= sg;
                up *= su;
            }
            // (values past F are zeros: gate is; what an infinity leaves is nothing)
            const float h = gate / (1.f + expf(-gate)) * up;
            const T hi = rows::from_f<T>(h);
            const float back = rows::to_f<T>(hi);
            T *to = static_cast<T *>(a.h) + 2 * c.choice[r0 + m] * a.ldh + f0 + f;
            to[0] = hi;
            to[a.ldh] = rows::from_f<T>(isfinite(back) ? (h - back) * kRestUp<T> : 0.f);
        }
    }
}

// -------------------------------------------------------------------- down

// (eight warps with twice the steps on their way: 16 tokens in 16 bits 72 us instead
// of 62, 32 tokens 133 instead of 114)
// (sixteen groups of columns: their sums take the registers of half the threads)
template <int NF>
constexpr int kDownWarps = NF <= 8 ? 16 : 8;
constexpr int kDownDepth = 3;

// The list of all used experts' steps, cut into `parts` of equal work: the first
// step of part w.  A step's work is its weights and its expert's rows (two columns
// of the matrix unit each), the weights' counted as kStepRows rows; the work before
// expert u is then steps (first[u] + kStepRows u).  (Cut into equal numbers of steps,
// the warp with a much-chosen expert is what the block waits for: 64 tokens, 2 of 8
// experts of 4096 x 2048, the fullest with 50, 8 bits 219 us, so 150; 16 bits 380 and
// 244.  With weights counted as 8 rows 156 and 258.)  Up to four tokens are one group
// of columns: equal numbers of steps.
constexpr int kStepRows = 4;
static_assert((kMaxSide / 64) * (kMaxRows + kStepRows * kMaxRows) < 0x7FFFFFFF / 16, "ints of work");
template <int NF>
__device__ __forceinline__ int first_step(const Choices &c, int steps, int w, int parts)
{
    const unsigned all = static_cast<unsigned>(c.used) * static_cast<unsigned>(steps);
    if (NF == 1 || w == parts) return static_cast<int>(all * w / parts);
    auto before = [&](int u) {
        return static_cast<unsigned>(steps) * static_cast<unsigned>(c.first[u] + kStepRows * u);
    };
    const unsigned goal = before(c.used) * w / parts;
    int u = 0, past = c.used;  // before(u) <= goal, and < before(past) where there are steps
    while (past - u > 1) {
        const int mid = (u + past) / 2;
        if (before(mid) <= goal)
            u = mid;
        else
            past = mid;
    }
    if (all == 0u) return 0;
    return u * steps + static_cast<int>((goal - before(u)) /
                                        static_cast<unsigned>(c.first[u + 1] - c.first[u] + kStepRows));
}

// grid: 16 channels of out.  The steps of all used experts form one list, a
// part of which, by work, is each warp's; a warp adds an expert's results, weighted, to
// sums of its own, and the block adds those in the warps' order.  The two parts of
// a row of h are neighbouring columns of the matrix unit, whose results one lane
// holds: up to four tokens of an expert cost no more than their columns.
template <class T, bool I8, int NF>
__global__ void __launch_bounds__(kDownWarps<NF> * 32, 1) down_kernel(const Args a)
{
    constexpr int WARPS = kDownWarps<NF>;
    using W = Weights<T, I8>;
    using P = Pieces<T, I8, 1, kDownDepth>;
    __shared__ Choices c;
    extern __shared__ __align__(16) unsigned char dyn[];  // the rings, [warp][token][channel] sums
    float *sums = reinterpret_cast<float *>(dyn + WARPS * P::BYTES);  // rows of kCh + 1
    dependent_release();
    // The up kernel releases its dependents after its own wait, so what it found
    // complete, ids and weights among it, is complete here too, and is read while
    // it still runs: on multiprocessors that its blocks have left, as a block of this
    // kernel does not fit beside them.  (F == 0: there is no up kernel.)
    if (a.F == 0) dependent_wait();
    find_choices<WARPS>(a, c);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int h0 = blockIdx.x * kCh;
    float *mine = sums + static_cast<long long>(warp) * a.T * (kCh + 1);
    for (int i = lane; i < a.T * (kCh + 1); i += 32) mine[i] = 0.f;
    const int steps = (a.F + W::STEP - 1) / W::STEP;
    int at = first_step<NF>(c, steps, warp, WARPS);
    const int end = first_step<NF>(c, steps, warp + 1, WARPS);
    P ring(dyn, warp, lane);
    // the step asked for next: expert au, its rows, step as
    int ask = at, au = steps > 0 ? at / steps : 0, as = at - au * steps;
    const char *arow[1][2];
    auto ask_rows = [&]() {
#pragma unroll
        for (int r = 0; r < 2; ++r)
            arow[0][r] = static_cast<const char *>(a.W2) + c.expert[au] * a.stride2 +
                         min(h0 + g + 8 * r, a.H - 1) * a.p2 + W::N * W::ES * t;
    };
    auto ask_next = [&](int slot) {
        if (ask < end) {
            ring.ask(slot, arow, as * W::STEP, a.F);
            ++ask;
            if (++as == steps) {
                as = 0;
                ++au;
                if (ask < end) ask_rows();
            }
        }
        P::commit();
    };
    if (ask < end) ask_rows();
    for (int d = 0; d < kDownDepth; ++d) ask_next(d);
    dependent_wait();  // h is complete
    __syncwarp();
    int slot = 0;
    while (at < end) {
        const int u = at / steps, lo = at - u * steps, hi = min(steps, lo + end - at);
        const int e = c.expert[u], r0 = c.first[u], n = c.first[u + 1] - r0;
        float scale[2] = {1.f, 1.f};
        if (I8)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                scale[r] = a.scale2[static_cast<long long>(e) * a.H + min(h0 + g + 8 * r, a.H - 1)];
        const char *trow[NF];
#pragma unroll
        for (int i = 0; i < NF; ++i)
            trow[i] = static_cast<const char *>(a.h) +
                      (2 * c.choice[r0 + min(4 * i + g / 2, n - 1)] + (g & 1)) * a.ldh * 2 +
                      2 * W::N * t;
        float acc[1][NF][4] = {};
        uint4 x[2][W::TOK];
        load_step<T, I8, true>(x, trow[0], lo * W::STEP, a.F, t);
        for (int s = lo; s < hi; ++s) {
            uint4 w[1][2][2], nx[2][W::TOK];
            if (s + 1 < hi) load_step<T, I8, true>(nx, trow[0], (s + 1) * W::STEP, a.F, t);
            P::arrived();
            ring.take(slot, w);
            ask_next(slot);
            multiply<T, I8, 1, NF, true>(acc, w, x, trow, s * W::STEP, a.F, t, 2 * n);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < W::TOK; ++j) x[i][j] = nx[i][j];
            slot = slot + 1 == kDownDepth ? 0 : slot + 1;
        }
#pragma unroll
        for (int m = 0; m < NF; ++m) {
            const int row = 4 * m + t;
            if (row < n)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    mine[c.token[r0 + row] * (kCh + 1) + 8 * r + g] +=
                        c.weight[r0 + row] *
                        (scale[r] *
                         fmaf(acc[0][m][2 * r + 1], 1.f / kRestUp<T>, acc[0][m][2 * r]));
        }
        __syncwarp();
        at += hi - lo;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * kCh; i += WARPS * 32) {
        const int m = i / kCh, ch = i % kCh;
        if (h0 + ch >= a.H) continue;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += sums[(w * a.T + m) * (kCh + 1) + ch];
        static_cast<T *>(a.out)[m * a.ldo + h0 + ch] = rows::from_f<T>(s);
    }
}

// NF: groups of eight tokens (up) and of four tokens' two columns (down: twice as
// many).
template <class T, bool I8, int NF>
int launch(const Args &a, bool x_vec, int num_sms, cudaStream_t st)
{
    if (a.F > 0) {
        constexpr int UF = NF > 1 ? NF / 2 : 1;
        using U = Up<T, I8, UF>;
        auto kern = x_vec ? up_kernel<T, I8, UF, true> : up_kernel<T, I8, UF, false>;
        if (!smem_attr_once(reinterpret_cast<const void *>(kern), U::SMEM)) return SGEMM_ERR_LAUNCH;
        const long long rows_ = static_cast<long long>(a.T) * a.k;
        const long long units = (a.E < rows_ ? a.E : rows_) * ((a.F + kCh - 1) / kCh);
        const long long room = static_cast<long long>(U::BLOCKS) * num_sms;
        const int s = launch_dependent(kern, dim3(static_cast<unsigned>(units < room ? units : room)),
                                       dim3(kUpWarps * 32), U::SMEM, 1, st, a);
        if (s != SGEMM_OK) return s;
    }
    constexpr int WARPS = kDownWarps<NF>;
    constexpr int ring = WARPS * Pieces<T, I8, 1, kDownDepth>::BYTES;
    constexpr int per_token = static_cast<int>(sizeof(float)) * WARPS * (kCh + 1);
    auto kern = down_kernel<T, I8, NF>;
    if (!smem_attr_once(reinterpret_cast<const void *>(kern), ring + per_token * 4 * NF))
        return SGEMM_ERR_LAUNCH;
    return launch_dependent(kern, dim3(static_cast<unsigned>((a.H + kCh - 1) / kCh)),
                            dim3(WARPS * 32), static_cast<size_t>(ring + per_token * a.T), 1, st, a);
}

template <class T, bool I8>
int run(const Args &a, bool x_vec, int num_sms, cudaStream_t st)
{
    if (a.T <= 4) return launch<T, I8, 1>(a, x_vec, num_sms, st);
    if (a.T <= 8) return launch<T, I8, 2>(a, x_vec, num_sms, st);
    if (a.T <= 16) return launch<T, I8, 4>(a, x_vec, num_sms, st);
    if (a.T <= 32) return launch<T, I8, 8>(a, x_vec, num_sms, st);
    return launch<T, I8, 16>(a, x_vec, num_sms, st);
}

bool sizes_ok(int T, int k, int H, int F)
{
    return choices_ok(T, k, 1) && T <= kMaxTokens && static_cast<long long>(T) * k <= kMaxRows &&
           H >= 0 && H <= kMaxSide && F >= 0 && F <= kMaxSide;
}
// A row of h: whole fragments, whose pad the kernel writes.
long long row_of_h(int F) { return (F + kCh - 1LL) / kCh * kCh; }

}  // namespace few
}  // namespace sg

using namespace sg;

extern "C" {

size_t sgemm_experts_layer_workspace_size(int T, int k, int H, int F)
{
    if (!few::sizes_ok(T, k, H, F)) return 0;
    return static_cast<size_t>(T) * k * static_cast<size_t>(few::row_of_h(F)) * 2 * 2;
}

int sgemm_experts_layer(int type, int wtype, int T, int k, int E, int H, int F, const void *x,
                        int ldx, const int *ids, const float *weights, const void *W1, int ld1,
                        long long stride1, const float *scale1, const void *W2, int ld2,
                        long long stride2, const float *scale2, void *out, int ldo,
                        void *workspace, size_t workspace_bytes, void *stream)
{
    return c_entry([&]() -> int {
        const bool i8 = wtype == SGEMM_EXPERTS_I8;
        if ((type != SGEMM_TYPE_BF16 && type != SGEMM_TYPE_FP16) ||
            (!i8 && wtype != SGEMM_EXPERTS_SAME) || !few::sizes_ok(T, k, H, F) || E < 1 ||
            E > kMaxExperts || ldx < 1 || ldx < H || ldo < 1 || ldo < H || ld1 < 1 || ld1 < H ||
            ld2 < 1 || ld2 < F || stride1 < 0 || stride2 < 0)
            return SGEMM_ERR_INVALID_ARG;
        if (E > 1 && ((F > 0 && stride1 < (2LL * F - 1) * ld1 + H) ||
                      (H > 0 && stride2 < (H - 1LL) * ld2 + F)))
            return SGEMM_ERR_INVALID_ARG;
        const long long ws = i8 ? 1 : 2;
        if (ld1 * ws % 16 != 0 || ld2 * ws % 16 != 0 || stride1 * ws % 16 != 0 ||
            stride2 * ws % 16 != 0 || !rows::aligned_to(W1, 16) || !rows::aligned_to(W2, 16) ||
            !rows::aligned_to(x, 2) || !rows::aligned_to(out, 2) || !rows::aligned_to(ids, 4) ||
            !rows::aligned_to(weights, 4) || !rows::aligned_to(scale1, 4) ||
            !rows::aligned_to(scale2, 4) || !rows::aligned_to(workspace, 16))
            return SGEMM_ERR_INVALID_ARG;
        if (T == 0 || H == 0) return SGEMM_OK;
        if (x == nullptr || ids == nullptr || out == nullptr) return SGEMM_ERR_INVALID_ARG;
        if (F > 0 && (W1 == nullptr || W2 == nullptr || (i8 && (scale1 == nullptr || scale2 == nullptr)) ||
                      workspace == nullptr ||
                      workspace_bytes < sgemm_experts_layer_workspace_size(T, k, H, F)))
            return SGEMM_ERR_INVALID_ARG;
        int num_sms = 0;
        unsigned int *status = nullptr;
        if (!current_sm103(&num_sms, &status)) return SGEMM_ERR_UNSUPPORTED;
        few::Args a{};
        a.T = T;
        a.k = k;
        a.E = E;
        a.H = H;
        a.F = F;
        a.x = x;
        a.ldx = ldx;
        a.ids = ids;
        a.weights = weights;
        a.W1 = W1;
        a.W2 = W2;
        a.p1 = ld1 * ws;
        a.stride1 = stride1 * ws;
        a.p2 = ld2 * ws;
        a.stride2 = stride2 * ws;
        a.scale1 = scale1;
        a.scale2 = scale2;
        a.out = out;
        a.ldo = ldo;
        a.h = workspace;
        a.ldh = few::row_of_h(F);
        const bool x_vec = rows::aligned_to(x, 16) && ldx % 8 == 0;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        if (type == SGEMM_TYPE_BF16)
            return i8 ? few::run<__nv_bfloat16, true>(a, x_vec, num_sms, st)
                      : few::run<__nv_bfloat16, false>(a, x_vec, num_sms, st);
        return i8 ? few::run<__half, true>(a, x_vec, num_sms, st) : few::run<__half, false>(a, x_vec, num_sms, st);
    });
}

}  // extern "C"

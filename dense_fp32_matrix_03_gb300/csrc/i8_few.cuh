// i8_few.cuh -- products of 8-bit integers with a scale for each token and
// channel, for few tokens:
//   C[m][n] = scaleA[m] * scaleB[n] * sum_k A[m][k] * B[n][k].
//
// What counts is to read the weights once, and soon: a decoding step's product
// takes little longer than HBM needs for them.  Both kernels here keep their
// sums in registers and need no tensor memory, barriers or pipeline, whose
// setting up is most of the time of the kernel in i8_tc.cuh for one token
// (4096 x 4096 on GB300: 11.0 us; 4.5 here, a plain read of the weights 4.1).
//   dots_kernel  up to four tokens at a time, integer dot products (dp4a):
//                16 instructions per 2 KB of weights and token, but on units
//                too slow for more (eight tokens took 16.7 us)
//   few_kernel   up to 8 * NF tokens at a time on the matrix units (mma.sync
//                m16n8k16, fp16 inputs, fp32 sums): 8-bit integers are exact
//                in fp16, widened in registers (widen4), the sums exact under
//                the same condition as in i8_tc.cuh; 80 instructions widen 2 KB
//                of weights.  (The integer matrix instruction needs none, but
//                its rate, about 115 products a clock and multiprocessor, made
//                16 tokens 7.9 us where this kernel takes 6.4.)
// In both the warps of a block share the steps of k of a few channels, add
// their sums in shared memory in order of k, and scale and store them; the
// weights of a dense call start on their way into L2 before the kernel waits
// for the one before it, and the scales are asked for before the weights.
#pragma once

#include "dependent.cuh"
#include "i8_gemm.h"
#include "i8_tc.cuh"

namespace sg {
namespace i8 {

// 16 bytes of a row from k on, zeros past K; nothing past K is read.
__device__ __forceinline__ uint4 load_tail(const signed char *row, int k, int K)
{
    if (k + 16 <= K) return *reinterpret_cast<const uint4 *>(row + k);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    for (int i = 0; i < 4; ++i)
        for (int b = 0; b < 4; ++b)
            if (k + 4 * i + b < K)
                w[i] |= (static_cast<uint32_t>(row[k + 4 * i + b]) & 255u) << (8 * b);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// (An ordinary load: the kernel before may still write the operands when this
// one starts, and a read-only load is defined for memory that stays as it is
// while the kernel lives.)
__device__ __forceinline__ uint4 load_row(const signed char *p)
{
    return *reinterpret_cast<const uint4 *>(p);
}

// Dense calls: asks L2 for the weights of `ch` channels from n0 on, a line of
// 128 bytes per thread and turn.  No value is read, so this may run before
// the kernel before has finished, even one that still writes them.
__device__ __forceinline__ void ask_weights(const Args &a, int n0, int ch)
{
    const int lines = (a.K + 127) / 128;
    for (int i = threadIdx.x; i < ch * lines; i += blockDim.x) {
        const int n = n0 + i / lines, k = i % lines * 128;
        if (n < a.N)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.B + static_cast<long long>(n) * a.ldb +
                                                          k));
    }
}

__device__ __forceinline__ int log2_of(int x) { return 31 - __clz(x); }

// The results of a block: `groups` runs of CH channels from n0 on, for the
// tokens of `tl`.  Thread tid makes results tid, tid + threads, ...;
// neighbours have neighbouring channels.
template <class T, int CH>
struct Results {
    const Args &a;
    const Tile &tl;
    int n0, shift, count;  // channels of a token: 1 << shift (CH and groups are powers of two)
    float sa, sb;          // the scales of this thread's first result
    __device__ __forceinline__ Results(const Args &args, const Tile &tile, int first, int groups)
        : a(args), tl(tile), n0(first), shift(log2_of(groups * CH)),
          count(groups * CH * tile.rows), sa(0.f), sb(0.f)
    {
        const int i = threadIdx.x;
        if (i < count && channel(i) < a.N) {
            sa = a.scaleA[tl.row0 + token(i)];
            sb = a.scaleB[static_cast<long long>(tl.e) * a.N + channel(i)];
        }
    }
    __device__ __forceinline__ int token(int i) const { return i >> shift; }
    __device__ __forceinline__ int of_token(int i) const { return i & ((1 << shift) - 1); }
    __device__ __forceinline__ int channel(int i) const { return n0 + of_token(i); }
    template <class F>
    __device__ __forceinline__ void put(int i, float x, float y, const F &sum)
    {
        static_cast<T *>(a.C)[(tl.row0 + token(i)) * a.ldc + channel(i)] =
            rows::from_f<T>(sum(of_token(i) / CH, token(i), of_token(i) % CH) * x * y);
    }
    // sum(group, token, channel of the group): the unscaled sum
    template <class F>
    __device__ __forceinline__ void store(const F &sum)
    {
        const int first = threadIdx.x, step = blockDim.x;
        if (first < count && channel(first) < a.N) put(first, sa, sb, sum);
        // (the scales of four results on their way together)
#pragma unroll 4
        for (int i = first + step; i < count; i += step)
            if (channel(i) < a.N)
                put(i, a.scaleA[tl.row0 + token(i)],
                    a.scaleB[static_cast<long long>(tl.e) * a.N + channel(i)], sum);
    }
};

// ------------------------------------------------------------------- dots
//
// A lane holds 16 bytes of each of the warp's channels and tokens, a step is
// 512 k: every load is 512 contiguous bytes.
constexpr int kDotK = 512, kDotCh = 4;
// (Seven blocks leave 72 registers: 18 words of the four-token form's spill, 4
// of the two-token form's; four tokens take 6.0 us at 4096 x 4096, two 5.0.)
constexpr int kDotWarps = 4, kDotBlocks = 7;  // of a block, of a multiprocessor

__device__ __forceinline__ int dot16(const uint4 &x, const uint4 &y, int s)
{
    s = __dp4a(static_cast<int>(x.x), static_cast<int>(y.x), s);
    s = __dp4a(static_cast<int>(x.y), static_cast<int>(y.y), s);
    s = __dp4a(static_cast<int>(x.z), static_cast<int>(y.z), s);
    return __dp4a(static_cast<int>(x.w), static_cast<int>(y.w), s);
}

// wk: warps that share the k of a group of channels.
template <class T, int MT>
__global__ void __launch_bounds__(kDotWarps * 32, kDotBlocks) dots_kernel(const Args a, int wk)
{
    __shared__ int part[kDotWarps][MT * kDotCh];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wc = kDotWarps / wk, cw = warp / wk, kw = warp % wk;
    const int x0 = blockIdx.x * wc * kDotCh, n0 = x0 + cw * kDotCh;
    dependent_release();
    if (a.offsets == nullptr) ask_weights(a, x0, wc * kDotCh);
    dependent_wait();
    const Tile tl = find_tile_warp(a, blockIdx.y, MT, lane);
    if (tl.e < 0) return;
    Results<T, kDotCh> out(a, tl, x0, wc);
    // this lane's rows; those past the last channel or token repeat it, and
    // their results are not stored
    const signed char *B[kDotCh], *A[MT];
#pragma unroll
    for (int c = 0; c < kDotCh; ++c)
        B[c] = a.B + tl.e * a.strideB +
               static_cast<long long>(min(n0 + c, a.N - 1)) * a.ldb + 16 * lane;
#pragma unroll
    for (int m = 0; m < MT; ++m)
        A[m] = a.A + (tl.row0 + min(m, tl.rows - 1)) * a.lda + 16 * lane;
    int acc[MT][kDotCh] = {};
    uint4 w[kDotCh], x[MT];
    auto use = [&]() {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < kDotCh; ++c) acc[m][c] = dot16(w[c], x[m], acc[m][c]);
    };
    // whole steps; then the warp whose turn it is takes what is left of k
    const int step = wk * kDotK, whole = a.K / kDotK * kDotK;
    int k = kw * kDotK;
    for (; k < whole; k += step) {
#pragma unroll
        for (int c = 0; c < kDotCh; ++c) w[c] = load_row(B[c] + k);
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = load_row(A[m] + k);
        use();
    }
    if (k == whole && whole < a.K) {
        const int K = a.K - 16 * lane;  // the rows start at 16 * lane
#pragma unroll
        for (int c = 0; c < kDotCh; ++c) w[c] = load_tail(B[c], whole, K);
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = load_tail(A[m], whole, K);
        use();
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < kDotCh; ++c) {
            const int s = __reduce_add_sync(0xffffffffu, acc[m][c]);
            if (lane == 0) part[warp][m * kDotCh + c] = s;
        }
    __syncthreads();
    out.store([&](int g, int m, int c) {
        int s = 0;
        for (int j = 0; j < wk; ++j) s += part[g * wk + j][m * kDotCh + c];
        return static_cast<float>(s);
    });
}

template <class T, int MT>
int launch_dots(const Args &a, cudaStream_t st)
{
    // at least two steps a warp
    const int wk = rows::pow2_threads((a.K + 2LL * kDotK - 1) / (2 * kDotK), 1, kDotWarps);
    const int ch = kDotWarps / wk * kDotCh;
    return launch_dependent(dots_kernel<T, MT>,
                            dim3(static_cast<unsigned>((a.N + ch - 1) / ch),
                                 static_cast<unsigned>(max_tiles(a, MT))),
                            dim3(kDotWarps * 32), 0, 1, st, a, wk);
}

// -------------------------------------------------------------------- few
//
// The matrix instruction's lane (g, t) = (lane / 4, lane % 4) holds row g and
// g + 8 of the weights and column g of the tokens, four values of k each.
// Which four is ours to choose as long as both operands agree: lane t takes
// bytes 16 t .. 16 t + 15 of either half of the step's 128, and feeds them to
// four instructions in order.  So every load is 16 bytes, a quad reads 64
// bytes of a row together, and nothing passes through shared memory.
constexpr int kFewK = 128;  // k per step and warp

__device__ __forceinline__ void widen16(const uint4 &v, uint32_t (&h)[8])
{
    widen4(v.x, h[0], h[1]);
    widen4(v.y, h[2], h[3]);
    widen4(v.z, h[4], h[5]);
    widen4(v.w, h[6], h[7]);
}
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// CF: times 16 channels per warp; WARPS: of a block; BLOCKS: of a
// multiprocessor, at least.
template <class T, int NF, int CF, int WARPS, int BLOCKS>
__global__ void __launch_bounds__(WARPS * 32, BLOCKS) few_kernel(const Args a, int wk)
{
    constexpr int CH = 16 * CF, TK = 8 * NF;
    __shared__ float part[WARPS][TK][CH + 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int wc = WARPS / wk, cw = warp / wk, kw = warp % wk;
    const int x0 = blockIdx.x * wc * CH, n0 = x0 + cw * CH;
    dependent_release();
    if (a.offsets == nullptr) ask_weights(a, x0, wc * CH);
    dependent_wait();
    const Tile tl = find_tile_warp(a, blockIdx.y, TK, lane);
    if (tl.e < 0) return;
    Results<T, CH> out(a, tl, x0, wc);
    // this lane's rows; those past the last channel or token repeat it, and
    // their results are not stored
    const signed char *B[CF][2], *A[NF];
#pragma unroll
    for (int c = 0; c < CF; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            B[c][h] = a.B + tl.e * a.strideB +
                      static_cast<long long>(min(n0 + 16 * c + 8 * h + g, a.N - 1)) * a.ldb +
                      16 * t;
#pragma unroll
    for (int n = 0; n < NF; ++n)
        A[n] = a.A + (tl.row0 + min(8 * n + g, tl.rows - 1)) * a.lda + 16 * t;
    float acc[CF][NF][4] = {};
    uint4 w[CF][2][2], x[NF][2];  // a step: [..][rows g, g + 8][half of k]
    auto use = [&]() {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t tok[NF][8];
#pragma unroll
            for (int n = 0; n < NF; ++n) widen16(x[n][i], tok[n]);
#pragma unroll
            for (int c = 0; c < CF; ++c) {
                uint32_t lo[8], hi[8];
                widen16(w[c][0][i], lo);
                widen16(w[c][1][i], hi);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int n = 0; n < NF; ++n)
                        if (n == 0 || 8 * n < tl.rows)
                            mma_16816(acc[c][n], lo[2 * j], hi[2 * j], lo[2 * j + 1],
                                      hi[2 * j + 1], tok[n][2 * j], tok[n][2 * j + 1]);
            }
        }
    };
    // whole steps; then the warp whose turn it is takes what is left of k
    const int step = wk * kFewK, whole = a.K / kFewK * kFewK;
    int k = kw * kFewK;
    for (; k < whole; k += step) {
#pragma unroll
        for (int c = 0; c < CF; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) w[c][h][i] = load_row(B[c][h] + k + 64 * i);
#pragma unroll
        for (int n = 0; n < NF; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) x[n][i] = load_row(A[n] + k + 64 * i);
        use();
    }
    if (k == whole && whole < a.K) {
        for (int i = 0; i < 2; ++i) {
            const int at = whole + 64 * i, K = a.K - 16 * t;  // the rows start at 16 * t
#pragma unroll
            for (int c = 0; c < CF; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) w[c][h][i] = load_tail(B[c][h], at, K);
#pragma unroll
            for (int n = 0; n < NF; ++n) x[n][i] = load_tail(A[n], at, K);
        }
        use();
    }
#pragma unroll
    for (int c = 0; c < CF; ++c)
#pragma unroll
        for (int n = 0; n < NF; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[warp][8 * n + 2 * t + (i & 1)][16 * c + 8 * (i >> 1) + g] = acc[c][n][i];
    __syncthreads();
    out.store([&](int gr, int m, int c) {
        float s = 0.f;
        for (int j = 0; j < wk; ++j) s += part[gr * wk + j][m][c];
        return s;
    });
}

template <class T, int NF, int CF, int WARPS, int BLOCKS>
int launch_few(const Args &a, cudaStream_t st)
{
    const int wk = rows::pow2_threads((a.K + kFewK - 1LL) / kFewK, 1, WARPS);
    const long long ch = WARPS / wk * 16LL * CF;
    return launch_dependent(few_kernel<T, NF, CF, WARPS, BLOCKS>,
                            dim3(static_cast<unsigned>((a.N + ch - 1) / ch),
                                 static_cast<unsigned>(max_tiles(a, 8 * NF))),
                            dim3(WARPS * 32), 0, 1, st, a, wk);
}

}  // namespace i8
}  // namespace sg

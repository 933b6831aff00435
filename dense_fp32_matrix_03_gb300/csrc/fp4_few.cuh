// fp4_few.cuh -- products in microscaled 4-bit floating point for up to four
// tokens (include/fp4_gemm.h).
//
// What counts is to read the weights once, and soon: sums stay in registers, and
// there is no tensor memory, barrier or pipeline, whose setting up is most of the
// time of the kernel in fp4_tc.cuh for one token.
//
// A code s eem, its sign put at bit 15 and eem at bits 11 .. 9 of a half, is the
// fp16 number 2^-14 times its value (subnormal where e is 0): two shifts and two
// logic instructions decode two codes.  (The conversion instruction for codes has
// a fraction of their rate: decoded by it and multiplied by mma.sync, one token
// through 4096 x 4096 took 7.9 us.)  Packed fp16 FMAs add the products of 16
// values exactly: each half of the sum takes eight, at most 1152 units of a
// quarter's product.  Then it is fp32: a block's two halves times both block scales
// (MX: in two steps).
//
// A warp takes four channels 32 apart, whose scales for 64 values are 16
// consecutive bytes of the layout, and 1024 k a step, 32 a lane.  The warps of a
// block share the steps of k of a few such channels and add their sums in order.
//
// Bound by instructions, about four a weight: one token through 1024 x 1024 2.8 us
// (the tensor-core kernel 3.7), 2048 x 2048 3.7 (4.8), 4096 x 4096 8.1 (5.8).
#pragma once

#include "fp4_tc.cuh"

namespace sg {
namespace fp4 {

constexpr int kFewTokens = 4;
constexpr int kFewK = 1024;                     // k per step and warp
constexpr int kFewWarps = 4, kFewCh = 4;        // of a block; channels of a warp

// Asks L2 for the weights of `groups` times four channels (first: their number)
// and their scales.  No value is read, so this may run before the kernel before
// has finished.
__device__ __forceinline__ void ask_weights(const Args &a, int first, int groups)
{
    const int lines = ((a.K + 1) / 2 + 127) / 128;
    for (int i = threadIdx.x; i < groups * kFewCh * lines; i += blockDim.x) {
        const int row = i / lines, q = first + row / kFewCh;
        const long long n = q / 32 * 128LL + q % 32 + row % kFewCh * 32;
        if (n < a.N)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.B + n * a.ldb + i % lines * 128));
    }
    for (int i = threadIdx.x; i < a.tiles; i += blockDim.x)
        if (first / 32 * 128LL < a.N)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                a.sfB + scale_row(first / 32 * 128LL + first % 32, a.tiles) + i * static_cast<long long>(kTileBytes)));
}

// 32 codes from k on (a multiple of 32); zeros from K on, nothing behind the
// 16 bytes that hold K - 1 is read.
__device__ __forceinline__ uint4 load_codes(const unsigned char *row, int k, int K)
{
    if (k >= K) return make_uint4(0u, 0u, 0u, 0u);
    uint4 v = *reinterpret_cast<const uint4 *>(row + k / 2);
    if (k + 32 > K) {
        const int left = K - k;  // 1 .. 31 codes
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = left - 8 * i;
            if (n <= 0)
                w[i] = 0u;
            else if (n < 8)
                w[i] &= (1u << (4 * n)) - 1u;
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}
// 2^-14 times the eight codes of a word: pairs (i, i + 4).
__device__ __forceinline__ void decode8(uint32_t w, __half2 (&h)[4])
{
    const uint32_t r[4] = {((w << 12) & 0x80008000u) | ((w << 9) & 0x0E000E00u),
                           ((w << 8) & 0x80008000u) | ((w << 5) & 0x0E000E00u),
                           ((w << 4) & 0x80008000u) | ((w << 1) & 0x0E000E00u),
                           (w & 0x80008000u) | ((w >> 3) & 0x0E000E00u)};
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const __half2 *>(&r[i]);
}
// The scales of 32 values from k on, out of the word of four blocks that holds them.
// NV: of its two halves of 16 values.  MX: one scale 2^e as two factors 2^(e / 2),
// rounded down and up, so that products of two operands' factors keep within fp32
// where the product of the scales does not (2^70 twice, times a code that is zero).
template <int FORMAT>
__device__ __forceinline__ float2 scales_of(uint32_t word, int k)
{
    if (FORMAT == SGEMM_FP4_NV) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(word >> (k % 64 / 2)), __NV_E4M3);
        return __half22float2(__half2(h));
    }
    const uint32_t b = word >> (k % 128 / 4) & 255u;  // e + 127
    return make_float2(__uint_as_float(b == 255u ? 0x7FC00000u : (b + 127u) >> 1 << 23),
                       __uint_as_float((b + 128u) >> 1 << 23));
}
constexpr int word_k(int format) { return kTileBlocks * (format == SGEMM_FP4_MX ? 32 : 16); }

// grid: wc * four channels.  wk: warps that share the k of a group of four.
template <class T, int FORMAT, int MT>
__global__ void __launch_bounds__(kFewWarps * 32, MT == 1 ? 6 : MT == 2 ? 5 : 3)
    few_kernel(const Args a, int wk)
{
    __shared__ float part[kFewWarps][MT * kFewCh];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wc = kFewWarps / wk, kw = warp % wk;
    const int first = blockIdx.x * wc, q = first + warp / wk;
    dependent_release();
    ask_weights(a, first, wc);
    dependent_wait();
    // this lane's rows; those past the last channel or token repeat another, and
    // their results are not stored
    const long long n0 = q / 32 * 128LL + q % 32;
    const unsigned char *B[kFewCh], *A[MT], *sfA[MT];
#pragma unroll
    for (int c = 0; c < kFewCh; ++c)
        B[c] = a.B + (n0 + 32 * c < a.N ? n0 + 32 * c : 0LL) * a.ldb;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        A[m] = a.A + min(m, a.M - 1) * a.lda;
        sfA[m] = a.sfA + scale_row(min(m, a.M - 1), a.tiles);
    }
    // (a row block's tile holds all four rows of a group, also past the last)
    const unsigned char *sfB = a.sfB + scale_row(n0 < a.N ? n0 : 0LL, a.tiles);
    float acc[MT][kFewCh] = {};
    for (int k = (kw * 32 + lane) * 32; k - lane * 32 < a.K; k += wk * kFewK) {
        const bool on = k < a.K;
        uint4 w[kFewCh], x[MT], ws = make_uint4(0u, 0u, 0u, 0u);
        uint32_t xs[MT];
        const long long tile = static_cast<long long>(k / word_k(FORMAT)) * kTileBytes;
#pragma unroll
        for (int c = 0; c < kFewCh; ++c) w[c] = load_codes(B[c], k, a.K);
        if (on) ws = *reinterpret_cast<const uint4 *>(sfB + tile);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            x[m] = load_codes(A[m], k, a.K);
            xs[m] = on ? *reinterpret_cast<const uint32_t *>(sfA[m] + tile) : 0u;
        }
        const uint32_t wsv[4] = {ws.x, ws.y, ws.z, ws.w};
        float2 sw[kFewCh], sx[MT];
#pragma unroll
        for (int c = 0; c < kFewCh; ++c) sw[c] = scales_of<FORMAT>(wsv[c], k);
#pragma unroll
        for (int m = 0; m < MT; ++m) sx[m] = scales_of<FORMAT>(xs[m], k);
#pragma unroll
        for (int b = 0; b < 2; ++b) {  // 16 values: two words
            __half2 xv[MT][8];
            // tokens times 2^13, so that a product is half of what it stands for and
            // sums of small scales keep off fp32's end
            const __half2 up = __half2half2(__ushort_as_half(0x7400));   // 2^14
            const __half2 up2 = __half2half2(__ushort_as_half(0x7000));  // 2^13
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                __half2 h[4];
                decode8(b ? x[m].z : x[m].x, h);
#pragma unroll
                for (int i = 0; i < 4; ++i) xv[m][i] = __hmul2(__hmul2(h[i], up), up2);
                decode8(b ? x[m].w : x[m].y, h);
#pragma unroll
                for (int i = 0; i < 4; ++i) xv[m][4 + i] = __hmul2(__hmul2(h[i], up), up2);
            }
#pragma unroll
            for (int c = 0; c < kFewCh; ++c) {
                __half2 h[4], g[4];
                decode8(b ? w[c].z : w[c].x, h);
                decode8(b ? w[c].w : w[c].y, g);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    __half2 s = __hmul2(h[0], xv[m][0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) s = __hfma2(h[i], xv[m][i], s);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s = __hfma2(g[i], xv[m][4 + i], s);
                    const float2 f = __half22float2(s);
                    if (FORMAT == SGEMM_FP4_NV) {
                        const float sc = (b ? sw[c].y : sw[c].x) * (b ? sx[m].y : sx[m].x);
                        acc[m][c] = fmaf(f.x + f.y, sc, acc[m][c]);
                    } else {
                        // (exact but for the sum, as all are powers of two of some 2^-127 to
                        // 2^127; where the first product leaves fp32, the second would)
                        acc[m][c] = fmaf((f.x + f.y) * (sw[c].x * sx[m].y), sw[c].y * sx[m].x,
                                         acc[m][c]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < kFewCh; ++c) {
            float s = acc[m][c];
#pragma unroll
            for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (lane == 0) part[warp][m * kFewCh + c] = s;
        }
    __syncthreads();
    const int i = threadIdx.x;  // group of channels, token, channel
    if (i < wc * MT * kFewCh) {
        const int gr = i / (MT * kFewCh), m = i / kFewCh % MT, c = i % kFewCh, qq = first + gr;
        const long long n = qq / 32 * 128LL + qq % 32 + 32 * c;
        if (m < a.M && n < a.N) {
            float s = 0.f;
            for (int j = 0; j < wk; ++j) s += part[gr * wk + j][m * kFewCh + c];
            const float sa = a.scaleA != nullptr ? a.scaleA[m] : 1.f;
            const float sb = a.scaleB != nullptr ? a.scaleB[n] : 1.f;
            static_cast<T *>(a.C)[m * a.ldc + n] = rows::from_f<T>(2.f * s * sa * sb);
        }
    }
}

template <class T, int FORMAT, int MT>
int launch_few(const Args &a, cudaStream_t st)
{
    const int wk = rows::pow2_threads((a.K + kFewK - 1LL) / kFewK, 1, kFewWarps);
    const int wc = kFewWarps / wk;
    const long long groups = (a.N + 127LL) / 128 * 32;
    return launch_dependent(few_kernel<T, FORMAT, MT>,
                            dim3(static_cast<unsigned>((groups + wc - 1) / wc)),
                            dim3(kFewWarps * 32), 0, 1, st, a, wk);
}

}  // namespace fp4
}  // namespace sg

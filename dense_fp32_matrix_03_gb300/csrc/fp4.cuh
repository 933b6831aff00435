// fp4.cuh -- the 4-bit format's layout and quantisation (include/fp4_gemm.h),
// shared by the kernels that write it (fp4_quant.cu, norm.cu) and read it
// (fp4_gemm.cu).
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/fp4_gemm.h"
#include "rows.cuh"

namespace sg {
namespace fp4 {

constexpr int kTileRows = 128, kTileBlocks = 4, kTileBytes = kTileRows * kTileBlocks;
constexpr int kLdStep = 32;  // a leading dimension's granule: 16 bytes of codes
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100

inline bool valid_format(int f) { return f == SGEMM_FP4_MX || f == SGEMM_FP4_NV; }
__host__ __device__ inline int block_of(int format) { return format == SGEMM_FP4_MX ? 32 : 16; }
// Tiles of block scales that K values of a row take.
__host__ __device__ inline long long scale_tiles(int format, long long K)
{
    const long long per = block_of(format) * kTileBlocks;
    return (K + per - 1) / per;
}
// Byte offset of a row's first scale word (four blocks); the next four blocks'
// word is kTileBytes further.
__host__ __device__ inline long long scale_row(long long row, long long tiles)
{
    return row / kTileRows * tiles * kTileBytes + row % 32 * 16 + row % kTileRows / 32 * 4;
}

// Eight (four: in the low half) fp32 values as 4-bit codes, value i in bits 4 i; to nearest, ties
// to the even code, 6 beyond 6.
__device__ __forceinline__ uint32_t pack_codes(const float (&v)[8])
{
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}
__device__ __forceinline__ uint32_t pack_codes(const float (&v)[4])
{
    uint32_t w;
    asm("{\n\t.reg .b8 a, b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b, a, b};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
    return w;
}

// What a row's quantisation hangs on.
struct RowScale {
    float c448, c2688;  // 448 / a_r and 2688 / a_r (NV); 0 for a row without values
    float scale;        // the row's own
    bool finite;
};
__device__ __forceinline__ RowScale row_scale(int format, unsigned amax_bits)
{
    const float amax = __uint_as_float(amax_bits);
    RowScale r;
    r.finite = amax_bits < 0x7F800000u;
    const bool some = r.finite && amax >= kTiny;
    r.c448 = some ? __fdiv_rn(448.f, amax) : 0.f;
    r.c2688 = some ? __fdiv_rn(2688.f, amax) : 0.f;
    r.scale = !r.finite ? __int_as_float(0x7FFFFFFF)
              : format == SGEMM_FP4_MX ? 1.f
                                       : (some ? __fdiv_rn(amax, 2688.f) : 0.f);
    return r;
}

// Quantises the warp's vectors of EV values of one row (EV = 4 or 8, lane l
// holds vector v = v0 + l, v0 a multiple of 32; values past the row are zeros)
// and stores codes and block scales.  The lanes of a block (16 or 32 values)
// find its largest magnitude together; those of four blocks send their scales
// out as one word.  All 32 lanes call; nvec: vectors of the row.
template <int FORMAT, int EV>
__device__ __forceinline__ void store_vectors(const float (&v)[EV], unsigned vec, unsigned nvec,
                                              const RowScale &rs, unsigned char *q_row,
                                              unsigned char *sf_row)
{
    constexpr int BL = (FORMAT == SGEMM_FP4_MX ? 32 : 16) / EV;  // lanes of a block
    const int lane = static_cast<int>(threadIdx.x) & 31;
    unsigned big = 0;
#pragma unroll
    for (int i = 0; i < EV; ++i) big = max(big, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = 1; d < BL; d *= 2) big = max(big, __shfl_xor_sync(0xffffffffu, big, d));
    unsigned byte;
    float up;
    if (FORMAT == SGEMM_FP4_MX) {
        const int e = static_cast<int>(big >> 23) - 2;
        byte = e > 0 ? e : 0;
        up = __uint_as_float((254u - byte) << 23);
    } else {
        byte = __nv_cvt_float_to_fp8(__uint_as_float(big) * rs.c448, __NV_SATFINITE, __NV_E4M3);
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte),
                                                     __NV_E4M3);
        up = byte != 0 ? __fdiv_rn(rs.c2688, __half2float(__half(h))) : 0.f;
    }
    if (!rs.finite) byte = 0;
    float u[EV];
#pragma unroll
    for (int i = 0; i < EV; ++i) u[i] = v[i] * up;
    const uint32_t codes = rs.finite ? pack_codes(u) : 0u;
    if constexpr (EV == 8) {
        if (vec < nvec) reinterpret_cast<uint32_t *>(q_row)[vec] = codes;
    } else {  // (eight codes together: the second four past an odd last vector are zeros)
        if (vec < ((nvec + 1) & ~1u))
            reinterpret_cast<uint16_t *>(q_row)[vec] = static_cast<uint16_t>(codes);
    }
    uint32_t word = byte << (8 * ((lane / BL) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, BL);
    word |= __shfl_xor_sync(0xffffffffu, word, 2 * BL);
    if (lane % (4 * BL) == 0 && vec < nvec)
        *reinterpret_cast<uint32_t *>(sf_row + static_cast<long long>(vec / (4 * BL)) * kTileBytes) =
            word;
}

}  // namespace fp4
}  // namespace sg

// rows.cuh -- rows of bf16, fp16 or fp32 values moved in vectors of 2 to 16
// bytes, and the host-side choice of the vector: shared by the row kernels
// (experts.cu, quant.cu: Vec; norm.cu, fp4_quant.cu: Words) and the products of
// few bits; the expert operators' limits.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/int8_gemm.h"
#include "../../include/sgemm.h"
#include "internal.h"

namespace sg {

// Limits of the expert operators and the products by expert.
constexpr int kMaxExperts = 1024;  // E
constexpr int kMaxChoices = 64;    // k

// T tokens with k choices out of E.
inline bool choices_ok(int T, int k, int E)
{
    return T >= 0 && k >= 1 && k <= kMaxChoices && E >= 1 && E <= kMaxExperts &&
           static_cast<long long>(T) * k <= 0x7FFFFFFFLL;
}

namespace rows {

// A vector of VB bytes.
template <int VB>
struct Raw;
template <>
struct Raw<16> {
    using T = uint4;
};
template <>
struct Raw<8> {
    using T = uint2;
};
template <>
struct Raw<4> {
    using T = uint32_t;
};
template <>
struct Raw<2> {
    using T = uint16_t;
};

template <class T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x)
{
    return x;
}
template <>
__device__ __forceinline__ float to_f<__half>(__half x)
{
    return __half2float(x);
}
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x)
{
    return __bfloat162float(x);
}
template <class T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x)
{
    return x;
}
template <>
__device__ __forceinline__ __half from_f<__half>(float x)
{
    return __float2half_rn(x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x)
{
    return __float2bfloat16_rn(x);
}

// VB bytes of values of type T, moved as one access.
template <class T, int VB>
struct Vec {
    static constexpr int N = VB / static_cast<int>(sizeof(T));
    union {
        typename Raw<VB>::T raw;
        T v[N];
    };
    __device__ __forceinline__ Vec() {}
    __device__ __forceinline__ void load(const void *p)
    {
        raw = *static_cast<const typename Raw<VB>::T *>(p);
    }
    // In pieces of LB bytes, the first `bytes` of them (a multiple of LB); zeros
    // for the rest.
    template <int LB>
    __device__ __forceinline__ void load_pieces(const char *p, unsigned bytes)
    {
        if constexpr (LB == VB) {
            load(p);
        } else {
            using P = typename Raw<LB>::T;
#pragma unroll
            for (int i = 0; i < VB / LB; ++i)
                reinterpret_cast<P *>(&raw)[i] =
                    static_cast<unsigned>(i * LB) < bytes
                        ? *reinterpret_cast<const P *>(p + i * LB)
                        : P{};
        }
    }
    __device__ __forceinline__ void store(void *p) const
    {
        *static_cast<typename Raw<VB>::T *>(p) = raw;
    }
    __device__ __forceinline__ void zero() { raw = typename Raw<VB>::T{}; }
    __device__ __forceinline__ float get(int i) const { return to_f<T>(v[i]); }
    __device__ __forceinline__ void set(int i, float x) { v[i] = from_f<T>(x); }
};

// A vector of VB bytes (8 or 16) as 32-bit words that are unpacked to fp32 and
// packed from it as a whole: values taken one by one out of a Vec of 16-bit
// values that lives in registers for long cost some five times the instructions.
template <class T, int VB>
struct Words {
    static constexpr int N = VB / static_cast<int>(sizeof(T));
    uint32_t w[VB / 4];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < VB / 4; ++i) w[i] = 0u;
    }
    // In pieces of LB bytes, the first `bytes` of them (a multiple of LB; all of
    // them where LB is VB); zeros for the rest.
    template <int LB>
    __device__ __forceinline__ void load(const char *p, unsigned bytes)
    {
        if constexpr (LB == 16) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        } else if constexpr (LB == 8) {
#pragma unroll
            for (int i = 0; i < VB / 8; ++i) {
                uint2 v = make_uint2(0u, 0u);
                if (VB == 8 || 8u * i < bytes) v = *reinterpret_cast<const uint2 *>(p + 8 * i);
                w[2 * i] = v.x;
                w[2 * i + 1] = v.y;
            }
        } else if constexpr (LB == 4) {
#pragma unroll
            for (int i = 0; i < VB / 4; ++i)
                w[i] = 4u * i < bytes ? *reinterpret_cast<const uint32_t *>(p + 4 * i) : 0u;
        } else {
#pragma unroll
            for (int i = 0; i < VB / 4; ++i) {
                const uint32_t lo =
                    4u * i < bytes ? *reinterpret_cast<const uint16_t *>(p + 4 * i) : 0u;
                const uint32_t hi =
                    4u * i + 2u < bytes ? *reinterpret_cast<const uint16_t *>(p + 4 * i + 2) : 0u;
                w[i] = lo | hi << 16;
            }
        }
    }
    template <int LB>
    __device__ __forceinline__ void store(char *p, unsigned bytes) const
    {
        if constexpr (LB == 16) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if constexpr (LB == 8) {
#pragma unroll
            for (int i = 0; i < VB / 8; ++i)
                if (VB == 8 || 8u * i < bytes)
                    *reinterpret_cast<uint2 *>(p + 8 * i) = make_uint2(w[2 * i], w[2 * i + 1]);
        } else if constexpr (LB == 4) {
#pragma unroll
            for (int i = 0; i < VB / 4; ++i)
                if (4u * i < bytes) *reinterpret_cast<uint32_t *>(p + 4 * i) = w[i];
        } else {
#pragma unroll
            for (int i = 0; i < VB / 4; ++i) {
                if (4u * i < bytes)
                    *reinterpret_cast<uint16_t *>(p + 4 * i) = static_cast<uint16_t>(w[i]);
                if (4u * i + 2u < bytes)
                    *reinterpret_cast<uint16_t *>(p + 4 * i + 2) = static_cast<uint16_t>(w[i] >> 16);
            }
        }
    }
    // The warp's vectors together (lane l's is vector v of the row, v - l a multiple
    // of 32), narrow pieces dealt to the lanes in turn: every access of the warp is
    // one run of bytes.  Piece i of vector v is then at piece_at(v, i); LB == VB is
    // vector v itself.  Zeros past the row's `bytes`.
    template <int LB>
    static __device__ __forceinline__ long long piece_at(unsigned v, int i)
    {
        return static_cast<long long>(v & ~31u) * VB + (i * 32 + static_cast<int>(v & 31u)) * LB;
    }
    template <int LB>
    __device__ __forceinline__ void load_dealt(const char *row, unsigned v, long long bytes)
    {
        if constexpr (LB == VB) {
            load<LB>(row + static_cast<long long>(v) * VB, VB);
        } else {
#pragma unroll
            for (int i = 0; i < VB / LB; ++i) {
                const long long at = piece_at<LB>(v, i);
                const bool in = at < bytes;
                if constexpr (LB == 8) {
                    uint2 x = make_uint2(0u, 0u);
                    if (in) x = *reinterpret_cast<const uint2 *>(row + at);
                    w[2 * i] = x.x;
                    w[2 * i + 1] = x.y;
                } else if constexpr (LB == 4) {
                    w[i] = in ? *reinterpret_cast<const uint32_t *>(row + at) : 0u;
                } else {
                    const uint32_t x = in ? *reinterpret_cast<const uint16_t *>(row + at) : 0u;
                    w[i / 2] = i % 2 ? w[i / 2] | x << 16 : x;
                }
            }
        }
    }
    template <int LB>
    __device__ __forceinline__ void store_dealt(char *row, unsigned v, long long bytes) const
    {
        if constexpr (LB == VB) {
            store<LB>(row + static_cast<long long>(v) * VB, VB);
        } else {
#pragma unroll
            for (int i = 0; i < VB / LB; ++i) {
                const long long at = piece_at<LB>(v, i);
                if (at >= bytes) continue;
                if constexpr (LB == 8)
                    *reinterpret_cast<uint2 *>(row + at) = make_uint2(w[2 * i], w[2 * i + 1]);
                else if constexpr (LB == 4)
                    *reinterpret_cast<uint32_t *>(row + at) = w[i];
                else
                    *reinterpret_cast<uint16_t *>(row + at) =
                        static_cast<uint16_t>(i % 2 ? w[i / 2] >> 16 : w[i / 2]);
            }
        }
    }
    // From here on unpacked anew: keeps the compiler from holding the values as
    // floats, twice the registers, over a wait.
    __device__ __forceinline__ void forget()
    {
#pragma unroll
        for (int i = 0; i < VB / 4; ++i) asm volatile("" : "+r"(w[i]));
    }
    __device__ __forceinline__ void unpack(float (&f)[N]) const
    {
#pragma unroll
        for (int i = 0; i < VB / 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(w[i]);
            } else if constexpr (std::is_same<T, __half>::value) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            } else {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
    __device__ __forceinline__ void pack(const float (&f)[N])
    {
#pragma unroll
        for (int i = 0; i < VB / 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                w[i] = __float_as_uint(f[i]);
            } else if constexpr (std::is_same<T, __half>::value) {
                const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&v);
            } else {
                const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&v);
            }
        }
    }
};

// Vectors of VB bytes that a thread moves at a time: up to 16 bytes, at most
// four.
template <int VB>
constexpr int kAhead = VB < 8 ? 4 : 16 / VB;

inline int elem_size(int type) { return type == SGEMM_TYPE_FP32 ? 4 : 2; }
inline bool valid_type(int type)
{
    return type == SGEMM_TYPE_BF16 || type == SGEMM_TYPE_FP16 || type == SGEMM_TYPE_FP32;
}
inline bool aligned_to(const void *p, int bytes)
{
    return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0;
}

// The widest access (16, 8, 4 or 2 bytes, at least one value) that every
// address and byte count of a call is a multiple of: feed it each base, row
// pitch and row length.
struct Width {
    uint64_t bits = 16;
    Width &add(uint64_t x)
    {
        bits |= x;
        return *this;
    }
    Width &add(const void *p) { return add(static_cast<uint64_t>(reinterpret_cast<uintptr_t>(p))); }
    int bytes() const { return static_cast<int>(bits & (~bits + 1)); }  // lowest set bit, <= 16
};

// Calls f with the row type and the vector width as template arguments
// (f.template run<T, VB>()).
template <class F>
int with_vec(int type, int vb, const F &f)
{
    if (type == SGEMM_TYPE_FP32) {
        if (vb == 16) return f.template run<float, 16>();
        if (vb == 8) return f.template run<float, 8>();
        return f.template run<float, 4>();
    }
    if (type == SGEMM_TYPE_BF16) {
        if (vb == 16) return f.template run<__nv_bfloat16, 16>();
        if (vb == 8) return f.template run<__nv_bfloat16, 8>();
        if (vb == 4) return f.template run<__nv_bfloat16, 4>();
        return f.template run<__nv_bfloat16, 2>();
    }
    if (vb == 16) return f.template run<__half, 16>();
    if (vb == 8) return f.template run<__half, 8>();
    if (vb == 4) return f.template run<__half, 4>();
    return f.template run<__half, 2>();
}

// Smallest power of two >= n, clamped to [lo, hi] (powers of two).
inline int pow2_threads(long long n, int lo, int hi)
{
    int t = lo;
    while (t < hi && t < n) t *= 2;
    return t;
}

}  // namespace rows
}  // namespace sg

// rows.cuh -- rows of bf16, fp16 or fp32 values moved in vectors of 2 to 16
// bytes, and the host-side choice of the vector: shared by the row kernels
// (experts.cu, quant.cu); the expert operators' limits.
#pragma once

#include <cstdint>
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

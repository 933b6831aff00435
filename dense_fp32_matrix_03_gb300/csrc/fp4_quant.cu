// fp4_quant.cu -- rows quantised to 4-bit floating point with a scale for each
// block of values, plain or of the gated activation (include/fp4_gemm.h).
//
// One pass, as the 8-bit quantiser (quant.cu): a row's values are held in
// registers between the row's maximum and the rounding.  A block of 16 or 32
// values spans two to eight lanes, which find its maximum by shuffles.
//
// Bound by instructions, not HBM: some 25 a value, among them NV's division for
// every block.  Measured on GB300, bf16: 8192 x 4096 22.4 us (NV; its bytes take
// 12.6) and 20.1 (MX), gated 43.7 (43.1), one row 1.8.
#include "../../include/fp4_gemm.h"
#include "dependent.cuh"
#include "fp4.cuh"
#include "rows.cuh"

namespace sg {
namespace fp4 {

using rows::Words;

constexpr int kHeld = 4;  // vectors per thread kept in registers

struct QuantArgs {
    int M, K;
    unsigned nvec;
    const char *x;
    long long x_pitch;  // bytes
    long long up;       // SwiGLU: bytes from the gates to the values
    unsigned char *q;
    long long q_pitch;  // bytes
    unsigned char *sf;
    long long tiles;
    float *scale;
};

// silu(x) = x / (1 + exp(-x)), by t = exp(-|x|): the divisor is 1 to 2, where the
// fast division holds to 2 units in the last place (it gives 0 for divisors beyond
// 2^126), and exp never leaves the range, so that the value is right down to where
// t is subnormal (|x| > 87: off by 2^-148 |x|, 2^-141 at most).  exp is the accurate one:
// the fast one is off by 2^-18 at 30, 2^-17 at 85.  In all within 8 units of
// fp32's last place.  An infinity or NaN of x gives one.  Gated 8192 x 4096 bf16
// 43.8 us (by the fast exponential 40, by x / (1 + expf(-x)) 53).
__device__ __forceinline__ float silu(float x)
{
    const float t = expf(-fabsf(x));
    return __fdividef(x < 0.f ? x * t : x, 1.f + t);
}

// One vector of the values to quantise, in fp32 (past the row: zeros).
template <class T, int VB, int LB, bool GATED>
__device__ __forceinline__ void load_values(const QuantArgs &a, const char *row, unsigned v,
                                            float (&f)[Words<T, VB>::N])
{
    constexpr unsigned EV = Words<T, VB>::N;
    const unsigned left =
        min(static_cast<unsigned>(a.K) - v * EV, EV) * static_cast<unsigned>(sizeof(T));
    Words<T, VB> g;
    g.template load<LB>(row + static_cast<long long>(v) * VB, left);
    g.unpack(f);
    if constexpr (GATED) {
        Words<T, VB> u;
        u.template load<LB>(row + a.up + static_cast<long long>(v) * VB, left);
        float h[EV];
        u.unpack(h);
#pragma unroll
        for (int i = 0; i < static_cast<int>(EV); ++i)
            f[i] = silu(f[i]) * h[i];
    }
}

// A vector of values kept until the maximum is known: as loaded, or, gated,
// as computed.
template <class T, int VB, int LB, bool GATED>
struct Held {
    static constexpr int EV = Words<T, VB>::N;
    Words<T, VB> w;
    __device__ __forceinline__ void zero() { w.zero(); }
    __device__ __forceinline__ void load(const QuantArgs &a, const char *row, unsigned v)
    {
        w.template load<LB>(row + static_cast<long long>(v) * VB,
                            min(static_cast<unsigned>(a.K) - v * EV, static_cast<unsigned>(EV)) *
                                static_cast<unsigned>(sizeof(T)));
    }
    __device__ __forceinline__ void get(float (&f)[EV]) const { w.unpack(f); }
    __device__ __forceinline__ void forget() { w.forget(); }
};
template <class T, int VB, int LB>
struct Held<T, VB, LB, true> {
    static constexpr int EV = Words<T, VB>::N;
    float f_[EV];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < EV; ++i) f_[i] = 0.f;
    }
    __device__ __forceinline__ void load(const QuantArgs &a, const char *row, unsigned v)
    {
        load_values<T, VB, LB, true>(a, row, v, f_);
    }
    __device__ __forceinline__ void get(float (&f)[EV]) const
    {
#pragma unroll
        for (int i = 0; i < EV; ++i) f[i] = f_[i];
    }
    __device__ __forceinline__ void forget() {}
};

template <class T, int VB, int LB, bool GATED, int FORMAT>
__global__ void __launch_bounds__(256, 4) quantize_kernel(const QuantArgs a)
{
    constexpr int EV = Words<T, VB>::N;
    __shared__ unsigned part[8];
    dependent_release();
    dependent_wait();
    const long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = r < a.M;
    const char *row = a.x + (live ? r : 0) * a.x_pitch;
    const unsigned tx = threadIdx.x, nx = blockDim.x, warps = nx >> 5;
    const unsigned nvec = live ? a.nvec : 0;

    Held<T, VB, LB, GATED> held[kHeld];
    unsigned big = 0;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        held[h].zero();
        if (tx + h * nx < nvec) held[h].load(a, row, tx + h * nx);
    }
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        float f[EV];
        held[h].get(f);
#pragma unroll
        for (int i = 0; i < EV; ++i) big = max(big, __float_as_uint(f[i]) & 0x7FFFFFFFu);
        held[h].forget();
    }
    for (unsigned v = tx + kHeld * nx; v < nvec; v += nx) {
        float f[EV];
        load_values<T, VB, LB, GATED>(a, row, v, f);
#pragma unroll
        for (int i = 0; i < EV; ++i) big = max(big, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    }
    big = __reduce_max_sync(0xffffffffu, big);
    if (warps > 1) {
        if ((tx & 31) == 0) part[threadIdx.y * warps + (tx >> 5)] = big;
        __syncthreads();
        for (unsigned w = 0; w < warps; ++w) big = max(big, part[threadIdx.y * warps + w]);
    }
    if (!live) return;
    const RowScale rs = row_scale(FORMAT, big);
    unsigned char *q = a.q + r * a.q_pitch, *sf = a.sf + scale_row(r, a.tiles);
    // (every lane of a warp that has a vector: blocks span lanes)
    const unsigned w0 = tx & ~31u;
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
        if (w0 + h * nx < nvec) {
            float f[EV];
            held[h].get(f);
            store_vectors<FORMAT>(f, tx + h * nx, nvec, rs, q, sf);
        }
    for (unsigned v = tx + kHeld * nx; (v & ~31u) < nvec; v += nx) {
        float f[EV] = {};
        if (v < nvec) load_values<T, VB, LB, GATED>(a, row, v, f);
        store_vectors<FORMAT>(f, v, nvec, rs, q, sf);
    }
    if (tx == 0) a.scale[r] = rs.scale;
}

struct QuantLaunch {
    const QuantArgs &args;
    bool gated;
    int format, num_sms;
    cudaStream_t st;
    template <class T, int LB, bool GATED, int FORMAT>
    int go() const
    {
        // at least four values a vector: narrower loads make one up
        constexpr int V4 = 4 * static_cast<int>(sizeof(T)), VB = LB > V4 ? LB : V4;
        constexpr int EV = Words<T, VB>::N;
        QuantArgs a = args;
        a.nvec = a.K > 0 ? (static_cast<unsigned>(a.K) - 1) / EV + 1 : 0;
        const int held = a.M <= num_sms ? 1 : kHeld;  // few rows: more threads on each
        const int tx = rows::pow2_threads((a.nvec + held - 1) / held, 32, 256), ty = 256 / tx;
        const dim3 block(static_cast<unsigned>(tx), static_cast<unsigned>(ty));
        const dim3 grid(static_cast<unsigned>((static_cast<long long>(a.M) + ty - 1) / ty));
        return launch_dependent(quantize_kernel<T, VB, LB, GATED, FORMAT>, grid, block, 0, 1, st,
                                a);
    }
    template <class T, int LB>
    int run() const
    {
        if (format == SGEMM_FP4_MX)
            return gated ? go<T, LB, true, SGEMM_FP4_MX>() : go<T, LB, false, SGEMM_FP4_MX>();
        return gated ? go<T, LB, true, SGEMM_FP4_NV>() : go<T, LB, false, SGEMM_FP4_NV>();
    }
};

}  // namespace fp4
}  // namespace sg

using namespace sg;

extern "C" {

size_t sgemm_fp4_scales_size(int format, int rows, int K)
{
    if (!fp4::valid_format(format) || rows < 0 || K < 0) return 0;
    return (static_cast<size_t>(rows) + fp4::kTileRows - 1) / fp4::kTileRows *
           static_cast<size_t>(fp4::scale_tiles(format, K)) * fp4::kTileBytes;
}

int sgemm_fp4_quantize_rows(int type, int act, int format, int M, int K, const void *X, int ldx,
                            unsigned char *Q, int ldq, unsigned char *sf, float *scale,
                            void *stream)
{
    return c_entry([&]() -> int {
        const bool gated = act == SGEMM_ACT_SWIGLU;
        if (!rows::valid_type(type) || (act != SGEMM_ACT_NONE && !gated) ||
            !fp4::valid_format(format) || M < 0 || K < 0 || ldx < 1 || ldq < 1 ||
            ldx < (gated ? 2LL * K : K) || ldq < K || ldq % fp4::kLdStep != 0)
            return SGEMM_ERR_INVALID_ARG;
        if (M == 0) return SGEMM_OK;
        const long long es = rows::elem_size(type);
        if (scale == nullptr || !rows::aligned_to(scale, 4) || !rows::aligned_to(Q, 16) ||
            !rows::aligned_to(sf, 16) || !rows::aligned_to(X, static_cast<int>(es)))
            return SGEMM_ERR_INVALID_ARG;
        if (K > 0 && (X == nullptr || Q == nullptr || sf == nullptr)) return SGEMM_ERR_INVALID_ARG;
        int num_sms = 0;
        unsigned int *status = nullptr;
        if (!current_sm103(&num_sms, &status)) return SGEMM_ERR_UNSUPPORTED;
        fp4::QuantArgs a{};
        a.M = M;
        a.K = K;
        a.x = static_cast<const char *>(X);
        a.x_pitch = ldx * es;
        a.up = K * es;
        a.q = Q;
        a.q_pitch = ldq / 2;
        a.sf = sf;
        a.tiles = fp4::scale_tiles(format, K);
        a.scale = scale;
        const int vb = K == 0 ? 16 : rows::Width().add(X).add(a.x_pitch).add(a.up).bytes();
        return rows::with_vec(type, vb, fp4::QuantLaunch{a, gated, format, num_sms,
                                                         static_cast<cudaStream_t>(stream)});
    });
}

}  // extern "C"

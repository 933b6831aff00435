// quant.cu -- rows quantised to 8-bit integers with one scale each
// (include/int8_gemm.h), plain, of the gated activation, or copied into
// expert order on the way (include/expert_layer.h).
//
// One pass: a row's values are held in registers between the maximum and the
// rounding, so each is read once and its code written once (a row longer
// than the block's registers reads its tail a second time, from L2).  The
// maximum is taken on the bit patterns of the magnitudes, where an infinity
// or NaN is larger than every finite value and so cannot be missed.
//
// Bound by HBM, with loads, reduction and stores of a row in sequence: four
// vectors a thread on blocks of at most 48 registers (five a multiprocessor)
// keep enough rows in flight.  Measured on GB300, bf16: 8192 x 4096 20.7 us
// (4.9 TB/s; with two or eight vectors a thread 22.5 and 21.0), 8192 x 8192 38 us
// (5.3), 65536 rows of 4096 in expert order from 8192 tokens 55 us (6.1), one
// row of 4096 1.5 us; fp32 8192 x 4096 27.8 us (6.0), 8192 x 8192 67 (5.0: half
// of a row is read a second time).
//
// Of the gated activation: 8192 x 4096 bf16 57 us (2.9 TB/s, 2.3 times its bytes'
// time), fp32 70 (4.3), 8192 x 4095 bf16 70, 65536 x 768 bf16 84 (3.0), one row of
// 4096 3.5 us.  An expf and an IEEE division a value, and values held in fp32 at
// three blocks a multiprocessor, keep it off the memory's rate.
//
// Rows off 16 bytes are loaded in pieces of what their alignment allows, into
// vectors of at least four values whose codes go out as one word: codes stored
// one by one cost more than the loads (one value / four values at a time, bf16:
// 8192 x 4095 80 / 30 us, 8192 x 4094 42 / 30, 32768 rows of 2001 in expert
// order from 8192 tokens 69 / 31, one row of 4095 3.9 / 1.6).
#include "../../include/expert_layer.h"
#include "dependent.cuh"
#include "rows.cuh"

namespace sg {
namespace qz {

using rows::Vec;

constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100
constexpr float kRound = 12582912.f;             // 1.5 * 2^23
constexpr int kHeld = 4;                         // vectors per thread kept in registers

struct Args {
    int M, K;               // rows, values (codes) per row
    unsigned nvec;          // vectors per row (unsigned: an index past the end of the longest
                            // row by a stride must not wrap below it)
    const char *x;
    long long x_pitch;      // bytes
    long long up;           // SwiGLU: bytes from the gates to the values
    signed char *q;
    long long ldq;
    float *scale;
    // expert order: row t goes to positions[t * k + j] for every j
    const int *positions, *total;
    int k, S;
};

// The low bytes of the first n of EV integers, as one access where QV says
// that q allows it and all are stored.
template <int EV, bool QV>
__device__ __forceinline__ void store_codes(signed char *p, const int (&c)[EV], int n)
{
    if (QV && n == EV) {
        uint32_t w[(EV + 3) / 4] = {};  // the low bytes side by side
        if constexpr (EV >= 4) {
#pragma unroll
            for (int i = 0; i < EV / 4; ++i)
                w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040),
                                   __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
        } else {
            w[0] = __byte_perm(c[0], c[1], 0x0040);
        }
        if constexpr (EV == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else if constexpr (EV == 4)
            *reinterpret_cast<uint32_t *>(p) = w[0];
        else
            *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(w[0]);
    } else {
#pragma unroll
        for (int i = 0; i < EV; ++i)
            if (i < n) p[i] = static_cast<signed char>(c[i]);
    }
}

// Bytes of the row from vector v on, as far as a vector goes.
template <class T, int VB>
__device__ __forceinline__ unsigned bytes_left(const Args &a, unsigned v)
{
    constexpr unsigned EV = Vec<T, VB>::N;
    return min(static_cast<unsigned>(a.K) - v * EV, EV) * static_cast<unsigned>(sizeof(T));
}

// One vector of the values to quantise, in fp32 (past the row: zeros).
template <class T, int VB, int LB, bool GATED>
__device__ __forceinline__ void load_values(const Args &a, const char *row, unsigned v,
                                            float (&f)[Vec<T, VB>::N])
{
    const unsigned left = bytes_left<T, VB>(a, v);
    Vec<T, VB> g;
    g.template load_pieces<LB>(row + static_cast<long long>(v) * VB, left);
    if constexpr (GATED) {
        Vec<T, VB> u;
        u.template load_pieces<LB>(row + a.up + static_cast<long long>(v) * VB, left);
#pragma unroll
        for (int i = 0; i < Vec<T, VB>::N; ++i) {
            const float x = g.get(i);
            f[i] = x / (1.f + expf(-x)) * u.get(i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < Vec<T, VB>::N; ++i) f[i] = g.get(i);
    }
}

// A vector of values kept until the maximum is known: as loaded, or, gated,
// as computed.
template <class T, int VB, int LB, bool GATED>
struct Held {
    Vec<T, VB> v;
    __device__ __forceinline__ void load(const Args &a, const char *row, unsigned i)
    {
        v.template load_pieces<LB>(row + static_cast<long long>(i) * VB, bytes_left<T, VB>(a, i));
    }
    __device__ __forceinline__ float get(int i) const { return v.get(i); }
};
template <class T, int VB, int LB>
struct Held<T, VB, LB, true> {
    float f[Vec<T, VB>::N];
    __device__ __forceinline__ void load(const Args &a, const char *row, unsigned i)
    {
        load_values<T, VB, LB, true>(a, row, i, f);
    }
    __device__ __forceinline__ float get(int i) const { return f[i]; }
};

template <class T, int VB, int LB, bool GATED, bool EXPERT, bool QV>
__global__ void __launch_bounds__(256, GATED ? 3 : 5) quantize_kernel(const Args a)
{
    constexpr int EV = Vec<T, VB>::N;
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
        const unsigned v = tx + h * nx;
        if (v < nvec) held[h].load(a, row, v);
    }
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
        if (tx + h * nx < nvec)
#pragma unroll
            for (int i = 0; i < EV; ++i)
                big = max(big, __float_as_uint(held[h].get(i)) & 0x7FFFFFFFu);
    for (unsigned v = tx + kHeld * nx; v < nvec; v += nx) {
        float g[EV];
        load_values<T, VB, LB, GATED>(a, row, v, g);
#pragma unroll
        for (int i = 0; i < EV; ++i) big = max(big, __float_as_uint(g[i]) & 0x7FFFFFFFu);
    }
    big = __reduce_max_sync(0xffffffffu, big);
    if (warps > 1) {
        if ((tx & 31) == 0) part[threadIdx.y * warps + (tx >> 5)] = big;
        __syncthreads();
        for (unsigned w = 0; w < warps; ++w) big = max(big, part[threadIdx.y * warps + w]);
    }
    if (!live) return;
    const float amax = __uint_as_float(big);
    const bool finite = big < 0x7F800000u, some = amax >= kTiny;
    const float inv = finite && some ? __fdiv_rn(127.f, amax) : 0.f;
    const float scale = !finite ? __int_as_float(0x7FFFFFFF)
                                : (some ? __fdiv_rn(amax, 127.f) : 0.f);

    // The nearest integer, ties to even, is in the low bits after 1.5 * 2^23 is
    // added (a conversion instruction has a quarter of the rate).
    auto codes = [&](const float (&x)[EV], int (&c)[EV]) {
#pragma unroll
        for (int i = 0; i < EV; ++i)
            c[i] = finite ? __float_as_int(__fadd_rn(__fmul_rn(x[i], inv), kRound)) : 0;
    };
    auto put = [&](unsigned v, const int (&c)[EV]) {
        const int n = LB == VB ? EV
                               : static_cast<int>(bytes_left<T, VB>(a, v) / sizeof(T));
        if constexpr (EXPERT) {
            const int total = *a.total;
            int none[EV] = {};
            for (int j = 0; j < a.k; ++j) {
                const int p = a.positions[r * a.k + j];
                if (p < 0 || p >= a.S) continue;
                signed char *dst = a.q + p * a.ldq + static_cast<long long>(v) * EV;
                if (p < total)
                    store_codes<EV, QV>(dst, c, n);
                else
                    store_codes<EV, QV>(dst, none, n);
            }
        } else {
            store_codes<EV, QV>(a.q + r * a.ldq + static_cast<long long>(v) * EV, c, n);
        }
    };
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        const unsigned v = tx + h * nx;
        if (v < nvec) {
            float f[EV];
            int c[EV];
#pragma unroll
            for (int i = 0; i < EV; ++i) f[i] = held[h].get(i);
            codes(f, c);
            put(v, c);
        }
    }
    for (unsigned v = tx + kHeld * nx; v < nvec; v += nx) {
        float g[EV];
        int c[EV];
        load_values<T, VB, LB, GATED>(a, row, v, g);
        codes(g, c);
        put(v, c);
    }
    if constexpr (EXPERT) {
        for (int j = tx; j < a.k; j += nx) {
            const int p = a.positions[r * a.k + j];
            if (p >= 0 && p < a.S) a.scale[p] = p < *a.total ? scale : 0.f;
        }
    } else {
        if (tx == 0) a.scale[r] = scale;
    }
}

struct Launch {
    const Args &args;
    bool gated, expert;
    cudaStream_t st;
    template <class T, int LB, bool GATED, bool EXPERT>
    int go() const
    {
        // at least four values a vector: narrower loads make one up
        constexpr int V4 = 4 * static_cast<int>(sizeof(T)), VB = LB > V4 ? LB : V4;
        constexpr int EV = Vec<T, VB>::N;
        Args a = args;
        a.nvec = a.K > 0 ? (static_cast<unsigned>(a.K) - 1) / EV + 1 : 0;
        const bool qv = rows::aligned_to(a.q, EV) && a.ldq % EV == 0;
        const int tx = rows::pow2_threads((a.nvec + kHeld - 1) / kHeld, 32, 256), ty = 256 / tx;
        const dim3 block(static_cast<unsigned>(tx), static_cast<unsigned>(ty));
        const dim3 grid(static_cast<unsigned>((static_cast<long long>(a.M) + ty - 1) / ty));
        auto kern = qv ? quantize_kernel<T, VB, LB, GATED, EXPERT, true>
                       : quantize_kernel<T, VB, LB, GATED, EXPERT, false>;
        return launch_dependent(kern, grid, block, 0, 1, st, a);
    }
    template <class T, int LB>
    int run() const
    {
        if (expert) return go<T, LB, false, true>();
        return gated ? go<T, LB, true, false>() : go<T, LB, false, false>();
    }
};

}  // namespace qz
}  // namespace sg

using namespace sg;

extern "C" {

int sgemm_i8_quantize_rows(int type, int act, int M, int K, const void *X, int ldx,
                           signed char *Q, int ldq, float *scale, void *stream)
{
    return c_entry([&]() -> int {
        const bool gated = act == SGEMM_ACT_SWIGLU;
        if (!rows::valid_type(type) || (act != SGEMM_ACT_NONE && !gated) || M < 0 || K < 0 ||
            ldx < 1 || ldq < 1 || ldx < (gated ? 2LL * K : K) || ldq < K)
            return SGEMM_ERR_INVALID_ARG;
        if (M == 0) return SGEMM_OK;
        const long long es = rows::elem_size(type);
        if (scale == nullptr || !rows::aligned_to(scale, 4)) return SGEMM_ERR_INVALID_ARG;
        if (K > 0 && (X == nullptr || Q == nullptr || !rows::aligned_to(X, static_cast<int>(es))))
            return SGEMM_ERR_INVALID_ARG;
        int num_sms = 0;
        unsigned int *status = nullptr;
        if (!current_sm103(&num_sms, &status)) return SGEMM_ERR_UNSUPPORTED;
        qz::Args a{};
        a.M = M;
        a.K = K;
        a.x = static_cast<const char *>(X);
        a.x_pitch = ldx * es;
        a.up = K * es;
        a.q = Q;
        a.ldq = ldq;
        a.scale = scale;
        const int vb = K == 0 ? 16 : rows::Width().add(X).add(a.x_pitch).add(a.up).bytes();
        return rows::with_vec(type, vb,
                              qz::Launch{a, gated, false, static_cast<cudaStream_t>(stream)});
    });
}

int sgemm_experts_dispatch_i8(int type, int T, int k, int E, int H, const void *x, int ldx,
                              const int *positions, const int *offsets, signed char *q, int ldq,
                              float *scale, void *stream)
{
    return c_entry([&]() -> int {
        if (!rows::valid_type(type) || !choices_ok(T, k, E) || H < 0 || ldx < 1 || ldq < 1 ||
            ldx < H || ldq < H)
            return SGEMM_ERR_INVALID_ARG;
        if (T == 0) return SGEMM_OK;
        const long long es = rows::elem_size(type);
        if (positions == nullptr || offsets == nullptr || scale == nullptr ||
            !rows::aligned_to(positions, 4) || !rows::aligned_to(offsets, 4) ||
            !rows::aligned_to(scale, 4))
            return SGEMM_ERR_INVALID_ARG;
        if (H > 0 && (x == nullptr || q == nullptr || !rows::aligned_to(x, static_cast<int>(es))))
            return SGEMM_ERR_INVALID_ARG;
        int num_sms = 0;
        unsigned int *status = nullptr;
        if (!current_sm103(&num_sms, &status)) return SGEMM_ERR_UNSUPPORTED;
        qz::Args a{};
        a.M = T;
        a.K = H;
        a.x = static_cast<const char *>(x);
        a.x_pitch = ldx * es;
        a.q = q;
        a.ldq = ldq;
        a.scale = scale;
        a.positions = positions;
        a.total = offsets + E;
        a.k = k;
        a.S = T * k;
        const int vb = H == 0 ? 16 : rows::Width().add(x).add(a.x_pitch).add(H * es).bytes();
        return rows::with_vec(type, vb,
                              qz::Launch{a, false, true, static_cast<cudaStream_t>(stream)});
    });
}

}  // extern "C"

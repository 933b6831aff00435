// fp4_gemm.cu -- products in microscaled 4-bit floating point
// (include/fp4_gemm.h): argument checks and kernels.
#include "../../include/fp4_gemm.h"
#include "dependent.cuh"
#include "fp4.cuh"
#include "rows.cuh"

namespace sg {
namespace fp4 {

constexpr int kMaxSide = 0x7FFFFFFF - 511;  // an index a tile past the last row or channel still is an int

struct Args {
    int M, N, K;
    const unsigned char *A, *sfA, *B, *sfB;
    long long lda, ldb;  // bytes
    long long tiles;     // of block scales, per row
    const float *scaleA, *scaleB;
    void *C;
    long long ldc;
    unsigned int *status;
    int num_sms;
};

// ------------------------------------------------------------ plain kernel
//
// C tiles of 64 x 64 by 256 threads, 4 x 4 each, over steps of 32 k decoded to
// fp32 in shared memory.
constexpr int kPT = 64, kPK = 32;

__device__ __forceinline__ float decode(unsigned code)
{
    const float m[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
    const float v = m[code & 7];
    return code & 8 ? -v : v;
}

template <int FORMAT>
__device__ __forceinline__ float block_scale(const unsigned char *sf, long long row,
                                             long long tiles, int block)
{
    const unsigned b = sf[scale_row(row, tiles) + static_cast<long long>(block / 4) * kTileBytes +
                          block % 4];
    if (FORMAT == SGEMM_FP4_MX)
        return b == 255u ? __int_as_float(0x7FFFFFFF)
                         : (b == 0u ? 5.877471754111438e-39f : __uint_as_float(b << 23));
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b),
                                                       __NV_E4M3)));
}

template <class T, int FORMAT>
__global__ void __launch_bounds__(256) plain_kernel(const Args a)
{
    __shared__ float As[kPK][kPT + 1], Bs[kPK][kPT + 1];
    dependent_release();
    dependent_wait();
    const int tid = threadIdx.x;
    const long long m0 = static_cast<long long>(blockIdx.y) * kPT;
    const long long n0 = static_cast<long long>(blockIdx.x) * kPT;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kPK) {
        for (int i = tid; i < kPT * kPK; i += 256) {
            const int r = i / kPK, c = i % kPK, k = k0 + c;
            float x = 0.f, y = 0.f;
            if (k < a.K && m0 + r < a.M)
                x = decode(a.A[(m0 + r) * a.lda + k / 2] >> (k % 2 * 4)) *
                    block_scale<FORMAT>(a.sfA, m0 + r, a.tiles, k / block_of(FORMAT));
            if (k < a.K && n0 + r < a.N)
                y = decode(a.B[(n0 + r) * a.ldb + k / 2] >> (k % 2 * 4)) *
                    block_scale<FORMAT>(a.sfB, n0 + r, a.tiles, k / block_of(FORMAT));
            As[c][r] = x;
            Bs[c][r] = y;
        }
        __syncthreads();
        for (int k = 0; k < kPK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(As[k][tid / 16 + 16 * i], Bs[k][tid % 16 + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long m = m0 + tid / 16 + 16 * i, n = n0 + tid % 16 + 16 * j;
            if (m >= a.M || n >= a.N) continue;
            const float sa = a.scaleA != nullptr ? a.scaleA[m] : 1.f;
            const float sb = a.scaleB != nullptr ? a.scaleB[n] : 1.f;
            static_cast<T *>(a.C)[m * a.ldc + n] = rows::from_f<T>(acc[i][j] * sa * sb);
        }
}

template <class T>
int run(const Args &a, int format, cudaStream_t st)
{
    const dim3 grid(static_cast<unsigned>((a.N + kPT - 1LL) / kPT),
                    static_cast<unsigned>((a.M + kPT - 1LL) / kPT));
    return launch_dependent(format == SGEMM_FP4_MX ? plain_kernel<T, SGEMM_FP4_MX>
                                                   : plain_kernel<T, SGEMM_FP4_NV>,
                            grid, dim3(256), 0, 1, st, a);
}

}  // namespace fp4
}  // namespace sg

using namespace sg;

extern "C" int sgemm_fp4(int type, int format, int M, int N, int K, const unsigned char *A,
                         int lda, const unsigned char *sfA, const float *scaleA,
                         const unsigned char *B, int ldb, const unsigned char *sfB,
                         const float *scaleB, void *C, int ldc, void *stream)
{
    return c_entry([&]() -> int {
        if (!rows::valid_type(type) || !fp4::valid_format(format) || M < 0 || N < 0 || K < 0 ||
            lda < 1 || ldb < 1 || ldc < 1 || lda < K || ldb < K || ldc < N ||
            lda % fp4::kLdStep != 0 || ldb % fp4::kLdStep != 0 || M > fp4::kMaxSide ||
            N > fp4::kMaxSide)
            return SGEMM_ERR_INVALID_ARG;
        if (M == 0 || N == 0) return SGEMM_OK;
        if (C == nullptr || !rows::aligned_to(C, rows::elem_size(type)) ||
            !rows::aligned_to(scaleA, 4) || !rows::aligned_to(scaleB, 4) ||
            !rows::aligned_to(A, 16) || !rows::aligned_to(B, 16) || !rows::aligned_to(sfA, 16) ||
            !rows::aligned_to(sfB, 16))
            return SGEMM_ERR_INVALID_ARG;
        if (K > 0 && (A == nullptr || B == nullptr || sfA == nullptr || sfB == nullptr))
            return SGEMM_ERR_INVALID_ARG;
        fp4::Args a{};
        if (!current_sm103(&a.num_sms, &a.status)) return SGEMM_ERR_UNSUPPORTED;
        a.M = M;
        a.N = N;
        a.K = K;
        a.A = A;
        a.sfA = sfA;
        a.B = B;
        a.sfB = sfB;
        a.lda = lda / 2;
        a.ldb = ldb / 2;
        a.tiles = fp4::scale_tiles(format, K);
        a.scaleA = scaleA;
        a.scaleB = scaleB;
        a.C = C;
        a.ldc = ldc;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        if (type == SGEMM_TYPE_BF16) return fp4::run<__nv_bfloat16>(a, format, st);
        if (type == SGEMM_TYPE_FP16) return fp4::run<__half>(a, format, st);
        return fp4::run<float>(a, format, st);
    });
}

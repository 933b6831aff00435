// fp4_gemm.cu -- products in microscaled 4-bit floating point
// (include/fp4_gemm.h): argument checks and kernels.
#include <atomic>

#include "../../include/fp4_gemm.h"
#include "dependent.cuh"
#include "fp4.cuh"
#include "fp4_few.cuh"
#include "fp4_tc.cuh"
#include "rows.cuh"

namespace sg {
namespace fp4 {

constexpr int kMaxSide = 0x7FFFFFFF - 511;  // an index a tile past the last row or channel still is an int
constexpr int kMaxK = 0x7FFFFFFF - 8191;    // and one a step of a whole block past the last value

// K == 0: zeros times the scales.
template <class T>
__global__ void __launch_bounds__(256) empty_kernel(const Args a)
{
    dependent_release();
    dependent_wait();
    const long long all = static_cast<long long>(a.M) * a.N;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < all; i += gridDim.x * 256LL) {
        const long long m = i / a.N, n = i - m * a.N;
        const float sa = a.scaleA != nullptr ? a.scaleA[m] : 1.f;
        const float sb = a.scaleB != nullptr ? a.scaleB[n] : 1.f;
        static_cast<T *>(a.C)[m * a.ldc + n] = rows::from_f<T>(0.f * sa * sb);
    }
}

// Clusters of `size` CTAs of C's kernel that the GPU runs at once: cached per
// device.  (A cluster stays within a processor group, so 152 multiprocessors hold
// fewer than 19 of 8.)
template <class C>
int room(int size, int num_sms)
{
    static std::atomic<int> known[64][4];  // sizes 1, 2, 4, 8; 0: not asked yet
    const int i = size == 1 ? 0 : size == 2 ? 1 : size == 4 ? 2 : 3;
    int dev = 0;
    if (size == 1) return num_sms;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return num_sms / size / 2;
    int n = known[dev][i].load();
    if (n == 0) {
        auto kern = fp4_kernel<C, float, SGEMM_FP4_NV>;
        if (smem_attr_once(reinterpret_cast<const void *>(kern), C::SMEM)) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(static_cast<unsigned>(num_sms / size * size));
            cfg.blockDim = dim3(C::THREADS);
            cfg.dynamicSmemBytes = C::SMEM;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = static_cast<unsigned>(size);
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) n = 0;
        }
        cudaGetLastError();
        if (n < 1) n = 1;
        known[dev][i].store(n);
    }
    return n;
}

std::atomic<int> g_force{SGEMM_FP4_KERNEL_AUTO};
std::atomic<int> g_last_kernel{SGEMM_FP4_KERNEL_AUTO}, g_last_split{1};

void note_product(int kernel, int split)
{
    g_last_kernel.store(kernel, std::memory_order_relaxed);
    g_last_split.store(split, std::memory_order_relaxed);
}

// CTAs that share a tile's k: worth their cluster (launched and met twice, 1.7 us)
// where k is long and tiles are few, and each keeps four stages or more.  us, alone /
// shared: 1 token 4096 x 1024 3.6 / 4.4, x 2048 4.8 / 4.8, x 4096 7.3 / 5.8; 48 tokens
// 2048 x 1024 3.8 / 4.7, 4096 x 4096 7.7 / 7.3, 8192 x 8192 13.5 / 11.9; the sums of
// two token tiles cost more than they save: 256 x 4096 x 4096 8.6 / 9.9.
template <class C>
int shared_k(const Args &a, long long tiles)
{
    const int stages = (a.K + kStageK - 1) / kStageK;
    int split = 1;
    if (a.M > C::NT || stages < (C::NT <= 32 ? 12 : 16)) return 1;
    while (split < 8 && tiles <= room<C>(2 * split, a.num_sms) && stages >= 8 * split) split *= 2;
    return split;
}

template <class T, int FORMAT>
int run(const Args &a, cudaStream_t st)
{
    if (a.K == 0) {
        note_product(SGEMM_FP4_KERNEL_AUTO, 1);
        return launch_dependent(empty_kernel<T>, dim3(static_cast<unsigned>(2 * a.num_sms)),
                                dim3(256), 0, 1, st, a);
    }
    const int c_bytes = rows::Width().add(a.C).add(a.ldc * sizeof(T)).bytes();
    const int stages = (a.K + kStageK - 1) / kStageK, pairs = ss_slots(a.num_sms);
    const long long cts = (a.N + kCh - 1LL) / kCh;  // channel tiles of one CTA
    const long long tiles = (a.M + Narrow::NT - 1LL) / Narrow::NT * cts;
    const bool few_can = a.M <= kFewTokens;
    // (one token tile: its scales begin with a tile of theirs)
    const bool slim_can = a.M <= Slim::NT;
    int kernel = g_force.load(std::memory_order_relaxed);
    if ((kernel == SGEMM_FP4_KERNEL_FEW && !few_can) || (kernel == SGEMM_FP4_KERNEL_SLIM && !slim_can))
        kernel = SGEMM_FP4_KERNEL_AUTO;
    int split = 1;
    if (kernel == SGEMM_FP4_KERNEL_AUTO || kernel == SGEMM_FP4_KERNEL_SLIM) {
        if (slim_can) split = shared_k<Slim>(a, cts);
        if (slim_can && kernel == SGEMM_FP4_KERNEL_AUTO) {
            kernel = SGEMM_FP4_KERNEL_SLIM;
            if (few_can) {
                // The kernels' times in us, as measured on GB300: few / slim, 1 token 1024
                // x 1024 2.8 / 3.7, 2048 x 1024 3.1 / 3.7, 2048 x 2048 3.6 / 4.8, 8192 x 512
                // 4.3 / 3.3, 4096 x 4096 8.1 / 5.8; 4 tokens 1024 x 1024 4.6 / 3.7
                const double per = a.M == 1 ? 0.33 : a.M == 2 ? 0.41 : 0.78;
                const double few = 2.4 + per * 1e-6 * a.N * a.K;
                const double waves = static_cast<double>((cts * split + a.num_sms - 1) / a.num_sms);
                const double slim = 2.5 + 0.31 * stages / split * waves + (split > 1 ? 1.7 : 0.);
                if (few < slim) kernel = SGEMM_FP4_KERNEL_FEW;
            }
        }
    }
    // us, narrow / wide: 128 x 4096 x 4096 8.2 / 9.9, 512 9.3 / 11.0, 1024 (256 tiles of the
    // narrow kernel) 14.2 / 11.5, 512 x 8192 x 8192 23.2 / 17.4, 2048 x 2048 x 1024 8.0 /
    // 7.4, 1024 x 4092 x 256 7.1 / 6.7: one wave of narrow tiles, or wide ones
    if (kernel == SGEMM_FP4_KERNEL_AUTO)
        kernel = tiles > a.num_sms ? SGEMM_FP4_KERNEL_WIDE : SGEMM_FP4_KERNEL_NARROW;
    if (kernel == SGEMM_FP4_KERNEL_NARROW) split = shared_k<Narrow>(a, tiles);
    note_product(kernel, kernel == SGEMM_FP4_KERNEL_SLIM || kernel == SGEMM_FP4_KERNEL_NARROW ? split : 1);
    switch (kernel) {
    case SGEMM_FP4_KERNEL_FEW:
        if (a.M == 1) return launch_few<T, FORMAT, 1>(a, st);
        if (a.M == 2) return launch_few<T, FORMAT, 2>(a, st);
        return launch_few<T, FORMAT, 4>(a, st);
    case SGEMM_FP4_KERNEL_SLIM:
        return launch_tc<Slim, T, FORMAT>(a, split > 1 || cts < a.num_sms ? cts : a.num_sms, split,
                                          c_bytes, st);
    case SGEMM_FP4_KERNEL_NARROW:
        return launch_tc<Narrow, T, FORMAT>(a, split > 1 || tiles < a.num_sms ? tiles : a.num_sms,
                                            split, c_bytes, st);
    default: {
        const long long wide = (a.M + Wide::NT - 1LL) / Wide::NT * ((a.N + 2LL * kCh - 1) / (2 * kCh));
        return launch_tc<Wide, T, FORMAT>(a, wide < pairs ? wide : pairs, 1, c_bytes, st);
    }
    }
}

template <class T>
int run(const Args &a, int format, cudaStream_t st)
{
    return format == SGEMM_FP4_MX ? run<T, SGEMM_FP4_MX>(a, st) : run<T, SGEMM_FP4_NV>(a, st);
}

}  // namespace fp4
}  // namespace sg

using namespace sg;

extern "C" {

int sgemm_fp4_tune_force(int kernel)
{
    if (kernel < SGEMM_FP4_KERNEL_AUTO || kernel > SGEMM_FP4_KERNEL_SLIM)
        return SGEMM_ERR_INVALID_ARG;
    fp4::g_force.store(kernel);
    return SGEMM_OK;
}

int sgemm_fp4_last_kernel(void) { return fp4::g_last_kernel.load(); }

int sgemm_fp4_last_split_count(void) { return fp4::g_last_split.load(); }

int sgemm_fp4(int type, int format, int M, int N, int K, const unsigned char *A,
                         int lda, const unsigned char *sfA, const float *scaleA,
                         const unsigned char *B, int ldb, const unsigned char *sfB,
                         const float *scaleB, void *C, int ldc, void *stream)
{
    return c_entry([&]() -> int {
        if (!rows::valid_type(type) || !fp4::valid_format(format) || M < 0 || N < 0 || K < 0 ||
            lda < 1 || ldb < 1 || ldc < 1 || lda < K || ldb < K || ldc < N ||
            lda % fp4::kLdStep != 0 || ldb % fp4::kLdStep != 0 || M > fp4::kMaxSide ||
            N > fp4::kMaxSide || K > fp4::kMaxK)
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

}  // extern "C"

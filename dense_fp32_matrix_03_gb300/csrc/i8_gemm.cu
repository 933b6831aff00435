// i8_gemm.cu -- products of 8-bit integers with a scale for each token and
// channel (include/int8_gemm.h): argument checks, the choice of the kernel
// and the integer dot-product kernel (the tensor-core one is i8_tc.cuh).
#include <atomic>
#include <cmath>
#include <cstring>

#include "../../include/int8_gemm.h"
#include "dependent.cuh"
#include "i8_few.cuh"
#include "i8_gemm.h"
#include "i8_tc.cuh"
#include "rows.cuh"

namespace sg {
namespace i8 {

// ------------------------------------------------- integer dot products
//
// C tiles of 64 tokens x 64 channels by 256 threads, 4 x 4 each, over steps
// of 64 k staged in shared memory as words of four 8-bit values (dp4a: four
// products and an exact 32-bit sum).  Any base and leading dimension: words
// are read whole where all allow it, byte by byte otherwise; bytes past K
// read as zero.  A plain kernel, bound by its loads, which nothing overlaps (us,
// by bytes / by words / the kernels for rows on 16 bytes; 4096 x 4096, 1 token
// 248 / 192 / 4.5, 16 266 / 203 / 6.4, 256 383 / 263 / 19, 1000 696 / 475 / 29;
// 8192 x 8192 x 4092 by words 6150, 317).  Weights are laid out once: rows padded
// to 16 bytes cost less than any kernel for rows that are not.
constexpr int kDT = 64, kDK = 64, kDW = kDK / 4;

template <bool WORDS>
__device__ __forceinline__ uint32_t load4(const signed char *row, int k, int K)
{
    if (k >= K) return 0u;
    if (WORDS && k + 4 <= K) return *reinterpret_cast<const uint32_t *>(row + k);
    uint32_t w = 0;
    for (int i = 0; i < 4 && k + i < K; ++i)
        w |= (static_cast<uint32_t>(row[k + i]) & 255u) << (8 * i);
    return w;
}

template <class T, bool WORDS>
__global__ void __launch_bounds__(256) dot_kernel(const Args a)
{
    __shared__ uint32_t As[kDW][kDT + 1], Bs[kDW][kDT + 1];
    __shared__ Tile tl;
    const int tid = threadIdx.x;
    dependent_release();
    dependent_wait();
    if (tid < 32) {
        const Tile t = find_tile_warp(a, blockIdx.y, kDT, tid);
        if (tid == 0) tl = t;
    }
    __syncthreads();
    if (tl.e < 0) return;
    const int n0 = blockIdx.x * kDT;
    const signed char *B = a.B + tl.e * a.strideB;
    int acc[4][4] = {};
    const int tm = (tid >> 4) * 4, tn = (tid & 15) * 4;
    for (int k0 = 0; k0 < a.K; k0 += kDK) {
        for (int i = tid; i < kDT * kDW; i += 256) {
            const int r = i / kDW, w = i % kDW;
            As[w][r] = r < tl.rows ? load4<WORDS>(a.A + (tl.row0 + r) * a.lda, k0 + 4 * w, a.K) : 0u;
            Bs[w][r] = n0 + r < a.N
                           ? load4<WORDS>(B + static_cast<long long>(n0 + r) * a.ldb, k0 + 4 * w, a.K)
                           : 0u;
        }
        __syncthreads();
#pragma unroll 4
        for (int w = 0; w < kDW; ++w) {
            int x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = static_cast<int>(As[w][tm + i]);
                y[i] = static_cast<int>(Bs[w][tn + i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(x[i], y[j], acc[i][j]);
        }
        __syncthreads();
    }
    const float *sb = a.scaleB + static_cast<long long>(tl.e) * a.N;
    for (int i = 0; i < 4; ++i) {
        if (tm + i >= tl.rows) break;
        const float sa = a.scaleA[tl.row0 + tm + i];
        T *c = static_cast<T *>(a.C) + (tl.row0 + tm + i) * a.ldc;
        for (int j = 0; j < 4; ++j)
            if (n0 + tn + j < a.N)
                c[n0 + tn + j] =
                    rows::from_f<T>(static_cast<float>(acc[i][j]) * sa * sb[n0 + tn + j]);
    }
}

template <class T>
int launch_dot(const Args &a, cudaStream_t st)
{
    const bool words = rows::aligned_to(a.A, 4) && rows::aligned_to(a.B, 4) && a.lda % 4 == 0 &&
                       a.ldb % 4 == 0 && a.strideB % 4 == 0;
    const long long gy = max_tiles(a, kDT), gx = (a.N + kDT - 1LL) / kDT;
    // grid.y holds 65535 tiles: longer calls go in pieces
    for (long long y0 = 0; y0 < gy; y0 += 65535) {
        Args b = a;
        b.tile0 = static_cast<int>(y0);
        const dim3 grid(static_cast<unsigned>(gx),
                        static_cast<unsigned>(gy - y0 < 65535 ? gy - y0 : 65535));
        const int rc = launch_dependent(words ? dot_kernel<T, true> : dot_kernel<T, false>, grid,
                                        dim3(256), 0, 1, st, b);
        if (rc != SGEMM_OK) return rc;
    }
    return SGEMM_OK;
}

// ------------------------------------------------- what a call looks like

// Whether the tensor-core kernel can read the operands: rows on 16-byte
// boundaries.
bool rows_on_16(const Args &a)
{
    return aligned16(a.A) && aligned16(a.B) && a.lda % 16 == 0 && a.ldb % 16 == 0 &&
           (a.E == 1 || a.strideB % 16 == 0);
}

// Output tiles of nt tokens x ch channels that a call is expected to have.
// Experts' counts are on the GPU: of equal ones each ends in one short tile (in
// one more where the mean is about a multiple of nt), of uneven ones in half a
// tile on average; the mean of the two.
double tiles_expected(const Args &a, int nt, int ch)
{
    const double cts = (a.N + ch - 1) / ch;
    if (a.offsets == nullptr) return (a.M + nt - 1LL) / nt * cts;
    const int used = a.E < a.M ? a.E : a.M;
    const double mean = static_cast<double>(a.M) / used / nt;
    const double uneven = mean > 0.5 ? mean + 0.5 : 1.;
    return used * 0.5 * (ceil(mean + 0.1) + uneven) * cts;
}

// Clusters of `size` CTAs of the narrow kernel that the GPU runs at once (a
// cluster stays within a processor group, so 152 multiprocessors hold fewer
// than 19 of 8): cached per device.
int narrow_room(int size, int num_sms)
{
    static std::atomic<int> room[64][4];  // sizes 1, 2, 4, 8; 0: not asked yet
    const int i = size == 1 ? 0 : size == 2 ? 1 : size == 4 ? 2 : 3;
    int dev = 0;
    if (size == 1) return num_sms;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return num_sms / size / 2;
    int n = room[dev][i].load();
    if (n == 0) {
        auto kern = i8_kernel<Narrow, float>;
        if (smem_attr_once(reinterpret_cast<const void *>(kern), Narrow::SMEM)) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(static_cast<unsigned>(num_sms / size * size));
            cfg.blockDim = dim3(Narrow::THREADS);
            cfg.dynamicSmemBytes = Narrow::SMEM;
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
        room[dev][i].store(n);
    }
    return n;
}

// ------------------------------------------------- the kernel for a call

// The kernel every later call is made to take (sgemm_i8_tune_force), and the
// kernel and split of the last product enqueued.
std::atomic<int> g_force{SGEMM_I8_KERNEL_AUTO};
std::atomic<int> g_last_kernel{SGEMM_I8_KERNEL_AUTO}, g_last_split{1};

void note_product(int kernel, int split)
{
    g_last_kernel.store(kernel, std::memory_order_relaxed);
    g_last_split.store(split, std::memory_order_relaxed);
}

// The few-token kernel's form for a dense call.
struct FewForm {
    bool once;   // blocks of 16 warps: all of them run at once, with two steps or
                 // more of k a warp (8 / 16 warps: 16 x 4096 x 4096 9.0 / 6.4,
                 // 16 x 8192 x 8192 20.7 / 21.2, 16 x 1024 x 1024 2.5 / 3.3)
    bool large;  // 32 tokens a block of 16 warps, likewise where all run at once
                 // (against the kernels chosen otherwise: 64 x 1024 x 4096 8.5 /
                 // 6.5, 64 x 1200 x 8192 12.7 / 9.1, 1024 x 64 x 4096 8.8 / 6.6,
                 // 17 x 2048 x 2048 5.7 / 5.0; with more blocks, 96 x 1024 x 4096
                 // 8.9 / 11.6; at shorter k, 64 x 1024 x 1024 3.7 / 5.3; with few
                 // blocks at that, 64 x 256 x 2048 3.2 / 4.6)
    explicit FewForm(const Args &a)
    {
        const long long blocks = (a.N + 15) / 16 * ((a.M + 31LL) / 32);
        once = a.K >= 2048 && a.N <= 2LL * a.num_sms * 16;
        large = a.M > 16 && blocks <= a.num_sms &&
                (a.K >= 4096 || (a.K >= 2048 && 4 * blocks >= a.num_sms));
    }
};

template <class T>
int launch_few_tokens(const Args &a, cudaStream_t st)
{
    if (a.offsets != nullptr) return launch_few<T, 1, 2, 4, 6>(a, st);
    const FewForm form(a);
    if (a.M <= 8)
        return form.once ? launch_few<T, 1, 1, 16, 2>(a, st) : launch_few<T, 1, 1, 8, 4>(a, st);
    if (a.M <= 16 && form.once) return launch_few<T, 2, 1, 16, 2>(a, st);
    if (form.large) return launch_few<T, 4, 1, 16, 1>(a, st);
    return launch_few<T, 2, 1, 8, 4>(a, st);
}

template <class T>
int run(const Args &a, cudaStream_t st)
{
    alignas(64) CUtensorMap tmW;
    alignas(64) CUtensorMap tmT;
    std::memset(&tmW, 0, sizeof(tmW));
    std::memset(&tmT, 0, sizeof(tmT));
    const int forced = g_force.load(std::memory_order_relaxed);
    if (a.K == 0 || !rows_on_16(a) || forced == SGEMM_I8_KERNEL_ANY_LAYOUT ||
        !encode_operand8(&tmW, a.B, a.N, a.K, a.ldb, a.E, a.strideB, kCh) ||
        !encode_operand8(&tmT, a.A, a.M, a.K, a.lda, 1, 0, kBoxRows)) {
        note_product(SGEMM_I8_KERNEL_ANY_LAYOUT, 1);
        return launch_dot<T>(a, st);
    }
    const int c_bytes = rows::Width().add(a.C).add(a.ldc * sizeof(T)).bytes();
    const int k_slots = (a.K + kSlotK - 1) / kSlotK;
    const int pairs = ss_slots(a.num_sms);
    const bool dense = a.offsets == nullptr;
    const bool dots_can = dense && a.M <= 4;
    // (a grid holds 65535 token tiles, of 8 rows by expert, of 16 or more else)
    const bool few_can = dense ? a.M <= 16 * 65535 : max_tiles(a, 8) <= 65535;
    int kernel = forced;
    if ((kernel == SGEMM_I8_KERNEL_DOTS && !dots_can) || (kernel == SGEMM_I8_KERNEL_FEW && !few_can))
        kernel = SGEMM_I8_KERNEL_AUTO;

    // The kernels' times in us, as measured on GB300 (bf16; M x N x K):
    //   few     2.9 us and a pass over the weights per 16 tokens, from HBM or
    //           L2, or the results: 17 .. 32 x 4096 x 4096 9.1, 48 13.5, 100 x
    //           1024 x 1024 4.1, 64 x 4096 x 128 5.8
    //   narrow  3.4 us (5 where a cluster's CTAs share a tile's slots, when tiles
    //           are few) and 0.8 a slot of 128 k and wave of tiles: 24 .. 64 x
    //           4096 x 4096 11.6 .. 12.6, 256 19.1, 512 25.2, 1024 45, 100 x 1024
    //           x 1024 8.4, 64 x 4096 x 128 4.3
    //   wide    about 0.7 a slot and wave, of tiles four times as large: 256 ..
    //           1024 x 4096 x 4096 27 .. 29, 2048 51; less when the GPU is full
    const double narrow_tiles = tiles_expected(a, Narrow::NT, kCh);
    const double wide_tiles = tiles_expected(a, Wide::NT, 2 * kCh);
    int split = 1;
    while (split < 8 && narrow_tiles <= narrow_room(2 * split, a.num_sms) && k_slots >= 4 * split)
        split *= 2;
    const double narrow_waves = ceil(narrow_tiles * split / a.num_sms) / split;
    if (kernel == SGEMM_I8_KERNEL_AUTO && dots_can) kernel = SGEMM_I8_KERNEL_DOTS;
    if (kernel == SGEMM_I8_KERNEL_AUTO && few_can) {
        if (dense) {
            const double passes = (a.M + 15) / 16 * (static_cast<double>(a.N) * a.K / 4.8e6);
            const double stores = static_cast<double>(a.M) * a.N / 7.5e4;
            if (a.M <= 16 || FewForm(a).large ||
                2.9 + (passes > stores ? passes : stores) <
                    (split > 1 ? 5. : 3.4) + 0.8 * narrow_waves * k_slots)
                kernel = SGEMM_I8_KERNEL_FEW;
        } else if (a.M <= 16LL * a.E) {
            // 32 experts of 2048 x 2048, few / narrow: 8 rows each 30 / 44 us, 12
            // rows 36 / 44 us, 16 rows 43 / 45.  The host knows the mean only.
            // Where rows gather on few experts, narrow would do better: 64 experts
            // of 2048 x 2048, rows in proportion to 1, 1/2, 1/3, ... 81 / 74, 256
            // rows on one and 16 on most others 69 / 65, all 1024 on one 66 / 18;
            // of small weights few keeps ahead (512 x 1024: 15 / 17, 13 / 18, 13 /
            // 11; even rows 10 / 16)
            kernel = SGEMM_I8_KERNEL_FEW;
        }
    }
    // A tile takes as long as its epilogue (short k) or its multiplies (long k),
    // whichever is longer, us by slots of k; K = 128, 512, 1024, 2048, narrow /
    // wide: 8192 x 8192 71 / 64, 92 / 73, 155 / 103, 286 / 175; 32 experts of
    // 3840 channels, 99 rows each, 22 / 30, 30 / 36, 48 / 51, 81 / 84, and of
    // 3837 channels, 128 rows each, 40 / 49, 50 / 61, 69 / 66, 113 / 90; fp32,
    // 8192 x 4096, 67 / 40, 78 / 52, - , 154 / 108.
    if (kernel == SGEMM_I8_KERNEL_AUTO) {
        const double s = k_slots, sn = s / split;
        const bool fp32 = sizeof(T) == 4, odd = c_bytes < 8 && !fp32;
        const double narrow_end = fp32 ? 4.1 + 0.27 * sn : odd ? 2.9 + 0.28 * sn : 2.2 + 0.25 * sn;
        const double narrow_mma = 0.8 + 0.6 * sn;
        const double wide_end = fp32 ? 4.6 + 0.5 * s : odd ? 6.0 + 0.4 * s : 4.2 + 0.2 * s;
        const double wide_mma = 1.9 + (fp32 ? 0.8 : 0.63) * s;
        const double narrow_cost = (narrow_end > narrow_mma ? narrow_end : narrow_mma) *
                                       ceil(narrow_tiles * split / a.num_sms) +
                                   (split > 1 ? 1.6 : 0.);
        const double wide_cost =
            (wide_end > wide_mma ? wide_end : wide_mma) * ceil(wide_tiles / pairs) + 0.8;
        // (experts of unknown counts: narrow where it is clearly ahead, since more of
        // its tiles may turn out to be needed: 60 experts of 200 rows x 1536 x 128
        // 37 / 27)
        kernel = (dense ? 1. : 0.9) * wide_cost < narrow_cost ? SGEMM_I8_KERNEL_WIDE
                                                              : SGEMM_I8_KERNEL_NARROW;
    }
    note_product(kernel, kernel == SGEMM_I8_KERNEL_NARROW ? split : 1);
    if (kernel == SGEMM_I8_KERNEL_DOTS) {
        if (a.M == 1) return launch_dots<T, 1>(a, st);
        if (a.M == 2) return launch_dots<T, 2>(a, st);
        return launch_dots<T, 4>(a, st);
    }
    if (kernel == SGEMM_I8_KERNEL_FEW) return launch_few_tokens<T>(a, st);
    if (kernel == SGEMM_I8_KERNEL_WIDE) {
        const long long tiles = max_tiles(a, Wide::NT) * ((a.N + 2 * kCh - 1) / (2 * kCh));
        return launch_tc_i8<Wide, T>(a, tmW, tmT, tiles < pairs ? tiles : pairs, 1, c_bytes, st);
    }
    // a cluster that shares a tile's k has one tile
    const long long tiles = max_tiles(a, Narrow::NT) * ((a.N + kCh - 1) / kCh);
    const long long clusters = split > 1 || tiles < a.num_sms ? tiles : a.num_sms;
    return launch_tc_i8<Narrow, T>(a, tmW, tmT, clusters, split, c_bytes, st);
}

// Checks and enqueues a product; offsets null: one dense group of M rows.
int product(int type, int M, int N, int K, int E, const int *offsets, const signed char *A,
            int lda, const float *scaleA, const signed char *B, int ldb, long long strideB,
            const float *scaleB, void *C, int ldc, void *stream)
{
    if (!rows::valid_type(type) || M < 0 || N < 0 || K < 0 || lda < 1 || ldb < 1 || ldc < 1 ||
        lda < K || ldb < K || ldc < N || K > kMaxK || M > kMaxSide || N > kMaxSide)
        return SGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (C == nullptr || scaleA == nullptr || scaleB == nullptr ||
        !rows::aligned_to(C, rows::elem_size(type)) || !rows::aligned_to(scaleA, 4) ||
        !rows::aligned_to(scaleB, 4))
        return SGEMM_ERR_INVALID_ARG;
    if (K > 0 && (A == nullptr || B == nullptr)) return SGEMM_ERR_INVALID_ARG;
    Args a{};
    if (!current_sm103(&a.num_sms, &a.status)) return SGEMM_ERR_UNSUPPORTED;
    a.M = M;
    a.N = N;
    a.K = K;
    a.E = E;
    a.offsets = offsets;
    a.A = A;
    a.B = B;
    a.lda = lda;
    a.ldb = ldb;
    a.strideB = strideB;
    a.scaleA = scaleA;
    a.scaleB = scaleB;
    a.C = C;
    a.ldc = ldc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (type == SGEMM_TYPE_BF16) return run<__nv_bfloat16>(a, st);
    if (type == SGEMM_TYPE_FP16) return run<__half>(a, st);
    return run<float>(a, st);
}

}  // namespace i8
}  // namespace sg

extern "C" {

int sgemm_i8_tune_force(int kernel)
{
    if (kernel < SGEMM_I8_KERNEL_AUTO || kernel > SGEMM_I8_KERNEL_ANY_LAYOUT)
        return SGEMM_ERR_INVALID_ARG;
    sg::i8::g_force.store(kernel);
    return SGEMM_OK;
}

int sgemm_i8_last_kernel(void) { return sg::i8::g_last_kernel.load(); }

int sgemm_i8_last_split_count(void) { return sg::i8::g_last_split.load(); }

int sgemm_i8(int type, int M, int N, int K, const signed char *A, int lda, const float *scaleA,
             const signed char *B, int ldb, const float *scaleB, void *C, int ldc, void *stream)
{
    return sg::c_entry([&]() -> int {
        return sg::i8::product(type, M, N, K, 1, nullptr, A, lda, scaleA, B, ldb, 0, scaleB, C, ldc,
                               stream);
    });
}

int sgemm_i8_experts(int type, int M, int N, int K, int E, const int *offsets,
                     const signed char *A, int lda, const float *scaleA, const signed char *B,
                     int ldb, long long strideB, const float *scaleB, void *C, int ldc,
                     void *stream)
{
    return sg::c_entry([&]() -> int {
        if (E < 1 || E > sg::kMaxExperts || offsets == nullptr ||
            !sg::rows::aligned_to(offsets, 4) || strideB < 0 ||
            (E > 1 && N > 0 && strideB < (N - 1LL) * ldb + K))
            return SGEMM_ERR_INVALID_ARG;
        return sg::i8::product(type, M, N, K, E, offsets, A, lda, scaleA, B, ldb, strideB, scaleB, C,
                               ldc, stream);
    });
}

}  // extern "C"

// i8_gemm.h -- what the 8-bit integer product's kernels share: the call's
// arguments and the map from token tiles to experts.
#pragma once

#include <cuda_runtime.h>

#include "rows.cuh"

namespace sg {
namespace i8 {

constexpr int kMaxK = 131071;  // 2^14 * K < 2^31: the 32-bit integer sums cannot overflow
constexpr int kMaxSide = 0x7FFFFFFF - 511;  // an index a tile past the last row or channel still is an int

struct Args {
    int M, N, K, E;
    const int *offsets;       // E + 1 row offsets; null: one group of all M rows
    const signed char *A, *B;
    long long lda, ldb, strideB;
    const float *scaleA, *scaleB;
    void *C;
    long long ldc;
    int tile0;                // first token tile of this launch (dot_kernel)
    unsigned int *status;     // device status word
    int num_sms;
};

// At most this many token tiles of `tm` rows: every expert may end in a
// short one, but none has one without a row.  (Of ascending offsets.  Others
// may give several experts the same rows; tiles from this number on are left
// out then, in every kernel.)
__host__ __device__ inline long long max_tiles(const Args &a, int tm)
{
    if (a.offsets == nullptr) return (static_cast<long long>(a.M) + tm - 1) / tm;
    return a.M / tm + (a.E < a.M ? a.E : a.M);
}

// Rows [lo, hi) of expert e, kept inside the M rows whatever offsets holds.
__device__ __forceinline__ void expert_rows(const Args &a, int e, int &lo, int &hi)
{
    if (a.offsets == nullptr) {
        lo = 0;
        hi = a.M;
        return;
    }
    lo = min(max(a.offsets[e], 0), a.M);
    hi = min(max(a.offsets[e + 1], lo), a.M);
}

// One token tile: `rows` rows from row0 on, of expert e (e < 0: no such tile).
struct Tile {
    int e, rows;
    long long row0;
};

// Token tile tile0 + u, found by one warp (every lane calls; the result is
// the same in all).
__device__ __forceinline__ Tile find_tile_warp(const Args &a, int u, int tm, int lane)
{
    Tile t{-1, 0, 0};
    long long want = static_cast<long long>(a.tile0) + u;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        int lo = 0, hi = 0;
        if (e0 + lane < a.E) expert_rows(a, e0 + lane, lo, hi);
        const int n = (hi - lo + tm - 1) / tm;
        int inc = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += x;
        }
        const unsigned has = __ballot_sync(0xffffffffu, want < inc);
        if (has) {
            const int src = __ffs(has) - 1;
            const int first = __shfl_sync(0xffffffffu, inc - n, src);
            const int l = __shfl_sync(0xffffffffu, lo, src);
            const int h = __shfl_sync(0xffffffffu, hi, src);
            const long long r = l + (want - first) * tm;
            t.e = e0 + src;
            t.row0 = r;
            t.rows = static_cast<int>(min(static_cast<long long>(tm), h - r));
            return t;
        }
        want -= __shfl_sync(0xffffffffu, inc, 31);
    }
    return t;
}

}  // namespace i8
}  // namespace sg

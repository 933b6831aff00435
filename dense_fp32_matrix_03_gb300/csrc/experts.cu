// experts.cu -- tokens sorted by expert and back (include/expert_layer.h):
// the stable sort, and the row kernels of dispatch, combine and their
// gradients.
#include <atomic>

#include "../../include/expert_layer.h"
#include "dependent.cuh"
#include "rows.cuh"

namespace sg {
namespace ex {

using rows::aligned_to;
using rows::Vec;

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortAhead = 8;     // steps of a warp's walk loaded at once
// Choices of a token whose rows are in flight together.  Four, on blocks small
// enough in registers that five or six share a multiprocessor, hide each
// other's chain of position, row and sum best (65536 rows of 4096 bf16
// combined, by choices x blocks: 8 x 4 97 us, 4 x 6 95, 4 x 8 (spills) 299,
// 2 x 8 112; the gradient of 32768 rows of 2048: 8 x 4 66, 4 x 5 48, 2 x 8 61).

// ------------------------------------------------------------------ sort
//
// position(s) = (choices of smaller experts) + (earlier choices of the same
// expert): a counting sort.  The choices are cut into one contiguous segment
// per warp, in order, over a cluster of CTAs, so that ranks within a segment
// need no atomics and the order is stable by construction:
//   1. each warp counts its segment into a histogram of its own (lanes of
//      equal key found with a warp match, the first adds their number);
//   2. a scan over the CTA's warps turns counts into the warp's first rank,
//      and the CTAs' totals, read through distributed shared memory, into
//      each expert's first position and each CTA's share of it;
//   3. each warp walks its segment again and hands out positions.
// One launch; the choices (4 bytes each) are read twice, the second time
// from L2.  The bytes are few (12 per choice): what bounds it is the chain
// of launch, two walks and two cluster barriers (32 choices 3.0 us), then the
// matches and scattered stores of the walks (65536 choices of 64 experts 12.0,
// of 8 experts 7.4, 262144 of 64 32 us).
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return static_cast<int>(r);
}
__device__ __forceinline__ int cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return static_cast<int>(r);
}
// An int of CTA `rank`'s shared memory, at this CTA's address p.
__device__ __forceinline__ int cluster_load(const int *p, int rank)
{
    uint32_t a, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(a)
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return static_cast<int>(v);
}

// The keys of this lane's choices i, i + 32, ... (dropped: E; past the
// segment: -1), all on their way at once.  (No pointer here is __restrict__:
// the router may still write ids when the kernel starts, and a const pointer
// so declared allows loads that are defined for unchanging memory only.)
__device__ __forceinline__ void load_keys(int (&key)[kSortAhead], const int *ids, long long i,
                                          long long hi, int E)
{
#pragma unroll
    for (int c = 0; c < kSortAhead; ++c) key[c] = i + 32 * c < hi ? ids[i + 32 * c] : -1;
#pragma unroll
    for (int c = 0; c < kSortAhead; ++c)
        key[c] = i + 32 * c >= hi ? -1 : (key[c] < 0 || key[c] >= E) ? E : key[c];
}

__global__ void __launch_bounds__(kSortThreads, 1)
    sort_kernel(const int *ids, int S, int E, int *offsets, int *slots, int *positions)
{
    extern __shared__ int sm[];
    const int E1 = E + 1;
    int *hist = sm;                       // [kSortWarps][E1]
    int *tot = hist + kSortWarps * E1;    // [E1] this CTA's counts
    int *base = tot + E1;                 // [E1] this CTA's first position of each key
    __shared__ int wsum[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = cluster_rank(), ncta = cluster_size();
    const int segs = ncta * kSortWarps;
    const long long len = ((static_cast<long long>(S) + segs - 1) / segs + 31) / 32 * 32;
    const long long lo = (static_cast<long long>(rank) * kSortWarps + warp) * len;
    const long long hi = min(lo + len, static_cast<long long>(S));
    int *mine = hist + warp * E1;

    dependent_release();
    for (int i = tid; i < kSortWarps * E1; i += kSortThreads) hist[i] = 0;
    dependent_wait();
    __syncthreads();
    for (long long i = lo; i < hi; i += 32 * kSortAhead) {
        int key[kSortAhead];
        load_keys(key, ids, i + lane, hi, E);
#pragma unroll
        for (int c = 0; c < kSortAhead; ++c) {
            if (i + 32 * c >= hi) break;
            const unsigned same = __match_any_sync(0xffffffffu, key[c]);
            if (key[c] >= 0 && lane == __ffs(same) - 1) mine[key[c]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int e = tid; e < E1; e += kSortThreads) {
        int run = 0;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const int n = hist[w * E1 + e];
            hist[w * E1 + e] = run;
            run += n;
        }
        tot[e] = run;
    }
    cluster_barrier();
    int before = 0, all = 0;  // key tid: in earlier CTAs, in all CTAs
    if (tid < E) {
        for (int c = 0; c < ncta; ++c) {
            const int n = cluster_load(&tot[tid], c);
            if (c < rank) before += n;
            all += n;
        }
    }
    // exclusive scan of `all` over the keys (E <= kSortThreads)
    int inc = all;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int n = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += n;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int ahead = 0, kept = 0;
    for (int w = 0; w < kSortWarps; ++w) {
        if (w < warp) ahead += wsum[w];
        kept += wsum[w];
    }
    const int first = ahead + inc - all;
    if (tid < E) base[tid] = first + before;
    if (tid == 0) {  // dropped choices: behind the kept ones
        int n = 0;
        for (int c = 0; c < rank; ++c) n += cluster_load(&tot[E], c);
        base[E] = kept + n;
    }
    if (rank == 0) {
        if (tid < E) offsets[tid] = first;
        if (tid == 0) offsets[E] = kept;
    }
    cluster_barrier();  // tot has been read by every CTA; base is written
    for (long long i = lo; i < hi; i += 32 * kSortAhead) {
        int key[kSortAhead];
        load_keys(key, ids, i + lane, hi, E);
#pragma unroll
        for (int c = 0; c < kSortAhead; ++c) {
            if (i + 32 * c >= hi) break;
            const unsigned same = __match_any_sync(0xffffffffu, key[c]);
            const int before_me = __popc(same & ((1u << lane) - 1u));
            int p = 0;
            if (key[c] >= 0) p = base[key[c]] + mine[key[c]] + before_me;
            __syncwarp();
            if (key[c] >= 0) {
                const int slot = static_cast<int>(i) + 32 * c + lane;
                positions[slot] = p;
                slots[p] = slot;
                if (before_me == 0) mine[key[c]] += __popc(same);
            }
            __syncwarp();
        }
    }
}

// CTAs of the sort's cluster: one for up to 512 choices (half a step per warp),
// 8 beyond, 16 from 8192 on where the GPU has room for such a cluster
// (64 experts: 2048 choices 7.0 us on one, 4104 6.6 us on 8, 65536 20 us on 8
// and 12 us on 16: what costs is a warp's match of up to 32 different keys and
// its stores to as many lines).
unsigned sort_cluster(int S)
{
    if (S <= 512) return 1u;
    static std::atomic<int> widest[64];  // per device: 0 not asked yet
    int dev = 0;
    if (S <= 8192 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 8u;
    int w = widest[dev].load();
    if (w == 0) {
        int n = 0;
        // the largest shared memory any call asks for
        const int most = (kSortWarps + 2) * (kMaxExperts + 1) * static_cast<int>(sizeof(int));
        if (cudaFuncSetAttribute(reinterpret_cast<const void *>(sort_kernel),
                                 cudaFuncAttributeNonPortableClusterSizeAllowed,
                                 1) == cudaSuccess &&
            smem_attr_once(reinterpret_cast<const void *>(sort_kernel), most)) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(16);
            cfg.blockDim = dim3(kSortThreads);
            cfg.dynamicSmemBytes = static_cast<size_t>(most);
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 16;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, sort_kernel, &cfg) != cudaSuccess) n = 0;
        }
        cudaGetLastError();
        w = n > 0 ? 16 : 8;
        widest[dev].store(w);
    }
    return static_cast<unsigned>(w);
}

// -------------------------------------------------------------- row kernels
//
// All move whole rows and compute next to nothing: bound by HBM.  A block
// takes blockDim.y tokens, blockDim.x threads over a row's vectors, and works
// token by token: a token's k rows are read (combine) or written (dispatch)
// together, G choices at a time, so its own row moves once.  A block lives for
// three dependent loads (kept count, position, row), so what counts is how
// many bytes each thread then has in flight: U vectors a block's width apart
// (neighbouring threads stay on neighbouring addresses) of each of G rows, 16
// bytes of each row where registers allow.  p(t,j) is checked against T * k,
// so a corrupt position cannot reach outside the rows.
//
// G and U by choices and alignment (us, one vector of four rows / as chosen):
//   k <= 2: two rows, two vectors or more: combine 8192 x 2 rows of 4096 bf16
//     43 / 38, 16384 x 1 of 1024 19.4 / 15, its gradient 56 / 51, 27 / 19
//   rows on 8 bytes or less: 16 bytes of four rows (at most four vectors):
//     3000 x 2 rows of 2825 fp16 49 / 21, 7252 x 3 of 2612 bf16 64 / 43, 1874 x
//     5 of 2825 fp16 51 / 28, dispatch of these 38 / 21, 35 / 32, 36 / 22
//   the gradient on 8 bytes: one vector, since it keeps a token's vector and
//     the sums too (7252 x 3 of 2612: 55; two vectors 73)
// (The register limits that keep five or six blocks on a multiprocessor spill in
// some of the forms chosen: combine's two-row form of 16-bit rows on 16 bytes 30
// words, its four-row form of bf16 on 8 bytes 12, the others 9 or fewer, the
// gradient's 1 or 2.)
//
// Measured on GB300, bf16 (us, share of the measured copy bandwidth for the
// bytes of kept rows, tokens' rows and results): 65536 rows of 4096 dispatched
// 93 (0.96), combined 95 (0.93), combine's gradient 170 (0.99); 32768 rows of
// 2048 28 (0.89), 31 (0.81), 48 (0.92).  Eight tokens of 2048: 1.7 to 2.3 us,
// launch and the three loads.

struct Args {
    int T, k, S;              // S = T * k
    unsigned nvec;            // vectors in a row (unsigned: an index past the end of the
                              // longest row by a stride must not wrap below it)
    const int *positions;
    const int *total;         // offsets[E]: the kept choices
    const float *weights;     // may be null: 1
    const char *tok;          // rows of tokens (x, dout)
    char *tok_out;            // rows of tokens written (out, dx)
    const char *row;          // rows by expert read
    char *row_out;            // rows by expert written
    float *dweights;
    long long tok_pitch, row_pitch, row_out_pitch;  // bytes
};

template <class T, int VB>
__global__ void __launch_bounds__(256) dispatch_kernel(const Args a)
{
    constexpr int G = 4, U = rows::kAhead<VB>;
    dependent_release();
    dependent_wait();
    const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (t >= a.T) return;
    const int total = *a.total;
    const char *tok = a.tok + t * a.tok_pitch;
    for (int j0 = 0; j0 < a.k; j0 += G) {
        int p[G];
#pragma unroll
        for (int j = 0; j < G; ++j)
            p[j] = j0 + j < a.k ? a.positions[t * a.k + j0 + j] : -1;
        for (unsigned v = blockIdx.y * U * blockDim.x + threadIdx.x; v < a.nvec;
             v += gridDim.y * U * blockDim.x) {
            Vec<T, VB> x[U], z;
            z.zero();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const unsigned i = v + u * blockDim.x;
                if (i < a.nvec) x[u].load(tok + static_cast<long long>(i) * VB);
            }
#pragma unroll
            for (int j = 0; j < G; ++j) {
                if (p[j] < 0 || p[j] >= a.S) continue;
                char *out = a.row_out + p[j] * a.row_out_pitch;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const unsigned i = v + u * blockDim.x;
                    if (i < a.nvec)
                        (p[j] < total ? x[u] : z).store(out + static_cast<long long>(i) * VB);
                }
            }
        }
    }
}

template <class T, int VB, int G, int U>
__global__ void __launch_bounds__(256, 6) combine_kernel(const Args a)
{
    using V = Vec<T, VB>;
    dependent_release();
    dependent_wait();
    const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (t >= a.T) return;
    const int total = min(*a.total, a.S);
    char *out = a.tok_out + t * a.tok_pitch;
    for (unsigned v = blockIdx.y * U * blockDim.x + threadIdx.x; v < a.nvec;
         v += gridDim.y * U * blockDim.x) {
        float acc[U][V::N];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < V::N; ++i) acc[u][i] = 0.f;
        for (int j0 = 0; j0 < a.k; j0 += G) {
            V x[G][U];
            float w[G];
            bool on[G];
#pragma unroll
            for (int j = 0; j < G; ++j) {
                on[j] = false;
                if (j0 + j < a.k) {
                    const int p = a.positions[t * a.k + j0 + j];
                    w[j] = a.weights ? a.weights[t * a.k + j0 + j] : 1.f;
                    on[j] = p >= 0 && p < total;
                    if (on[j]) {
                        const char *row = a.row + p * a.row_pitch;
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const unsigned i = v + u * blockDim.x;
                            if (u == 0 || i < a.nvec)
                                x[j][u].load(row + static_cast<long long>(i) * VB);
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < G; ++j)
                if (on[j]) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (u == 0 || v + u * blockDim.x < a.nvec)
#pragma unroll
                            for (int i = 0; i < V::N; ++i)
                                acc[u][i] = fmaf(w[j], x[j][u].get(i), acc[u][i]);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned c = v + u * blockDim.x;
            V o;
#pragma unroll
            for (int i = 0; i < V::N; ++i) o.set(i, acc[u][i]);
            if (u == 0 || c < a.nvec) o.store(out + static_cast<long long>(c) * VB);
        }
    }
}

// DW: dweights wanted (rows is read).  blockDim.x threads of one token sum
// their products over the row, then over lanes and warps in a fixed order.
template <class T, int VB, int G, int U, bool DW>
__global__ void __launch_bounds__(256, G * U == 16 ? 4 : 5) combine_grad_kernel(const Args a)
{
    using V = Vec<T, VB>;
    __shared__ float part[8][G];  // one row per warp of the block
    dependent_release();
    dependent_wait();
    const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = t < a.T;
    const int total = min(*a.total, a.S);
    const int wid = (threadIdx.y * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    const char *tok = a.tok + t * a.tok_pitch;
    for (int j0 = 0; j0 < a.k; j0 += G) {
        float w[G], dw[G];
        int p[G];
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const bool in = live && j0 + j < a.k;
            p[j] = in ? a.positions[t * a.k + j0 + j] : -1;
            if (p[j] >= a.S) p[j] = -1;
            w[j] = in && a.weights ? a.weights[t * a.k + j0 + j] : 1.f;
            dw[j] = 0.f;
        }
        for (unsigned v = threadIdx.x; live && v < a.nvec; v += U * blockDim.x) {
            V g[U], x[G][U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const unsigned i = v + u * blockDim.x;
                if (u == 0 || i < a.nvec) g[u].load(tok + static_cast<long long>(i) * VB);
            }
            if (DW) {
#pragma unroll
                for (int j = 0; j < G; ++j)
                    if (p[j] >= 0 && p[j] < total) {
                        const char *row = a.row + p[j] * a.row_pitch;
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const unsigned i = v + u * blockDim.x;
                            if (u == 0 || i < a.nvec)
                                x[j][u].load(row + static_cast<long long>(i) * VB);
                        }
                    }
            }
#pragma unroll
            for (int j = 0; j < G; ++j) {
                if (p[j] < 0) continue;
                char *out = a.row_out + p[j] * a.row_out_pitch;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const unsigned at = v + u * blockDim.x;
                    if (u > 0 && at >= a.nvec) continue;
                    V o;
                    if (p[j] < total) {
#pragma unroll
                        for (int i = 0; i < V::N; ++i) {
                            if (DW) dw[j] = fmaf(x[j][u].get(i), g[u].get(i), dw[j]);
                            o.set(i, w[j] * g[u].get(i));
                        }
                    } else {
                        o.zero();
                    }
                    o.store(out + static_cast<long long>(at) * VB);
                }
            }
        }
        if (DW) {
#pragma unroll
            for (int j = 0; j < G; ++j) {
#pragma unroll
                for (int d = 16; d > 0; d /= 2) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], d);
                if (lane == 0) part[wid][j] = dw[j];
            }
            __syncthreads();
            const int warps = blockDim.x >> 5;
            if (live && threadIdx.x < G && j0 + static_cast<int>(threadIdx.x) < a.k) {
                float s = 0.f;
                for (int i = 0; i < warps; ++i) s += part[threadIdx.y * warps + i][threadIdx.x];
                a.dweights[t * a.k + j0 + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

// Threads over a row (per_thread vectors each) and tokens per block (256
// threads, at least a warp per token), and blocks over a row's columns: enough
// that few tokens still spread over the GPU.
struct Grid {
    dim3 grid, block;
};
Grid row_grid(int T, unsigned nvec, unsigned per_thread, bool split_columns)
{
    const unsigned pieces = nvec == 0 ? 1 : (nvec + per_thread - 1) / per_thread;
    const unsigned turns = (pieces + 255) / 256;
    const int tx = ((pieces + turns - 1) / turns + 31) / 32 * 32, ty = 256 / tx;
    const unsigned gx = static_cast<unsigned>((static_cast<long long>(T) + ty - 1) / ty);
    unsigned gy = 1;
    if (split_columns) {
        gy = (pieces + tx - 1) / tx;
        if (gy > 64) gy = 64;
    }
    return {dim3(gx, gy), dim3(static_cast<unsigned>(tx), static_cast<unsigned>(ty))};
}

enum Op { kDispatch, kCombine, kCombineGrad };

struct Launch {
    Op op;
    const Args &a;
    cudaStream_t st;
    template <class T, int VB>
    int run() const
    {
        constexpr int U = rows::kAhead<VB>, U2 = U > 2 ? U : 2;
        constexpr int UG = VB < 8 ? U : 1;  // combine's gradient, beyond two choices
        const bool two = op != kDispatch && a.k <= 2, dw = a.dweights != nullptr;
        const Grid g =
            row_grid(a.T, a.nvec, two ? U2 : op == kCombineGrad ? UG : U, op != kCombineGrad);
        auto kern = op == kDispatch ? dispatch_kernel<T, VB>
                    : op == kCombine
                        ? (two ? combine_kernel<T, VB, 2, U2> : combine_kernel<T, VB, 4, U>)
                    : dw ? (two ? combine_grad_kernel<T, VB, 2, U2, true>
                                : combine_grad_kernel<T, VB, 4, UG, true>)
                         : (two ? combine_grad_kernel<T, VB, 2, U2, false>
                                : combine_grad_kernel<T, VB, 4, UG, false>);
        return launch_dependent(kern, g.grid, g.block, 0, 1, st, a);
    }
};

}  // namespace ex
}  // namespace sg

using namespace sg;
using ex::Args;

namespace {

bool int_aligned(const void *p) { return rows::aligned_to(p, 4); }

// The checks every row call shares; run = false: return rc as it is.
struct Checked {
    int rc;
    bool run;
};
Checked check_rows(int type, int T, int k, int E, int H, const void *tok, int ld_tok,
                   const void *row, int ld_row, const int *positions, const int *offsets)
{
    if (!rows::valid_type(type) || !choices_ok(T, k, E) || H < 0 || ld_tok < 1 || ld_row < 1 ||
        ld_tok < H || ld_row < H)
        return {SGEMM_ERR_INVALID_ARG, false};
    if (T == 0) return {SGEMM_OK, false};
    const int es = rows::elem_size(type);
    if (positions == nullptr || offsets == nullptr || !int_aligned(positions) ||
        !int_aligned(offsets))
        return {SGEMM_ERR_INVALID_ARG, false};
    if (H > 0 && (tok == nullptr || row == nullptr || !rows::aligned_to(tok, es) ||
                  !rows::aligned_to(row, es)))
        return {SGEMM_ERR_INVALID_ARG, false};
    return {SGEMM_OK, true};
}

Args base_args(int T, int k, int E, const int *positions, const int *offsets)
{
    Args a{};
    a.T = T;
    a.k = k;
    a.S = T * k;
    a.positions = positions;
    a.total = offsets + E;
    return a;
}

bool on_gpu()
{
    int num_sms = 0;
    unsigned int *status = nullptr;
    return current_sm103(&num_sms, &status);
}

int combine(int type, int T, int k, int E, int H, const void *rws, int ldr, const int *positions,
            const int *offsets, const float *weights, void *out, int ldo, void *stream)
{
    const Checked c = check_rows(type, T, k, E, H, out, ldo, rws, ldr, positions, offsets);
    if (!c.run) return c.rc;
    if (!int_aligned(weights)) return SGEMM_ERR_INVALID_ARG;
    if (H == 0) return SGEMM_OK;
    if (!on_gpu()) return SGEMM_ERR_UNSUPPORTED;
    const long long es = rows::elem_size(type);
    Args a = base_args(T, k, E, positions, offsets);
    a.weights = weights;
    a.row = static_cast<const char *>(rws);
    a.tok_out = static_cast<char *>(out);
    a.row_pitch = ldr * es;
    a.tok_pitch = ldo * es;
    const int vb = rows::Width().add(rws).add(out).add(a.row_pitch).add(a.tok_pitch).add(H * es).bytes();
    a.nvec = static_cast<unsigned>(H * es / vb);
    return rows::with_vec(type, vb, ex::Launch{ex::kCombine, a, static_cast<cudaStream_t>(stream)});
}

}  // namespace

extern "C" {

int sgemm_experts_sort(int T, int k, int E, const int *ids, int *offsets, int *slots,
                       int *positions, void *stream)
{
    return c_entry([&]() -> int {
        if (!choices_ok(T, k, E) || offsets == nullptr || !int_aligned(offsets))
            return SGEMM_ERR_INVALID_ARG;
        const int S = T * k;
        if (S > 0 && (ids == nullptr || slots == nullptr || positions == nullptr ||
                      !int_aligned(ids) || !int_aligned(slots) || !int_aligned(positions)))
            return SGEMM_ERR_INVALID_ARG;
        if (!on_gpu()) return SGEMM_ERR_UNSUPPORTED;
        const int smem = (ex::kSortWarps + 2) * (E + 1) * static_cast<int>(sizeof(int));
        if (!smem_attr_once(reinterpret_cast<const void *>(ex::sort_kernel), smem))
            return SGEMM_ERR_LAUNCH;
        const unsigned ncta = ex::sort_cluster(S);
        return launch_dependent(ex::sort_kernel, dim3(ncta), dim3(ex::kSortThreads),
                                static_cast<size_t>(smem), ncta, static_cast<cudaStream_t>(stream),
                                ids, S, E, offsets, slots, positions);
    });
}

int sgemm_experts_dispatch(int type, int T, int k, int E, int H, const void *x, int ldx,
                           const int *positions, const int *offsets, void *rws, int ldr,
                           void *stream)
{
    return c_entry([&]() -> int {
        const Checked c = check_rows(type, T, k, E, H, x, ldx, rws, ldr, positions, offsets);
        if (!c.run || H == 0) return c.rc;
        if (!on_gpu()) return SGEMM_ERR_UNSUPPORTED;
        const long long es = rows::elem_size(type);
        Args a = base_args(T, k, E, positions, offsets);
        a.tok = static_cast<const char *>(x);
        a.row_out = static_cast<char *>(rws);
        a.tok_pitch = ldx * es;
        a.row_out_pitch = ldr * es;
        const int vb =
            rows::Width().add(x).add(rws).add(a.tok_pitch).add(a.row_out_pitch).add(H * es).bytes();
        a.nvec = static_cast<unsigned>(H * es / vb);
        return rows::with_vec(type, vb, ex::Launch{ex::kDispatch, a, static_cast<cudaStream_t>(stream)});
    });
}

int sgemm_experts_dispatch_grad(int type, int T, int k, int E, int H, const void *drows, int ldr,
                                const int *positions, const int *offsets, void *dx, int ldx,
                                void *stream)
{
    return c_entry([&]() -> int {
        return combine(type, T, k, E, H, drows, ldr, positions, offsets, nullptr, dx, ldx, stream);
    });
}

int sgemm_experts_combine(int type, int T, int k, int E, int H, const void *rws, int ldr,
                          const int *positions, const int *offsets, const float *weights,
                          void *out, int ldo, void *stream)
{
    return c_entry([&]() -> int {
        return combine(type, T, k, E, H, rws, ldr, positions, offsets, weights, out, ldo, stream);
    });
}

int sgemm_experts_combine_grad(int type, int T, int k, int E, int H, const void *dout, int ldo,
                               const void *rws, int ldr, const int *positions,
                               const int *offsets, const float *weights, void *drows, int ldd,
                               float *dweights, void *stream)
{
    return c_entry([&]() -> int {
        const Checked c = check_rows(type, T, k, E, H, dout, ldo, drows, ldd, positions, offsets);
        if (!c.run) return c.rc;
        const long long es = rows::elem_size(type);
        if (!int_aligned(weights) || !int_aligned(dweights)) return SGEMM_ERR_INVALID_ARG;
        if (dweights != nullptr && H > 0 &&
            (rws == nullptr || ldr < H || !rows::aligned_to(rws, static_cast<int>(es))))
            return SGEMM_ERR_INVALID_ARG;
        if (H == 0 && dweights == nullptr) return SGEMM_OK;
        if (!on_gpu()) return SGEMM_ERR_UNSUPPORTED;
        Args a = base_args(T, k, E, positions, offsets);
        a.weights = weights;
        a.tok = static_cast<const char *>(dout);
        a.row_out = static_cast<char *>(drows);
        a.dweights = dweights;
        a.tok_pitch = ldo * es;
        a.row_out_pitch = ldd * es;
        rows::Width w;
        w.add(dout).add(drows).add(a.tok_pitch).add(a.row_out_pitch).add(H * es);
        if (dweights != nullptr) {
            a.row = static_cast<const char *>(rws);
            a.row_pitch = ldr * es;
            w.add(rws).add(a.row_pitch);
        }
        // H == 0: pointers may be null; the kernel writes zero dweights only
        const int vb = H == 0 ? 16 : w.bytes();
        a.nvec = static_cast<unsigned>(H * es / vb);
        return rows::with_vec(type, vb,
                              ex::Launch{ex::kCombineGrad, a, static_cast<cudaStream_t>(stream)});
    });
}

}  // extern "C"

// norm.cu -- the root-mean-square norm of a residual stream, with an output in
// the rows' type, in 8 bits or in 4 bits, and its gradient (include/rms_norm.h).
//
// Forward: one pass.  A row's vectors (the sum s, rounded as it is kept, and
// the weight) stay in registers between the reduction and the output, so each
// value is read once; a row longer than the registers reads its tail a second
// time.  The codes of a quantised row hang on s and the weight alone: rho, whose
// last bits depend on the order of a sum, only enters the row's scale.
//
// Bound by HBM: a thread has eight to twelve 16-byte loads in flight, four
// vectors of x, the residual and the weight (one of each where there are no more
// rows than multiprocessors: more threads on a row, 8 x 4096 1.9 us).  Measured on
// GB300, 8192 x 4096 bf16: row 40.0 us (6.7 TB/s), 8 bits 39.0 (6.0), 4 bits 42.5
// (5.2, where the rounding's instructions count); rows on 8, 4 and 2 bytes (8192 x
// 4092, 4094, 4095) 40.4, 41.8 and 78 us, their narrow pieces dealt to a warp's lanes
// in turn (each lane its own vector's: 106 on 2 bytes).  Values held as floats, or taken
// out of 16-bit vectors one by one, cost registers and instructions: 8 bits 42.9,
// 4 bits 48.
#include "../../include/rms_norm.h"
#include "dependent.cuh"
#include "fp4.cuh"
#include "rows.cuh"

namespace sg {
namespace norm {

using rows::Words;

constexpr float kI8Tiny = 7.888609052210118e-31f;  // 2^-100
constexpr float kRound = 12582912.f;               // 1.5 * 2^23
constexpr int kHeld = 4;                           // vectors per thread kept in registers
enum Out { kRow = 0, kI8 = 1, kFp4Mx = 2, kFp4Nv = 3 };

struct Args {
    int M, H;
    unsigned nvec;  // vectors per row
    float eps;
    const char *x, *res, *w;
    char *sum, *y;
    long long px, pr, ps, py;  // row pitches in bytes
    unsigned char *q;          // few bits: codes, bytes per row
    long long pq;
    bool whole_codes;  // 8 bits: a vector's codes on a boundary of theirs
    unsigned char *sf;
    long long sf_tiles;
    float *scale;
};

// Bytes of a row from vector v on, as far as a vector goes.
template <class T, int VB>
__device__ __forceinline__ unsigned bytes_left(int H, unsigned v)
{
    constexpr unsigned EV = Words<T, VB>::N;
    return min(static_cast<unsigned>(H) - v * EV, EV) * static_cast<unsigned>(sizeof(T));
}

// A vector of a row, and back: DEALT, with narrow pieces dealt to the warp's lanes.
// (4 bits want neighbouring values in a lane.)
template <class T, int VB, int LB, bool DEALT>
__device__ __forceinline__ void get(Words<T, VB> &w, const char *row, unsigned v, int H)
{
    if constexpr (DEALT)
        w.template load_dealt<LB>(row, v, static_cast<long long>(H) * static_cast<int>(sizeof(T)));
    else
        w.template load<LB>(row + static_cast<long long>(v) * VB, bytes_left<T, VB>(H, v));
}
template <class T, int VB, int LB, bool DEALT>
__device__ __forceinline__ void set(const Words<T, VB> &w, char *row, unsigned v, int H)
{
    if constexpr (DEALT)
        w.template store_dealt<LB>(row, v, static_cast<long long>(H) * static_cast<int>(sizeof(T)));
    else
        w.template store<LB>(row + static_cast<long long>(v) * VB, bytes_left<T, VB>(H, v));
}
// The column of a dealt vector's value i.
template <class T, int VB, int LB>
__device__ __forceinline__ long long column(unsigned v, int i)
{
    constexpr int PE = LB / static_cast<int>(sizeof(T));  // values of a piece
    return Words<T, VB>::template piece_at<LB>(v, i / PE) / static_cast<int>(sizeof(T)) + i % PE;
}
// Vectors of a row: all lanes of the last warp where pieces are dealt.
template <class T, int VB, int LB, bool DEALT>
unsigned vectors(int H)
{
    constexpr unsigned EV = Words<T, VB>::N;
    const unsigned n = H > 0 ? (static_cast<unsigned>(H) - 1) / EV + 1 : 0;
    return DEALT && LB < VB ? (n + 31) / 32 * 32 : n;
}

template <class T, int VB, int LB, bool DEALT>
__device__ __forceinline__ void load_weight(const Args &a, unsigned v, Words<T, VB> &w)
{
    if (a.w != nullptr) {
        get<T, VB, LB, DEALT>(w, a.w, v, a.H);
    } else {
        float one[Words<T, VB>::N];
#pragma unroll
        for (int i = 0; i < Words<T, VB>::N; ++i) one[i] = 1.f;
        w.pack(one);
    }
}
// x + res as the row type keeps it.
template <class T, int VB>
__device__ __forceinline__ void add(Words<T, VB> &x, const Words<T, VB> &r)
{
    float f[Words<T, VB>::N], g[Words<T, VB>::N];
    x.unpack(f);
    r.unpack(g);
#pragma unroll
    for (int i = 0; i < Words<T, VB>::N; ++i) f[i] += g[i];
    x.pack(f);
}

template <class T, int VB, int LB, int OUT>
__global__ void __launch_bounds__(256, 3) norm_kernel(const Args a)
{
    constexpr int EV = Words<T, VB>::N;
    constexpr bool DEALT = OUT == kRow || OUT == kI8;
    __shared__ float part_sum[8];
    __shared__ unsigned part_max[8];
    dependent_release();
    dependent_wait();
    const long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = r < a.M;
    const long long row = live ? r : 0;
    const char *x = a.x + row * a.px, *res = a.res + row * a.pr;
    char *sum = a.sum + row * a.ps;
    const unsigned tx = threadIdx.x, nx = blockDim.x, warps = nx >> 5;
    const unsigned nvec = live ? a.nvec : 0;

    Words<T, VB> s[kHeld], w[kHeld];
    {
        Words<T, VB> t[kHeld];
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const unsigned v = tx + h * nx;
            s[h].zero();
            w[h].zero();
            t[h].zero();
            if (v < nvec) {
                get<T, VB, LB, DEALT>(s[h], x, v, a.H);
                if (a.res != nullptr) get<T, VB, LB, DEALT>(t[h], res, v, a.H);
                load_weight<T, VB, LB, DEALT>(a, v, w[h]);
            }
        }
        if (a.res != nullptr)
#pragma unroll
            for (int h = 0; h < kHeld; ++h) add(s[h], t[h]);
    }
    float square = 0.f;
    unsigned big = 0;
    auto gather = [&](const Words<T, VB> &sv, const Words<T, VB> &wv) {
        float f[EV], g[EV];
        sv.unpack(f);
        if (OUT != kRow) wv.unpack(g);
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            square = fmaf(f[i], f[i], square);
            if (OUT != kRow) big = max(big, __float_as_uint(f[i] * g[i]) & 0x7FFFFFFFu);
        }
    };
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        const unsigned v = tx + h * nx;
        if (v < nvec) {
            gather(s[h], w[h]);
            if (a.sum != nullptr) set<T, VB, LB, DEALT>(s[h], sum, v, a.H);
        }
    }
    // a vector of a long row's tail; again: in the second pass, when the sum, if
    // it is kept, may have taken the place of x or res
    auto tail = [&](unsigned v, bool again, Words<T, VB> &sv, Words<T, VB> &wv) {
        load_weight<T, VB, LB, DEALT>(a, v, wv);
        if (again && a.sum != nullptr) {
            get<T, VB, LB, DEALT>(sv, sum, v, a.H);
            return;
        }
        get<T, VB, LB, DEALT>(sv, x, v, a.H);
        if (a.res != nullptr) {
            Words<T, VB> t;
            get<T, VB, LB, DEALT>(t, res, v, a.H);
            add(sv, t);
        }
    };
    for (unsigned v = tx + kHeld * nx; v < nvec; v += nx) {
        Words<T, VB> sv, wv;
        tail(v, false, sv, wv);
        gather(sv, wv);
        if (a.sum != nullptr) set<T, VB, LB, DEALT>(sv, sum, v, a.H);
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) square += __shfl_xor_sync(0xffffffffu, square, d);
    if (OUT != kRow) big = __reduce_max_sync(0xffffffffu, big);
    if (warps > 1) {
        const unsigned first = threadIdx.y * warps;
        if ((tx & 31) == 0) {
            part_sum[first + (tx >> 5)] = square;
            part_max[first + (tx >> 5)] = big;
        }
        __syncthreads();
        square = 0.f;
        for (unsigned i = 0; i < warps; ++i) {
            square += part_sum[first + i];
            big = max(big, part_max[first + i]);
        }
    }
    if (!live) return;
    const float rho = rsqrtf(__fdiv_rn(square, static_cast<float>(a.H)) + a.eps);

    if constexpr (OUT == kRow) {
        char *y = a.y + r * a.py;
        auto put = [&](unsigned v, const Words<T, VB> &sv, const Words<T, VB> &wv) {
            float f[EV], g[EV];
            sv.unpack(f);
            wv.unpack(g);
#pragma unroll
            for (int i = 0; i < EV; ++i) f[i] = f[i] * rho * g[i];
            Words<T, VB> o;
            o.pack(f);
            set<T, VB, LB, DEALT>(o, y, v, a.H);
        };
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (tx + h * nx < nvec) put(tx + h * nx, s[h], w[h]);
        for (unsigned v = tx + kHeld * nx; v < nvec; v += nx) {
            Words<T, VB> sv, wv;
            tail(v, true, sv, wv);
            put(v, sv, wv);
        }
    } else if constexpr (OUT == kI8) {
        const float amax = __uint_as_float(big);
        const bool finite = big < 0x7F800000u, some = finite && amax >= kI8Tiny;
        const float inv = some ? __fdiv_rn(127.f, amax) : 0.f;
        unsigned char *q = a.q + r * a.pq;
        auto put = [&](unsigned v, const Words<T, VB> &sv, const Words<T, VB> &wv) {
            // (the nearest integer, ties to even, is in the low byte after 1.5 * 2^23
            // is added)
            float f[EV], g[EV];
            sv.unpack(f);
            wv.unpack(g);
            uint32_t c[EV];
#pragma unroll
            for (int i = 0; i < EV; ++i)
                c[i] = some ? __float_as_uint(__fadd_rn(__fmul_rn(f[i] * g[i], inv), kRound)) : 0u;
            if (LB == VB && a.whole_codes) {
#pragma unroll
                for (int i = 0; i < EV; i += 4)
                    c[i / 4] = __byte_perm(__byte_perm(c[i], c[i + 1], 0x0040),
                                           __byte_perm(c[i + 2], c[i + 3], 0x0040), 0x5410);
                if constexpr (EV == 8)
                    reinterpret_cast<uint2 *>(q)[v] = make_uint2(c[0], c[1]);
                else
                    reinterpret_cast<uint32_t *>(q)[v] = c[0];
            } else {
#pragma unroll
                for (int i = 0; i < EV; ++i) {
                    const long long at = column<T, VB, LB>(v, i);
                    if (at < a.H) q[at] = static_cast<unsigned char>(c[i]);
                }
            }
        };
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (tx + h * nx < nvec) put(tx + h * nx, s[h], w[h]);
        for (unsigned v = tx + kHeld * nx; v < nvec; v += nx) {
            Words<T, VB> sv, wv;
            tail(v, true, sv, wv);
            put(v, sv, wv);
        }
        if (tx == 0)
            a.scale[r] = !finite ? __int_as_float(0x7FFFFFFF)
                                 : (some ? __fdiv_rn(amax, 127.f) * rho : 0.f);
    } else {
        constexpr int FORMAT = OUT == kFp4Mx ? SGEMM_FP4_MX : SGEMM_FP4_NV;
        const fp4::RowScale rs = fp4::row_scale(FORMAT, big);
        unsigned char *q = a.q + r * a.pq, *sf = a.sf + fp4::scale_row(r, a.sf_tiles);
        auto put = [&](unsigned v, const Words<T, VB> &sv, const Words<T, VB> &wv) {
            float f[EV], g[EV];
            sv.unpack(f);
            wv.unpack(g);
#pragma unroll
            for (int i = 0; i < EV; ++i) f[i] *= g[i];
            fp4::store_vectors<FORMAT>(f, v, nvec, rs, q, sf);
        };
        // (every lane of a warp that has a vector: blocks span lanes)
        const unsigned w0 = tx & ~31u;
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (w0 + h * nx < nvec) put(tx + h * nx, s[h], w[h]);
        for (unsigned v = tx + kHeld * nx; (v & ~31u) < nvec; v += nx) {
            Words<T, VB> sv, wv;
            sv.zero();
            wv.zero();
            if (v < nvec) tail(v, true, sv, wv);
            put(v, sv, wv);
        }
        if (tx == 0) a.scale[r] = a.H > 0 ? rs.scale * rho : 0.f;
    }
}

struct Launch {
    const Args &args;
    int out, num_sms;
    cudaStream_t st;
    template <class T, int LB, int OUT>
    int go() const
    {
        // narrower loads make up a vector of 16 bytes (4 bits: of four values)
        constexpr int V4 = 4 * static_cast<int>(sizeof(T));
        constexpr int VB = OUT == kRow || OUT == kI8 ? 16 : LB > V4 ? LB : V4;
        constexpr int EV = Words<T, VB>::N;
        Args a = args;
        a.nvec = vectors<T, VB, LB, OUT == kRow || OUT == kI8>(a.H);
        a.whole_codes = OUT == kI8 && rows::aligned_to(a.q, EV) && a.pq % EV == 0;
        const int held = a.M <= num_sms ? 1 : kHeld;  // few rows: more threads on each
        const int tx = rows::pow2_threads((a.nvec + held - 1) / held, 32, 256), ty = 256 / tx;
        const dim3 block(static_cast<unsigned>(tx), static_cast<unsigned>(ty));
        const dim3 grid(static_cast<unsigned>((static_cast<long long>(a.M) + ty - 1) / ty));
        return launch_dependent(norm_kernel<T, VB, LB, OUT>, grid, block, 0, 1, st, a);
    }
    template <class T, int LB>
    int run() const
    {
        if (out == kI8) return go<T, LB, kI8>();
        if (out == kFp4Mx) return go<T, LB, kFp4Mx>();
        if (out == kFp4Nv) return go<T, LB, kFp4Nv>();
        return go<T, LB, kRow>();
    }
};

// ---------------------------------------------------------------- gradient
//
// A block takes every gridDim.x-th group of rows; a thread keeps its columns'
// sums for dweight in registers over all of them, and the block writes one
// partial row, which the second kernel adds in the blocks' order.  (Columns
// past the registers' are added up in the partial row itself.)  With two vectors a
// thread, the next rows are on their way while these are reduced: two blocks of
// 256 threads a multiprocessor, 8192 x 4096 bf16 51.4 us (5.2 TB/s; without the rows
// ahead 64, on three blocks, whose registers spill, 77, with one vector on 512
// threads 72).

constexpr int kGradRows = 608;  // partial rows, at most

struct GradArgs {
    int M, H;
    unsigned nvec;
    float eps;
    const char *s, *w, *dy, *ds;
    char *dx;
    long long ps, pdy, pds, pdx;
    float *part;  // null: dweight is not wanted
};

// HELD: vectors of a row that a thread keeps.
template <class T, int VB, int LB, int HELD>
__global__ void __launch_bounds__(256, 2) grad_kernel(const GradArgs a)
{
    constexpr int EV = Words<T, VB>::N;
    __shared__ float2 part[2][8];
    extern __shared__ float columns[];  // half the groups' columns
    dependent_release();
    dependent_wait();
    const unsigned tx = threadIdx.x, nx = blockDim.x, ny = blockDim.y, warps = nx >> 5;
    const unsigned first = threadIdx.y * warps;
    float acc[HELD][EV];
    Words<T, VB> w[HELD];
    auto weight = [&](unsigned v, Words<T, VB> &wv) {
        if (a.w != nullptr) {
            get<T, VB, LB, true>(wv, a.w, v, a.H);
        } else {
            float one[EV];
#pragma unroll
            for (int i = 0; i < EV; ++i) one[i] = 1.f;
            wv.pack(one);
        }
    };
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
        w[h].zero();
        if (tx + h * nx < a.nvec) weight(tx + h * nx, w[h]);
#pragma unroll
        for (int i = 0; i < EV; ++i) acc[h][i] = 0.f;
    }
    float *mine = a.part + static_cast<long long>(blockIdx.x) * a.H;
    const long long step = static_cast<long long>(gridDim.x) * ny;
    const long long turns = (a.M + step - 1) / step;
    auto row_of = [&](long long turn) { return (turn * gridDim.x + blockIdx.x) * ny + threadIdx.y; };
    Words<T, VB> sv[HELD], gv[HELD], dv[HELD];
    // this thread's vectors of row r (zeros past the last row)
    auto load = [&](long long r, Words<T, VB> (&x)[HELD], Words<T, VB> (&g)[HELD],
                    Words<T, VB> (&d)[HELD]) {
#pragma unroll
        for (int h = 0; h < HELD; ++h) {
            const unsigned v = tx + h * nx;
            x[h].zero();
            g[h].zero();
            d[h].zero();
            if (r < a.M && v < a.nvec) {
                get<T, VB, LB, true>(x[h], a.s + r * a.ps, v, a.H);
                get<T, VB, LB, true>(g[h], a.dy + r * a.pdy, v, a.H);
                if (a.ds != nullptr) get<T, VB, LB, true>(d[h], a.ds + r * a.pds, v, a.H);
            }
        }
    };
    constexpr bool AHEAD = HELD <= 2;
    if (AHEAD) load(row_of(0), sv, gv, dv);
    int buf = 0;
    for (long long turn = 0; turn < turns; ++turn, buf ^= 1) {
        const long long r = row_of(turn);
        const bool live = r < a.M;
        const long long row = live ? r : 0;
        const unsigned nvec = live ? a.nvec : 0;
        const char *s = a.s + row * a.ps, *dy = a.dy + row * a.pdy, *ds = a.ds + row * a.pds;
        char *dx = a.dx + row * a.pdx;
        Words<T, VB> ns[HELD], ng[HELD], nd[HELD];
        if (AHEAD)
            load(turn + 1 < turns ? row_of(turn + 1) : a.M, ns, ng, nd);
        else
            load(r, sv, gv, dv);
        float square = 0.f, inner = 0.f;
        auto gather = [&](const Words<T, VB> &x, const Words<T, VB> &g, const Words<T, VB> &wv) {
            float fx[EV], fg[EV], fw[EV];
            x.unpack(fx);
            g.unpack(fg);
            wv.unpack(fw);
#pragma unroll
            for (int i = 0; i < EV; ++i) {
                square = fmaf(fx[i], fx[i], square);
                inner = fmaf(fw[i] * fg[i], fx[i], inner);
            }
        };
#pragma unroll
        for (int h = 0; h < HELD; ++h) gather(sv[h], gv[h], w[h]);
        for (unsigned v = tx + HELD * nx; v < nvec; v += nx) {
            Words<T, VB> x, g, wv;
            get<T, VB, LB, true>(x, s, v, a.H);
            get<T, VB, LB, true>(g, dy, v, a.H);
            weight(v, wv);
            gather(x, g, wv);
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
            square += __shfl_xor_sync(0xffffffffu, square, d);
            inner += __shfl_xor_sync(0xffffffffu, inner, d);
        }
        if (warps > 1) {
            // (two buffers: a thread still reads one while the next turn fills the other)
            if ((tx & 31) == 0) part[buf][first + (tx >> 5)] = make_float2(square, inner);
            __syncthreads();
            // (a warp's lanes take the warps' sums: eight of them at most)
            float2 p = make_float2(0.f, 0.f);
            if ((tx & 31) < warps) p = part[buf][first + (tx & 31)];
#pragma unroll
            for (int d = 4; d > 0; d /= 2) {
                p.x += __shfl_xor_sync(0xffffffffu, p.x, d);
                p.y += __shfl_xor_sync(0xffffffffu, p.y, d);
            }
            square = __shfl_sync(0xffffffffu, p.x, 0);
            inner = __shfl_sync(0xffffffffu, p.y, 0);
        }
        const float n = static_cast<float>(a.H);
        const float rho = rsqrtf(__fdiv_rn(square, n) + a.eps);
        // (where the squares leave the range, so may s dy and its sum: rho 0 takes them
        // out by s, not by a product that is an infinity already)
        const float c = rho == 0.f ? 0.f : rho * rho * __fdiv_rn(inner, n);
        const float one = rho == 0.f ? 0.f : 1.f;
        auto put = [&](unsigned v, const Words<T, VB> &x, const Words<T, VB> &g, const Words<T, VB> &wv,
                       const Words<T, VB> &d, float (&dyx)[EV]) {
            float fx[EV], fg[EV], f[EV], fd[EV];
            x.unpack(fx);
            g.unpack(fg);
            wv.unpack(f);
            d.unpack(fd);
#pragma unroll
            for (int i = 0; i < EV; ++i) {
                f[i] = fmaf(rho, f[i] * fg[i] - fx[i] * c, fd[i]);
                dyx[i] = fg[i] * (fx[i] * one);
            }
            Words<T, VB> o;
            o.pack(f);
            set<T, VB, LB, true>(o, dx, v, a.H);
        };
#pragma unroll
        for (int h = 0; h < HELD; ++h) {
            sv[h].forget();
            gv[h].forget();
            w[h].forget();
        }
#pragma unroll
        for (int h = 0; h < HELD; ++h)
            if (tx + h * nx < nvec) {
                float dyx[EV];
                put(tx + h * nx, sv[h], gv[h], w[h], dv[h], dyx);
#pragma unroll
                for (int i = 0; i < EV; ++i) acc[h][i] = fmaf(dyx[i], rho, acc[h][i]);
            }
        for (unsigned v = tx + HELD * nx; v < nvec; v += nx) {
            Words<T, VB> x, g, wv, d;
            get<T, VB, LB, true>(x, s, v, a.H);
            get<T, VB, LB, true>(g, dy, v, a.H);
            d.zero();
            if (a.ds != nullptr) get<T, VB, LB, true>(d, ds, v, a.H);
            weight(v, wv);
            float dyx[EV];
            put(v, x, g, wv, d, dyx);
            if (a.part != nullptr) {  // (a row of its own: one group here)
#pragma unroll
                for (int i = 0; i < EV; ++i) {
                    const long long at = column<T, VB, LB>(v, i);
                    if (at < a.H) mine[at] = fmaf(dyx[i], rho, turn > 0 ? mine[at] : 0.f);
                }
            }
        }
        if (AHEAD)
#pragma unroll
            for (int h = 0; h < HELD; ++h) {
                sv[h] = ns[h];
                gv[h] = ng[h];
                dv[h] = nd[h];
            }
    }
    if (a.part == nullptr) return;
    // the groups' sums, the upper half added to the lower until one is left, to the
    // block's partial row
    for (unsigned half = ny / 2; half > 0; half /= 2) {
        if (threadIdx.y >= half && threadIdx.y < 2 * half)
#pragma unroll
            for (int h = 0; h < HELD; ++h)
#pragma unroll
                for (int i = 0; i < EV; ++i)
                    columns[((threadIdx.y - half) * HELD * EV + h * EV + i) * nx + tx] = acc[h][i];
        __syncthreads();
        if (threadIdx.y < half)
#pragma unroll
            for (int h = 0; h < HELD; ++h)
#pragma unroll
                for (int i = 0; i < EV; ++i)
                    acc[h][i] += columns[(threadIdx.y * HELD * EV + h * EV + i) * nx + tx];
        __syncthreads();
    }
    if (threadIdx.y == 0)
#pragma unroll
        for (int h = 0; h < HELD; ++h) {
            const unsigned v = tx + h * nx;
#pragma unroll
            for (int i = 0; i < EV; ++i) {
                const long long at = column<T, VB, LB>(v, i);
                if (v < a.nvec && at < a.H) mine[at] = acc[h][i];
            }
        }
}

// dweight: the partial rows added in order, 32 columns a block, 32 threads a
// column.
__global__ void __launch_bounds__(1024) columns_kernel(int H, int parts, const float *part,
                                                       float *dweight)
{
    __shared__ float sums[32][33];
    dependent_release();
    dependent_wait();
    const int c = static_cast<int>(threadIdx.x) & 31, g = static_cast<int>(threadIdx.x) >> 5;
    const long long h = static_cast<long long>(blockIdx.x) * 32 + c;
    float s = 0.f;
    if (h < H)
#pragma unroll 8
        for (int p = g; p < parts; p += 32) s += part[static_cast<long long>(p) * H + h];
    sums[g][c] = s;
    __syncthreads();
    s = sums[c][g];
#pragma unroll
    for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
    const long long to = static_cast<long long>(blockIdx.x) * 32 + g;
    if (c == 0 && to < H) dweight[to] = s;
}

// Partial rows of a call.
inline int partial_rows(int M) { return M < kGradRows ? M : kGradRows; }

struct GradLaunch {
    const GradArgs &args;
    int num_sms;
    float *dweight;
    cudaStream_t st;
    // The kernel for a.nvec vectors a row; parts: its blocks.
    template <class T, int VB, int LB, int HELD>
    int rows_pass(const GradArgs &a, int &parts) const
    {
        constexpr int EV = Words<T, VB>::N;
        const int tx = rows::pow2_threads((a.nvec + HELD - 1) / HELD, 32, 256), ty = 256 / tx;
        const long long groups = (static_cast<long long>(a.M) + ty - 1) / ty;
        parts = static_cast<int>(groups < 2LL * num_sms ? groups : 2LL * num_sms);
        if (parts > partial_rows(a.M)) parts = partial_rows(a.M);
        const dim3 block(static_cast<unsigned>(tx), static_cast<unsigned>(ty));
        const size_t smem = sizeof(float) * HELD * EV * tx * (ty / 2);
        return launch_dependent(grad_kernel<T, VB, LB, HELD>,
                                dim3(static_cast<unsigned>(parts)), block, smem, 1, st, a);
    }
    template <class T, int LB>
    int run() const
    {
        constexpr int VB = 16;
        GradArgs a = args;
        a.nvec = vectors<T, VB, LB, true>(a.H);
        int parts = 0;
        if (a.M > 0) {
            const int st_ = a.nvec <= 512 ? rows_pass<T, VB, LB, 2>(a, parts)
                                          : rows_pass<T, VB, LB, 4>(a, parts);
            if (st_ != SGEMM_OK) return st_;
        }
        if (dweight == nullptr) return SGEMM_OK;
        return launch_dependent(columns_kernel, dim3(static_cast<unsigned>((a.H + 31LL) / 32)),
                                dim3(1024), 0, 1, st, a.H, parts,
                                static_cast<const float *>(a.part), dweight);
    }
};

// ------------------------------------------------------------ entry points

struct Stream {  // the arguments the three forward calls share
    int type, M, H;
    float eps;
    const void *x;
    int ldx;
    const void *res;
    int ldr;
    const void *weight;
    void *sum;
    int lds;
};

bool eps_ok(float eps) { return eps >= 1.17549435e-38f && eps <= 3.402823466e38f; }

bool stream_ok(const Stream &s)
{
    if (!rows::valid_type(s.type) || s.M < 0 || s.H < 0 || !eps_ok(s.eps) || s.ldx < 1 ||
        s.ldx < s.H || (s.res != nullptr && (s.ldr < 1 || s.ldr < s.H)) ||
        (s.sum != nullptr && (s.lds < 1 || s.lds < s.H)))
        return false;
    const int es = rows::elem_size(s.type);
    return rows::aligned_to(s.x, es) && rows::aligned_to(s.res, es) &&
           rows::aligned_to(s.weight, es) && rows::aligned_to(s.sum, es) &&
           (s.M == 0 || s.H == 0 || s.x != nullptr);
}

int forward(const Stream &s, Args a, int out, rows::Width width, void *stream)
{
    int num_sms = 0;
    unsigned int *status = nullptr;
    if (!current_sm103(&num_sms, &status)) return SGEMM_ERR_UNSUPPORTED;
    const long long es = rows::elem_size(s.type);
    a.M = s.M;
    a.H = s.H;
    a.eps = s.eps;
    a.x = static_cast<const char *>(s.x);
    a.res = static_cast<const char *>(s.res);
    a.w = static_cast<const char *>(s.weight);
    a.sum = static_cast<char *>(s.sum);
    a.px = s.ldx * es;
    a.pr = s.res != nullptr ? s.ldr * es : 0;
    a.ps = s.sum != nullptr ? s.lds * es : 0;
    width.add(a.x).add(a.px).add(a.res).add(a.pr).add(a.w).add(a.sum).add(a.ps).add(s.H * es);
    return rows::with_vec(s.type, s.H == 0 ? 16 : width.bytes(),
                          Launch{a, out, num_sms, static_cast<cudaStream_t>(stream)});
}

}  // namespace norm
}  // namespace sg

using namespace sg;

extern "C" {

int sgemm_rms_norm(int type, int M, int H, float eps, const void *x, int ldx, const void *res,
                   int ldr, const void *weight, void *sum, int lds, void *y, int ldy, void *stream)
{
    return c_entry([&]() -> int {
        const norm::Stream s{type, M, H, eps, x, ldx, res, ldr, weight, sum, lds};
        if (!norm::stream_ok(s) || ldy < 1 || ldy < H ||
            !rows::aligned_to(y, rows::elem_size(type)))
            return SGEMM_ERR_INVALID_ARG;
        if (M == 0 || H == 0) return SGEMM_OK;
        if (y == nullptr) return SGEMM_ERR_INVALID_ARG;
        norm::Args a{};
        a.y = static_cast<char *>(y);
        a.py = static_cast<long long>(ldy) * rows::elem_size(type);
        return norm::forward(s, a, norm::kRow, rows::Width().add(a.y).add(a.py), stream);
    });
}

int sgemm_rms_norm_i8(int type, int M, int H, float eps, const void *x, int ldx, const void *res,
                      int ldr, const void *weight, void *sum, int lds, signed char *q, int ldq,
                      float *scale, void *stream)
{
    return c_entry([&]() -> int {
        const norm::Stream s{type, M, H, eps, x, ldx, res, ldr, weight, sum, lds};
        if (!norm::stream_ok(s) || ldq < 1 || ldq < H || !rows::aligned_to(scale, 4))
            return SGEMM_ERR_INVALID_ARG;
        if (M == 0) return SGEMM_OK;
        if (scale == nullptr || (H > 0 && q == nullptr)) return SGEMM_ERR_INVALID_ARG;
        norm::Args a{};
        a.q = reinterpret_cast<unsigned char *>(q);
        a.pq = ldq;
        a.scale = scale;
        return norm::forward(s, a, norm::kI8, rows::Width(), stream);
    });
}

int sgemm_rms_norm_fp4(int type, int format, int M, int H, float eps, const void *x, int ldx,
                       const void *res, int ldr, const void *weight, void *sum, int lds,
                       unsigned char *q, int ldq, unsigned char *sf, float *scale, void *stream)
{
    return c_entry([&]() -> int {
        const norm::Stream s{type, M, H, eps, x, ldx, res, ldr, weight, sum, lds};
        if (!norm::stream_ok(s) || !fp4::valid_format(format) || ldq < 1 || ldq < H ||
            ldq % fp4::kLdStep != 0 || !rows::aligned_to(scale, 4) || !rows::aligned_to(q, 16) ||
            !rows::aligned_to(sf, 16))
            return SGEMM_ERR_INVALID_ARG;
        if (M == 0) return SGEMM_OK;
        if (scale == nullptr || (H > 0 && (q == nullptr || sf == nullptr)))
            return SGEMM_ERR_INVALID_ARG;
        norm::Args a{};
        a.q = q;
        a.pq = ldq / 2;
        a.sf = sf;
        a.sf_tiles = fp4::scale_tiles(format, H);
        a.scale = scale;
        return norm::forward(s, a, format == SGEMM_FP4_MX ? norm::kFp4Mx : norm::kFp4Nv,
                             rows::Width(), stream);
    });
}

size_t sgemm_rms_norm_grad_workspace_size(int M, int H)
{
    if (M < 0 || H < 0) return 0;
    return static_cast<size_t>(norm::partial_rows(M)) * static_cast<size_t>(H) * sizeof(float);
}

int sgemm_rms_norm_grad(int type, int M, int H, float eps, const void *s, int lds,
                        const void *weight, const void *dy, int ldy, const void *dsum, int ldds,
                        void *dx, int ldx, float *dweight, void *workspace,
                        size_t workspace_bytes, void *stream)
{
    return c_entry([&]() -> int {
        if (!rows::valid_type(type) || M < 0 || H < 0 || !norm::eps_ok(eps) || lds < 1 ||
            lds < H || ldy < 1 || ldy < H || ldx < 1 || ldx < H ||
            (dsum != nullptr && (ldds < 1 || ldds < H)))
            return SGEMM_ERR_INVALID_ARG;
        const int es = rows::elem_size(type);
        if (!rows::aligned_to(s, es) || !rows::aligned_to(weight, es) ||
            !rows::aligned_to(dy, es) || !rows::aligned_to(dsum, es) ||
            !rows::aligned_to(dx, es) || !rows::aligned_to(dweight, 4) ||
            !rows::aligned_to(workspace, 16))
            return SGEMM_ERR_INVALID_ARG;
        if (H == 0 || (M == 0 && dweight == nullptr)) return SGEMM_OK;
        if (M > 0 && (s == nullptr || dy == nullptr || dx == nullptr))
            return SGEMM_ERR_INVALID_ARG;
        if (M > 0 && dweight != nullptr &&
            (workspace == nullptr ||
             workspace_bytes < sgemm_rms_norm_grad_workspace_size(M, H)))
            return SGEMM_ERR_INVALID_ARG;
        int num_sms = 0;
        unsigned int *status = nullptr;
        if (!current_sm103(&num_sms, &status)) return SGEMM_ERR_UNSUPPORTED;
        norm::GradArgs a{};
        a.M = M;
        a.H = H;
        a.eps = eps;
        a.s = static_cast<const char *>(s);
        a.w = static_cast<const char *>(weight);
        a.dy = static_cast<const char *>(dy);
        a.ds = static_cast<const char *>(dsum);
        a.dx = static_cast<char *>(dx);
        a.ps = static_cast<long long>(lds) * es;
        a.pdy = static_cast<long long>(ldy) * es;
        a.pds = dsum != nullptr ? static_cast<long long>(ldds) * es : 0;
        a.pdx = static_cast<long long>(ldx) * es;
        a.part = dweight != nullptr ? static_cast<float *>(workspace) : nullptr;
        const int vb = rows::Width()
                           .add(a.s).add(a.w).add(a.dy).add(a.ds).add(a.dx)
                           .add(a.ps).add(a.pdy).add(a.pds).add(a.pdx)
                           .add(static_cast<uint64_t>(H) * es)
                           .bytes();
        return rows::with_vec(type, vb, norm::GradLaunch{a, num_sms, dweight,
                                                         static_cast<cudaStream_t>(stream)});
    });
}

}  // extern "C"

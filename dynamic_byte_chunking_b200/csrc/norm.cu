// Residual RMS norm, its 8-bit form, row quantisation and the norm's backward
// pass (formulas at the declarations in dbc.h).
//
// All of it is bound by HBM.  A row is read once into registers, its sum of
// squares (and the maximum under the 8-bit code) is reduced over the threads
// that hold it, and it is written from there.  Sums are fp32; a row whose sum
// of squares leaves [1e-30, 1e37] (squares that overflow or vanish in fp32, or
// something not finite) is summed again in fp64 from the registers.
//
// Rows of up to 128 fragments of 16 bytes belong to a team of 8, 16 or 32
// lanes, R rows at a time so that each thread keeps about four loads per input
// in flight; wider rows belong to a CTA that copies the next ones ahead.  The
// backward pass, whose threads keep their columns' dw sums in registers, copies
// ahead at every width.  Rows off the 16-byte grid are in norm_odd.cuh.
//
// Measured (us on the device, of a copy's time for the same bytes; all inputs
// larger than L2): 2.2 M x 256 bf16 with residual 650 (107 %), 262144 x 512 159
// (104 %), 20000 x 4096 104 (98 %); the 8-bit form 155 (94 %) and 104 (86 %),
// where the arithmetic of the codes shows (two issue slots of three are taken);
// backward 2.2 M x 256 521 (101 %), 100000 x 512 with ds 67 (95 %), 65536 x 256
// with ds 26.7 (78 %, with the join of the dw lines), 32749 x 1536 with fp32 dy 90
// (69 %: its 136 registers leave an SM 12 warps; fewer registers spill (153 us),
// fewer columns per thread pay more barriers (100 us)).
#include "norm.cuh"
#include "norm_odd.cuh"

namespace dbc {
namespace nm {

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// One row from registers to memory (s, then y or q), fragment column `col`.
template <class T, int NE, int MODE, bool RES>
__device__ __forceinline__ void write_frag(const FwdArgs &a, int64_t r, int col, const Frag<T, NE> &f,
                                           const float (&w)[NE], const RowFactor &k, const Quant &qn) {
    if (RES && a.s) f.store(static_cast<T *>(a.s) + r * a.ss + col);
    float o[NE];
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) {
        const float2 wi = make_float2(w[2 * i], w[2 * i + 1]);
        float2 v = f.pair(i);
        if (MODE == kPlain) {
            if (k.pre != 1.f) v = mul2(v, both(k.pre));
            v = mul2(mul2(v, both(k.rstd)), wi);
        } else if (weighs(MODE)) {
            v = mul2(v, wi);
        }
        o[2 * i] = v.x, o[2 * i + 1] = v.y;
    }
    if (MODE == kPlain) store_as<NE>(a.y, a.y_bf16, r * a.ys + col, o);
    else qn.template store<narrow<T>(MODE), NE>(a.q + r * a.qs + col, o);
}

// Sum of squares (two chains) and largest |p| of a fragment.
template <int MODE, class T, int NE>
__device__ __forceinline__ void stats(const Frag<T, NE> &f, const float (&w)[NE], float2 &ss, float &m) {
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) {
        const float2 v = f.pair(i);
        if (norms(MODE)) ss = fma2(v, v, ss);
        if (MODE != kPlain) m = abs_max(m, weighs(MODE) ? mul2(v, make_float2(w[2 * i], w[2 * i + 1])) : v);
    }
}

// More dynamic shared memory than any launch here asks for (the tiles of odd rows take up to 197 KB, at eight
// rows of 1024 fp32 elements), and with what the kernels declare beside it within a CTA's 227 KB.
constexpr int kMostSmem = 208 * 1024;

// Rows in shared memory at a time of kernels that copy ahead: B bytes per thread and row, up to MAXT
// threads; 64 KB a CTA of 256 threads (three to an SM), and what fits beside `other` bytes for the wide ones.
constexpr int block_stages(int B, int MAXT, int other = 0) {
    const int s = MAXT > 256 ? (kMostSmem - other) / (B * MAXT) : 64 * 1024 / (B * MAXT);
    return s < 1 ? 1 : s > 4 ? 4 : s;
}

// R rows per team of W lanes, NV fragments per lane and row.
template <class T, int NE, int MODE, bool RES, int W, int NV, int R>
__global__ void __launch_bounds__(kThreads, weighs(MODE) ? 4 : 0) team_kernel(const FwdArgs a) {
    const int64_t team = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / W;
    const int t = threadIdx.x % W;
    if ((((int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31)) / W) * R >= a.N) return;   // a whole warp
    const int64_t r0 = team * R;
    Frag<T, NE> f[R][NV], g[R][NV];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * W + t) * NE;
            f[i][j].zero();
            if (r0 + i < a.N && col < a.d) {
                f[i][j].load(static_cast<const T *>(a.x) + (r0 + i) * a.xs + col);
                if (RES) g[i][j].load(static_cast<const T *>(a.res) + (r0 + i) * a.rs + col);
            }
        }
    constexpr bool LATE = MODE == kPlain && NV > 2;          // the weight, where registers are short
    float w[NV][NE];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (j * W + t) * NE;
#pragma unroll
        for (int i = 0; i < NE; ++i) w[j][i] = 1.f;
        if (norms(MODE) && !LATE && col < a.d) a.w.get<NE>(col, w[j]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float2 s2 = make_float2(0.f, 0.f);
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (RES && r0 + i < a.N && (j * W + t) * NE < a.d) f[i][j].add(g[i][j]);
            stats<MODE>(f[i][j], w[j], s2, m);
        }
        const float ss = norms(MODE) ? team_reduce<W>(s2.x + s2.y, Add()) : 1.f;
        if (MODE != kPlain) m = team_reduce<W>(m, AbsMax());
        RowFactor k(ss, a);
        if (norms(MODE) && __any_sync(0xffffffffu, !(ss >= kLow && ss <= kHigh))) {
            double t2 = 0;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < NE; ++e) t2 += (double)f[i][j].at(e) * f[i][j].at(e);
            t2 = team_reduce<W>(t2, Add());
            if (!(ss >= kLow && ss <= kHigh)) k = RowFactor(t2, a);   // not the warp's other rows
            if (!isfinite(t2)) {
                m = __int_as_float(0x7fc00000);
                if (t == 0) flag(a.st, DBC_ERR_NONFINITE);
            }
        }
        const Quant qn(m);
        if (r0 + i < a.N) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = (j * W + t) * NE;
                if (LATE && col < a.d) a.w.get<NE>(col, w[j]);
                if (col < a.d) write_frag<T, NE, MODE, RES>(a, r0 + i, col, f[i][j], w[j], k, qn);
            }
            if (MODE != kPlain && t == 0) {
                a.scale[r0 + i] = row_scale<MODE>(qn, k);
                if (qn.bad) flag(a.st, DBC_ERR_NONFINITE);
            }
        }
    }
}

// Rows on their way to a thread: the fragments that it will work on, copied by itself into its own slots
// of shared memory some rows ahead (cp.async; nobody else reads them, so no barrier).  An array's
// fragments are `threads` 16-byte units (or one smaller unit) apart, so that a warp's accesses are whole
// lines; `at` is the offset per thread of the fragment inside a stage.
template <int NE, class V>
__device__ __forceinline__ void ring_copy(uint32_t stage, int at, int threads, const V *src, bool in) {
    constexpr int bytes = NE * (int)sizeof(V), u = bytes < 16 ? bytes : 16;
    const uint32_t dst = stage + at * threads + threadIdx.x * u;
    if constexpr (bytes >= 16) {
#pragma unroll
        for (int i = 0; i < bytes / 16; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * threads * 16),
                         "l"(reinterpret_cast<const char *>(src) + i * 16), "r"(in ? 16 : 0)
                         : "memory");
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(in ? bytes : 0), "n"(bytes)
                     : "memory");
    }
}
template <int NE, class V>
__device__ __forceinline__ void ring_read(Frag<V, NE> &f, const char *stage, int at, int threads) {
    constexpr int bytes = NE * (int)sizeof(V), u = bytes < 16 ? bytes : 16;
    const char *p = stage + at * threads + threadIdx.x * u;
    uint32_t w[bytes / 4];
    if constexpr (u == 16) {
#pragma unroll
        for (int i = 0; i < bytes / 16; ++i) {
            const uint4 x = *reinterpret_cast<const uint4 *>(p + i * threads * 16);
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
    } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x, w[1] = x.y;
    }
    f.from_words(w);
}
template <int S>
__device__ __forceinline__ void ring_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
}

// Wide rows, forward: CTAs of blockDim.x threads walk the rows, NV fragments of one row per thread, the
// next S - 1 rows on their way.
template <class T, int NE, int MODE, bool RES, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) block_kernel(const FwdArgs a) {
    constexpr int U = NE * (int)sizeof(T), B = NV * U * (RES ? 2 : 1);       // bytes of a fragment, of a thread's row
    constexpr int S = block_stages(B, MAXT);
    extern __shared__ __align__(16) char smem[];
    __shared__ float2 part[2][32];
    __shared__ double wide[32];
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
    const int t = threadIdx.x, W = blockDim.x, lane = t & 31, warp = t >> 5, warps = W >> 5;
    auto start = [&](int64_t r, int st) {
        const bool row = r < a.N;
        const T *const x = static_cast<const T *>(a.x) + (row ? r : 0) * a.xs;
        const T *const g = RES ? static_cast<const T *>(a.res) + (row ? r : 0) * a.rs : x;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * W + t) * NE;
            const bool in = row && col < a.d;
            ring_copy<NE>(base + st * B * W, j * U, W, x + (in ? col : 0), in);
            if (RES) ring_copy<NE>(base + st * B * W, (NV + j) * U, W, g + (in ? col : 0), in);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int k = 0; k < S - 1; ++k) start(blockIdx.x + (int64_t)k * gridDim.x, k);
    // The weight stays in registers, but in the plain norm of up to 512 fragments, which does better
    // with more warps than with them (20000 x 4096: 105 us against 114; 8192 x 8192: 99 against 96).
    constexpr bool LATE = MODE == kPlain && MAXT <= 256;
    float w[NV][NE];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (j * W + t) * NE;
#pragma unroll
        for (int i = 0; i < NE; ++i) w[j][i] = 1.f;
        if (norms(MODE) && !LATE && col < a.d) a.w.get<NE>(col, w[j]);
    }
    int ph = 0, st = 0;
    for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x, ph ^= 1) {
        start(r + (int64_t)(S - 1) * gridDim.x, st == 0 ? S - 1 : st - 1);
        ring_wait<S>();
        Frag<T, NE> f[NV];
        float2 s2 = make_float2(0.f, 0.f);
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            ring_read<NE>(f[j], smem + st * B * W, j * U, W);
            if constexpr (RES) {
                Frag<T, NE> g;
                ring_read<NE>(g, smem + st * B * W, (NV + j) * U, W);
                f[j].add(g);                             // zeros past the row's end
            }
            stats<MODE>(f[j], w[j], s2, m);
        }
        float ss = norms(MODE) ? team_reduce<32>(s2.x + s2.y, Add()) : 0.f;
        if (MODE != kPlain) m = team_reduce<32>(m, AbsMax());
        if (lane == 0) part[ph][warp] = make_float2(ss, m);
        __syncthreads();             // the other buffer's readers are past the row before's barrier
        const float2 v = lane < warps ? part[ph][lane] : make_float2(0.f, 0.f);
        if (norms(MODE)) ss = team_reduce<32>(v.x, Add());
        if (MODE != kPlain) m = team_reduce<32>(v.y, AbsMax());
        RowFactor k(ss, a);
        if (norms(MODE) && !(ss >= kLow && ss <= kHigh)) {     // the same in every thread
            double t2 = 0;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < NE; ++e) t2 += (double)f[j].at(e) * f[j].at(e);
            t2 = team_reduce<32>(t2, Add());
            if (lane == 0) wide[warp] = t2;
            __syncthreads();
            t2 = team_reduce<32>(lane < warps ? wide[lane] : 0.0, Add());
            k = RowFactor(t2, a);
            if (!isfinite(t2)) {
                m = __int_as_float(0x7fc00000);
                if (t == 0) flag(a.st, DBC_ERR_NONFINITE);
            }
        }
        const Quant qn(m);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * W + t) * NE;
            if (col < a.d) {
                if (LATE) a.w.get<NE>(col, w[j]);
                write_frag<T, NE, MODE, RES>(a, r, col, f[j], w[j], k, qn);
            }
        }
        if (MODE != kPlain && t == 0) {
            a.scale[r] = row_scale<MODE>(qn, k);
            if (qn.bad) flag(a.st, DBC_ERR_NONFINITE);
        }
        if (++st == S) st = 0;
    }
}

// The same for the backward pass: dy, s and ds of a thread's row; SUMS: with the fp64 sums of the threads' columns
// behind them.
template <class TY, class T, int NE, int NV, int MAXT, bool SUMS>
struct Ring {
    static constexpr int UY = NE * (int)sizeof(TY), U = NE * (int)sizeof(T), kS = NV * UY, kDs = kS + NV * U;
    static constexpr int kSums = SUMS ? NV * NE * (int)sizeof(double) : 0;          // of a thread
    static constexpr int B = kDs + NV * U, S = block_stages(B, MAXT, kSums * MAXT);
    static constexpr int smem(int threads) { return (S * B + kSums) * threads; }
    static __device__ __forceinline__ double *sums(char *smem, int threads) {
        return reinterpret_cast<double *>(smem + S * B * threads);
    }
    // Where the next row to copy lies; advanced by `step` rows at a time (pointers, not products of rows
    // and strides: three of those a row were a tenth of the instructions).
    struct Walk {
        const TY *y;
        const T *s, *ds;
        int64_t left, step, dy, dss, dds;
        __device__ __forceinline__ Walk(const BwdArgs &a, int64_t r, int64_t step_)
            : y(static_cast<const TY *>(a.dy) + r * a.ys), s(static_cast<const T *>(a.s) + r * a.ss),
              ds(a.ds ? static_cast<const T *>(a.ds) + r * a.ds_s : nullptr), left(a.N - r), step(step_),
              dy(step_ * a.ys), dss(step_ * a.ss), dds(step_ * a.ds_s) {}
    };
    // Starts the copies of that row (nothing, but still a group, when it is past the end).
    static __device__ __forceinline__ void start(const BwdArgs &a, Walk &k, uint32_t base, int stage, int t, int W,
                                                 int threads) {
        const uint32_t st = base + stage * B * threads;
        const bool row = k.left > 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * W + t) * NE;
            const bool in = row && col < a.d;
            ring_copy<NE>(st, j * UY, threads, in ? k.y + col : static_cast<const TY *>(a.dy), in);
            ring_copy<NE>(st, kS + j * U, threads, in ? k.s + col : static_cast<const T *>(a.s), in);
            if (a.ds) ring_copy<NE>(st, kDs + j * U, threads, in ? k.ds + col : static_cast<const T *>(a.ds), in);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        k.y += k.dy;
        k.s += k.dss;
        if (a.ds) k.ds += k.dds;
        k.left -= k.step;
    }
    static __device__ __forceinline__ void wait() { ring_wait<S>(); }
    // Fragment j of the row's dy and s; then of its ds.
    static __device__ __forceinline__ void get(const char *smem, int stage, int j, int threads, Frag<TY, NE> &y,
                                               Frag<T, NE> &f) {
        ring_read<NE>(y, smem + stage * B * threads, j * UY, threads);
        ring_read<NE>(f, smem + stage * B * threads, kS + j * U, threads);
    }
    static __device__ __forceinline__ void get_ds(const char *smem, int stage, int j, int threads, Frag<T, NE> &g) {
        ring_read<NE>(g, smem + stage * B * threads, kDs + j * U, threads);
    }
};

template <class TY, class T, int NE>
__device__ __forceinline__ void bwd_stats(const Frag<TY, NE> &y, const Frag<T, NE> &f, const float (&w)[NE],
                                          float2 &ss, float2 &sg) {
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) {
        const float2 v = f.pair(i);
        ss = fma2(v, v, ss);
        sg = fma2(mul2(y.pair(i), make_float2(w[2 * i], w[2 * i + 1])), v, sg);
    }
}
template <class TY, class T, int NE>
__device__ __forceinline__ void bwd_stats_wide(const Frag<TY, NE> &y, const Frag<T, NE> &f, const float (&w)[NE],
                                               double &ss, double &sg) {
#pragma unroll 1
    for (int i = 0; i < NE; ++i) {
        float v = 0.f, g = 0.f;
#pragma unroll
        for (int k = 0; k < NE; ++k)
            if (k == i) v = f.at(k), g = y.at(k) * w[k];
        ss += (double)v * v;
        sg += (double)g * v;
    }
}
// Whether the fragment has a g = dy w that is not zero.
template <class TY, int NE>
__device__ __forceinline__ bool any_g(const Frag<TY, NE> &y, const float (&w)[NE]) {
    bool any = false;
#pragma unroll
    for (int i = 0; i < NE; ++i) any |= y.at(i) * w[i] != 0.f;
    return any;
}
template <class Q, bool DW, class TY, class T, int NE>
__device__ __forceinline__ void bwd_frag(const BwdArgs &a, const char *smem, int stage, T *dx, int j, int threads,
                                         const Frag<TY, NE> &y, const Frag<T, NE> &f, const float (&w)[NE],
                                         const BwdFactor &k, float (&acc)[NE]) {
    float o[NE];
    const bool scaled = k.k.pre != 1.f;
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) {
        const float2 wi = make_float2(w[2 * i], w[2 * i + 1]), yi = y.pair(i);
        float2 xh = mul2(f.pair(i), both(k.k.rstd));
        if (scaled) xh = mul2(mul2(f.pair(i), both(k.k.pre)), both(k.k.rstd));
        float2 v = mul2(fma2(xh, both(-k.c), mul2(yi, wi)), both(k.k.rstd));
        if (scaled) v = mul2(v, both(k.k.pre));
        o[2 * i] = v.x, o[2 * i + 1] = v.y;
        if (DW) {
            const float2 s2 = fma2(yi, xh, make_float2(acc[2 * i], acc[2 * i + 1]));
            acc[2 * i] = s2.x, acc[2 * i + 1] = s2.y;
        }
    }
    Frag<T, NE> q;
    if (a.ds) {
        Q::get_ds(smem, stage, j, threads, q);
#pragma unroll
        for (int i = 0; i < NE / 2; ++i) {
            const float2 v = add2(make_float2(o[2 * i], o[2 * i + 1]), q.pair(i));
            o[2 * i] = v.x, o[2 * i + 1] = v.y;
        }
    }
    q.set(o);
    q.store(dx);
}

// Teams of W lanes walk the rows; a lane keeps the dw sums of its own columns
// (fp32 in registers, fp64 in shared memory behind the ring), the CTA joins
// them at the end (a fixed order).
template <class TY, class T, int NE, bool DW, int W, int NV>
__global__ void __launch_bounds__(kThreads, 2) bwd_team_kernel(const BwdArgs a) {
    using Q = Ring<TY, T, NE, NV, kThreads, DW>;
    extern __shared__ __align__(16) char smem[];
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
    const int t = threadIdx.x % W, lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kThreads / W);
    double *const sums = Q::sums(smem, kThreads);         // element i of fragment j at (j * NE + i) * kThreads + thread
    float w[NV][NE], acc[NV][NE];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (j * W + t) * NE;
#pragma unroll
        for (int i = 0; i < NE; ++i) w[j][i] = 1.f, acc[j][i] = 0.f;
        if (col < a.d) a.w.get<NE>(col, w[j]);
    }
    // all teams of a warp take the same number of steps: the first team's row decides
    const int64_t first = (int64_t)blockIdx.x * (kThreads / W) + (threadIdx.x & ~31) / W, mine = lane / W;
    typename Q::Walk walk(a, first + mine, step);
    T *px = static_cast<T *>(a.dx) + (first + mine) * a.xs;
    const int64_t dpx = step * a.xs;
    for (int k = 0; k < Q::S - 1; ++k) Q::start(a, walk, base, k, t, W, kThreads);
    if (DW) {
#pragma unroll
        for (int i = 0; i < NV * NE; ++i) sums[i * kThreads + threadIdx.x] = 0;
    }
    int stage = 0;
    for (int64_t rw = first; rw < a.N;) {
        // kFold rows at a time (all of them where no dw is wanted), then the fold
        const int64_t end = DW ? min(a.N, rw + kFold * step) : a.N;
        for (; rw < end; rw += step, px += dpx) {
            const int64_t r = rw + mine;
            Q::start(a, walk, base, stage == 0 ? Q::S - 1 : stage - 1, t, W, kThreads);
            Q::wait();
            Frag<TY, NE> y[NV];
            Frag<T, NE> f[NV];
            float2 pss = make_float2(0.f, 0.f), psg = pss;
#pragma unroll
            for (int j = 0; j < NV; ++j) Q::get(smem, stage, j, kThreads, y[j], f[j]);
#pragma unroll
            for (int j = 0; j < NV; ++j) bwd_stats(y[j], f[j], w[j], pss, psg);
            const float ss = team_reduce<W>(pss.x + pss.y, Add()), sg = team_reduce<W>(psg.x + psg.y, Add());
            BwdFactor k(ss, sg, a);
            bool odd = !in_range(ss, sg);
            if (__any_sync(0xffffffffu, faint(sg))) {
                bool some = false;
#pragma unroll
                for (int j = 0; j < NV; ++j) some |= any_g(y[j], w[j]);
                odd |= team_any<W>(some) && faint(sg);
            }
            if (__any_sync(0xffffffffu, odd)) {
                double s2 = 0, g2 = 0;
#pragma unroll
                for (int j = 0; j < NV; ++j) bwd_stats_wide(y[j], f[j], w[j], s2, g2);
                s2 = team_reduce<W>(s2, Add());
                g2 = team_reduce<W>(g2, Add());
                if (odd) k = BwdFactor(s2, g2, a);           // not the warp's other rows
                if (t == 0 && (!isfinite(s2) || !isfinite(g2))) flag(a.st, DBC_ERR_NONFINITE);
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = (j * W + t) * NE;
                // read again rather than held (100000 x 512 with ds: 67 us against 71, which spilled)
                if constexpr (NV > 1) Q::get(smem, stage, j, kThreads, y[j], f[j]);
                if (r < a.N && col < a.d)
                    bwd_frag<Q, DW>(a, smem, stage, px + col, j, kThreads, y[j], f[j], w[j], k, acc[j]);
            }
            if (++stage == Q::S) stage = 0;
        }
        if (DW) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                fold_sums<NE, false>(sums + j * NE * kThreads + threadIdx.x, kThreads, acc[j], false);
        }
    }
    if constexpr (DW) {
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += kThreads) {
            const int v = c / NE, e = c % NE;            // lane v % W's fragment v / W has the column
            const double *const at = sums + (v / W * NE + e) * kThreads + v % W;
            double sum = 0;
#pragma unroll
            for (int k = 0; k < kThreads / W; ++k) sum += at[k * W];
            a.part[(int64_t)blockIdx.x * a.d + c] = sum;
        }
    }
}

// Wide rows: one row per CTA at a time, NV fragments per thread.  A thread's fp64 dw sums are in shared memory
// behind the ring or, where that has no room for them (1024 threads), its columns of the CTA's line.  In the
// line element i of fragment v, of V of them, is at i * V + v: whole sectors to a warp.
template <class TY, class T, int NE, bool DW, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > 512 ? 1 : 0)     // (unbounded, 1024 threads got 32 registers and spilled)
    bwd_block_kernel(const BwdArgs a) {
    constexpr bool OWN = DW && MAXT <= 512;
    using Q = Ring<TY, T, NE, NV, MAXT, OWN>;
    extern __shared__ __align__(16) char smem[];
    __shared__ float2 part[2][32];
    __shared__ double2 wide[32];
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
    const int t = threadIdx.x, W = blockDim.x, lane = t & 31, warp = t >> 5, warps = W >> 5;
    float w[NV][NE], acc[NV][NE];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (j * W + t) * NE;
#pragma unroll
        for (int i = 0; i < NE; ++i) w[j][i] = 1.f, acc[j][i] = 0.f;
        if (col < a.d) a.w.get<NE>(col, w[j]);
    }
    typename Q::Walk walk(a, blockIdx.x, gridDim.x);
    T *px = static_cast<T *>(a.dx) + (int64_t)blockIdx.x * a.xs;
    const int64_t dpx = (int64_t)gridDim.x * a.xs;
    for (int k = 0; k < Q::S - 1; ++k) Q::start(a, walk, base, k, t, W, W);
    double *const sums = Q::sums(smem, W), *const line = DW ? a.part + (int64_t)blockIdx.x * a.d : nullptr;
    const int V = a.d / NE;
    int ph = 0, stage = 0;
    bool first = true;
    for (int64_t r = blockIdx.x; r < a.N; first = false) {
        // kFold rows at a time (all of them where no dw is wanted), then the fold
        const int64_t end = DW ? min(a.N, r + kFold * (int64_t)gridDim.x) : a.N;
        for (; r < end; r += gridDim.x, ph ^= 1, px += dpx) {
            Q::start(a, walk, base, stage == 0 ? Q::S - 1 : stage - 1, t, W, W);
            Q::wait();
            Frag<TY, NE> y[NV];
            Frag<T, NE> f[NV];
            float2 pss = make_float2(0.f, 0.f), psg = pss;
#pragma unroll
            for (int j = 0; j < NV; ++j) Q::get(smem, stage, j, W, y[j], f[j]);
#pragma unroll
            for (int j = 0; j < NV; ++j) bwd_stats(y[j], f[j], w[j], pss, psg);
            float ss = team_reduce<32>(pss.x + pss.y, Add()), sg = team_reduce<32>(psg.x + psg.y, Add());
            if (lane == 0) part[ph][warp] = make_float2(ss, sg);
            __syncthreads();             // the other buffer's readers are past the row before's barrier
            const float2 v = lane < warps ? part[ph][lane] : make_float2(0.f, 0.f);
            ss = team_reduce<32>(v.x, Add());
            sg = team_reduce<32>(v.y, Add());
            BwdFactor k(ss, sg, a);
            bool odd = !in_range(ss, sg);                    // the same in every thread
            if (faint(sg)) {
                bool some = false;
#pragma unroll
                for (int j = 0; j < NV; ++j) some |= any_g(y[j], w[j]);
                odd |= __syncthreads_or(some) != 0;
            }
            if (odd) {
                double s2 = 0, g2 = 0;
#pragma unroll
                for (int j = 0; j < NV; ++j) bwd_stats_wide(y[j], f[j], w[j], s2, g2);
                s2 = team_reduce<32>(s2, Add());
                g2 = team_reduce<32>(g2, Add());
                if (lane == 0) wide[warp] = make_double2(s2, g2);
                __syncthreads();
                const double2 v2 = lane < warps ? wide[lane] : make_double2(0, 0);
                s2 = team_reduce<32>(v2.x, Add());
                g2 = team_reduce<32>(v2.y, Add());
                k = BwdFactor(s2, g2, a);
                if (t == 0 && (!isfinite(s2) || !isfinite(g2))) flag(a.st, DBC_ERR_NONFINITE);
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = (j * W + t) * NE;
                if (col < a.d) {
                    // Fragments are read again after the barrier rather than held across it (20000 x 4096 bf16: 109
                    // us against 114; 8192 x 16384 with fp32 dy: 419 against 505), but for fp32 dy at up to 256 threads,
                    // where that costs (32749 x 1536: 95 against 87)
                    if constexpr (sizeof(TY) == 2 || MAXT > 256) Q::get(smem, stage, j, W, y[j], f[j]);
                    bwd_frag<Q, DW>(a, smem, stage, px + col, j, W, y[j], f[j], w[j], k, acc[j]);
                }
            }
            if (++stage == Q::S) stage = 0;
        }
        if (DW) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (OWN) fold_sums<NE, false>(sums + j * NE * W + t, W, acc[j], first);
                else if (j * W + t < V) fold_sums<NE, true>(line + j * W + t, V, acc[j], first);
            }
        }
    }
    if (OWN) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * W + t < V) {
#pragma unroll
                for (int i = 0; i < NE; ++i) line[i * V + j * W + t] = sums[(j * NE + i) * W + t];
            }
    }
}

// dw = the CTAs' lines added up, in a fixed order: 8 columns (two 32-byte
// sectors of every line) per CTA, 128 threads per column.  The lines hold
// element i of fragment v, of V of them, at i * V + v.
__global__ void __launch_bounds__(1024) dw_kernel(const double *part, int lines, int d, int V, float *dw) {
    __shared__ double sm[32][8];
    const int c = threadIdx.x & 7, k = threadIdx.x >> 3, col = blockIdx.x * 8 + c;
    double v[10];                                    // lines <= 148 * 8 < 128 * 10
#pragma unroll
    for (int i = 0; i < 10; ++i) v[i] = col < d && k + i * 128 < lines ? part[(int64_t)(k + i * 128) * d + col] : 0.0;
    double t = 0;
#pragma unroll
    for (int i = 0; i < 10; ++i) t += v[i];
    t += __shfl_xor_sync(0xffffffffu, t, 8);
    t += __shfl_xor_sync(0xffffffffu, t, 16);
    if ((threadIdx.x & 31) < 8) sm[threadIdx.x >> 5][c] = t;
    __syncthreads();
    if (threadIdx.x < 256) {                         // warp w: column w
        t = team_reduce<32>(sm[threadIdx.x & 31][threadIdx.x >> 5], Add());
        const int out = blockIdx.x * 8 + (threadIdx.x >> 5);
        if ((threadIdx.x & 31) == 0 && out < d) dw[out % V * (d / V) + out / V] = (float)t;
    }
}

inline bool aligned_to(const void *p, int64_t e) { return (reinterpret_cast<uintptr_t>(p) % e) == 0; }
inline int64_t esize(int dtype) { return dtype == DBC_BF16 ? 2 : 4; }
inline bool known(int dtype) { return dtype == DBC_F32 || dtype == DBC_BF16; }

// Argument checks shared by the forward entries (shapes first, then pointers,
// which are not looked at for an empty batch).
inline dbc_status check_fwd(const FwdArgs &a, int dtype, int w_dtype, int64_t d, bool norm) {
    if (a.N < 0 || d <= 0) return DBC_ERR_INVALID_ARG;
    if (norm && (!(a.eps > 0.f) || !std::isfinite(a.eps))) return DBC_ERR_INVALID_ARG;
    if (!known(dtype) || (a.w.p && !known(w_dtype)) || d > kMaxD) return DBC_ERR_UNSUPPORTED;
    if (a.s && !a.res) return DBC_ERR_INVALID_ARG;
    if (a.xs < d || (a.res && a.rs < d) || (a.s && a.ss < d)) return DBC_ERR_INVALID_ARG;
    if (a.N == 0) return DBC_OK;
    const int64_t e = esize(dtype);
    if (!a.x || !aligned_to(a.x, e) || !aligned_to(a.res, e) || !aligned_to(a.s, e)) return DBC_ERR_INVALID_ARG;
    if (a.w.p && !aligned_to(a.w.p, esize(w_dtype))) return DBC_ERR_INVALID_ARG;
    return DBC_OK;
}

// Whether rows of `stride` elements of `esz` bytes at p all start on multiples
// of `unit` bytes.
inline bool on_grid(const void *p, int64_t stride, int64_t esz, int64_t unit) {
    return !p || (reinterpret_cast<uintptr_t>(p) % unit == 0 && stride * esz % unit == 0);
}

template <class T, int NE, int MODE, int W, int NV, int R>
dbc_status launch_team(const FwdArgs &a, cudaStream_t st) {
    const int64_t teams = (a.N + R - 1) / R, grid = (teams * W + kThreads - 1) / kThreads;
    if (grid > INT32_MAX) return DBC_ERR_UNSUPPORTED;
    if constexpr (norms(MODE)) {
        if (a.res) {
            team_kernel<T, NE, MODE, true, W, NV, R><<<(unsigned)grid, kThreads, 0, st>>>(a);
            return DBC_OK;
        }
    }
    team_kernel<T, NE, MODE, false, W, NV, R><<<(unsigned)grid, kThreads, 0, st>>>(a);
    return DBC_OK;
}

// As many CTAs as are resident at once, at most `most`; 0 after a CUDA error.
// The runtime's occupancy query costs a third of a small call's host time, so
// each host thread remembers its last answers (they depend on the kernel and
// the launch alone).
constexpr int kSms = 148;
template <class K>
int resident(K kernel, int threads, int smem, int64_t most) {
    struct Answer {
        const void *kernel;
        int threads, smem, per_sm;
    };
    static thread_local Answer known[8] = {};
    static thread_local int at = 0;
    const void *key = reinterpret_cast<const void *>(kernel);
    if (!allow_smem(kernel, kMostSmem)) return 0;
    int per_sm = 0;
    for (const Answer &k : known)
        if (k.kernel == key && k.threads == threads && k.smem == smem) per_sm = k.per_sm;
    if (!per_sm) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1) {
            cudaGetLastError();
            return 0;
        }
        known[at] = {key, threads, smem, per_sm};
        at = (at + 1) % 8;
    }
    return (int)std::min<int64_t>(most, (int64_t)per_sm * kSms);
}

template <class T, int NE, int MODE, bool RES, int NV, int MAXT>
dbc_status launch_block_res(const FwdArgs &a, cudaStream_t st) {
    constexpr int B = NV * NE * (int)sizeof(T) * (RES ? 2 : 1);
    const int threads = ((a.d + NE * NV - 1) / (NE * NV) + 31) / 32 * 32, smem = block_stages(B, MAXT) * B * threads;
    auto *k = block_kernel<T, NE, MODE, RES, NV, MAXT>;
    const int ctas = resident(k, threads, smem, a.N);
    if (!ctas) return DBC_ERR_CUDA;
    k<<<ctas, threads, smem, st>>>(a);
    return DBC_OK;
}
template <class T, int NE, int MODE, int NV, int MAXT>
dbc_status launch_block(const FwdArgs &a, cudaStream_t st) {
    if constexpr (norms(MODE)) {
        if (a.res) return launch_block_res<T, NE, MODE, true, NV, MAXT>(a, st);
    }
    return launch_block_res<T, NE, MODE, false, NV, MAXT>(a, st);
}

// Threads, rows in shared memory (two where that leaves room for a second CTA)
// and bytes of the kernels that give a row to a CTA.
struct OddPlan {
    int threads, stages, smem;
};
inline OddPlan odd_plan(int d, int nv, int in_bytes, int out_bytes) {
    const int stages = 2 * in_bytes + out_bytes <= 100 * 1024 ? 2 : 1;
    return {((d + nv - 1) / nv + 31) / 32 * 32, stages, stages * in_bytes + out_bytes};
}
// Rows of a tile: whole passes of the teams, `budget` bytes of shared memory at `row_bytes` a row, and
// not so many that SMs stay without a tile.  Four CTAs to an SM forward (100000 x 257: 78 us with 56 KB,
// 85 with 28, 94 with 78), two backward, where the fp64 sums take their part of 112 KB (94 us; without those
// sums 92 us with 91 KB, 117 with 30).
inline int odd_tile_rows(int64_t N, int row_bytes, int teams, int budget) {
    return std::max(1, (int)std::min<int64_t>(budget / row_bytes, N / (kSms * 4)) / teams) * teams;
}

template <class T, int MODE, bool RES, int NV, int MAXT>
dbc_status launch_odd_row(const FwdArgs &a, cudaStream_t st) {
    const int slot = slot_bytes(a.d, sizeof(T));
    const OddPlan p = odd_plan(a.d, NV, (RES ? 2 : 1) * slot, slot_bytes(a.d, MODE != kPlain ? 1 : a.y_bf16 ? 2 : 4));
    auto *k = odd_kernel<T, MODE, RES, NV, MAXT>;
    const int ctas = resident(k, p.threads, p.smem, a.N);
    if (!ctas) return DBC_ERR_CUDA;
    k<<<ctas, p.threads, p.smem, st>>>(a, slot, p.stages);
    return DBC_OK;
}
template <class T, int MODE, bool RES, int W>
dbc_status launch_odd_tile(const FwdArgs &a, cudaStream_t st) {
    constexpr int TEAMS = kThreads / W;
    const int slot = slot_bytes(a.d, sizeof(T)), oslot = slot_bytes(a.d, MODE != kPlain ? 1 : a.y_bf16 ? 2 : 4);
    constexpr int IN = RES ? 2 : 1;
    const int row = (2 * IN + (RES && a.s ? 1 : 0)) * slot + oslot;
    const int R = odd_tile_rows(a.N, row, TEAMS, 56 * 1024 - 4 * a.d), smem = R * row + a.d * 4;
    auto *k = odd_tile_kernel<T, MODE, RES, W>;
    const int ctas = resident(k, kThreads, smem, (a.N + R - 1) / R);
    if (!ctas) return DBC_ERR_CUDA;
    k<<<ctas, kThreads, smem, st>>>(a, R, slot, oslot);
    return DBC_OK;
}
template <class T, int MODE, bool RES>
dbc_status launch_odd_res(const FwdArgs &a, cudaStream_t st) {
    if (a.d <= 64) return launch_odd_tile<T, MODE, RES, 8>(a, st);
    if (a.d <= 128) return launch_odd_tile<T, MODE, RES, 16>(a, st);
    if (a.d <= 1024) return launch_odd_tile<T, MODE, RES, 32>(a, st);
    if (a.d <= 2048) return launch_odd_row<T, MODE, RES, 8, 256>(a, st);
    return launch_odd_row<T, MODE, RES, 16, 1024>(a, st);
}
template <class T, int MODE>
dbc_status launch_odd(const FwdArgs &a, cudaStream_t st) {
    if constexpr (norms(MODE)) {
        if (a.res) return launch_odd_res<T, MODE, true>(a, st);
    }
    return launch_odd_res<T, MODE, false>(a, st);
}

// Several rows per team pay once every SM has work without them.
inline bool many(int64_t rows, int lanes, int R) { return rows * lanes / 32 / R >= 148 * 16; }

template <class T, int MODE>
dbc_status launch_rows(const FwdArgs &a, cudaStream_t st) {
    constexpr int E = 16 / sizeof(T);
    const int64_t e = sizeof(T), ysz = a.y_bf16 ? 2 : 4;
    const bool vec = a.d % E == 0 && on_grid(a.x, a.xs, e, 16) && on_grid(a.res, a.rs, e, 16) &&
                     on_grid(a.s, a.ss, e, 16) && on_grid(a.y, a.ys, ysz, std::min<int64_t>(16, E * ysz)) &&
                     on_grid(a.q, a.qs, 1, E) && on_grid(a.w.p, 0, 1, a.w.bf16 ? E * 2 : 16);
    if (!vec) return launch_odd<T, MODE>(a, st);
    const int V = a.d / E;
    if (V <= 8)
        return many(a.N, 8, 4) ? launch_team<T, E, MODE, 8, 1, 4>(a, st) : launch_team<T, E, MODE, 8, 1, 1>(a, st);
    if (V <= 16)
        return many(a.N, 16, 4) ? launch_team<T, E, MODE, 16, 1, 4>(a, st) : launch_team<T, E, MODE, 16, 1, 1>(a, st);
    if (V <= 32)
        return many(a.N, 32, 4) ? launch_team<T, E, MODE, 32, 1, 4>(a, st) : launch_team<T, E, MODE, 32, 1, 1>(a, st);
    if (V <= 64)
        return many(a.N, 32, 2) ? launch_team<T, E, MODE, 32, 2, 2>(a, st) : launch_team<T, E, MODE, 32, 2, 1>(a, st);
    if (V <= 128) return launch_team<T, E, MODE, 32, 4, 1>(a, st);
    if (V <= 512) return launch_block<T, E, MODE, 2, 256>(a, st);
    if (V <= 1024) return launch_block<T, E, MODE, 2, 512>(a, st);
    if constexpr (sizeof(T) == 4) {
        if (V > 2048) return launch_block<T, E, MODE, 4, 1024>(a, st);
    }
    return launch_block<T, E, MODE, 2, 1024>(a, st);
}

template <int MODE>
dbc_status launch_fwd(const FwdArgs &a, int dtype, cudaStream_t st) {
    // bf16 rows under a bf16 weight (or none) give products of 16 significant bits
    constexpr int kBf16Mode = MODE == kI8 ? kI8Narrow : MODE;
    const dbc_status c = dtype != DBC_BF16              ? launch_rows<float, MODE>(a, st)
                         : !a.w.p || a.w.bf16 ? launch_rows<__nv_bfloat16, kBf16Mode>(a, st)
                                              : launch_rows<__nv_bfloat16, MODE>(a, st);
    if (c != DBC_OK) return c;
    count_launches(1);
    return launch_status();
}

// The most CTAs of a backward call, and with them the lines of dw sums: up to
// 8 per SM, fewer for wide rows, whose lines would otherwise outweigh the rows.
inline int bwd_lines(int64_t N, int64_t d) {
    return (int)std::min<int64_t>(N, kSms * std::min<int64_t>(8, std::max<int64_t>(1, kMaxD / d)));
}

template <class K>
int launch_resident(K kernel, const BwdArgs &a, int threads, int smem, int64_t most, cudaStream_t st) {
    const int ctas = resident(kernel, threads, smem, most);
    if (ctas) kernel<<<ctas, threads, smem, st>>>(a);
    return ctas;
}

template <class TY, class T, int NV, int MAXT>
int launch_odd_bwd_row(const BwdArgs &a, cudaStream_t st) {
    const int yslot = slot_bytes(a.d, sizeof(TY)), slot = slot_bytes(a.d, sizeof(T));
    const int sums = a.part && NV <= 8 ? (a.d + NV * 32 - 1) / (NV * 32) * 32 * NV * (int)sizeof(double) : 0;
    const OddPlan p = odd_plan(a.d, NV, yslot + (a.ds ? 2 : 1) * slot, sums);
    auto *k = a.part ? odd_bwd_kernel<TY, T, true, NV, MAXT> : odd_bwd_kernel<TY, T, false, NV, MAXT>;
    const int ctas = resident(k, p.threads, p.smem, bwd_lines(a.N, a.d));
    if (ctas) k<<<ctas, p.threads, p.smem, st>>>(a, yslot, slot, p.stages);
    return ctas;
}
template <class TY, class T, int W, int NV>
int launch_odd_bwd_tile(const BwdArgs &a, cudaStream_t st) {
    const int yslot = slot_bytes(a.d, sizeof(TY)), slot = slot_bytes(a.d, sizeof(T));
    const int row = 2 * (yslot + (a.ds ? 2 : 1) * slot) + slot;
    const int sums = a.part ? (a.d + W - 1) / W * kThreads * (int)sizeof(double) : 0;
    const int R = std::min(kFold * kThreads / W, odd_tile_rows(a.N, row, kThreads / W, 112 * 1024 - sums));
    const int smem = sums + R * row;
    auto *k = a.part ? odd_bwd_tile_kernel<TY, T, true, W, NV> : odd_bwd_tile_kernel<TY, T, false, W, NV>;
    const int ctas = resident(k, kThreads, smem, std::min<int64_t>(bwd_lines(a.N, a.d), (a.N + R - 1) / R));
    if (ctas) k<<<ctas, kThreads, smem, st>>>(a, R, yslot, slot);
    return ctas;
}

template <class TY, class T, int NE, int W, int NV>
int launch_bwd_team(const BwdArgs &a, cudaStream_t st) {
    constexpr int rows = kThreads / W;
    const int64_t most = std::min<int64_t>(bwd_lines(a.N, a.d), (a.N + rows - 1) / rows);
    return a.part ? launch_resident(bwd_team_kernel<TY, T, NE, true, W, NV>, a, kThreads,
                                    Ring<TY, T, NE, NV, kThreads, true>::smem(kThreads), most, st)
                  : launch_resident(bwd_team_kernel<TY, T, NE, false, W, NV>, a, kThreads,
                                    Ring<TY, T, NE, NV, kThreads, false>::smem(kThreads), most, st);
}

template <class TY, class T, int NE, int NV, int MAXT>
int launch_bwd_block(const BwdArgs &a, cudaStream_t st) {
    const int threads = ((a.d + NE * NV - 1) / (NE * NV) + 31) / 32 * 32;
    const int most = bwd_lines(a.N, a.d);
    return a.part ? launch_resident(bwd_block_kernel<TY, T, NE, true, NV, MAXT>, a, threads,
                                    Ring<TY, T, NE, NV, MAXT, MAXT <= 512>::smem(threads), most, st)
                  : launch_resident(bwd_block_kernel<TY, T, NE, false, NV, MAXT>, a, threads,
                                    Ring<TY, T, NE, NV, MAXT, false>::smem(threads), most, st);
}

// (V: fragments of a line, see dw_kernel)
template <class TY, class T>
int launch_bwd(const BwdArgs &a, int &V, cudaStream_t st) {
    constexpr int E = 16 / sizeof(T);
    const int64_t e = sizeof(T), ey = sizeof(TY);
    const bool vec = a.d % E == 0 && on_grid(a.s, a.ss, e, 16) && on_grid(a.ds, a.ds_s, e, 16) &&
                     on_grid(a.dx, a.xs, e, 16) && on_grid(a.dy, a.ys, ey, std::min<int64_t>(16, E * ey)) &&
                     on_grid(a.w.p, 0, 1, a.w.bf16 ? E * 2 : 16);
    V = a.d;
    if (!vec) {
        if (a.d <= 64) return launch_odd_bwd_tile<TY, T, 8, 8>(a, st);
        if (a.d <= 128) return launch_odd_bwd_tile<TY, T, 16, 8>(a, st);
        if (a.d <= 256) return launch_odd_bwd_tile<TY, T, 32, 8>(a, st);
        if (a.d <= 512) return launch_odd_bwd_tile<TY, T, 32, 16>(a, st);
        if (a.d <= 2048) return launch_odd_bwd_row<TY, T, 8, 256>(a, st);
        if (a.d <= 8192) return launch_odd_bwd_row<TY, T, 8, 1024>(a, st);
        return launch_odd_bwd_row<TY, T, 16, 1024>(a, st);
    }
    if (a.d <= 8 * E) return launch_bwd_team<TY, T, E, 8, 1>(a, st);
    if (a.d <= 16 * E) return launch_bwd_team<TY, T, E, 16, 1>(a, st);
    if (a.d <= 32 * E) return launch_bwd_team<TY, T, E, 32, 1>(a, st);
    if (a.d <= 64 * E) return launch_bwd_team<TY, T, E, 32, 2>(a, st);
    V = a.d / E;
    if (V <= 512) return launch_bwd_block<TY, T, E, 2, 256>(a, st);
    if (V <= 1024) return launch_bwd_block<TY, T, E, 2, 512>(a, st);
    if constexpr (sizeof(T) == 4) {
        if (V > 2048) return launch_bwd_block<TY, T, E, 4, 1024>(a, st);
    }
    return launch_bwd_block<TY, T, E, 2, 1024>(a, st);
}

}  // namespace nm
}  // namespace dbc

using namespace dbc;

extern "C" dbc_status rms_norm(const void *x, int64_t x_stride, int dtype, const void *residual, int64_t r_stride,
                               const void *weight, int w_dtype, int64_t N, int64_t d, float eps, void *s,
                               int64_t s_stride, void *y, int64_t y_stride, int y_dtype, int32_t *dev_status,
                               dbc_stream_t stream) {
    DBC_NVTX_RANGE("rms_norm");
    nm::FwdArgs a{x, residual, s, y, nullptr, nullptr, {weight, w_dtype == DBC_BF16}, x_stride, r_stride, s_stride,
                  y_stride, 0, N, (int)d, y_dtype == DBC_BF16, eps, 1.f / (float)d, dev_status};
    const dbc_status c = nm::check_fwd(a, dtype, w_dtype, d, true);
    if (c != DBC_OK) return c;
    if (!nm::known(y_dtype)) return DBC_ERR_UNSUPPORTED;
    if (y_stride < d) return DBC_ERR_INVALID_ARG;
    if (N == 0) return DBC_OK;
    if (!y || y == s || !nm::aligned_to(y, nm::esize(y_dtype))) return DBC_ERR_INVALID_ARG;
    return nm::launch_fwd<nm::kPlain>(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" dbc_status rms_norm_i8(const void *x, int64_t x_stride, int dtype, const void *residual, int64_t r_stride,
                                  const void *weight, int w_dtype, int64_t N, int64_t d, float eps, void *s,
                                  int64_t s_stride, int8_t *q, int64_t q_stride, float *scale, int32_t *dev_status,
                                  dbc_stream_t stream) {
    DBC_NVTX_RANGE("rms_norm_i8");
    nm::FwdArgs a{x, residual, s, nullptr, q, scale, {weight, w_dtype == DBC_BF16}, x_stride, r_stride, s_stride,
                  0, q_stride, N, (int)d, 0, eps, 1.f / (float)d, dev_status};
    const dbc_status c = nm::check_fwd(a, dtype, w_dtype, d, true);
    if (c != DBC_OK) return c;
    if (q_stride < d) return DBC_ERR_INVALID_ARG;
    if (N == 0) return DBC_OK;
    if (!q || !scale || !nm::aligned_to(scale, 4)) return DBC_ERR_INVALID_ARG;
    return nm::launch_fwd<nm::kI8>(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" dbc_status quantize_rows_i8(const void *x, int64_t x_stride, int dtype, int64_t N, int64_t d, int8_t *q,
                                       int64_t q_stride, float *scale, int32_t *dev_status, dbc_stream_t stream) {
    DBC_NVTX_RANGE("quantize_rows_i8");
    nm::FwdArgs a{x, nullptr, nullptr, nullptr, q, scale, {nullptr, 0}, x_stride, 0, 0, 0, q_stride, N, (int)d, 0,
                  1.f, 1.f, dev_status};
    const dbc_status c = nm::check_fwd(a, dtype, DBC_F32, d, false);
    if (c != DBC_OK) return c;
    if (q_stride < d) return DBC_ERR_INVALID_ARG;
    if (N == 0) return DBC_OK;
    if (!q || !scale || !nm::aligned_to(scale, 4)) return DBC_ERR_INVALID_ARG;
    return nm::launch_fwd<nm::kQuant>(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t rms_norm_backward_workspace(int64_t N, int64_t d) {
    if (N <= 0 || d <= 0) return 0;
    return align_up((size_t)nm::bwd_lines(N, d) * (size_t)d * sizeof(double));
}

extern "C" dbc_status rms_norm_backward(const void *dy, int64_t dy_stride, int dy_dtype, const void *s,
                                        int64_t s_stride, int dtype, const void *weight, int w_dtype, const void *ds,
                                        int64_t ds_stride, int64_t N, int64_t d, float eps, void *dx,
                                        int64_t dx_stride, float *dw, void *ws, size_t ws_bytes, int32_t *dev_status,
                                        dbc_stream_t stream) {
    DBC_NVTX_RANGE("rms_norm_backward");
    if (N < 0 || d <= 0 || !(eps > 0.f) || !std::isfinite(eps)) return DBC_ERR_INVALID_ARG;
    if (!nm::known(dtype) || !nm::known(dy_dtype) || (weight && !nm::known(w_dtype)) || d > nm::kMaxD)
        return DBC_ERR_UNSUPPORTED;
    if (dy_stride < d || s_stride < d || dx_stride < d || (ds && ds_stride < d)) return DBC_ERR_INVALID_ARG;
    const int64_t e = nm::esize(dtype);
    if (N > 0 && (!dy || !s || !dx || !nm::aligned_to(dy, nm::esize(dy_dtype)) || !nm::aligned_to(s, e) ||
                  !nm::aligned_to(dx, e) || !nm::aligned_to(ds, e)))
        return DBC_ERR_INVALID_ARG;
    if ((weight && !nm::aligned_to(weight, nm::esize(w_dtype))) || !nm::aligned_to(dw, 4)) return DBC_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) {
        if (dw && cudaMemsetAsync(dw, 0, (size_t)d * sizeof(float), st) != cudaSuccess) return DBC_ERR_CUDA;
        return DBC_OK;
    }
    if (dw && (!ws || !nm::aligned_to(ws, 16) || ws_bytes < rms_norm_backward_workspace(N, d)))
        return DBC_ERR_WORKSPACE;
    const nm::BwdArgs a{dy, s, ds, dx, {weight, w_dtype == DBC_BF16}, dy_stride, s_stride, ds_stride, dx_stride, N,
                        (int)d, eps, 1.f / (float)d, dw ? static_cast<double *>(ws) : nullptr, dev_status};
    using B = __nv_bfloat16;
    const bool by = dy_dtype == DBC_BF16, bs = dtype == DBC_BF16;
    int V = 0;
    const int lines = by && bs ? nm::launch_bwd<B, B>(a, V, st)
                      : by     ? nm::launch_bwd<B, float>(a, V, st)
                      : bs     ? nm::launch_bwd<float, B>(a, V, st)
                               : nm::launch_bwd<float, float>(a, V, st);
    if (!lines) return DBC_ERR_CUDA;
    if (dw) nm::dw_kernel<<<(unsigned)((d + 7) / 8), 1024, 0, st>>>(a.part, lines, (int)d, V, dw);
    count_launches(dw ? 2 : 1);
    return launch_status();
}

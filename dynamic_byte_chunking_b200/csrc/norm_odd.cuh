// The norm kernels for rows off the 16-byte grid: odd widths, odd strides,
// shifted bases.
//
// Element by element from global memory such rows move 64 bytes per bf16
// instruction and stay at a fifth of HBM's rate (30000 x 777 with a residual:
// 142 us; 500000 x 33: 374).  Here a row travels as the
// aligned 16-byte pieces that cover it (asynchronous copies into shared memory
// one row ahead, whole pieces back out, elements only at its two ends) and only
// the arithmetic goes element by element, column j * W + t by thread t of the W
// that share the row: 68 and 63 us, two fifths of the rate; what is left is the
// latency of the tiles' barriers and of the element-wise shared-memory accesses
// between them.  Nothing outside the row is written, and nothing in front
// of the array or behind the row is read.
#pragma once

#include "norm.cuh"

namespace dbc {
namespace nm {

// Bytes of a shared-memory slot for a row of d elements, at any misalignment.
__host__ __device__ inline int slot_bytes(int64_t d, int esz) { return (int)((d * esz + 15) / 16 * 16 + 16); }

__device__ __forceinline__ int off16(const void *p) { return (int)(reinterpret_cast<uintptr_t>(p) & 15); }

// Starts the copies of a row at p (of an array that begins at `base`) into a
// slot; the row's first element lands at the slot's byte off16(p).
template <class T>
__device__ __forceinline__ void row_in(char *slot, const T *base, const T *p, int d, int t, int W) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), a0 = a & ~(uintptr_t)15, e = a + (uintptr_t)d * sizeof(T);
    const int n = (int)((e - a0 + 15) >> 4);
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(slot);
    for (int i = t; i < n; i += W) {
        const uintptr_t src = a0 + (uintptr_t)i * 16;
        if (src >= reinterpret_cast<uintptr_t>(base)) {
            const int bytes = (int)min((uintptr_t)16, e - src);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s + i * 16), "l"(src), "r"(bytes) : "memory");
        } else {                                     // the piece begins in front of the array
            for (uintptr_t b = a; b < min(src + 16, e); b += sizeof(T))
                *reinterpret_cast<T *>(slot + i * 16 + (b - src)) = *reinterpret_cast<const T *>(b);
        }
    }
}

// A row from a slot (first element at byte off16(p)) to p.
template <class T>
__device__ __forceinline__ void row_out(T *p, const char *slot, int d, int t, int W) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), a0 = a & ~(uintptr_t)15, e = a + (uintptr_t)d * sizeof(T);
    const int n = (int)((e - a0 + 15) >> 4);
    for (int i = t; i < n; i += W) {
        const uintptr_t dst = a0 + (uintptr_t)i * 16;
        if (dst >= a && dst + 16 <= e) {
            *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(slot + i * 16);
        } else {
            for (uintptr_t b = max(dst, a); b < min(dst + 16, e); b += sizeof(T))
                *reinterpret_cast<T *>(b) = *reinterpret_cast<const T *>(slot + i * 16 + (b - dst));
        }
    }
}

// Lanes for a row of so many bytes: a power of two up to 32 that covers its pieces.
__device__ __forceinline__ int lanes_for(int bytes) {
    const int n = bytes / 16 + 2;
    return n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : 32;
}

// The same for `rows` rows that are `stride` apart, by a whole CTA: one long
// row where they touch, else row by row, `slot` bytes apart.
template <class T>
__device__ __forceinline__ void tile_in(char *tile, int slot, const T *base, const T *p, int64_t stride, int rows, int d) {
    if (stride == d) {
        row_in(tile, base, p, rows * d, threadIdx.x, blockDim.x);
    } else {
        const int W = lanes_for(d * (int)sizeof(T));
        for (int r = threadIdx.x / W; r < rows; r += blockDim.x / W)
            row_in(tile + r * slot, base, p + r * stride, d, threadIdx.x % W, W);
    }
}
template <class T>
__device__ __forceinline__ void tile_out(T *p, int64_t stride, const char *tile, int slot, int rows, int d) {
    if (stride == d) {
        row_out(p, tile, rows * d, threadIdx.x, blockDim.x);
    } else {
        const int W = lanes_for(d * (int)sizeof(T));
        for (int r = threadIdx.x / W; r < rows; r += blockDim.x / W)
            row_out(p + r * stride, tile + r * slot, d, threadIdx.x % W, W);
    }
}
// Where row r of a tile begins in shared memory; p is the first row's address.
template <class T>
__device__ __forceinline__ T *tile_row(char *tile, int slot, const T *p, int64_t stride, int r, int d) {
    return reinterpret_cast<T *>(stride == d ? tile + off16(p) + r * d * (int)sizeof(T)
                                             : tile + r * slot + off16(p + r * stride));
}

__device__ __forceinline__ void st_f(float *p, float v) { *p = v; }
__device__ __forceinline__ void st_f(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void copies_done(int ahead) {
    if (ahead) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Reduces a pair of values over the CTA (one barrier; `sh` is free again after the next one).
template <class V2, class F, class G>
__device__ __forceinline__ V2 team_pair(V2 v, F f, G g, V2 *sh) {
    v.x = team_reduce<32>(v.x, f);
    v.y = team_reduce<32>(v.y, g);
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    const V2 u = lane < warps ? sh[lane] : V2{0, 0};
    return V2{team_reduce<32>(u.x, f), team_reduce<32>(u.y, g)};
}

// Forward, narrow rows: tiles of R rows, W lanes to a row, everything read from
// shared memory twice (statistics, outputs).  Buffers: x (and the residual) for
// two tiles, then s, then y or q, then the weight as fp32.
template <class T, int MODE, bool RES, int W>
__global__ void __launch_bounds__(kThreads) odd_tile_kernel(const FwdArgs a, int R, int slot, int oslot) {
    extern __shared__ __align__(16) char smem[];
    const int t = threadIdx.x % W, team = threadIdx.x / W;
    constexpr int IN = RES ? 2 : 1, TEAMS = kThreads / W;
    const T *const X = static_cast<const T *>(a.x);
    const T *const G = static_cast<const T *>(a.res);
    T *const S = static_cast<T *>(a.s);
    const int tile_bytes = R * slot;
    char *const sbuf = smem + 2 * IN * tile_bytes;
    char *const obuf = sbuf + (RES && S ? tile_bytes : 0);
    float *const w = reinterpret_cast<float *>(obuf + R * oslot);
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
        float o[1] = {1.f};
        if (norms(MODE)) a.w.get<1>(c, o);
        w[c] = o[0];
    }
    const int64_t tiles = (a.N + R - 1) / R;
    auto start = [&](int64_t i, int st) {
        if (i < tiles) {
            const int64_t r0 = i * R;
            const int rows = (int)min((int64_t)R, a.N - r0);
            char *const in = smem + st * IN * tile_bytes;
            tile_in(in, slot, X, X + r0 * a.xs, a.xs, rows, a.d);
            if (RES) tile_in(in + tile_bytes, slot, G, G + r0 * a.rs, a.rs, rows, a.d);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int st = 0;
    start(blockIdx.x, 0);
    for (int64_t i = blockIdx.x; i < tiles; i += gridDim.x, st ^= 1) {
        __syncthreads();                                 // the tile before has left its buffers
        start(i + gridDim.x, st ^ 1);
        copies_done(1);
        __syncthreads();
        const int64_t r0 = i * R;
        const int rows = (int)min((int64_t)R, a.N - r0);
        char *const in = smem + st * IN * tile_bytes;
        for (int k0 = 0; k0 < rows; k0 += TEAMS) {       // all lanes of a warp together
            const int k = k0 + team;
            const bool live = k < rows;
            const int n = live ? a.d : 0;
            const T *const x = tile_row(in, slot, X + r0 * a.xs, a.xs, k, a.d);
            const T *const g = RES ? tile_row(in + tile_bytes, slot, G + r0 * a.rs, a.rs, k, a.d) : x;
            auto val = [&](int c) { return RES ? round_to<T>(ld_f(x + c) + ld_f(g + c)) : ld_f(x + c); };
            float ss = 0.f, m = 0.f;
#pragma unroll 4
            for (int c = t; c < n; c += W) {
                const float v = val(c);
                if (norms(MODE)) ss = fmaf(v, v, ss);
                if (MODE != kPlain) m = abs_max(m, weighs(MODE) ? v * w[c] : v);
            }
            if (norms(MODE)) ss = team_reduce<W>(ss, Add());
            if (MODE != kPlain) m = team_reduce<W>(m, AbsMax());
            RowFactor f(ss, a);
            const bool odd = norms(MODE) && live && !(ss >= kLow && ss <= kHigh);
            if (norms(MODE) && __any_sync(0xffffffffu, odd)) {
                double t2 = 0;
                for (int c = t; c < n; c += W) {
                    const double v = val(c);
                    t2 += v * v;
                }
                t2 = team_reduce<W>(t2, Add());
                if (odd) f = RowFactor(t2, a);
                if (odd && !isfinite(t2)) {
                    m = __int_as_float(0x7fc00000);
                    if (t == 0) flag(a.st, DBC_ERR_NONFINITE);
                }
            }
            const Quant qn(m);
            T *const so = RES && S ? tile_row(sbuf, slot, S + r0 * a.ss, a.ss, k, a.d) : nullptr;
            if (MODE == kPlain && a.y_bf16) {
                __nv_bfloat16 *const o =
                    tile_row(obuf, oslot, static_cast<__nv_bfloat16 *>(a.y) + r0 * a.ys, a.ys, k, a.d);
#pragma unroll 4
                for (int c = t; c < n; c += W) {
                    const float v = val(c);
                    if (RES && S) st_f(so + c, v);
                    o[c] = __float2bfloat16_rn(v * f.pre * f.rstd * w[c]);
                }
            } else if (MODE == kPlain) {
                float *const o = tile_row(obuf, oslot, static_cast<float *>(a.y) + r0 * a.ys, a.ys, k, a.d);
#pragma unroll 4
                for (int c = t; c < n; c += W) {
                    const float v = val(c);
                    if (RES && S) st_f(so + c, v);
                    o[c] = v * f.pre * f.rstd * w[c];
                }
            } else {
                int8_t *const o = tile_row(obuf, oslot, a.q + r0 * a.qs, a.qs, k, a.d);
                // two columns at a time: loads, packed arithmetic, stores
#pragma unroll 2
                for (int c = t; c < n; c += 2 * W) {
                    const bool two = c + W < n;
                    const float v[2] = {val(c), two ? val(c + W) : 0.f};
                    const float p[2] = {weighs(MODE) ? v[0] * w[c] : v[0], weighs(MODE) && two ? v[1] * w[c + W] : v[1]};
                    uint32_t u[2];
                    qn.template codes<narrow<T>(MODE)>(p, u);
                    if (RES && S) st_f(so + c, v[0]);
                    o[c] = qn.bad ? 0 : (int8_t)u[0];
                    if (two) {
                        if (RES && S) st_f(so + c + W, v[1]);
                        o[c + W] = qn.bad ? 0 : (int8_t)u[1];
                    }
                }
                if (t == 0 && live) {
                    a.scale[r0 + k] = row_scale<MODE>(qn, f);
                    if (qn.bad) flag(a.st, DBC_ERR_NONFINITE);
                }
            }
        }
        __syncthreads();
        if (RES && S) tile_out(S + r0 * a.ss, a.ss, sbuf, slot, rows, a.d);
        if (MODE != kPlain) tile_out(a.q + r0 * a.qs, a.qs, obuf, oslot, rows, a.d);
        else if (a.y_bf16) tile_out(static_cast<__nv_bfloat16 *>(a.y) + r0 * a.ys, a.ys, obuf, oslot, rows, a.d);
        else tile_out(static_cast<float *>(a.y) + r0 * a.ys, a.ys, obuf, oslot, rows, a.d);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Forward, wide rows: one row per CTA at a time.  Slots: x (and the residual)
// for `stages` rows, then y or q; s goes back into x's slot, whose values are in
// registers by then.
template <class T, int MODE, bool RES, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) odd_kernel(const FwdArgs a, int slot, int stages) {
    extern __shared__ __align__(16) char smem[];
    __shared__ float2 sh[32];
    __shared__ double2 shw[32];
    const int W = blockDim.x, t = threadIdx.x;
    constexpr int IN = RES ? 2 : 1;
    char *const out = smem + stages * IN * slot;
    const T *const X = static_cast<const T *>(a.x);
    const T *const Rs = static_cast<const T *>(a.res);
    float w[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float o[1] = {1.f};
        if (norms(MODE) && j * W + t < a.d) a.w.get<1>(j * W + t, o);
        w[j] = o[0];
    }
    auto start = [&](int64_t r, int st) {
        if (r < a.N) {
            char *const in = smem + st * IN * slot;
            row_in(in, X, X + r * a.xs, a.d, t, W);
            if (RES) row_in(in + slot, Rs, Rs + r * a.rs, a.d, t, W);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int ahead = stages - 1;
    int st = 0;
    if (ahead) start(blockIdx.x, 0);
    for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x) {
        __syncthreads();                              // the row before has left its slots
        if (ahead) start(r + gridDim.x, st ^ 1);
        else start(r, 0);
        copies_done(ahead);
        __syncthreads();
        char *const in = smem + st * IN * slot;
        const T *const x = reinterpret_cast<const T *>(in + off16(X + r * a.xs));
        const T *const g = reinterpret_cast<const T *>(in + slot + (RES ? off16(Rs + r * a.rs) : 0));
        float v[NV], ss = 0.f, m = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * W + t;
            v[j] = 0.f;
            if (c < a.d) {
                v[j] = ld_f(x + c);
                if (RES) v[j] = round_to<T>(v[j] + ld_f(g + c));
            }
            if (norms(MODE)) ss = fmaf(v[j], v[j], ss);
            if (MODE != kPlain) m = abs_max(m, weighs(MODE) ? v[j] * w[j] : v[j]);
        }
        const float2 sm = team_pair(make_float2(ss, m), Add(), AbsMax(), sh);
        ss = sm.x, m = sm.y;
        RowFactor k(ss, a);
        if (norms(MODE) && !(ss >= kLow && ss <= kHigh)) {   // the same in the whole team
            double t2 = 0;
#pragma unroll
            for (int j = 0; j < NV; ++j) t2 += (double)v[j] * v[j];
            t2 = team_pair(make_double2(t2, 0), Add(), Add(), shw).x;
            k = RowFactor(t2, a);
            if (!isfinite(t2)) {
                m = __int_as_float(0x7fc00000);
                if (t == 0) flag(a.st, DBC_ERR_NONFINITE);
            }
        }
        const Quant qn(m);
        T *const sp = RES && a.s ? static_cast<T *>(a.s) + r * a.ss : nullptr;
        T *const so = reinterpret_cast<T *>(in + off16(sp));
        if (MODE == kPlain) {
            if (a.y_bf16) {
                __nv_bfloat16 *const y = static_cast<__nv_bfloat16 *>(a.y) + r * a.ys;
                __nv_bfloat16 *const yo = reinterpret_cast<__nv_bfloat16 *>(out + off16(y));
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (j * W + t < a.d) yo[j * W + t] = __float2bfloat16_rn(v[j] * k.pre * k.rstd * w[j]);
            } else {
                float *const y = static_cast<float *>(a.y) + r * a.ys;
                float *const yo = reinterpret_cast<float *>(out + off16(y));
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (j * W + t < a.d) yo[j * W + t] = v[j] * k.pre * k.rstd * w[j];
            }
        } else {
            int8_t *const qo = reinterpret_cast<int8_t *>(out + off16(a.q + r * a.qs));
#pragma unroll
            for (int j = 0; j < NV; j += 4) {
                float p[4];
                uint32_t u[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) p[q] = weighs(MODE) ? v[j + q] * w[j + q] : v[j + q];
                qn.template codes<narrow<T>(MODE)>(p, u);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if ((j + q) * W + t < a.d) qo[(j + q) * W + t] = qn.bad ? 0 : (int8_t)u[q];
            }
            if (t == 0) {
                a.scale[r] = row_scale<MODE>(qn, k);
                if (qn.bad) flag(a.st, DBC_ERR_NONFINITE);
            }
        }
        if (RES && sp) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j * W + t < a.d) {
                    Frag<T, 1> f;
                    const float u[1] = {v[j]};
                    f.set(u);
                    f.store(so + j * W + t);
                }
        }
        __syncthreads();
        if (RES && sp) row_out(sp, in, a.d, t, W);
        if (MODE != kPlain) row_out(a.q + r * a.qs, out, a.d, t, W);
        else if (a.y_bf16) row_out(static_cast<__nv_bfloat16 *>(a.y) + r * a.ys, out, a.d, t, W);
        else row_out(static_cast<float *>(a.y) + r * a.ys, out, a.d, t, W);
        if (ahead) st ^= 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Backward, narrow rows: tiles of R rows, W lanes to a row.  Buffers: the lanes' fp64
// dw sums, then dy, s (and ds) for two tiles, then dx; a lane keeps the dw sums of
// its NV columns, the CTA joins them at the end (a fixed order).
template <class TY, class T, bool DW, int W, int NV>
__global__ void __launch_bounds__(kThreads, 2) odd_bwd_tile_kernel(const BwdArgs a, int R, int yslot, int slot) {
    extern __shared__ __align__(16) char all[];
    constexpr int TEAMS = kThreads / W;
    const int t = threadIdx.x % W, team = threadIdx.x / W;
    double *const sums = reinterpret_cast<double *>(all);     // column j's at sums[j * kThreads + thread]
    const int nj = (a.d + W - 1) / W;                         // a lane's columns
    char *const smem = all + (DW ? nj * kThreads * (int)sizeof(double) : 0);
    const TY *const Y = static_cast<const TY *>(a.dy);
    const T *const S = static_cast<const T *>(a.s);
    const T *const D = static_cast<const T *>(a.ds);
    T *const X = static_cast<T *>(a.dx);
    const int stage = R * (yslot + (D ? 2 : 1) * slot);
    char *const obuf = smem + 2 * stage;
    float w[NV], acc[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float o[1] = {0.f};
        if (j * W + t < a.d) a.w.get<1>(j * W + t, o);
        w[j] = o[0];
        acc[j] = 0.f;
        if (DW && j < nj) sums[j * kThreads + threadIdx.x] = 0;
    }
    auto fold = [&] {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (j < nj) sums[j * kThreads + threadIdx.x] += acc[j];
            acc[j] = 0.f;
        }
    };
    const int passes = R / TEAMS;                             // rows of a team in a tile, at most kFold
    int done = 0;                                             // rows since the fold before
    const int64_t tiles = (a.N + R - 1) / R;
    auto start = [&](int64_t i, int st) {
        if (i < tiles) {
            const int64_t r0 = i * R;
            const int rows = (int)min((int64_t)R, a.N - r0);
            char *const in = smem + st * stage;
            tile_in(in, yslot, Y, Y + r0 * a.ys, a.ys, rows, a.d);
            tile_in(in + R * yslot, slot, S, S + r0 * a.ss, a.ss, rows, a.d);
            if (D) tile_in(in + R * (yslot + slot), slot, D, D + r0 * a.ds_s, a.ds_s, rows, a.d);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int st = 0;
    start(blockIdx.x, 0);
    for (int64_t i = blockIdx.x; i < tiles; i += gridDim.x, st ^= 1) {
        __syncthreads();                                 // the tile before has left its buffers
        start(i + gridDim.x, st ^ 1);
        copies_done(1);
        __syncthreads();
        const int64_t r0 = i * R;
        const int rows = (int)min((int64_t)R, a.N - r0);
        char *const in = smem + st * stage;
        for (int k0 = 0; k0 < rows; k0 += TEAMS) {       // all lanes of a warp together
            const int k = k0 + team;
            const int n = k < rows ? a.d : 0;
            const TY *const dy = tile_row(in, yslot, Y + r0 * a.ys, a.ys, k, a.d);
            const T *const s = tile_row(in + R * yslot, slot, S + r0 * a.ss, a.ss, k, a.d);
            float y[NV], f[NV], ss = 0.f, sg = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = j * W + t;
                y[j] = c < n ? ld_f(dy + c) : 0.f;
                f[j] = c < n ? ld_f(s + c) : 0.f;
                ss = fmaf(f[j], f[j], ss);
                sg = fmaf(y[j] * w[j], f[j], sg);
            }
            ss = team_reduce<W>(ss, Add());
            sg = team_reduce<W>(sg, Add());
            BwdFactor b(ss, sg, a);
            bool odd = !in_range(ss, sg);
            if (__any_sync(0xffffffffu, faint(sg))) {
                bool some = false;
#pragma unroll
                for (int j = 0; j < NV; ++j) some |= y[j] * w[j] != 0.f;
                odd |= team_any<W>(some) && faint(sg);
            }
            odd &= k < rows;
            if (__any_sync(0xffffffffu, odd)) {
                double s2 = 0, g2 = 0;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    s2 += (double)f[j] * f[j];
                    g2 += (double)(y[j] * w[j]) * f[j];
                }
                s2 = team_reduce<W>(s2, Add());
                g2 = team_reduce<W>(g2, Add());
                if (odd) b = BwdFactor(s2, g2, a);
                if (odd && t == 0 && (!isfinite(s2) || !isfinite(g2))) flag(a.st, DBC_ERR_NONFINITE);
            }
            T *const o = tile_row(obuf, slot, X + r0 * a.xs, a.xs, k, a.d);
            const T *const ds = D ? tile_row(in + R * (yslot + slot), slot, D + r0 * a.ds_s, a.ds_s, k, a.d) : s;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = j * W + t;
                if (c < n) {
                    const float xh = f[j] * b.k.pre * b.k.rstd;
                    if (DW) acc[j] = fmaf(y[j], xh, acc[j]);
                    float u = fmaf(-xh, b.c, y[j] * w[j]) * b.k.rstd * b.k.pre;
                    if (D) u += ld_f(ds + c);
                    st_f(o + c, u);
                }
            }
        }
        __syncthreads();
        if (DW && (done += passes) > kFold - passes) {
            fold();
            done = 0;
        }
        tile_out(X + r0 * a.xs, a.xs, obuf, slot, rows, a.d);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (DW) {
        fold();
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += kThreads) {
            const double *const at = sums + c / W * kThreads + c % W;
            double v = 0;
#pragma unroll
            for (int i = 0; i < TEAMS; ++i) v += at[i * W];
            a.part[(int64_t)blockIdx.x * a.d + c] = v;
        }
    }
}

// Backward, wide rows: one row per CTA at a time.  Slots: dy, s (and ds) for
// `stages` rows; dx goes back into s's slot.  dw sums stay with the threads that
// own the columns: in fp64 behind the slots or, where those leave no room (NV = 16), in the CTA's line.
template <class TY, class T, bool DW, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > 512 ? 1 : 3) odd_bwd_kernel(const BwdArgs a, int yslot, int slot, int stages) {
    extern __shared__ __align__(16) char smem[];
    __shared__ float2 sh[32];
    __shared__ double2 shw[32];
    const int W = blockDim.x, t = threadIdx.x;
    const int stage = yslot + (a.ds ? 2 : 1) * slot;
    const TY *const Y = static_cast<const TY *>(a.dy);
    const T *const S = static_cast<const T *>(a.s);
    const T *const D = static_cast<const T *>(a.ds);
    float w[NV], acc[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float o[1] = {1.f};
        if (j * W + t < a.d) a.w.get<1>(j * W + t, o);
        w[j] = o[0];
        acc[j] = 0.f;
    }
    auto start = [&](int64_t r, int st) {
        if (r < a.N) {
            char *const in = smem + st * stage;
            row_in(in, Y, Y + r * a.ys, a.d, t, W);
            row_in(in + yslot, S, S + r * a.ss, a.d, t, W);
            if (D) row_in(in + yslot + slot, D, D + r * a.ds_s, a.d, t, W);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    constexpr bool OWN = DW && NV <= 8;
    double *const sums = reinterpret_cast<double *>(smem + stages * stage);
    double *const line = DW ? a.part + (int64_t)blockIdx.x * a.d : nullptr;
    const int ahead = stages - 1;
    int st = 0;
    if (ahead) start(blockIdx.x, 0);
    bool first = true;
    for (int64_t r = blockIdx.x; r < a.N; first = false) {
        // kFold rows at a time (all of them where no dw is wanted), then the fold
        const int64_t end = DW ? min(a.N, r + kFold * (int64_t)gridDim.x) : a.N;
        for (; r < end; r += gridDim.x) {
            __syncthreads();                              // the row before has left its slots
            if (ahead) start(r + gridDim.x, st ^ 1);
            else start(r, 0);
            copies_done(ahead);
            __syncthreads();
            char *const in = smem + st * stage;
            const TY *const dy = reinterpret_cast<const TY *>(in + off16(Y + r * a.ys));
            const T *const s = reinterpret_cast<const T *>(in + yslot + off16(S + r * a.ss));
            const T *const ds = reinterpret_cast<const T *>(in + yslot + slot + (D ? off16(D + r * a.ds_s) : 0));
            float y[NV], f[NV];
            float2 p = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = j * W + t;
                y[j] = c < a.d ? ld_f(dy + c) : 0.f;
                f[j] = c < a.d ? ld_f(s + c) : 0.f;
                p.x = fmaf(f[j], f[j], p.x);
                p.y = fmaf(y[j] * w[j], f[j], p.y);
            }
            p = team_pair(p, Add(), Add(), sh);       // (its barrier: everybody has read s)
            BwdFactor k(p.x, p.y, a);
            bool odd = !in_range(p.x, p.y);                  // the same in the whole team
            if (faint(p.y)) {
                bool some = false;
#pragma unroll
                for (int j = 0; j < NV; ++j) some |= y[j] * w[j] != 0.f;
                odd |= __syncthreads_or(some) != 0;
            }
            if (odd) {
                double2 q = make_double2(0, 0);
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    q.x += (double)f[j] * f[j];
                    q.y += (double)(y[j] * w[j]) * f[j];
                }
                q = team_pair(q, Add(), Add(), shw);
                k = BwdFactor(q.x, q.y, a);
                if (t == 0 && (!isfinite(q.x) || !isfinite(q.y))) flag(a.st, DBC_ERR_NONFINITE);
            }
            T *const dx = static_cast<T *>(a.dx) + r * a.xs;
            T *const o = reinterpret_cast<T *>(in + yslot + off16(dx));
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = j * W + t;
                const float xh = f[j] * k.k.pre * k.k.rstd;
                if (DW) acc[j] = fmaf(y[j], xh, acc[j]);
                if (c < a.d) {
                    float u[1] = {fmaf(-xh, k.c, y[j] * w[j]) * k.k.rstd * k.k.pre};
                    if (D) u[0] += ld_f(ds + c);
                    Frag<T, 1> q;
                    q.set(u);
                    q.store(o + c);
                }
            }
            __syncthreads();
            row_out(dx, in + yslot, a.d, t, W);
            if (ahead) st ^= 1;
        }
        if (DW) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float one[1] = {acc[j]};
                if (OWN) fold_sums<1, false>(sums + j * W + t, 0, one, first);
                else if (j * W + t < a.d) fold_sums<1, true>(line + j * W + t, 0, one, first);
                acc[j] = 0.f;
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (OWN) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * W + t < a.d) line[j * W + t] = sums[j * W + t];
    }
}

}  // namespace nm
}  // namespace dbc

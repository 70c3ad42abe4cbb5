// The norm kernels for rows off the 16-byte grid: odd widths, odd strides,
// shifted bases.
//
// Element by element from global memory such rows move 64 bytes per bf16
// instruction and stay at a fifth of HBM's rate.  Here a row travels as the
// aligned 16-byte pieces that cover it (asynchronous copies into shared memory
// one row ahead, whole pieces back out, elements only at its two ends) and only
// the arithmetic goes element by element, column j * W + t by thread t of the W
// that share the row.  Nothing outside the row is written, and nothing in front
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

template <bool BLOCK>
__device__ __forceinline__ void team_sync() {
    if constexpr (BLOCK) __syncthreads();
    else __syncwarp();
}
__device__ __forceinline__ void copies_done(int ahead) {
    if (ahead) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Sums two values over the team; `sh` is this team's, two buffers of 32 pairs
// used in turn by BLOCK teams (one barrier each).
template <bool BLOCK, class V2, class F, class G>
__device__ __forceinline__ V2 team_pair(V2 v, F f, G g, V2 *sh) {
    v.x = team_reduce<32>(v.x, f);
    v.y = team_reduce<32>(v.y, g);
    if constexpr (BLOCK) {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) sh[threadIdx.x >> 5] = v;
        __syncthreads();
        V2 u = lane < warps ? sh[lane] : V2{0, 0};
        v.x = team_reduce<32>(u.x, f);
        v.y = team_reduce<32>(u.y, g);
    }
    return v;
}

// Forward: teams of one warp (eight per CTA) or of a CTA.  Slots per team: x
// (and the residual) for `stages` rows, then y or q; s goes back into x's slot,
// whose values are in registers by then.
template <class T, int MODE, bool RES, int NV, bool BLOCK, int MAXT>
__global__ void __launch_bounds__(MAXT) odd_kernel(const FwdArgs a, int slot, int stages, int team_bytes) {
    extern __shared__ __align__(16) char smem[];
    __shared__ float2 sh[32];
    __shared__ double2 shw[32];
    const int W = BLOCK ? blockDim.x : 32, t = BLOCK ? threadIdx.x : threadIdx.x & 31;
    const int64_t teams = (int64_t)gridDim.x * (BLOCK ? 1 : blockDim.x / 32);
    const int64_t team = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
    char *const mine = smem + (BLOCK ? 0 : (threadIdx.x >> 5) * team_bytes);
    constexpr int IN = RES ? 2 : 1;
    char *const out = mine + stages * IN * slot;
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
            char *const in = mine + st * IN * slot;
            row_in(in, X, X + r * a.xs, a.d, t, W);
            if (RES) row_in(in + slot, Rs, Rs + r * a.rs, a.d, t, W);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int ahead = stages - 1;
    int st = 0;
    if (ahead) start(team, 0);
    for (int64_t r = team; r < a.N; r += teams) {
        team_sync<BLOCK>();                              // the row before has left its slots
        if (ahead) start(r + teams, st ^ 1);
        else start(r, 0);
        copies_done(ahead);
        team_sync<BLOCK>();
        char *const in = mine + st * IN * slot;
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
        const float2 sm = team_pair<BLOCK>(make_float2(ss, m), Add(), AbsMax(), sh);
        ss = sm.x, m = sm.y;
        RowFactor k(ss, a.d, a.eps);
        if (norms(MODE) && !(ss >= kLow && ss <= kHigh)) {   // the same in the whole team
            double t2 = 0;
#pragma unroll
            for (int j = 0; j < NV; ++j) t2 += (double)v[j] * v[j];
            t2 = team_pair<BLOCK>(make_double2(t2, 0), Add(), Add(), shw).x;
            k = RowFactor(t2, a.d, a.eps);
            if (!isfinite(t2)) {
                m = __int_as_float(0x7fc00000);
                if (t == 0) flag(a.st, DBC_ERR_NONFINITE);
            }
        }
        const Quant qn(m);
        T *const sp = RES && a.s ? static_cast<T *>(a.s) + r * a.ss : nullptr;
        T *const so = reinterpret_cast<T *>(in + off16(sp));
        if (!BLOCK) __syncwarp();                        // s overwrites x (a CTA has had its barrier in the sums)
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
            for (int j = 0; j < NV; ++j)
                if (j * W + t < a.d) {
                    const float p[1] = {weighs(MODE) ? v[j] * w[j] : v[j]};
                    qn.template store<narrow<T>(MODE), 1>(qo + j * W + t, p);
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
        team_sync<BLOCK>();
        if (RES && sp) row_out(sp, in, a.d, t, W);
        if (MODE != kPlain) row_out(a.q + r * a.qs, out, a.d, t, W);
        else if (a.y_bf16) row_out(static_cast<__nv_bfloat16 *>(a.y) + r * a.ys, out, a.d, t, W);
        else row_out(static_cast<float *>(a.y) + r * a.ys, out, a.d, t, W);
        if (ahead) st ^= 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Backward.  Slots per team: dy, s (and ds) for `stages` rows; dx goes back
// into s's slot.  dw sums stay with the threads that own the columns.
template <class TY, class T, bool DW, int NV, bool BLOCK, int MAXT>
__global__ void __launch_bounds__(MAXT)
    odd_bwd_kernel(const BwdArgs a, int yslot, int slot, int stages, int team_bytes) {
    extern __shared__ __align__(16) char smem[];
    __shared__ float2 sh[32];
    __shared__ double2 shw[32];
    const int W = BLOCK ? blockDim.x : 32, t = BLOCK ? threadIdx.x : threadIdx.x & 31;
    const int64_t teams = (int64_t)gridDim.x * (BLOCK ? 1 : blockDim.x / 32);
    const int64_t team = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
    char *const mine = smem + (BLOCK ? 0 : (threadIdx.x >> 5) * team_bytes);
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
            char *const in = mine + st * stage;
            row_in(in, Y, Y + r * a.ys, a.d, t, W);
            row_in(in + yslot, S, S + r * a.ss, a.d, t, W);
            if (D) row_in(in + yslot + slot, D, D + r * a.ds_s, a.d, t, W);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int ahead = stages - 1;
    int st = 0;
    if (ahead) start(team, 0);
    for (int64_t r = team; r < a.N; r += teams) {
        team_sync<BLOCK>();                              // the row before has left its slots
        if (ahead) start(r + teams, st ^ 1);
        else start(r, 0);
        copies_done(ahead);
        team_sync<BLOCK>();
        char *const in = mine + st * stage;
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
        p = team_pair<BLOCK>(p, Add(), Add(), sh);       // (its barrier: everybody has read s)
        BwdFactor k(p.x, p.y, a.d, a.eps);
        if (!in_range(p.x, p.y)) {                       // the same in the whole team
            double2 q = make_double2(0, 0);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                q.x += (double)f[j] * f[j];
                q.y += (double)(y[j] * w[j]) * f[j];
            }
            q = team_pair<BLOCK>(q, Add(), Add(), shw);
            k = BwdFactor(q.x, q.y, a.d, a.eps);
            if (t == 0 && (!isfinite(q.x) || !isfinite(q.y))) flag(a.st, DBC_ERR_NONFINITE);
        }
        T *const dx = static_cast<T *>(a.dx) + r * a.xs;
        T *const o = reinterpret_cast<T *>(in + yslot + off16(dx));
        if (!BLOCK) __syncwarp();
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
        team_sync<BLOCK>();
        row_out(dx, in + yslot, a.d, t, W);
        if (ahead) st ^= 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (DW && BLOCK) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * W + t < a.d) a.part[(int64_t)blockIdx.x * a.d + j * W + t] = acc[j];
    } else if constexpr (DW) {
        __syncthreads();                                 // the slots become the warps' lines
        float *const line = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * 32 + t < a.d) line[(threadIdx.x >> 5) * a.d + j * 32 + t] = acc[j];
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
            float v = 0.f;
            for (int i = 0; i < (int)blockDim.x / 32; ++i) v += line[i * a.d + c];
            a.part[(int64_t)blockIdx.x * a.d + c] = v;
        }
    }
}

}  // namespace nm
}  // namespace dbc

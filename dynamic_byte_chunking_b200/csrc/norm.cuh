// Building blocks of the norm kernels: row fragments in registers, team
// reductions, the 8-bit code.
#pragma once

#include "common.cuh"
#include "pairs.cuh"

namespace dbc {
namespace nm {

// NE consecutive elements of a row in registers: 16 bytes of the row's type (8
// bf16 or 4 fp32; 8 fp32 or 4 bf16 of an array of the other type beside it), or
// one element.  Rows bypass L1 (read once); what all rows share is kept there.
template <class T, int NE>
struct Frag;

template <>
struct Frag<__nv_bfloat16, 8> {
    uint32_t w[4];
    __device__ __forceinline__ float2 pair(int i) const {
        return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    // bf16(fp32(a + b)) is bf16(a + b): where the exponents are so far apart that fp32 rounds the sum,
    // it rounds to the larger operand either way.
    __device__ __forceinline__ void add(const Frag &g) {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(g.w[i]));
    }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(p));
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    }
    __device__ __forceinline__ void load_shared_by_rows(const __nv_bfloat16 *p) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void from_words(const uint32_t (&u)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = u[i];
    }
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
    __device__ __forceinline__ float at(int i) const {
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
};

template <>
struct Frag<__nv_bfloat16, 4> {
    uint32_t w[2];
    __device__ __forceinline__ float2 pair(int i) const {
        return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    // bf16(fp32(a + b)) is bf16(a + b): where the exponents are so far apart that fp32 rounds the sum,
    // it rounds to the larger operand either way.
    __device__ __forceinline__ void add(const Frag &g) {
#pragma unroll
        for (int i = 0; i < 2; ++i) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(g.w[i]));
    }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(p));
        w[0] = u.x, w[1] = u.y;
    }
    __device__ __forceinline__ void load_shared_by_rows(const __nv_bfloat16 *p) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = u.x, w[1] = u.y;
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
    __device__ __forceinline__ void from_words(const uint32_t (&u)[2]) { w[0] = u[0], w[1] = u[1]; }
    __device__ __forceinline__ void zero() { w[0] = w[1] = 0; }
    __device__ __forceinline__ float at(int i) const {
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ void set(const float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
};

template <>
struct Frag<__nv_bfloat16, 1> {
    __nv_bfloat16 b;
    __device__ __forceinline__ void load_shared_by_rows(const __nv_bfloat16 *p) {
        b = __ushort_as_bfloat16(__ldg(reinterpret_cast<const unsigned short *>(p)));
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *p = b; }
    __device__ __forceinline__ float at(int) const { return __bfloat162float(b); }
    __device__ __forceinline__ void set(const float (&v)[1]) { b = __float2bfloat16_rn(v[0]); }
};

template <int NE>
struct Frag<float, NE> {
    static_assert(NE == 8 || NE == 4 || NE == 1, "");
    float v[NE];
    __device__ __forceinline__ float2 pair(int i) const { return make_float2(v[2 * i], v[2 * i + 1]); }
    __device__ __forceinline__ void add(const Frag &g) {
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] += g.v[i];
    }
    __device__ __forceinline__ void load(const float *p) {
        if constexpr (NE == 1) {
            v[0] = __ldcg(p);
        } else {
#pragma unroll
            for (int i = 0; i < NE / 4; ++i) {
                const float4 u = __ldcg(reinterpret_cast<const float4 *>(p) + i);
                v[4 * i] = u.x, v[4 * i + 1] = u.y, v[4 * i + 2] = u.z, v[4 * i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ void load_shared_by_rows(const float *p) {
        if constexpr (NE == 1) {
            v[0] = __ldg(p);
        } else {
#pragma unroll
            for (int i = 0; i < NE / 4; ++i) {
                const float4 u = __ldg(reinterpret_cast<const float4 *>(p) + i);
                v[4 * i] = u.x, v[4 * i + 1] = u.y, v[4 * i + 2] = u.z, v[4 * i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ void store(float *p) const {
        if constexpr (NE == 1) {
            *p = v[0];
        } else {
#pragma unroll
            for (int i = 0; i < NE / 4; ++i)
                reinterpret_cast<float4 *>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
    }
    __device__ __forceinline__ void from_words(const uint32_t (&u)[NE]) {
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] = __uint_as_float(u[i]);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] = 0.f;
    }
    __device__ __forceinline__ float at(int i) const { return v[i]; }
    __device__ __forceinline__ void set(const float (&u)[NE]) {
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] = u[i];
    }
};

// The weight: fp32 or bf16, NULL reads as ones.
struct Weight {
    const void *p;
    int bf16;
    template <int NE>
    __device__ __forceinline__ void get(int64_t i, float (&out)[NE]) const {
        if (!p) {
#pragma unroll
            for (int k = 0; k < NE; ++k) out[k] = 1.f;
        } else if (bf16) {
            Frag<__nv_bfloat16, NE> f;
            f.load_shared_by_rows(static_cast<const __nv_bfloat16 *>(p) + i);
#pragma unroll
            for (int k = 0; k < NE; ++k) out[k] = f.at(k);
        } else {
            Frag<float, NE> f;
            f.load_shared_by_rows(static_cast<const float *>(p) + i);
#pragma unroll
            for (int k = 0; k < NE; ++k) out[k] = f.at(k);
        }
    }
};

template <int NE>
__device__ __forceinline__ void store_as(void *base, int bf16, int64_t i, const float (&v)[NE]) {
    if (bf16) {
        Frag<__nv_bfloat16, NE> f;
        f.set(v);
        f.store(static_cast<__nv_bfloat16 *>(base) + i);
    } else {
        Frag<float, NE> f;
        f.set(v);
        f.store(static_cast<float *>(base) + i);
    }
}

// max(m, |v|), NaN if either is.
__device__ __forceinline__ float abs_max(float m, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}

__device__ __forceinline__ float abs_max(float m, float2 v) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(v.x), "f"(v.y));
    return r;
}

// How a row is quantised, from its m = max |p|.
//
// The code is rint(127 p / m), halves to even, and it has to be the exact
// quotient's: with bf16 inputs one quotient in a few hundred IS a half.  The
// quotient t of a = 127 p comes from the reciprocal and one residual step, so
// it is a / m rounded once (but for 2^-23 of a step); adding 1.5 * 2^23 rounds t to a whole number
// (halves to even) and leaves it in the low bits.
//   NARROW (p has 16 significant bits: a bf16 value, or a product of two): a is
//   exact, and a / m is a half-integer h or at least h 2^-23.99 away from it
//   (254 P 2^e - (2k + 1) M is a multiple of 2^e, and 2^e >= h M / (127 * 2^16)),
//   more than the h 2^-24 that t is rounded by: t decides.
//   Otherwise t is off by up to 1.6e-5, and quotients closer than that to a half
//   (one fp32 value in ten thousand) are settled by the sign of 127 p - h m, with
//   127 p in two exact pieces; the difference from h m cancels to a few bits, so
//   it is exact too.
struct Quant {
    float m, rinv;
    bool bad;
    __device__ __forceinline__ explicit Quant(float m_) {
        bad = !(m_ <= 3.4028234e38f);
        m = bad ? 0.f : m_;
        rinv = m > 0.f ? 1.f / m : 0.f;
    }
    template <bool NARROW>
    __device__ __forceinline__ static float settle(float p, float m, float v, float t) {
        constexpr float kMagic = 12582912.f;
        const float r = v - kMagic, e = t - r;
        if (NARROW || fabsf(e) < 0.5f - 4e-5f) return v;
        const float h = r + copysignf(0.5f, e);
        const float hi = 127.f * p, lo = fmaf(127.f, p, -hi);
        const float d = fmaf(-h, m, hi) + lo;
        // just above or below h, or on it: the even neighbour (h + 1.5 * 2^23 would round to it too)
        const float f = d > 0.f ? h + 0.5f : d < 0.f ? h - 0.5f : rintf(h);
        return f + kMagic;
    }
    // Codes in the low bytes of u (anything for a bad row).
    template <bool NARROW, int NE>
    __device__ __forceinline__ void codes(const float (&p_)[NE], uint32_t (&u)[NE]) const {
        constexpr float kMagic = 12582912.f;
        float p[NE], ms = m, rs = rinv;
#pragma unroll
        for (int i = 0; i < NE; ++i) p[i] = p_[i];
        if (ms < 0x1p-60f || ms > 0x1p100f) {          // reciprocal or residual could leave fp32's range
            const float k = ms < 1.f ? 0x1p80f : 0x1p-80f;
            ms *= k;
            rs = ms > 0.f ? 1.f / ms : 0.f;
#pragma unroll
            for (int i = 0; i < NE; ++i) p[i] *= k;    // exact, or too small to matter
        }
        const float2 c127 = make_float2(127.f, 127.f), mm = make_float2(-ms, -ms), rr = make_float2(rs, rs);
#pragma unroll
        for (int i = 0; i < NE; i += 2) {
            const float2 a = mul2(make_float2(p[i], p[i + 1]), c127);
            const float2 t0 = mul2(a, rr);
            const float2 t = fma2(fma2(t0, mm, a), rr, t0);
            const float2 v = add2(t, make_float2(kMagic, kMagic));
            u[i] = __float_as_uint(settle<NARROW>(p[i], ms, v.x, t.x));
            u[i + 1] = __float_as_uint(settle<NARROW>(p[i + 1], ms, v.y, t.y));
        }
    }
    template <bool NARROW, int NE>
    __device__ __forceinline__ void store(int8_t *q, const float (&p)[NE]) const {
        uint32_t u[NE], w[NE / 4];
        codes<NARROW>(p, u);
#pragma unroll
        for (int i = 0; i < NE / 4; ++i)
            w[i] = bad ? 0u
                       : __byte_perm(__byte_perm(u[4 * i], u[4 * i + 1], 0x0040),
                                     __byte_perm(u[4 * i + 2], u[4 * i + 3], 0x0040), 0x5410);
        if constexpr (NE == 8) *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(q) = w[0];
    }
};

struct Add {
    template <class V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};
struct AbsMax {
    __device__ __forceinline__ float operator()(float a, float b) const { return abs_max(a, b); }
};

// Reduction over teams of W consecutive lanes (a power of two up to 32); all
// 32 lanes take part, every lane gets its team's result.
template <int W, class V, class F>
__device__ __forceinline__ V team_reduce(V v, F f) {
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Whether `v` holds in any lane of the team (all 32 lanes take part).
template <int W>
__device__ __forceinline__ bool team_any(bool v) {
    const uint32_t b = __ballot_sync(0xffffffffu, v);
    return ((b >> (threadIdx.x & 31 & ~(W - 1))) & (0xffffffffu >> (32 - W))) != 0;
}

// ---------------------------------------------------------------- what the kernels share
template <class T>
__device__ __forceinline__ float round_to(float v);
template <>
__device__ __forceinline__ float round_to<float>(float v) { return v; }
template <>
__device__ __forceinline__ float round_to<__nv_bfloat16>(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }

constexpr int kThreads = 256;
constexpr int64_t kMaxD = 16384;
constexpr float kLow = 1e-30f, kHigh = 1e37f;

// kI8Narrow: the norm's 8-bit form where s * w has 16 significant bits (bf16
// rows, bf16 weight or none); kQuant: no norm, p = x.
enum { kPlain = 0, kI8 = 1, kI8Narrow = 2, kQuant = 3 };
constexpr bool norms(int mode) { return mode != kQuant; }
constexpr bool weighs(int mode) { return mode == kI8 || mode == kI8Narrow; }
template <class T>
constexpr bool narrow(int mode) { return mode == kI8Narrow || (mode == kQuant && sizeof(T) == 2); }

struct FwdArgs {
    const void *x, *res;
    void *s, *y;
    int8_t *q;
    float *scale;
    Weight w;
    int64_t xs, rs, ss, ys, qs, N;
    int d, y_bf16;
    float eps, inv_d;
    int32_t *st;
};

// What the row's statistics say: the factors of y = (s * pre) * rstd * w (pre
// is 1 unless rstd would be subnormal) and the 8-bit scale.
struct RowFactor {
    float pre, rstd;
    template <class A>
    __device__ __forceinline__ RowFactor(float ss, const A &a) : pre(1.f) {
        rstd = rsqrtf(fmaf(ss, a.inv_d, a.eps));
    }
    template <class A>
    __device__ __forceinline__ RowFactor(double ss, const A &a) {
        const double r = 1.0 / sqrt(ss / a.d + (double)a.eps);
        pre = r < 0x1p-120 ? 0x1p-16f : 1.f;
        rstd = (float)(r / (double)pre);
    }
};

template <int MODE>
__device__ __forceinline__ float row_scale(const Quant &q, const RowFactor &k) {
    if (q.bad) return __int_as_float(0x7fc00000);
    const float m = q.m;
    if (!norms(MODE)) return m / 127.f;
    // the order that leaves fp32's normal range only where the scale itself does
    return m < 1.f ? m * k.rstd * k.pre / 127.f : m / 127.f * k.pre * k.rstd;
}

struct BwdArgs {
    const void *dy, *s, *ds;
    void *dx;
    Weight w;
    int64_t ys, ss, ds_s, xs, N;
    int d;
    float eps, inv_d;
    double *part;                // one line of d dw sums per CTA, or NULL
    int32_t *st;
};

__device__ __forceinline__ bool in_range(float ss, float sg) { return ss >= kLow && ss <= kHigh && isfinite(sg); }
// sum(g s) that is this small may have lost products below fp32's range: each loses up to 2^-150, up to 2^-136
// over the longest row, which a sum of 2^-110 does not notice (2^-26 of it).  Such a row is summed again in fp64
// unless all its g are zero (padding), where the fp32 sum is exact.
__device__ __forceinline__ bool faint(float sg) { return fabsf(sg) < 0x1p-110f; }

// dx = rstd (g - xhat c) + ds with xhat = s rstd and c = mean(g xhat); rstd as in RowFactor.
struct BwdFactor {
    RowFactor k;
    float c;
    __device__ __forceinline__ BwdFactor(float ss, float sg, const BwdArgs &a) : k(ss, a) {
        c = sg * a.inv_d * k.rstd;
    }
    __device__ __forceinline__ BwdFactor(double ss, double sg, const BwdArgs &a) : k(ss, a) {
        c = (float)(sg / a.d * (double)k.rstd * (double)k.pre);
    }
};

// dw: a thread adds the rows' terms of its columns in fp32 for this many rows, then adds that to fp64 sums.  One
// fp32 chain over all its rows would be off by a third of the square root of their number, in roundings of the
// result.  Measured with normal gradients: 9e-8 of dw at 65536 to 524288 rows, 2.9e-7 as one chain (fp64 sums of
// the same fp32 terms 6e-8; folds every 8 rows 8e-8 and up to 5 % slower).  Compensated fp32 sums are more exact,
// but their seven operations a term took 2200003 x 256 from 540 to 702 us; this takes 521.
constexpr int kFold = 16;
// Adds the fp32 sums of a thread's NE columns to its fp64 sums (or starts those), `step` apart, and clears them.
// Only this thread uses them, so the order is the program's.  LINE: in global memory, where the addition is sent
// off without waiting for the old value.
template <int NE, bool LINE>
__device__ __forceinline__ void fold_sums(double *sum, int step, float (&acc)[NE], bool first) {
#pragma unroll
    for (int i = 0; i < NE; ++i, sum += step) {
        if (first) *sum = acc[i];
        else if (LINE) atomicAdd(sum, (double)acc[i]);
        else *sum += acc[i];
        acc[i] = 0.f;
    }
}

}  // namespace nm
}  // namespace dbc

// Residual RMS norm, its 8-bit form, row quantisation and the norm's backward
// pass (formulas at the declarations in dbc.h).
//
// All of it is bound by HBM: a row is read, two row sums or a sum and a
// maximum are taken, and the row is written.  Sums are fp32; a row whose sum
// of squares leaves [1e-30, 1e37] (squares that overflow or vanish in fp32) is
// summed again in fp64 and finished there.
#include "common.cuh"

namespace dbc {
namespace nm {

constexpr int kThreads = 256;
constexpr int64_t kMaxD = 16384;

template <class T>
__device__ __forceinline__ float round_to(float v);
template <>
__device__ __forceinline__ float round_to<float>(float v) { return v; }
template <>
__device__ __forceinline__ float round_to<__nv_bfloat16>(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }

__device__ __forceinline__ void st_f(float *p, float v) { *p = v; }
__device__ __forceinline__ void st_f(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// An fp32 or bf16 array read element by element; NULL reads as ones.
struct Weight {
    const void *p;
    int bf16;
    __device__ __forceinline__ float at(int64_t i) const {
        if (!p) return 1.f;
        return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
    }
};

// The code of p for a row maximum m: rint(127 p / m), halves to even.  The
// fp32 quotient is off by less than 127 * 2^-23 = 1.6e-5; where that could
// decide the rounding, fp64 does: 127 p is exact there, and a quotient of two
// 24-bit numbers that is not a half-integer is at least 2^-34 away from one
// (|q| <= 127), far more than the division's rounding.
__device__ __noinline__ int code_exact(float p, float m) { return (int)rint((double)p * 127.0 / (double)m); }
__device__ __forceinline__ int code(float p, float m, float inv) {
    const float t = p * inv, r = rintf(t);
    if (fabsf(fabsf(t - r) - 0.5f) < 4e-5f) return code_exact(p, m);
    return (int)r;
}

// How a row is quantised, from m = max |p|: tiny rows are scaled by 2^100
// (exact) so that 127 / m stays in range.
struct Quant {
    float pre, m, inv;
    bool bad;
    __device__ __forceinline__ explicit Quant(float m_, bool nonfinite) {
        bad = nonfinite || !(m_ <= 3.4028234e38f);
        pre = m_ < 0x1p-60f ? 0x1p100f : 1.f;
        m = m_ * pre;
        inv = m > 0.f ? 127.f / m : 0.f;
    }
    __device__ __forceinline__ int operator()(float p) const { return bad || m == 0.f ? 0 : code(p * pre, m, inv); }
};

template <class F>
__device__ __forceinline__ double block_reduce(double v, F f, double *sm) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sm[0];
    for (int i = 1; i < kThreads / 32; ++i) v = f(v, sm[i]);
    return v;
}

enum { kPlain = 0, kI8 = 1, kQuantOnly = 2 };

struct FwdArgs {
    const void *x, *res;
    void *s, *y;
    int8_t *q;
    float *scale;
    Weight w;
    int64_t xs, rs, ss, ys, qs, N;
    int d, y_bf16;
    float eps;
    int32_t *st;
};

// One CTA per row; the row is read twice (the second time from L2).
template <class T, int MODE>
__global__ void __launch_bounds__(kThreads) norm_kernel(const FwdArgs a) {
    __shared__ double sm[kThreads / 32];
    auto add = [](double u, double v) { return u + v; };
    auto mx = [](double u, double v) { return fmax(u, v); };
    for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + r * a.xs;
        const T *res = a.res ? static_cast<const T *>(a.res) + r * a.rs : nullptr;
        T *s = a.s ? static_cast<T *>(a.s) + r * a.ss : nullptr;
        auto val = [&](int i) { return res ? round_to<T>(ld_f(x + i) + ld_f(res + i)) : ld_f(x + i); };
        float acc = 0.f, m = 0.f;
        bool fin = true;
        for (int i = threadIdx.x; i < a.d; i += kThreads) {
            const float v = val(i);
            acc = fmaf(v, v, acc);
            fin &= isfinite(v);
            if (MODE != kPlain) {
                const float p = fabsf(MODE == kI8 ? v * a.w.at(i) : v);
                fin &= isfinite(p);
                m = fmaxf(m, p);
            }
        }
        double ss = block_reduce(acc, add, sm);
        fin = __syncthreads_and(fin) != 0;
        if (!fin && threadIdx.x == 0) flag(a.st, DBC_ERR_NONFINITE);
        if (MODE != kPlain) m = (float)block_reduce(m, mx, sm);
        if (MODE != kQuantOnly && fin && !(ss >= 1e-30 && ss <= 1e37)) {
            double t = 0;
            for (int i = threadIdx.x; i < a.d; i += kThreads) {
                const double v = val(i);
                t += v * v;
            }
            ss = block_reduce(t, add, sm);
        }
        const double rstd = 1.0 / sqrt(ss / a.d + (double)a.eps);
        const Quant q(m, !fin);
        for (int i = threadIdx.x; i < a.d; i += kThreads) {
            const float v = val(i);
            if (s) st_f(s + i, v);
            if (MODE == kPlain) {
                const float o = (float)(v * rstd * a.w.at(i));
                if (a.y_bf16) st_f(static_cast<__nv_bfloat16 *>(a.y) + r * a.ys + i, o);
                else st_f(static_cast<float *>(a.y) + r * a.ys + i, o);
            } else {
                a.q[r * a.qs + i] = (int8_t)q(MODE == kI8 ? v * a.w.at(i) : v);
            }
        }
        if (MODE != kPlain && threadIdx.x == 0)
            a.scale[r] = !fin ? __int_as_float(0x7fc00000) : MODE == kI8 ? (float)(m * rstd / 127.0) : m / 127.f;
        __syncthreads();
    }
}

struct BwdArgs {
    const void *dy, *s, *ds;
    void *dx;
    Weight w;
    int64_t ys, ss, ds_s, xs, N;
    int d;
    float eps;
    float *part;
    int32_t *st;
};

// One CTA walks rows r = blockIdx.x, + gridDim.x, ...; thread t owns columns
// t, t + 256, ... and adds its rows' dw terms into its own line of `part`.
template <class TY, class T>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const BwdArgs a) {
    __shared__ double sm[kThreads / 32];
    auto add = [](double u, double v) { return u + v; };
    float *part = a.part ? a.part + (int64_t)blockIdx.x * a.d : nullptr;
    if (part)
        for (int i = threadIdx.x; i < a.d; i += kThreads) part[i] = 0.f;
    for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x) {
        const TY *dy = static_cast<const TY *>(a.dy) + r * a.ys;
        const T *s = static_cast<const T *>(a.s) + r * a.ss;
        const T *ds = a.ds ? static_cast<const T *>(a.ds) + r * a.ds_s : nullptr;
        T *dx = static_cast<T *>(a.dx) + r * a.xs;
        double t2 = 0, tg = 0;
        bool fin = true;
        for (int i = threadIdx.x; i < a.d; i += kThreads) {
            const double v = ld_f(s + i), g = (double)ld_f(dy + i) * a.w.at(i);
            fin &= isfinite(v) && isfinite(g);
            t2 += v * v;
            tg += v * g;
        }
        t2 = block_reduce(t2, add, sm);
        tg = block_reduce(tg, add, sm);
        if (!__syncthreads_and(fin) && threadIdx.x == 0) flag(a.st, DBC_ERR_NONFINITE);
        const double rstd = 1.0 / sqrt(t2 / a.d + (double)a.eps);
        const double c = tg / a.d * rstd * rstd;
        for (int i = threadIdx.x; i < a.d; i += kThreads) {
            const double v = ld_f(s + i), y = ld_f(dy + i);
            double o = rstd * (y * a.w.at(i) - v * c);
            if (ds) o += ld_f(ds + i);
            st_f(dx + i, (float)o);
            if (part) part[i] += (float)(y * v * rstd);
        }
    }
}

__global__ void __launch_bounds__(kThreads) dw_kernel(const float *part, int rows, int d, float *dw) {
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= d) return;
    double t = 0;
    for (int r = 0; r < rows; ++r) t += part[(int64_t)r * d + i];
    dw[i] = (float)t;
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

template <int MODE>
dbc_status launch_fwd(const FwdArgs &a, int dtype, cudaStream_t st) {
    const int grid = (int)std::min<int64_t>(a.N, (int64_t)num_sms() * 8);
    if (dtype == DBC_BF16) norm_kernel<__nv_bfloat16, MODE><<<grid, kThreads, 0, st>>>(a);
    else norm_kernel<float, MODE><<<grid, kThreads, 0, st>>>(a);
    count_launches(1);
    return launch_status();
}

inline int bwd_grid(int64_t N) { return (int)std::min<int64_t>(std::max<int64_t>(N, 1), 148 * 4); }

}  // namespace nm
}  // namespace dbc

using namespace dbc;

extern "C" dbc_status rms_norm(const void *x, int64_t x_stride, int dtype, const void *residual, int64_t r_stride,
                               const void *weight, int w_dtype, int64_t N, int64_t d, float eps, void *s,
                               int64_t s_stride, void *y, int64_t y_stride, int y_dtype, int32_t *dev_status,
                               dbc_stream_t stream) {
    DBC_NVTX_RANGE("rms_norm");
    nm::FwdArgs a{x, residual, s, y, nullptr, nullptr, {weight, w_dtype == DBC_BF16}, x_stride, r_stride, s_stride,
                  y_stride, 0, N, (int)d, y_dtype == DBC_BF16, eps, dev_status};
    const dbc_status c = nm::check_fwd(a, dtype, w_dtype, d, true);
    if (c != DBC_OK) return c;
    if (!nm::known(y_dtype)) return DBC_ERR_UNSUPPORTED;
    if (y_stride < d) return DBC_ERR_INVALID_ARG;
    if (N == 0) return DBC_OK;
    if (!y || !nm::aligned_to(y, nm::esize(y_dtype))) return DBC_ERR_INVALID_ARG;
    return nm::launch_fwd<nm::kPlain>(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" dbc_status rms_norm_i8(const void *x, int64_t x_stride, int dtype, const void *residual, int64_t r_stride,
                                  const void *weight, int w_dtype, int64_t N, int64_t d, float eps, void *s,
                                  int64_t s_stride, int8_t *q, int64_t q_stride, float *scale, int32_t *dev_status,
                                  dbc_stream_t stream) {
    DBC_NVTX_RANGE("rms_norm_i8");
    nm::FwdArgs a{x, residual, s, nullptr, q, scale, {weight, w_dtype == DBC_BF16}, x_stride, r_stride, s_stride,
                  0, q_stride, N, (int)d, 0, eps, dev_status};
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
                  1.f, dev_status};
    const dbc_status c = nm::check_fwd(a, dtype, DBC_F32, d, false);
    if (c != DBC_OK) return c;
    if (q_stride < d) return DBC_ERR_INVALID_ARG;
    if (N == 0) return DBC_OK;
    if (!q || !scale || !nm::aligned_to(scale, 4)) return DBC_ERR_INVALID_ARG;
    return nm::launch_fwd<nm::kQuantOnly>(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t rms_norm_backward_workspace(int64_t N, int64_t d) {
    if (N <= 0 || d <= 0) return 0;
    return align_up((size_t)nm::bwd_grid(N) * (size_t)d * sizeof(float));
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
    const int grid = nm::bwd_grid(N);
    nm::BwdArgs a{dy, s, ds, dx, {weight, w_dtype == DBC_BF16}, dy_stride, s_stride, ds_stride, dx_stride, N, (int)d,
                  eps, dw ? static_cast<float *>(ws) : nullptr, dev_status};
    using B = __nv_bfloat16;
    if (dy_dtype == DBC_BF16 && dtype == DBC_BF16) nm::bwd_kernel<B, B><<<grid, nm::kThreads, 0, st>>>(a);
    else if (dy_dtype == DBC_BF16) nm::bwd_kernel<B, float><<<grid, nm::kThreads, 0, st>>>(a);
    else if (dtype == DBC_BF16) nm::bwd_kernel<float, B><<<grid, nm::kThreads, 0, st>>>(a);
    else nm::bwd_kernel<float, float><<<grid, nm::kThreads, 0, st>>>(a);
    count_launches(dw ? 2 : 1);
    if (dw)
        nm::dw_kernel<<<(unsigned)((d + nm::kThreads - 1) / nm::kThreads), nm::kThreads, 0, st>>>(
            static_cast<const float *>(ws), grid, (int)d, dw);
    return launch_status();
}

// matmul_i8: out = a_scale * b_scale * (a b^T) (+ bias), int8 operands with
// exact int32 sums (formula and arguments at the declaration in dbc.h).
#include "common.cuh"

namespace dbc {
namespace mi {

constexpr int64_t kMaxK = 131071;                // K * 128 * 128 < 2^31
constexpr int64_t kMaxMN = (1ll << 31) - 1024;   // tile origins stay in 32 bits

struct Args {
    const int8_t *a, *b;
    const float *as, *bs;
    const void *bias;
    void *out;
    int64_t lda, ldb, ldo, M, N;
    int K, bias_bf16, out_bf16;
    int32_t *st;
};

__device__ __forceinline__ float bias_at(const Args &p, int64_t j) {
    if (!p.bias) return 0.f;
    return p.bias_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.bias)[j])
                       : static_cast<const float *>(p.bias)[j];
}

// 64 x 64 outputs per CTA of 256 threads, 4 x 4 each, with the packed 4-byte
// dot product; K in steps of 64 bytes through shared memory.
__global__ void __launch_bounds__(256) dot_kernel(const Args p) {
    __shared__ int A[64][17], B[64][17];
    const int64_t m0 = (int64_t)blockIdx.x * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t n0 = (int64_t)blockIdx.y * 64; n0 < p.N; n0 += (int64_t)gridDim.y * 64) {
        int acc[4][4] = {};
        for (int k0 = 0; k0 < p.K; k0 += 64) {
            const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 16;
            auto fetch = [&](const int8_t *base, int64_t ld, int64_t row, int64_t rows, int *dst) {
                int4 v = make_int4(0, 0, 0, 0);
                // rows start on 16 bytes and ld >= K is a multiple of 16, so the piece that holds
                // byte k0 + c < K lies inside the row
                if (row < rows && k0 + c < p.K) v = *reinterpret_cast<const int4 *>(base + row * ld + k0 + c);
                int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int left = p.K - (k0 + c + 4 * i);   // bytes of this word inside the row
                    dst[i] = left >= 4 ? w[i] : left <= 0 ? 0 : w[i] & ((1 << (8 * left)) - 1);
                }
            };
            fetch(p.a, p.lda, m0 + r, p.M, &A[r][c / 4]);
            fetch(p.b, p.ldb, n0 + r, p.N, &B[r][c / 4]);
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 16; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(A[ty + 16 * i][k], B[tx + 16 * j][k], acc[i][j]);
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + ty + 16 * i;
            for (int j = 0; j < 4; ++j) {
                const int64_t n = n0 + tx + 16 * j;
                if (m >= p.M || n >= p.N) continue;
                const float v = (float)acc[i][j] * p.as[m] * p.bs[n] + bias_at(p, n);
                if (p.out_bf16) static_cast<__nv_bfloat16 *>(p.out)[m * p.ldo + n] = __float2bfloat16_rn(v);
                else static_cast<float *>(p.out)[m * p.ldo + n] = v;
            }
        }
    }
}

}  // namespace mi
}  // namespace dbc

using namespace dbc;

extern "C" dbc_status matmul_i8(const int8_t *a, int64_t lda, const float *a_scale, const int8_t *b, int64_t ldb,
                                const float *b_scale, const void *bias, int bias_dtype, int64_t M, int64_t N,
                                int64_t K, void *out, int64_t ldo, int out_dtype, int32_t *dev_status,
                                dbc_stream_t stream) {
    DBC_NVTX_RANGE("matmul_i8");
    if (M < 0 || N < 0 || K < 0) return DBC_ERR_INVALID_ARG;
    if ((out_dtype != DBC_F32 && out_dtype != DBC_BF16) ||
        (bias && bias_dtype != DBC_F32 && bias_dtype != DBC_BF16) || K > mi::kMaxK || M > mi::kMaxMN ||
        N > mi::kMaxMN)
        return DBC_ERR_UNSUPPORTED;
    if (lda < K || ldb < K || lda % 16 || ldb % 16 || ldo < N) return DBC_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return DBC_OK;
    if (!a_scale || !b_scale || !out || (K && (!a || !b || !aligned16(a) || !aligned16(b))))
        return DBC_ERR_INVALID_ARG;
    const uintptr_t oa = out_dtype == DBC_BF16 ? 2 : 4, ba = bias_dtype == DBC_BF16 ? 2 : 4;
    if ((reinterpret_cast<uintptr_t>(out) % oa) || (bias && reinterpret_cast<uintptr_t>(bias) % ba) ||
        (reinterpret_cast<uintptr_t>(a_scale) % 4) || (reinterpret_cast<uintptr_t>(b_scale) % 4))
        return DBC_ERR_INVALID_ARG;
    const mi::Args p{a, b, a_scale, b_scale, bias, out, lda, ldb, ldo, M, N, (int)K, bias_dtype == DBC_BF16,
                     out_dtype == DBC_BF16, dev_status};
    const dim3 grid((unsigned)((M + 63) / 64), (unsigned)std::min<int64_t>((N + 63) / 64, 32768));
    mi::dot_kernel<<<grid, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    count_launches(1);
    return launch_status();
}

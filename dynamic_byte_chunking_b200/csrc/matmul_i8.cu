// matmul_i8: out = a_scale * b_scale * (a b^T) (+ bias), int8 operands with
// exact int32 sums (formula and arguments at the declaration in dbc.h).
//
// Both kernels feed kind::i8 tcgen05 MMAs (128 x N x 32 per instruction, sums
// in TMEM) from a ring of TMA-loaded, 128-byte swizzled stages of 128 bytes of
// K; TMA's zero fill pads odd depths and row counts.
//   * wide_kernel: 256 tokens x 256 channels per tile and pair of CTAs
//     (cta_group::2: each CTA loads half of both operands, so that a byte of
//     shared memory feeds twice the products of a single CTA's tile), one
//     persistent CTA per SM; loads, MMAs and the epilogue of the tile before (two
//     accumulators) run at the same time.  Outputs leave through swizzled staging
//     and TMA tile stores.
//   * split_kernel: for few tokens or few tiles.  128 CHANNELS sit on the TMEM
//     lanes and the tokens on its columns, so that one token costs 16 columns
//     and not 128 lanes; the depth is split over a cluster of up to 8 CTAs,
//     whose partial sums (integers: any order gives the same) are joined through
//     distributed shared memory.
// Measured (us on the device): 8192 x 4096 x 4096 94 in short runs (2.9 P op/s, 86 % of twice the
// measured bf16 rate; the tensor pipe is fed without a pause: a stage of 512 cycles' MMAs every 541) and
// 108 in long ones, where the power cap holds the clock near 1.45 GHz (torch._int_mm, without scales: 106);
// 32768 x 1536 x 512 34 (outputs and their staging share the time with the loads: 28 without the stores,
// 24 without the epilogue's arithmetic); 4 x 8192 x 8192 15.9 with the weight in HBM (66 % of the copy's
// rate) and 10.7 with it in L2.
// Every wait is bounded; a timeout flags DBC_ERR_TIMEOUT and the CTA skips its
// remaining work, after waiting for its copies and MMAs in flight.
#include <cuda.h>
#include <string.h>

#include "pairs.cuh"
#include "tc.cuh"
#include "tma_host.cuh"

namespace dbc {
namespace mi {

constexpr int64_t kMaxK = 131071;                // K * 128 * 128 < 2^31
constexpr int64_t kMaxMN = (1ll << 31) - 1024;   // tile origins stay in 32 bits

struct Args {
    const float *as, *bs;
    const void *bias;
    void *out;
    int64_t ldo;
    int M, N, K, bias_bf16, out_bf16;
    int32_t *st;
};

__device__ __forceinline__ float bias_at(const Args &p, int64_t j) {
    if (!p.bias) return 0.f;
    return p.bias_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.bias)[j])
                       : static_cast<const float *>(p.bias)[j];
}

// sum * a_scale * b_scale (+ bias).  The smaller scale comes first: 2^31 times it overflows only where the result
// does, and its product with a whole number keeps fp32's precision at any size.
__device__ __forceinline__ float scaled(float sum, float as, float bs, float bias) {
    const bool a = fabsf(as) < fabsf(bs);
    return fmaf(sum * (a ? as : bs), a ? bs : as, bias);
}
// Up to this the token's scale may come first whatever the other is.
constexpr float kBigScale = 0x1p96f;

// The four (at the end of the depth: fewer) K steps of one stage.
__device__ __forceinline__ void mma_stage(uint32_t d, uint32_t sa, uint32_t sb, uint32_t idesc, int left, bool first) {
    const uint64_t da = tc::sdesc(sa, 16, 1024), db = tc::sdesc(sb, 16, 1024);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k * 32 < left)
            tc::mma_i8(d, tc::sdesc_add(da, k * 32), tc::sdesc_add(db, k * 32), idesc, first && k == 0 ? 0u : 1u);
}

// ---------------------------------------------------------------- many tiles
struct Wide {
    static constexpr int BM = 256, BN = 256;                              // of a pair; each CTA loads half of both
    static constexpr int NS = 5, EPI = 16, THREADS = 64 + EPI * 32;
    static constexpr uint32_t HALF = 128 * 128, STAGE = 2 * HALF;
    static constexpr uint32_t SLAB = 32 * 64;                             // one warp's 32 rows x 64 bytes
    static constexpr size_t SMEM = NS * STAGE + EPI * SLAB + 1024;
};

struct Tile {
    int m, n;
};
// Tiles in groups of 16 column blocks, rows outermost inside a group: the CTAs
// that run together share their rows of a and a group's rows of b in L2.
// Divisions by a group's width go by its reciprocal (exact: fewer than 2^28
// tiles to a group of at most 16 columns); as divisions they were a quarter of
// the epilogue's time.
struct Tiles {
    uint32_t full, last, inv16, inv_last, groups;        // tiles of a full group; the last group's width
    __device__ __forceinline__ Tiles(uint32_t mt, uint32_t nt)
        : full(mt * 16), last((nt - 1) % 16 + 1), inv16(1u << 28), inv_last(0xffffffffu / last + 1), groups((nt + 15) / 16) {}
    __device__ __forceinline__ Tile at(uint32_t i) const {
        const uint32_t g = groups == 1 ? 0 : i / full, rem = i - g * full;
        const bool tail = g + 1 == groups;
        const uint32_t w = tail ? last : 16, m = w == 1 ? rem : __umulhi(rem, tail ? inv_last : inv16);
        return {(int)m, (int)(g * 16 + rem - m * w)};
    }
};

template <bool TMA_OUT, bool BF16, bool BIAS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Wide::THREADS, 1)
    wide_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                const __grid_constant__ CUtensorMap to, const Args p) {
    using C = Wide;
    extern __shared__ uint8_t smraw[];
    // full: CTA 0's, both producers' copies; empty, tfull: each CTA's, committed by CTA 0's MMAs;
    // tempty: CTA 0's, the epilogue warps of both CTAs
    __shared__ uint64_t full[C::NS], empty[C::NS], tfull[2], tempty[2], drain;
    __shared__ uint32_t tmem_base;
    __shared__ __align__(16) float s_scale[C::EPI][64], s_bias[C::EPI][64];       // each epilogue warp's channels
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = tc::cluster_rank();
    const uint32_t base = (tc::smem_u32(smraw) + 1023u) & ~1023u;
    uint8_t *const sgen = smraw + (base - tc::smem_u32(smraw));
    if (warp == 1) tc::tmem_alloc_pair(&tmem_base, 2 * C::BN);
    if (tid == 0) {
        for (int i = 0; i < C::NS; ++i) {
            tc::mbar_init(&full[i], 2);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&tfull[i], 1);
            tc::mbar_init(&tempty[i], 2 * C::EPI);
        }
        tc::mbar_init(&drain, 1);
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&ta);
        tc::tma_prefetch_desc(&tb);
        if (TMA_OUT) tc::tma_prefetch_desc(&to);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();                                  // both CTAs' barriers exist
    tc::fence_after_sync();
    const uint32_t tbase = tmem_base;
    const int mt = (p.M + C::BM - 1) / C::BM, nt = (p.N + C::BN - 1) / C::BN, ks = (p.K + 127) / 128;
    const int tiles = mt * nt, pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    const Tiles order((uint32_t)mt, (uint32_t)nt);

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, issued = 0;                       // stage; stages in use, up to NS
            uint32_t ph = 1;                             // parity of the stage's last release
            bool ok = true;
            for (int i = pair; i < tiles && ok; i += pairs) {
                const Tile t = order.at(i);
                const int y0 = t.m * C::BM + (int)rank * 128, x0 = t.n * C::BN + (int)rank * 128;
                for (int k = 0; k < ks; ++k) {
                    if (issued == C::NS && !(ok = tc::mbar_wait(&empty[s], ph, p.st))) break;
                    issued += issued < C::NS;
                    const uint32_t sa = base + s * C::STAGE, bar = tc::map_to(tc::smem_u32(&full[s]), 0);
                    tc::mbar_arrive_expect_tx_at(bar, C::STAGE);
                    tc::tma_load_2d_pair(sa, &ta, bar, k * 128, y0);
                    tc::tma_load_2d_pair(sa + C::HALF, &tb, bar, k * 128, x0);
                    if (++s == C::NS) s = 0, ph ^= 1;
                }
            }
            // all stages released: no arrival is under way to a CTA that has ended
            for (int k = 0; k < issued && ok; ++k) {
                const bool wrap = issued == C::NS && s + k >= C::NS;
                ok = issued == C::NS ? tc::mbar_wait(&empty[wrap ? s + k - C::NS : s + k], wrap ? ph ^ 1 : ph, p.st)
                                     : tc::mbar_wait(&empty[k], 0, p.st);
            }
            // after a timeout: copies under way (microseconds) land before the CTA ends
            if (!ok)
                for (const long long t0 = clock64(); clock64() - t0 < (1ll << 22);) {
                }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // The whole warp walks the loop and one elected lane issues: descriptors stay in uniform
            // registers (issued from a single-lane branch an MMA took 80 cycles, its work takes 128).
            // The next stage's barrier is asked before this stage's MMAs are issued.
            constexpr uint32_t idesc = tc::idesc_i8(C::BM, C::BN);
            const bool issuer = tc::elect_one();
            int s = 0;
            uint32_t ph = 0;
            int n = 0;
            bool ok = true, ready = false;
            for (int i = pair; i < tiles && ok; i += pairs, ++n) {
                const int b = (int)(n & 1);
                if (n >= 2) ok = tc::mbar_wait(&tempty[b], (uint32_t)(n / 2 - 1) & 1u, p.st);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                for (int k = 0; k < ks; ++k) {
                    if (!ready) ok = tc::mbar_wait(&full[s], ph, p.st);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    const int s1 = s + 1 == C::NS ? 0 : s + 1;
                    const uint32_t ph1 = s + 1 == C::NS ? ph ^ 1 : ph;
                    ready = tc::mbar_try_wait(&full[s1], ph1);
                    tc::fence_after_sync();
                    const uint32_t sa = base + s * C::STAGE;
                    const uint64_t da = tc::sdesc(sa, 16, 1024), db = tc::sdesc(sa + C::HALF, 16, 1024);
                    const int left = p.K - k * 128;
                    if (issuer) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j * 32 < left)
                                tc::mma_i8_pair(tbase + b * C::BN, tc::sdesc_add(da, j * 32), tc::sdesc_add(db, j * 32),
                                                idesc, k || j ? 1u : 0u);
                        tc::mma_commit_pair(&empty[s]);
                    }
                    __syncwarp();
                    s = s1, ph = ph1;
                }
                if (ok && issuer) tc::mma_commit_pair(&tfull[b]);
                __syncwarp();
            }
            if (!ok) {
                if (issuer) {
                    tc::mma_commit_pair(&drain);
                    tc::mbar_wait(&drain, 0, p.st);
                }
                __syncwarp();
            }
        }
    } else {
        // Warp w owns TMEM lanes (w % 4) * 32 .. + 31 (its tokens) and 64 of the 256 columns.  It takes
        // them into registers at once and releases the accumulator, so that the MMAs of the tile
        // after next do not wait for the arithmetic.
        const int q = warp & 3, cg = ((warp - 2) >> 2) * 64;
        uint8_t *const slab = sgen + C::NS * C::STAGE + (warp - 2) * C::SLAB;
        float *const sc = s_scale[warp - 2], *const sb = s_bias[warp - 2];
        const uint32_t release[2] = {tc::map_to(tc::smem_u32(&tempty[0]), 0), tc::map_to(tc::smem_u32(&tempty[1]), 0)};
        constexpr int COLS = BF16 ? 32 : 16;             // columns of a slab
        constexpr int E = COLS / 4;                      // elements of 16 bytes
        bool ok = true;
        // The next tile's scales are fetched while this one is computed: a lane's four rows' and two of the
        // warp's 64 channels', which the warp shares.  No barrier joins the warps, so that they drift apart
        // and fill each other's waits.
        float as[4] = {0.f, 0.f, 0.f, 0.f}, cs[2] = {0.f, 0.f};
        uint32_t cb[2] = {0, 0};
        Tile next = {0, 0};
        auto fetch = [&](int i) {
            if (i >= tiles) return;
            next = order.at(i);
            const int row = next.m * C::BM + (int)rank * 128 + q * 32 + (lane >> 2), j0 = next.n * C::BN + cg + lane;
#pragma unroll
            for (int h = 0; h < 4; ++h)
                if (row + h * 8 < p.M) as[h] = p.as[row + h * 8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = j0 + h * 32;
                if (j < p.N) {
                    cs[h] = p.bs[j];
                    if (BIAS) cb[h] = p.bias_bf16 ? static_cast<const uint16_t *>(p.bias)[j] : static_cast<const uint32_t *>(p.bias)[j];
                }
            }
        };
        fetch(pair);
        int b = 0;
        uint32_t ph = 0;
        for (int i = pair; i < tiles; i += pairs, ph ^= b, b ^= 1) {
            const int r0 = next.m * C::BM + (int)rank * 128 + q * 32, n0 = next.n * C::BN + cg;
            const float ra[4] = {as[0], as[1], as[2], as[3]};
            __syncwarp();                                // the tile before has read the channels' scales
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sc[h * 32 + lane] = cs[h];
                if (BIAS) sb[h * 32 + lane] = __uint_as_float(p.bias_bf16 ? cb[h] << 16 : cb[h]);
            }
            __syncwarp();
            fetch(i + pairs);
            // (one lane polls: 32 of them slow the barriers that the MMA thread waits on)
            if (ok && lane == 0) ok = tc::mbar_wait(&tfull[b], ph, p.st);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            tc::fence_after_sync();
            uint32_t v[2][32];                           // rows q * 32 .. + 15 and + 16 .. + 31
            const uint32_t tad = tbase + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * C::BN + cg);
            tc::tmem_ld_16x64_nw(tad, v[0]);
            tc::tmem_ld_16x64_nw(tad + (16u << 16), v[1]);
            tc::tmem_wait_ld();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_at(release[b]);
            if (n0 >= p.N || r0 >= p.M) continue;
            if (__any_sync(0xffffffffu, fmaxf(fmaxf(fabsf(ra[0]), fabsf(ra[1])), fmaxf(fabsf(ra[2]), fabsf(ra[3]))) > kBigScale)) {
                // a scale that may have to come second: the sums go through the staging, element by element
                // (the order chosen in the loop below would cost every call 4 to 6 %)
#pragma unroll
                for (int c0 = 0; c0 < 64; c0 += 16) {
                    if (TMA_OUT && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    __syncwarp();
#pragma unroll
                    for (int i = c0 / 8; i < c0 / 8 + 2; ++i)
#pragma unroll
                        for (int h = 0; h < 4; ++h)
                            *reinterpret_cast<uint2 *>(slab + ((lane >> 2) + h * 8) * 64 + (i & 1) * 32 + (lane & 3) * 8) =
                                make_uint2(v[h >> 1][i * 4 + (h & 1) * 2], v[h >> 1][i * 4 + (h & 1) * 2 + 1]);
                    __syncwarp();
                    const int j = n0 + c0 + lane % 16, rows = min(32, p.M - r0);
                    for (int r = lane / 16; r < rows && j < p.N; r += 2) {
                        const int sum = *reinterpret_cast<const int *>(slab + r * 64 + lane % 16 * 4);
                        const float o = scaled((float)sum, p.as[r0 + r], p.bs[j], BIAS ? bias_at(p, j) : 0.f);
                        const int64_t at = (int64_t)(r0 + r) * p.ldo + j;
                        if constexpr (BF16) static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(o);
                        else static_cast<float *>(p.out)[at] = o;
                    }
                }
                continue;
            }
#pragma unroll
            for (int c0 = 0; c0 < 64; c0 += COLS) {
                if (TMA_OUT && lane == 0)                // the store before has read the staging
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
                // blocks of 8 columns: this lane has two of them, of rows lane / 4 + 0, 8, 16, 24 (so that it
                // needs the scales of 16 channels and not of 64)
#pragma unroll
                for (int i = c0 / 8; i < (c0 + COLS) / 8; ++i) {
                    const int c = i * 8 + (lane & 3) * 2;
                    const float2 s2 = *reinterpret_cast<const float2 *>(sc + c);
                    const float2 b2 = BIAS ? *reinterpret_cast<const float2 *>(sb + c) : make_float2(0.f, 0.f);
                    uint32_t w[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const uint32_t *x = &v[h >> 1][i * 4 + (h & 1) * 2];
                        float2 o = mul2(make_float2((float)(int)x[0], (float)(int)x[1]), make_float2(ra[h], ra[h]));
                        o = BIAS ? fma2(o, s2, b2) : mul2(o, s2);
                        if constexpr (BF16) {
                            const __nv_bfloat162 z = __floats2bfloat162_rn(o.x, o.y);
                            w[h] = *reinterpret_cast<const uint32_t *>(&z);
                        } else {
                            const int r = (lane >> 2) + h * 8, ch = (i & 1) * 2 + ((lane & 3) >> 1);
                            *reinterpret_cast<float2 *>(slab + r * 64 + ((ch ^ ((r >> 1) & 3)) * 16) + (lane & 1) * 8) = o;
                        }
                    }
                    // 64-byte swizzle: chunk c of row r at c ^ (r / 2 % 4); here lane l's is row l of chunk i
                    if constexpr (BF16)
                        tc::stmatrix4(tc::smem_u32(slab) + lane * 64 + (((i & 3) ^ ((lane >> 1) & 3)) * 16), w[0], w[1],
                                      w[2], w[3]);
                }
                if (n0 + c0 < p.N) {
                    if (TMA_OUT) {
                        tc::fence_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            asm volatile(
                                "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                                    &to),
                                "r"(n0 + c0), "r"(r0), "r"(tc::smem_u32(slab))
                                : "memory");
                            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        }
                    } else {
                        // output rows or widths off the 16-byte grid: element by element, row after row of the slab
                        __syncwarp();
                        const int cols = min(COLS, p.N - n0 - c0), rows = min(32, p.M - r0);
                        constexpr int STEP = 32 / COLS;  // rows at a time
                        const int j = lane % COLS;
                        for (int r = lane / COLS; r < rows; r += STEP) {
                            if (j >= cols) continue;
                            const int64_t at = (int64_t)(r0 + r) * p.ldo + n0 + c0 + j;
                            const uint8_t *src = slab + r * 64 + (((j / E) ^ ((r >> 1) & 3)) * 16);
                            if constexpr (BF16)
                                static_cast<__nv_bfloat16 *>(p.out)[at] =
                                    reinterpret_cast<const __nv_bfloat16 *>(src)[j % E];
                            else
                                static_cast<float *>(p.out)[at] = reinterpret_cast<const float *>(src)[j % E];
                        }
                        __syncwarp();
                    }
                }
            }
        }
        // the staging outlives the stores' reads; the writes complete with the kernel
        if (TMA_OUT && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();                                  // nothing of the pair is under way to this CTA
    if (warp == 1) tc::tmem_dealloc_pair(tbase, 2 * C::BN);
}

// ---------------------------------------------------------------- few tokens or few tiles
// BT tokens (TMEM columns) x 128 channels (lanes) per cluster of CTAs that
// split the depth.
template <int BT>
struct Split {
    static constexpr int NS = BT <= 32 ? 5 : 4;
    static constexpr uint32_t W = 128 * 128, X = BT * 128, STAGE = W + X;
    static constexpr int PITCH = 132;                                     // words per token of the partial sums
    static constexpr uint32_t RING = NS * STAGE, PART = BT * PITCH * 4;
    static constexpr size_t SMEM = (RING > PART ? RING : PART) + 1024;
    static constexpr int TCOLS = BT < 32 ? 32 : BT;
};

__device__ __forceinline__ int4 ld_cluster(uint32_t addr, uint32_t rank) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(tc::map_to(addr, rank)));
    return v;
}

// Joins the partial sums of tokens rank, rank + S, ... of a cluster of S CTAs: a warp takes a token at a
// time, a lane four channels; four tokens' loads from all CTAs are in flight together.
template <int S, int PITCH, class F>
__device__ __forceinline__ void join(uint32_t base, uint32_t rank, int rows, F put) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int m0 = (int)rank + S * warp; m0 < rows; m0 += S * 16) {
        int4 v[4][S];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < S; ++r) {
                const int m = m0 + S * 4 * i;
                v[i][r] = m < rows ? ld_cluster(base + (uint32_t)(m * PITCH + lane * 4) * 4u, r) : make_int4(0, 0, 0, 0);
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int4 t = v[i][0];
#pragma unroll
            for (int r = 1; r < S; ++r) t.x += v[i][r].x, t.y += v[i][r].y, t.z += v[i][r].z, t.w += v[i][r].w;
            if (m0 + S * 4 * i < rows) put(m0 + S * 4 * i, t);
        }
    }
}

__device__ __forceinline__ void store_one(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

template <int BT>
__global__ void __launch_bounds__(128)
    split_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx, const Args p,
                 const int splits) {
    using C = Split<BT>;
    extern __shared__ uint8_t smraw[];
    __shared__ uint64_t full[C::NS], empty[C::NS], done;
    __shared__ uint32_t tmem_base;
    __shared__ int s_ok;
    __shared__ float s_as[BT];                           // the tokens' scales
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (tc::smem_u32(smraw) + 1023u) & ~1023u;
    int *const part = reinterpret_cast<int *>(smraw + (base - tc::smem_u32(smraw)));
    const uint32_t rank = splits > 1 ? tc::cluster_rank() : 0;
    const int n0 = (int)(blockIdx.x / splits) * 128, m0 = blockIdx.y * BT;
    const int ks = (p.K + 127) / 128;
    const int k0 = (int)((int64_t)ks * rank / splits), k1 = (int)((int64_t)ks * (rank + 1) / splits);
    if (warp == 0) tc::tmem_alloc(&tmem_base, C::TCOLS);
    if (tid == 0) {
        for (int i = 0; i < C::NS; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        tc::mbar_init(&done, 1);
        tc::fence_mbar_init();
        s_ok = 1;
        if (p.K) {
            tc::tma_prefetch_desc(&tw);
            tc::tma_prefetch_desc(&tx);
        }
    }
    const int rows = min(BT, p.M - m0);
    const float my_as = tid < rows ? p.as[m0 + tid] : 0.f;
    if (tid < BT) s_as[tid] = my_as;
    tc::fence_before_sync();
    const bool order = __syncthreads_or(fabsf(my_as) > kBigScale) != 0;
    tc::fence_after_sync();
    const uint32_t tbase = tmem_base;

    if (warp == 0) {
        // warp 0 loads, warp 1 issues the MMAs: whole warps, one elected lane acting (see wide_kernel)
        const bool issuer = tc::elect_one();
        bool ok = true;
        int s = 0;
        uint32_t ph = 1;
        for (int k = k0; k < k1; ++k) {
            if (k - k0 >= C::NS) ok = tc::mbar_wait(&empty[s], ph, p.st);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            if (issuer) {
                const uint32_t sw = base + s * C::STAGE;
                tc::mbar_arrive_expect_tx(&full[s], C::STAGE);
                tc::tma_load_2d(sw, &tw, &full[s], k * 128, n0);
                tc::tma_load_2d(sw + C::W, &tx, &full[s], k * 128, m0);
            }
            __syncwarp();
            if (++s == C::NS) s = 0, ph ^= 1;
        }
        if (!ok) {
            // after a timeout: every stage's last copies land before the shared memory is reused
            for (int k = 0; k < C::NS; ++k) tc::mbar_wait(&full[k], k < s ? ph ^ 1 : ph, p.st);
            s_ok = 0;
        }
    } else if (warp == 1) {
        constexpr uint32_t idesc = tc::idesc_i8(128, BT);
        const bool issuer = tc::elect_one();
        bool ok = true;
        int s = 0;
        uint32_t ph = 0;
        for (int k = k0; k < k1; ++k) {
            ok = tc::mbar_wait(&full[s], ph, p.st);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc::fence_after_sync();
            const uint32_t sw = base + s * C::STAGE;
            if (issuer) {
                mma_stage(tbase, sw, sw + C::W, idesc, p.K - k * 128, k == k0);
                tc::mma_commit(&empty[s]);
            }
            __syncwarp();
            if (++s == C::NS) s = 0, ph ^= 1;
        }
        if (issuer) tc::mma_commit(&done);
        __syncwarp();
        ok &= tc::mbar_wait(&done, 0, p.st);
        if (!__all_sync(0xffffffffu, ok)) s_ok = 0;
    }
    __syncthreads();
    tc::fence_after_sync();
    const bool ok = s_ok != 0;
    auto put = [&](int m, int n, int sum, float as, float bs, float bias) {
        const float v = order ? scaled((float)sum, as, bs, bias) : fmaf((float)sum * as, bs, bias);
        const int64_t at = (int64_t)(m0 + m) * p.ldo + n;
        if (p.out_bf16) static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(v);
        else static_cast<float *>(p.out)[at] = v;
    };
    if (splits == 1) {
        const int n = n0 + tid;                         // this thread's channel
        const float bs = n < p.N ? p.bs[n] : 0.f, bias = n < p.N ? bias_at(p, n) : 0.f;
        auto column = [&](auto *o) {
            o += (int64_t)m0 * p.ldo + n;
            for (int c0 = 0; c0 < rows && ok; c0 += 16) {
                uint32_t v[16];
                tc::tmem_ld16_nw(tbase + ((uint32_t)(warp * 32) << 16) + c0, v);
                tc::tmem_wait_ld();
                float f[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] = fmaf((p.K ? (float)(int)v[j] : 0.f) * s_as[c0 + j], bs, bias);
                if (order) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) f[j] = scaled(p.K ? (float)(int)v[j] : 0.f, s_as[c0 + j], bs, bias);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j, o += p.ldo)
                    if (c0 + j < rows && n < p.N) store_one(o, f[j]);
            }
        };
        if (p.out_bf16) column(static_cast<__nv_bfloat16 *>(p.out));
        else column(static_cast<float *>(p.out));
    } else {
        for (int c0 = 0; c0 < rows; c0 += 16) {
            uint32_t v[16];
            tc::tmem_ld16_nw(tbase + ((uint32_t)(warp * 32) << 16) + c0, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) part[(c0 + j) * C::PITCH + tid] = (int)v[j];
        }
        const int n = n0 + lane * 4;                    // the first of this lane's channels
        float bs[4], bias[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bs[j] = n + j < p.N ? p.bs[n + j] : 0.f;
            bias[j] = n + j < p.N ? bias_at(p, n + j) : 0.f;
        }
        auto put4 = [&](int m, const int4 &t) {
            const float as = s_as[m];
            const int s[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < p.N) put(m, n + j, s[j], as, bs[j], bias[j]);
        };
        tc::cluster_sync();
        if (ok) {
            if (splits == 2) join<2, C::PITCH>(base, rank, rows, put4);
            else if (splits == 4) join<4, C::PITCH>(base, rank, rows, put4);
            else join<8, C::PITCH>(base, rank, rows, put4);
        }
        tc::cluster_sync();                              // the others have read this CTA's sums
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) tc::tmem_dealloc(tbase, C::TCOLS);
}

template <int BT>
dbc_status launch_split(const int8_t *a, int64_t lda, const int8_t *b, int64_t ldb, const Args &p, cudaStream_t st) {
    using C = Split<BT>;
    CUtensorMap tw, tx;
    memset(&tw, 0, sizeof tw);
    memset(&tx, 0, sizeof tx);
    if (p.K && (!tma::encode_i8_rows(&tw, b, p.N, p.K, ldb, 128) || !tma::encode_i8_rows(&tx, a, p.M, p.K, lda, BT)))
        return DBC_ERR_CUDA;
    const int nt = (p.N + 127) / 128, mt = (p.M + BT - 1) / BT, ks = (p.K + 127) / 128;
    int splits = 1;
    // At least two steps of depth to a CTA, and no more CTAs than run at once: one to an SM with 128
    // tokens' stages (200 x 4096 x 4096 takes 12.2 us so, 17.9 with up to two; 100 x 5000 x 5000 13.9 and
    // 19.6), else two (64 x 8192 x 8192 takes 12.2 us with up to two to an SM, 15.3 with one; 4 x 8192 x 8192
    // 10.7 and 13.1).
    while (splits < 8 && splits * 4 <= ks && (int64_t)nt * mt * splits * 2 <= 148 * (BT > 64 ? 1 : 2)) splits *= 2;
    if (cudaFuncSetAttribute(split_kernel<BT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM) !=
        cudaSuccess) {
        cudaGetLastError();                              // not the next call's
        return DBC_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(nt * splits), (unsigned)mt);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)splits;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, split_kernel<BT>, tw, tx, p, splits) != cudaSuccess) {
        cudaGetLastError();
        return DBC_ERR_CUDA;
    }
    return DBC_OK;
}

dbc_status launch_wide(const int8_t *a, int64_t lda, const int8_t *b, int64_t ldb, const Args &p, cudaStream_t st) {
    using C = Wide;
    CUtensorMap ta, tb, to;
    memset(&to, 0, sizeof to);
    if (!tma::encode_i8_rows(&ta, a, p.M, p.K, lda, 128) || !tma::encode_i8_rows(&tb, b, p.N, p.K, ldb, 128))
        return DBC_ERR_CUDA;
    const int64_t esz = p.out_bf16 ? 2 : 4;
    // (a tile store writes whole 16-byte pieces: with a width that ends inside one it would write behind the row)
    const bool tma_out = aligned16(p.out) && p.ldo * esz % 16 == 0 && p.N * esz % 16 == 0 &&
                         tma::encode_out_rows(&to, p.out, p.out_bf16, p.M, p.N, p.ldo, 32);
    using K = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, Args);
    static const K kernels[8] = {wide_kernel<false, false, false>, wide_kernel<false, false, true>,
                                 wide_kernel<false, true, false>,  wide_kernel<false, true, true>,
                                 wide_kernel<true, false, false>,  wide_kernel<true, false, true>,
                                 wide_kernel<true, true, false>,   wide_kernel<true, true, true>};
    const K k = kernels[(tma_out ? 4 : 0) + (p.out_bf16 ? 2 : 0) + (p.bias ? 1 : 0)];
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM) != cudaSuccess) {
        cudaGetLastError();                              // not the next call's
        return DBC_ERR_CUDA;
    }
    const int64_t tiles = (int64_t)((p.M + C::BM - 1) / C::BM) * ((p.N + C::BN - 1) / C::BN);
    if (tiles > (1 << 30)) return DBC_ERR_UNSUPPORTED;   // outputs of 10^14 bytes
    k<<<(unsigned)(2 * std::min<int64_t>(tiles, num_sms() / 2)), C::THREADS, C::SMEM, st>>>(ta, tb, to, p);
    return DBC_OK;
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
    mi::Args p{a_scale, b_scale, bias, out, ldo, (int)M, (int)N, (int)K, bias_dtype == DBC_BF16,
               out_dtype == DBC_BF16, dev_status};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // From 24 of the 74 pairs' tiles on.  Where the split kernel needs a second wave (more than 148 of its
    // tiles of 128 x 128) the wide one is ahead but for the shortest depths: 2048 x 2048 (64 wide tiles) takes
    // 10.5, 12.2 and 19.5 us at depths 256, 1024 and 4096, split 10.2, 13.8 and 27.1; 3000 x 1024 (48) 10.4,
    // 12.0 and 19.1, split 10.1, 13.4 and 26.8.  Below 24 it is behind: 1280 x 1024 (20) 10.3, 11.9 and 18.6,
    // split 5.7, 7.4 and 14.4.  Between 24 and 37 tiles the split kernel, since its epilogue is short, would
    // still be ahead (2048 x 1024, 32 tiles: 5.7, 7.6 and 14.6 against 10.3, 12.0 and 18.9; 4096 x 512 x 512:
    // 6.2 against 10.7).
    const int64_t wide_tiles = ((M + 255) / 256) * ((N + 255) / 256);
    if (K > 0 && M > 128 && wide_tiles >= 24) {
        const dbc_status c = mi::launch_wide(a, lda, b, ldb, p, st);
        if (c != DBC_OK) return c;
        count_launches(1);
        return launch_status();
    }
    // The split kernel's token tiles are the grid's second dimension (65535); only a depth of zero leaves
    // it more of them than 24.
    const int64_t most = 65535 * 128, nt = (N + 127) / 128;
    // Tokens of a tile: as few as leave at most 74 tiles, so that short epilogues run side by side (us with at
    // most 37, 74 and 148 tiles: 300 x 1536 x 512 7.8, 6.4 and 6.5; 200 x 1024 x 2048 8.3, 7.4 and 7.9) and
    // long weights are not read by many tiles (64 x 8192 x 8192 12.4, 12.4 and 15.5; 64 x 4096 x 4096 9.5, 8.9
    // and 10.0).  Where the weight is short and the depth long, 37 is a little ahead (61 x 1543 x 1531 5.9
    // against 6.2, 128 x 1024 x 1024 5.9 against 6.5).
    int tile = 16;
    while (tile < 128 && tile < M && ((M + tile - 1) / tile) * nt > 74) tile *= 2;
    for (int64_t m0 = 0; m0 < M; m0 += most) {
        p.M = (int)std::min<int64_t>(M - m0, most);
        p.as = a_scale + m0;
        p.out = static_cast<char *>(out) + m0 * ldo * (int64_t)oa;
        const dbc_status c = tile <= 16   ? mi::launch_split<16>(a, lda, b, ldb, p, st)
                             : tile <= 32 ? mi::launch_split<32>(a, lda, b, ldb, p, st)
                             : tile <= 64 ? mi::launch_split<64>(a, lda, b, ldb, p, st)
                                          : mi::launch_split<128>(a, lda, b, ldb, p, st);
        if (c != DBC_OK) return c;
        count_launches(1);
    }
    return launch_status();
}

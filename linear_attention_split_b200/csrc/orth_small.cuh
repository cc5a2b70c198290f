// orth_small.cuh -- Newton-Schulz steps of small matrices, one block per matrix, and the TTT-Linear
// step whose inner update is orthogonalised (its gradient, its update, the general output pass).
//
// A matrix of at most 64 rows stays in shared memory through all steps, so nothing but the input and
// the result touches HBM and a step costs three products of 64 x 64 x 64 (more along a long side)
// with a block barrier after each: the chain of launches of orth.cuh costs 4 to 5 us a product.  The
// operands are hi + lo fp16 as there; at this size the warp-level mma is the faster one (a tcgen05
// product of one 64 x 64 tile spends most of its time on the way into and out of tensor memory).
// The cross terms hi lo + lo hi have an accumulator of their own: the tensor cores drop the bits
// below the accumulator's last at every addition, and shorter chains keep that below fp32 rounding.
#pragma once
#include "common.cuh"
#include "orth.cuh"

namespace orth {

constexpr int SM_M = 64;                 // rows of a small matrix
constexpr int SM_N = 256;                // its longer side at most
constexpr int SM_TPB = 256;              // 8 warps: 2 x 4 tiles of 32 x 16
constexpr int SM_LD = SM_M + 8;          // padded row of A and P, in halves (16-byte rows, no bank conflicts)
__host__ __device__ constexpr int sm_ldx(int N) { return (N + 63) / 64 * 64 + 8; }
constexpr int SM_SQ = SM_M * SM_LD * 2;  // halves of A (hi and lo)
constexpr int small_smem_bytes(int N) { return (2 * SM_SQ + SM_M * sm_ldx(N) * 2) * 2; }

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A 32 x 16 tile of a product: rows row0.. of a ([64][lda], lo parts a_lo halves behind) times columns
// col0.. of b, which is [n][k] (b symmetric or itself transposed) or, TRANS, [k][n].
template <bool TRANS>
__device__ __forceinline__ void tile_product(float (&acc)[2][2][4], const __half* a, int lda, int a_lo, int row0, const __half* b,
                                             int ldb, int b_lo, int col0, int k16) {
    const int lane = threadIdx.x & 31;
    float low[2][2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = low[i][j][e] = 0.f;
    const uint32_t pa = smem_u32(a + (row0 + (lane & 15)) * lda + (lane >> 4) * 8);
    const uint32_t pb = TRANS ? smem_u32(b + (((lane >> 3) & 1) * 8 + (lane & 7)) * ldb + col0 + (lane >> 4) * 8)
                              : smem_u32(b + (col0 + (lane >> 4) * 8 + (lane & 7)) * ldb + ((lane >> 3) & 1) * 8);
    const uint32_t sb = TRANS ? 32u * ldb : 32u;  // bytes of 16 k
#pragma unroll 4
    for (int k = 0; k < k16; ++k) {
        uint32_t ah[2][4], al[2][4], bh[4], bl[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t at = pa + 32u * i * lda + 32u * k;
            ldsm_x4(at, ah[i][0], ah[i][1], ah[i][2], ah[i][3]);
            ldsm_x4(at + 2u * a_lo, al[i][0], al[i][1], al[i][2], al[i][3]);
        }
        if (TRANS) {
            ldsm_x4_t(pb + sb * k, bh[0], bh[1], bh[2], bh[3]);
            ldsm_x4_t(pb + sb * k + 2u * b_lo, bl[0], bl[1], bl[2], bl[3]);
        } else {
            ldsm_x4(pb + sb * k, bh[0], bh[1], bh[2], bh[3]);
            ldsm_x4(pb + sb * k + 2u * b_lo, bl[0], bl[1], bl[2], bl[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mma_f16(acc[i][j], ah[i], bh[2 * j], bh[2 * j + 1]);
                mma_f16(low[i][j], ah[i], bl[2 * j], bl[2 * j + 1]);
                mma_f16(low[i][j], al[i], bh[2 * j], bh[2 * j + 1]);
            }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] += low[i][j][e];
}

__device__ __forceinline__ void put2(__half* hi, int lo, float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    *reinterpret_cast<__half2*>(hi) = h;
    *reinterpret_cast<__half2*>(hi + lo) = __floats2half2_rn(x - f.x, y - f.y);
}

// All steps on X ([64][ldx] hi, then lo; zero outside the matrix) with A and P as scratch; the last
// product goes to last(row, col, v, w): the values at (row, col) and (row, col + 1), times SX SP.
// Enter with X written and not yet synchronised.
template <typename Last>
__device__ __forceinline__ void small_steps(__half* X, int ldx, __half* A, __half* P, int N, int steps, float ca, float cb,
                                            float cc, Last last) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = (warp & 1) * 32, col0 = (warp >> 1) * 16, gr = lane >> 2, gc = (lane & 3) * 2;
    const int x_lo = SM_M * ldx, s_lo = SM_M * SM_LD, k16 = (N + 15) / 16, strips = (N + 63) / 64;
    for (int step = 0; step < steps; ++step) {
        float acc[2][2][4], a[2][2][4];
        __syncthreads();  // X is written
        tile_product<false>(acc, X, ldx, x_lo, row0, X, ldx, x_lo, col0, k16);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float v = acc[i][j][2 * h] * (1.f / SX), w = acc[i][j][2 * h + 1] * (1.f / SX);
                    a[i][j][2 * h] = v;
                    a[i][j][2 * h + 1] = w;
                    put2(A + (row0 + 16 * i + 8 * h + gr) * SM_LD + col0 + 8 * j + gc, s_lo, v, w);
                }
        __syncthreads();  // A is written
        tile_product<false>(acc, A, SM_LD, s_lo, row0, A, SM_LD, s_lo, col0, SM_M / 16);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = row0 + 16 * i + 8 * h + gr, c = col0 + 8 * j + gc;
                    float v[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        v[e] = SP * (fmaf(cc / (SX * SX), acc[i][j][2 * h + e], cb / SX * a[i][j][2 * h + e]) +
                                     (r == c + e ? ca : 0.f));
                    put2(P + r * SM_LD + c, s_lo, v[0], v[1]);
                }
        __syncthreads();  // P is written
        const bool done = step + 1 == steps;
        for (int s = 0; s < strips; ++s) {
            tile_product<true>(acc, P, SM_LD, s_lo, row0, X, ldx, x_lo, 64 * s + col0, SM_M / 16);
            if (!done) __syncthreads();  // every warp has read this strip of X
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = row0 + 16 * i + 8 * h + gr, c = 64 * s + col0 + 8 * j + gc;
                        if (done)
                            last(r, c, acc[i][j][2 * h], acc[i][j][2 * h + 1]);
                        else
                            put2(X + r * ldx + c, x_lo, acc[i][j][2 * h] * (1.f / SP), acc[i][j][2 * h + 1] * (1.f / SP));
                    }
        }
    }
}

// sum over the block, in warp order
__device__ __forceinline__ double block_sum(double s, double* sm) {
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < SM_TPB / 32; ++w) s += sm[w];
    return s;
}

// one block per matrix: X [M][N] of the shorter side M <= 64, N <= 256
template <typename T>
__global__ void __launch_bounds__(SM_TPB, 2)
    small_kernel(const T* x, T* out, int M, int N, int tall, int steps, float ca, float cb, float cc, float eps, float scale) {
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ double sums[SM_TPB / 32];
    __half *A = reinterpret_cast<__half*>(raw), *P = A + SM_SQ, *X = P + SM_SQ;
    const int ldx = sm_ldx(N), wide = ldx - 8, mn = M * N;
    griddep_wait();
    griddep_launch();
    x += (long long)blockIdx.x * mn;
    out += (long long)blockIdx.x * mn;
    double s = 0.0;
    for (int i = threadIdx.x; i < mn; i += SM_TPB) {
        const double v = (double)to_f(x[i]);
        s = fma(v, v, s);
    }
    const double inv = inverse_norm(block_sum(s, sums), eps) * SX;
    // zero around the matrix, then the matrix (a tall one transposed)
    if (M < SM_M || N < wide)
        for (int i = threadIdx.x; i < SM_M * wide; i += SM_TPB) {
            const int r = i / wide, c = i % wide;
            if (r >= M || c >= N) X[r * ldx + c] = X[SM_M * ldx + r * ldx + c] = __float2half_rn(0.f);
        }
    for (int i = threadIdx.x; i < mn; i += SM_TPB) {
        const int r = tall ? i % M : i / N, c = tall ? i / M : i % N;
        split((float)((double)to_f(x[i]) * inv), X[r * ldx + c], X[SM_M * ldx + r * ldx + c]);
    }
    const float f = scale / (SX * SP);
    small_steps(X, ldx, A, P, N, steps, ca, cb, cc, [&](int r, int c, float v, float w) {
        if (r >= M || c >= N) return;
        T* o = out + (tall ? c * M + r : r * N + c);
        o[0] = from_f<T>(v * f);
        if (c + 1 < N) o[tall ? M : 1] = from_f<T>(w * f);
    });
}

// ------------------------------------------------------------------ TTT-Linear, orthogonalised step
constexpr int D = 64, DD = D * D, ROWB = 128, TILE = TM * ROWB;

// G and C^T of one split of a unit's tokens, bf16, d = 64: [V | K]^T K on the tcgen05 tensor cores.
// Grid (S, U); part [U][S][2][64][64] (G, C^T).
constexpr int G_STAGES = 3, G_THREADS = 64 + 128;  // producer, issuer, four epilogue warps
constexpr uint32_t IDESC_GRAM = tc::idesc_bf16(128, 64, 1, 1);
struct GBars {
    uint64_t full[G_STAGES], empty[G_STAGES], done;
    uint32_t tmem_base;
};
constexpr int g_smem_bytes() { return G_STAGES * 2 * TILE + (int)sizeof(GBars) + 1024; }

__global__ void __launch_bounds__(G_THREADS)
    gram_tc_kernel(const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k, float* __restrict__ part,
                   int TT, int n_tiles) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_align<1024>(smem_raw);
    GBars* bars = reinterpret_cast<GBars*>(ring + G_STAGES * 2 * TILE);
    const int S = gridDim.x, r = blockIdx.x, u = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_t = r < n_tiles ? (n_tiles - r + S - 1) / S : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < G_STAGES; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        mbar_init(&bars->done, 1);
        mbar_fence_init();
        // the first tiles into L2 while the previous grid may still run; loads come after its end
        for (int i = 0; i < min(G_STAGES, n_t); ++i) {
            tma_prefetch_l2_3d(&tm_v, 0, (r + i * S) * TT, u);
            tma_prefetch_l2_3d(&tm_k, 0, (r + i * S) * TT, u);
        }
    }
    if (warp == 1) tc::alloc(&bars->tmem_base, 64);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    griddep_wait();
    griddep_launch();
    const uint32_t tmem = bars->tmem_base;
    if (warp == 0) {
        if (lane == 0)
            for (int i = 0; i < n_t; ++i) {
                const int slot = i % G_STAGES, use = i / G_STAGES;
                if (use > 0) mbar_wait(&bars->empty[slot], (use - 1) & 1, TTT_DEVERR_TIMEOUT_TMA);
                uint8_t* dst = ring + slot * 2 * TILE;
                mbar_expect_tx(&bars->full[slot], 2 * TT * ROWB);
                tma_load_3d(dst, &tm_v, 0, (r + i * S) * TT, u, &bars->full[slot]);
                tma_load_3d(dst + TILE, &tm_k, 0, (r + i * S) * TT, u, &bars->full[slot]);
            }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int i = 0; i < n_t; ++i) {
                const int slot = i % G_STAGES;
                mbar_wait(&bars->full[slot], (i / G_STAGES) & 1, TTT_DEVERR_TIMEOUT_TMA);
                tc::fence_after();
                const uint32_t vb = smem_u32(ring + slot * 2 * TILE);
                const uint64_t a = tc::smem_desc(vb, TILE, 1024, 2), b = tc::smem_desc(vb + TILE, TILE, 1024, 2);
                for (int ks = 0; ks < TT / 16; ++ks)
                    tc::mma_bf16(tmem, a + (uint64_t)(ks * 128), b + (uint64_t)(ks * 128), IDESC_GRAM, i > 0 || ks > 0);
                tc::commit(&bars->empty[slot]);
            }
            tc::commit(&bars->done);
        }
    } else {
        const int q4 = warp & 3, row = q4 * 32 + lane;  // rows 0-63: C^T, rows 64-127: G
        const uint32_t lane_base = tmem + ((uint32_t)(q4 * 32) << 16);
        float* dst = part + ((size_t)u * S + r) * 2 * DD + (row >= D ? (row - D) * D : DD + row * D);
        if (n_t > 0) {
            mbar_wait(&bars->done, 0, TTT_DEVERR_TIMEOUT_TMA);
            tc::fence_after();
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float x[16];
            if (n_t > 0) {
                tc::ld16(lane_base + c * 16, x);
                tc::wait_ld();
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<float4*>(dst + c * 16 + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) tc::dealloc(tmem, 64);
}

// The same for any d <= 128 and type on the CUDA cores: grid (S, U, blocks of 64 x 64 of the d x 2d
// sums [G | C]), 256 threads with 4 x 4 values each, 32 tokens at a time through shared memory.
// part [U][S][2][d][d] (G, C^T).
template <typename T>
__global__ void __launch_bounds__(256)
    gram_kernel(const T* __restrict__ k, const T* __restrict__ v, float* __restrict__ part, int N, int d) {
    __shared__ float ks[32][68], xs[32][68];
    const int S = gridDim.x, r = blockIdx.x;
    const long long u = blockIdx.y;
    const int nb = (d + 63) / 64, i0 = blockIdx.z / (2 * nb) * 64, jb = blockIdx.z % (2 * nb);
    const bool is_c = jb >= nb;
    const int j0 = (is_c ? jb - nb : jb) * 64;
    griddep_wait();
    griddep_launch();
    const int per = (N + S - 1) / S, t0 = r * per, t1 = min(N, t0 + per);
    const T* ku = k + u * N * d;
    const T* xu = (is_c ? v : k) + u * N * d;
    const int ti = threadIdx.x / 16 * 4, tj = threadIdx.x % 16 * 4;
    float acc[4][4] = {};
    for (int t = t0; t < t1; t += 32) {
        for (int e = threadIdx.x; e < 32 * 64; e += 256) {
            const int row = e / 64, c = e % 64;
            const bool in = t + row < t1;
            ks[row][c] = in && i0 + c < d ? to_f(ku[(long long)(t + row) * d + i0 + c]) : 0.f;
            xs[row][c] = in && j0 + c < d ? to_f(xu[(long long)(t + row) * d + j0 + c]) : 0.f;
        }
        __syncthreads();
#pragma unroll 8
        for (int row = 0; row < 32; ++row) {
            const float4 a = *reinterpret_cast<const float4*>(&ks[row][ti]), b = *reinterpret_cast<const float4*>(&xs[row][tj]);
            const float ax[4] = {a.x, a.y, a.z, a.w}, bx[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(ax[i], bx[j], acc[i][j]);
        }
        __syncthreads();
    }
    float* p = part + (u * S + r) * 2 * d * d + (is_c ? (long long)d * d : 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = i0 + ti + i, col = j0 + tj + j;
            if (row < d && col < d) p[is_c ? (long long)col * d + row : (long long)row * d + col] = acc[i][j];
        }
}

// One block per unit, d <= 64: the partials are added in split order, g = (1/N)(G W0 - C) is formed in
// fp32, orthogonalised (small_steps), and W* = W0 - eta U written.
constexpr int FLD = D + 4;
constexpr int update_smem_bytes() { return small_smem_bytes(D); }
__global__ void __launch_bounds__(SM_TPB, 2)
    update_kernel(const float* __restrict__ part, const float* __restrict__ w0, float* __restrict__ w_star, int S, int H, int d,
                  float inv_n, float eta, int steps, float ca, float cb, float cc, float eps) {
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ double sums[SM_TPB / 32];
    __half *A = reinterpret_cast<__half*>(raw), *P = A + SM_SQ, *X = P + SM_SQ;
    float *G = reinterpret_cast<float*>(A), *W = reinterpret_cast<float*>(P);  // [k][64 + 4], before the steps
    static_assert(SM_SQ * 2 >= D * FLD * 4, "G and W0 fit where A and P go");
    const long long u = blockIdx.x;
    const int dd = d * d, tid = threadIdx.x, ldx = sm_ldx(D);
    w0 += (u % H) * dd;
    for (int e = tid; e < DD; e += SM_TPB) {
        const int r = e / D, c = e % D;
        W[r * FLD + c] = r < d && c < d ? __ldg(w0 + r * d + c) : 0.f;
    }
    griddep_wait();  // the partials
    griddep_launch();
    part += u * S * 2 * dd;
    for (int e = tid; e < DD; e += SM_TPB) {  // G is symmetric: rows are its k
        const int r = e / D, c = e % D;
        float s = 0.f;
        if (r < d && c < d)
            for (int i = 0; i < S; ++i) s += part[(size_t)i * 2 * dd + r * d + c];
        G[r * FLD + c] = s;
    }
    const int tr = (tid >> 4) * 4, tc = (tid & 15) * 4;
    float acc[4][4];  // -C first: rows tr.., columns tc..
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float s = 0.f;
            if (tr + i < d && tc + j < d)
                for (int q = 0; q < S; ++q) s += part[((size_t)q * 2 + 1) * dd + (tc + j) * d + tr + i];
            acc[i][j] = -s;
        }
    __syncthreads();
    float gw[4][4] = {};
#pragma unroll 4
    for (int k = 0; k < D; ++k) {
        const float4 a = *reinterpret_cast<const float4*>(G + k * FLD + tr), b = *reinterpret_cast<const float4*>(W + k * FLD + tc);
        const float ax[4] = {a.x, a.y, a.z, a.w}, bx[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) gw[i][j] = fmaf(ax[i], bx[j], gw[i][j]);
    }
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[i][j] = (acc[i][j] + gw[i][j]) * inv_n;
            s = fma((double)acc[i][j], (double)acc[i][j], s);
        }
    const double inv = inverse_norm(block_sum(s, sums), eps) * SX;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; j += 2)
            put2(X + (tr + i) * ldx + tc + j, SM_M * ldx, (float)(acc[i][j] * inv), (float)(acc[i][j + 1] * inv));
    w_star += u * dd;
    small_steps(X, ldx, A, P, D, steps, ca, cb, cc, [&](int r, int c, float v, float w) {
        if (r >= d || c >= d) return;
        const float f = -eta / (SX * SP);
        w_star[r * d + c] = fmaf(f, v, __ldg(w0 + r * d + c));
        if (c + 1 < d) w_star[r * d + c + 1] = fmaf(f, w, __ldg(w0 + r * d + c + 1));
    });
}

// O = Q W on the CUDA cores for any d <= 128 and type: 64 tokens x 64 output features per block,
// 4 x 4 values a thread, 32 input features at a time through shared memory.  Grid (token tiles, U,
// feature tiles).
template <typename T>
__global__ void __launch_bounds__(256)
    apply_kernel(const T* __restrict__ q, const float* __restrict__ w, T* __restrict__ out, int N, int d) {
    __shared__ float qs[32][68], ws[32][68];
    const long long u = blockIdx.y;
    const int t0 = blockIdx.x * 64, j0 = blockIdx.z * 64;
    const int ti = threadIdx.x / 16 * 4, tj = threadIdx.x % 16 * 4;
    griddep_wait();
    griddep_launch();
    float acc[4][4] = {};
    for (int k0 = 0; k0 < d; k0 += 32) {
        for (int e = threadIdx.x; e < 32 * 64; e += 256) {
            const int t = e / 32, c = e % 32;
            qs[c][t] = t0 + t < N && k0 + c < d ? to_f(q[(u * N + t0 + t) * d + k0 + c]) : 0.f;
            const int r = e / 64, j = e % 64;
            ws[r][j] = k0 + r < d && j0 + j < d ? w[u * d * d + (long long)(k0 + r) * d + j0 + j] : 0.f;
        }
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
            const float4 a = *reinterpret_cast<const float4*>(&qs[k][ti]), b = *reinterpret_cast<const float4*>(&ws[k][tj]);
            const float ax[4] = {a.x, a.y, a.z, a.w}, bx[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(ax[i], bx[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (t0 + ti + i < N && j0 + tj + j < d) out[(u * N + t0 + ti + i) * d + j0 + tj + j] = from_f<T>(acc[i][j]);
}

// ---- d > 64: the steps of the general path between these two
// g[u] = (1/N)(G W0[h] - C), the partials added in split order
__global__ void __launch_bounds__(TPB)
    gradient_kernel(const float* __restrict__ part, const float* __restrict__ w0, float* __restrict__ g, int S, int H, int d,
                    float inv_n) {
    const long long u = blockIdx.x;
    const int dd = d * d, e = blockIdx.y * TPB + threadIdx.x;
    griddep_wait();
    griddep_launch();
    if (e >= dd) return;
    const int i = e / d, j = e % d;
    const float* W0 = w0 + (u % H) * dd;
    float gw = 0.f, c = 0.f;
    for (int m = 0; m < d; ++m) {
        float s = 0.f;
        for (int q = 0; q < S; ++q) s += part[(u * S + q) * 2 * dd + i * d + m];
        gw = fmaf(s, W0[m * d + j], gw);
    }
    for (int q = 0; q < S; ++q) c += part[((u * S + q) * 2 + 1) * dd + j * d + i];
    g[u * dd + e] = (gw - c) * inv_n;
}

// W* = W0[h] - eta U
__global__ void __launch_bounds__(TPB)
    step_kernel(const float* __restrict__ upd, const float* __restrict__ w0, float* __restrict__ w_star, int H, int dd, float eta) {
    const long long u = blockIdx.x;
    const int e = blockIdx.y * TPB + threadIdx.x;
    griddep_wait();
    griddep_launch();
    if (e < dd) w_star[u * dd + e] = w0[(u % H) * dd + e] - eta * upd[u * dd + e];
}

}  // namespace orth

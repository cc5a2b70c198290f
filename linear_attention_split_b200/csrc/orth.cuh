// orth.cuh -- the orthogonal factor of an update by Newton-Schulz products.
//
// X_0 = X / max(|X|_F, eps), then `steps` times
//     A = X X^T,   P = a I + b A + c A^2,   X <- P X,
// which sends every singular value s of X_0 to p(s) = a s + b s^3 + c s^5 and leaves its singular
// vectors.  Everything is done on the side that is shorter (X is taken transposed when it is
// tall), so A and P are M x M with M = min(m, n).  Sums of squares are formed in fp64, so that no
// finite X overflows its norm.
//
// The products run on the fp16 tensor cores with every operand held as hi + lo, two fp16 numbers
// (about 22 bits), and hi hi + hi lo + lo hi accumulated in fp32: bf16 operands would leave 3e-2
// of the result's norm wrong, fp16 alone 3e-3 (the iteration enlarges what is lost early by up to
// a^5, and at s = 1 the polynomial cancels 3.4 - 4.8 + 2.0), three products 1e-6.  Values are
// bounded (|s| <= 2 throughout, checked on the host), so fixed powers of two keep them inside
// fp16: X and A are stored times 2^12, P times 2^10.
//
// product_kernel: one 128 x 128 tile of a product per cluster; the K range is split over the S
// CTAs of the cluster when there are few tiles, and the partial tiles are exchanged through
// distributed shared memory (each CTA adds one slice of columns, in rank order: deterministic).
// Per CTA a TMA producer and a tcgen05 issuer over a ring of 64-wide K blocks, and four epilogue
// warps.  A and P are symmetric: only tiles on or above the diagonal are formed, and written twice.
#pragma once
#include "common.cuh"
#include <cuda_fp16.h>

namespace orth {

constexpr int TPB = 256;
constexpr int MAX_PARTS = 64;
constexpr float SX = 4096.f, SP = 1024.f;  // scale of stored X and A, and of stored P

// part[u][p] = sum of squares of piece p of matrix u
template <typename T>
__global__ void __launch_bounds__(TPB) square_kernel(const T* __restrict__ x, double* __restrict__ part, long long mn) {
    __shared__ double sm[TPB / 32];
    griddep_wait();
    griddep_launch();
    const T* xu = x + blockIdx.y * mn;
    double s = 0.0;
    for (long long i = (long long)blockIdx.x * TPB + threadIdx.x; i < mn; i += (long long)gridDim.x * TPB) {
        const double v = (double)to_f(xu[i]);
        s = fma(v, v, s);
    }
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < TPB / 32; ++w) s += sm[w];
        part[(long long)blockIdx.y * gridDim.x + blockIdx.x] = s;
    }
}

__device__ __forceinline__ void split(float v, __half& hi, __half& lo) {
    hi = __float2half_rn(v);
    lo = __float2half_rn(v - __half2float(hi));
}
// 1 / max(norm, eps); a norm that is not finite gives NaN, which then fills the matrix
__device__ __forceinline__ double inverse_norm(double squares, float eps) {
    const double n = sqrt(squares);
    return isfinite(n) ? 1.0 / fmax(n, (double)eps) : (double)NAN;
}

// X [u][hi, lo][M][ld] from x (transposed on the way when tall), zero in columns N .. ld - 1.
// 32 x 32 tiles through shared memory, so that both sides are read and written along rows.
template <typename T>
__global__ void __launch_bounds__(256)
    start_kernel(const T* __restrict__ x, const double* __restrict__ part, __half* __restrict__ y, int parts, int M,
                 int N, int ld, int tall, float eps) {
    __shared__ float sm[32][33];
    griddep_wait();
    griddep_launch();
    const int u = blockIdx.z, i0 = blockIdx.y * 32, j0 = blockIdx.x * 32;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    double s = 0.0;
    for (int p = 0; p < parts; ++p) s += part[(long long)u * parts + p];
    const double inv = inverse_norm(s, eps);
    const T* xu = x + (long long)u * M * N;
    for (int r = ty; r < 32; r += 8) {
        const int i = tall ? i0 + tx : i0 + r, j = tall ? j0 + r : j0 + tx;
        float v = 0.f;
        if (i < M && j < N) v = (float)((double)to_f(xu[tall ? (long long)j * M + i : (long long)i * N + j]) * inv * SX);
        if (tall)
            sm[tx][r] = v;
        else
            sm[r][tx] = v;
    }
    __syncthreads();
    for (int r = ty; r < 32; r += 8) {
        const int i = i0 + r, j = j0 + tx;
        if (i >= M || j >= ld) continue;
        __half* yu = y + (long long)u * 2 * M * ld + (long long)i * ld + j;
        split(sm[r][tx], yu[0], yu[(long long)M * ld]);
    }
}

constexpr int TM = 128, KB = 64;                     // tile of the output, K block
constexpr int OPB = TM * KB * 2;                     // one operand's K block, 16 KB
constexpr int STAGES = 3;
constexpr int MAX_SPLIT = 8;
constexpr int THREADS = 64 + 128;                    // producer, issuer, four epilogue warps
constexpr uint32_t IDESC_K = tc::idesc_f16(128, 128, 0, 0);   // both operands K-major
constexpr uint32_t IDESC_MN = tc::idesc_f16(128, 128, 0, 1);  // the second MN-major

enum Kind { GRAM = 0, POLY = 1, NEXT = 2, OUT_F32 = 3, OUT_BF16 = 4 };

struct PParams {
    int kblocks;             // K blocks of the whole product
    int M, tiles_n;          // rows of X, A and P; tiles along the columns (not used by GRAM, POLY)
    int kind;
    int ld;                  // row stride of the halves that are written (GRAM, POLY, NEXT), columns written
    __half* y;               // where they go, [u][hi, lo][M][ld]
    const __half* a;         // POLY: A, same shape
    void* out;               // OUT: [u][M][N], or [u][N][M] when tall
    int N, tall;
    float ca, cb, cc, scale;
};
struct PBars {
    uint64_t full[STAGES], empty[STAGES], done;
    uint32_t tmem_base;
};
constexpr int p_smem_bytes() { return STAGES * 4 * OPB + (int)sizeof(PBars) + 1024; }

__device__ __forceinline__ void put8(__half* hi, __half* lo, const float* v) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 x = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        const float2 f = __half22float2(x);
        const __half2 r = __floats2half2_rn(v[2 * i] - f.x, v[2 * i + 1] - f.y);
        h[i] = *reinterpret_cast<const uint32_t*>(&x);
        l[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
    *reinterpret_cast<uint4*>(hi) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(lo) = make_uint4(l[0], l[1], l[2], l[3]);
}

// What becomes of 16 adjacent values v of the product at (row, col), the tile being (bi, bj)
__device__ __forceinline__ void finish16(const PParams& p, int u, int row, int col, bool mirror, float (&v)[16]) {
    if (row >= p.M) return;
    const long long mat = (long long)p.M * p.ld;
    if (p.kind == OUT_F32 || p.kind == OUT_BF16) {
        const float f = p.scale / (SX * SP);
        const long long mn = (long long)p.M * p.N;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (col + e < p.N) {
                const long long at = u * mn + (p.tall ? (long long)(col + e) * p.M + row : (long long)row * p.N + col + e);
                if (p.kind == OUT_F32)
                    static_cast<float*>(p.out)[at] = v[e] * f;
                else
                    static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v[e] * f);
            }
        return;
    }
    __half* hi = p.y + u * 2 * mat + (long long)row * p.ld + col;
    __half* lo = hi + mat;
    if (p.kind == GRAM) {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] *= 1.f / SX;
    } else if (p.kind == NEXT) {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] *= 1.f / SP;
    } else {
        const __half* ah = p.a + u * 2 * mat + (long long)row * p.ld + col;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (col + 8 * h < p.ld) {
                const uint4 x = *reinterpret_cast<const uint4*>(ah + 8 * h), y = *reinterpret_cast<const uint4*>(ah + mat + 8 * h);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&xs[i]));
                    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&ys[i]));
                    const int e = 8 * h + 2 * i;
                    v[e] = fmaf(p.cc / (SX * SX), v[e], p.cb / SX * (f.x + g.x));
                    v[e + 1] = fmaf(p.cc / (SX * SX), v[e + 1], p.cb / SX * (f.y + g.y));
                }
            }
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = SP * (v[e] + (row == col + e ? p.ca : 0.f));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (col + 8 * h < p.ld) put8(hi + 8 * h, lo + 8 * h, v + 8 * h);
    if (mirror)
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (col + e < p.M) {
                __half* m = p.y + u * 2 * mat + (long long)(col + e) * p.ld + row;
                split(v[e], m[0], m[mat]);
            }
}

// first, second: the operands' tensor maps over [2 u + part][rows][ld]; the second is the first's
// own kind (K-major, box 64 x 128) for GRAM and POLY, MN-major (box 64 x 64, X itself) otherwise
__global__ void __launch_bounds__(THREADS, 1)
    product_kernel(const __grid_constant__ CUtensorMap first, const __grid_constant__ CUtensorMap second, const PParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_align<1024>(smem_raw);
    PBars* bars = reinterpret_cast<PBars*>(ring + STAGES * 4 * OPB);
    const int S = gridDim.x, r = blockIdx.x, u = blockIdx.z;  // cluster (S, 1, 1)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool sym = p.kind <= POLY;
    int bi, bj;
    if (sym) {  // tile of the upper triangle, column by column
        bj = 0;
        int t = blockIdx.y;
        while (t > bj) t -= ++bj;
        bi = t;
    } else {
        bi = blockIdx.y / p.tiles_n;
        bj = blockIdx.y % p.tiles_n;
    }
    const int per = (p.kblocks + S - 1) / S, k0 = min(r * per, p.kblocks), nk = min(per, p.kblocks - k0);
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        mbar_init(&bars->done, 1);
        mbar_fence_init();
    }
    if (warp == 1) tc::alloc(&bars->tmem_base, 128);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    griddep_wait();
    griddep_launch();
    const uint32_t tmem = bars->tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < nk; ++i) {
                const int slot = i % STAGES, use = i / STAGES;
                if (use > 0) mbar_wait(&bars->empty[slot], (use - 1) & 1, TTT_DEVERR_TIMEOUT_TMA);
                uint8_t* dst = ring + slot * 4 * OPB;
                uint64_t* bar = &bars->full[slot];
                const int k = (k0 + i) * KB;
                mbar_expect_tx(bar, 4 * OPB);
                for (int part = 0; part < 2; ++part) {
                    tma_load_3d(dst + part * OPB, &first, k, bi * TM, 2 * u + part, bar);
                    if (sym) {
                        tma_load_3d(dst + (2 + part) * OPB, &second, k, bj * TM, 2 * u + part, bar);
                    } else {
                        tma_load_3d(dst + (2 + part) * OPB, &second, bj * TM, k, 2 * u + part, bar);
                        tma_load_3d(dst + (2 + part) * OPB + OPB / 2, &second, bj * TM + 64, k, 2 * u + part, bar);
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int i = 0; i < nk; ++i) {
                const int slot = i % STAGES;
                mbar_wait(&bars->full[slot], (i / STAGES) & 1, TTT_DEVERR_TIMEOUT_TMA);
                tc::fence_after();
                const uint32_t base = smem_u32(ring + slot * 4 * OPB);
                const uint64_t ah = tc::smem_desc(base, 16, 1024, 2), al = tc::smem_desc(base + OPB, 16, 1024, 2);
                const uint32_t lbo = sym ? 16 : OPB / 2;
                const uint64_t bh = tc::smem_desc(base + 2 * OPB, lbo, 1024, 2);
                const uint64_t bl = tc::smem_desc(base + 3 * OPB, lbo, 1024, 2);
                const uint64_t bstep = sym ? 2 : 128;
                const uint32_t idesc = sym ? IDESC_K : IDESC_MN;
#pragma unroll
                for (int ks = 0; ks < KB / 16; ++ks) {
                    tc::mma_bf16(tmem, ah + 2 * ks, bl + bstep * ks, idesc, i > 0 || ks > 0);
                    tc::mma_bf16(tmem, al + 2 * ks, bh + bstep * ks, idesc, 1);
                    tc::mma_bf16(tmem, ah + 2 * ks, bh + bstep * ks, idesc, 1);
                }
                tc::commit(&bars->empty[slot]);
            }
            tc::commit(&bars->done);
        }
    }
    const int q4 = warp & 3, row = q4 * 32 + lane;  // the row of the tile that an epilogue thread holds
    const uint32_t lane_base = tmem + ((uint32_t)(q4 * 32) << 16);
    const bool mirror = sym && bi != bj;
    if (warp >= 2) {
        if (nk > 0) {
            mbar_wait(&bars->done, 0, TTT_DEVERR_TIMEOUT_TMA);
            tc::fence_after();
        }
        if (S == 1) {
            for (int c = 0; c < TM; c += 16) {
                float v[16];
                tc::ld16(lane_base + c, v);
                tc::wait_ld();
                finish16(p, u, bi * TM + row, bj * TM + c, mirror, v);
            }
        }
    }
    if (S > 1) {
        const int w = TM / S, pitch = w + 4;  // columns of a slice; padded row of the exchange buffer
        float* buf = reinterpret_cast<float*>(ring);  // [S][128][pitch], over the ring
        cluster_sync_all();  // every CTA's MMAs have read their operands: the rings are free
        if (warp >= 2) {
            for (int c = 0; c < TM; c += 16) {
                float v[16];
                if (nk > 0) {
                    tc::ld16(lane_base + c, v);
                    tc::wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = 0.f;
                }
                const uint32_t at = dsmem_map(buf + ((size_t)r * TM + row) * pitch + c % w, c / w);
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + 4 * e), "f"(v[e]),
                                 "f"(v[e + 1]), "f"(v[e + 2]), "f"(v[e + 3])
                                 : "memory");
            }
        }
        cluster_sync_all();
        if (warp >= 2) {
            for (int c = 0; c < w; c += 16) {
                float v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = 0.f;
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 x = *reinterpret_cast<const float4*>(buf + ((size_t)s * TM + row) * pitch + c + e);
                        v[e] += x.x, v[e + 1] += x.y, v[e + 2] += x.z, v[e + 3] += x.w;
                    }
                finish16(p, u, bi * TM + row, bj * TM + r * w + c, mirror, v);
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) tc::dealloc(tmem, 128);
}

}  // namespace orth

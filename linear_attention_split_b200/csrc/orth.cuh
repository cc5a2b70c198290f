// orth.cuh -- the orthogonal factor of an update by Newton-Schulz products.
//
// X_0 = X / max(|X|_F, eps), then `steps` times
//     A = X X^T,   Q = b I + c A,   P = a I + A Q  (= a I + b A + c A^2),   X <- P X,
// which sends every singular value s of X_0 to p(s) = a s + b s^3 + c s^5 and leaves its singular
// vectors.  Everything is done on the side that is shorter (X is taken transposed when it is
// tall), so A, Q and P are M x M with M = min(m, n).  Sums of squares are formed in fp64, so that no
// finite X overflows its norm.
//
// The products run on the fp16 tensor cores.  An operand is held as hi + lo, two fp16 numbers (about
// 22 bits), and a product is hi hi + hi lo + lo hi accumulated in fp32.  fp32 matrices take all three
// (result good to about 1e-6 of its norm).  For bf16 ones X is held as hi alone and only A Q, the
// cheap product, and P hi + lo are taken in full: the iteration enlarges what is lost early by up to
// a^5, and at s = 1 the polynomial cancels 3.4 - 4.8 + 2.0; in simulation bf16 operands leave 3e-2 of
// the norm wrong, hi hi throughout 2e-3 to 3e-3, this choice 4e-4 to 8e-4, below the 1.7e-3 that
// rounding the result to bf16 costs.  Values are bounded (|s| <= 2 throughout, checked on the host), so
// fixed powers of two keep them inside fp16: X and A are stored times 2^12, P times 2^10, Q times 2^9.
//
// product_kernel: one 128 x 128 tile of a product per cluster; the K range is split over the S
// CTAs of the cluster when there are few tiles, and the partial tiles are exchanged through
// distributed shared memory (each CTA adds one slice of rows, in rank order: deterministic).  Per CTA
// a TMA producer and a tcgen05 issuer over a ring of 64-wide K blocks, and four epilogue warps, which
// stage what they write so that rows go out whole (straight from the accumulator's layout, one row per
// lane, a tile took 5300 cycles; staged about a third).  A, Q and P are symmetric: only tiles on or
// above the diagonal are formed, and an operand block below it is read from its mirror image as an
// MN-major operand.  The tensor cores cut what falls below the accumulator's last bit at every
// addition, about 1e-7 of the result for each: a full product therefore spreads its K blocks over
// three accumulators and keeps the cross terms in a fourth, added in fp32 in the epilogue (1024 x 4096,
// one accumulator: 2.4e-5 of the norm).
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

// X [u][hi, lo][M][ld] (hi alone with halves = 1) from x (transposed on the way when tall), zero in columns N .. ld - 1.
// 32 x 32 tiles through shared memory, so that both sides are read and written along rows.
template <typename T>
__global__ void __launch_bounds__(256)
    start_kernel(const T* __restrict__ x, const double* __restrict__ part, __half* __restrict__ y, int parts, int M,
                 int N, int ld, int tall, int halves, float eps) {
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
        __half lo;
        split(sm[r][tx], yu[0], lo);
        if (halves == 2) yu[(long long)M * ld] = lo;
    }
}

constexpr int TM = 128, KB = 64;                     // tile of the output, K block
constexpr int OPB = TM * KB * 2;                     // one operand's K block, 16 KB
constexpr int MAX_SPLIT = 8;
constexpr int THREADS = 64 + 128;                    // producer, issuer, four epilogue warps
constexpr float SQ = 512.f;                          // scale of stored Q

enum Kind { GRAM = 0, POLY = 1, NEXT = 2, OUT_F32 = 3, OUT_BF16 = 4 };

struct PParams {
    int kblocks;             // K blocks of the whole product
    int M, tiles_n;          // rows of X, A, Q and P; tiles along the columns (NEXT, OUT)
    int kind;
    int ld;                  // row stride of the halves that are written (GRAM, POLY, NEXT), columns written
    int parts;               // 2: hi and lo are written, 1: hi alone
    __half* y;               // where they go, [u][hi, lo][M][ld]
    __half* y2;              // GRAM: Q, same shape
    void* out;               // OUT: [u][M][N], or [u][N][M] when tall
    int N, tall;
    float ca, cb, cc, scale;
};
constexpr int MAX_STAGES = 4;
struct PBars {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES], done;
    uint32_t tmem_base;
};
constexpr int STG = 72;  // padded row of the staged halves (64 columns); floats: 68
constexpr int EXCHANGE = TM * TM * 4;               // the S partial slices of a tile
constexpr int STAGED = TM / 2 * STG * 2 * 4;        // up to four arrays of half a tile's rows
// What a product takes: FL, SL: the first / second operand's lo part as well; ACC accumulators for hi hi
// (and one for the cross terms, if any); STAGES K blocks in flight; MINB CTAs on an SM.
template <bool FL_, bool SL_, int ACC_, int STAGES_, int MINB_>
struct Config {
    static constexpr bool FL = FL_, SL = SL_;
    static constexpr int ACC = ACC_, STAGES = STAGES_, MINB = MINB_;
    static constexpr int STAGE = (2 + FL + SL) * OPB;
    static constexpr int ACCS = ACC + (FL || SL);
    static constexpr int COLS = ACCS == 1 ? 128 : ACCS == 2 ? 256 : 512;  // of tensor memory
    // the ring; over it the exchange and what is staged
    static constexpr int RING = STAGES * STAGE > EXCHANGE + STAGED ? STAGES * STAGE : EXCHANGE + STAGED;
    static constexpr int SMEM = RING + (int)sizeof(PBars) + 1024;
    static_assert(MINB * COLS <= 512 && STAGES <= MAX_STAGES, "");
};
using Full = Config<true, true, 3, 3, 1>;      // hi hi + hi lo + lo hi, 192 KB ring
using High = Config<false, false, 1, 3, 2>;    // hi hi, 96 KB
using Left = Config<true, false, 1, 2, 2>;     // hi hi + lo hi, 96 KB
__device__ __forceinline__ void split8(const float* v, uint4& hi, uint4& lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 x = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        const float2 f = __half22float2(x);
        const __half2 r = __floats2half2_rn(v[2 * i] - f.x, v[2 * i + 1] - f.y);
        h[i] = *reinterpret_cast<const uint32_t*>(&x);
        l[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// 16 adjacent values of the product at (row, col) of the matrix into the staging area: `sr` is the
// row there, `sc` the column of the 64 that are staged.  Tall results go straight out: a warp's lanes
// are adjacent rows, which are adjacent in memory.
__device__ __forceinline__ void stage16(const PParams& p, int u, int row, int col, uint8_t* area, int rows, int sr, int sc,
                                        float (&v)[16]) {
    const float f = p.scale / (SX * SP);
    if (p.kind >= OUT_F32) {
        if (p.tall) {
            if (row < p.M)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (col + e < p.N) {
                        const long long at = ((long long)u * p.N + col + e) * p.M + row;
                        if (p.kind == OUT_F32)
                            static_cast<float*>(p.out)[at] = v[e] * f;
                        else
                            static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v[e] * f);
                    }
        } else if (p.kind == OUT_F32) {
            float* o = reinterpret_cast<float*>(area) + sr * 68 + sc;
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<float4*>(o + e) = make_float4(v[e] * f, v[e + 1] * f, v[e + 2] * f, v[e + 3] * f);
        } else {
            uint32_t* o = reinterpret_cast<uint32_t*>(area) + (sr * STG + sc) / 2;
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                *reinterpret_cast<uint4*>(o + e) =
                    make_uint4(pack_bf16(v[2 * e] * f, v[2 * e + 1] * f), pack_bf16(v[2 * e + 2] * f, v[2 * e + 3] * f),
                               pack_bf16(v[2 * e + 4] * f, v[2 * e + 5] * f), pack_bf16(v[2 * e + 6] * f, v[2 * e + 7] * f));
        }
        return;
    }
    __half* o = reinterpret_cast<__half*>(area) + sr * STG + sc;
    const int arr = rows * STG;  // halves of one staged array: y hi, y lo, y2 hi, y2 lo
    uint4 hi, lo;
    float w[16];
    const float m = p.kind == GRAM ? 1.f / SX : p.kind == NEXT ? 1.f / SP : SP / (SX * SQ);
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = v[e] * m + (p.kind == POLY && row == col + e ? SP * p.ca : 0.f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        split8(w + 8 * h, hi, lo);
        *reinterpret_cast<uint4*>(o + 8 * h) = hi;
        if (p.parts == 2) *reinterpret_cast<uint4*>(o + arr + 8 * h) = lo;
    }
    if (p.kind == GRAM) {
        // Q = b I + c A of the A that was computed, not of its rounded parts
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = SQ * (p.cc / (SX * SX) * v[e] + (row == col + e ? p.cb : 0.f));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            split8(w + 8 * h, hi, lo);
            *reinterpret_cast<uint4*>(o + 2 * arr + 8 * h) = hi;
            *reinterpret_cast<uint4*>(o + 3 * arr + 8 * h) = lo;
        }
    }
}
// The staged 64 columns of `rows` rows (matrix rows row0.., columns col0..) out to memory, by 128 threads
__device__ __forceinline__ void flush64(const PParams& p, int u, int row0, int col0, const uint8_t* area, int rows, int tid) {
    const long long mat = (long long)p.M * p.ld;
    if (p.kind >= OUT_F32) {
        if (p.tall) return;
        const long long base = (long long)u * p.M * p.N;
        const int per = p.kind == OUT_F32 ? 4 : 8, lanes = 64 / per;  // 16-byte pieces of a row
        const bool whole = p.N % per == 0;
        for (int i = tid; i < rows * lanes; i += 128) {
            const int r = i / lanes, c = i % lanes * per;
            if (row0 + r >= p.M) continue;
            const long long at = base + (long long)(row0 + r) * p.N + col0 + c;
            if (p.kind == OUT_F32) {
                const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(area) + r * 68 + c);
                float* o = static_cast<float*>(p.out) + at;
                if (whole) {
                    if (col0 + c < p.N) *reinterpret_cast<float4*>(o) = x;
                } else {
                    const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col0 + c + e < p.N) o[e] = xs[e];
                }
            } else {
                const __nv_bfloat16* s = reinterpret_cast<const __nv_bfloat16*>(area) + r * STG + c;
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
                if (whole) {
                    if (col0 + c < p.N) *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(s);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (col0 + c + e < p.N) o[e] = s[e];
                }
            }
        }
        return;
    }
    const int arrays = p.kind == GRAM ? 4 : p.parts;
    for (int a = 0; a < arrays; ++a) {
        __half* y = (a < 2 ? p.y : p.y2) + ((long long)u * 2 + (a & 1)) * mat;
        if (a == 1 && p.parts == 1) continue;
        const __half* s = reinterpret_cast<const __half*>(area) + a * rows * STG;
        for (int i = tid; i < rows * 8; i += 128) {
            const int r = i / 8, c = i % 8 * 8;
            if (row0 + r < p.M && col0 + c < p.ld)
                *reinterpret_cast<uint4*>(y + (long long)(row0 + r) * p.ld + col0 + c) =
                    *reinterpret_cast<const uint4*>(s + r * STG + c);
        }
    }
}

// One K block of a symmetric operand's rows t * 128 ..: K-major from its own tiles, which lie on or
// above the diagonal, or from the mirror image, MN-major
__device__ __forceinline__ void load_symmetric(uint8_t* dst, const CUtensorMap* km, const CUtensorMap* mn, int t, int k, int z,
                                               uint64_t* bar) {
    if (k / TM >= t) {
        tma_load_3d(dst, km, k, t * TM, z, bar);
    } else {
        tma_load_3d(dst, mn, t * TM, k, z, bar);
        tma_load_3d(dst + OPB / 2, mn, t * TM + 64, k, z, bar);
    }
}

// Operands' tensor maps over [2 u + part][rows][ld], by rows of K (box 64 x 128: k) and by 64 x 64 blocks
// (mn).  GRAM: both operands X, K-major.  POLY: A and Q, symmetric.  NEXT, OUT: P, symmetric, and X, MN-major.
struct Maps {
    CUtensorMap first_k, first_mn, second_k, second_mn;
};
template <typename C>
__global__ void __launch_bounds__(THREADS, C::MINB) product_kernel(const __grid_constant__ Maps maps, const PParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_align<1024>(smem_raw);
    PBars* bars = reinterpret_cast<PBars*>(ring + C::RING);
    const int S = gridDim.x, r = blockIdx.x, u = blockIdx.z;  // cluster (S, 1, 1)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int bi, bj;
    if (p.kind <= POLY) {  // tile of the upper triangle, column by column
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
        tma_prefetch_desc(&maps.first_k);
        tma_prefetch_desc(p.kind <= POLY ? &maps.second_k : &maps.second_mn);
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        mbar_init(&bars->done, 1);
        mbar_fence_init();
    }
    if (warp == 1) tc::alloc(&bars->tmem_base, C::COLS);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    griddep_wait();
    griddep_launch();
    const uint32_t tmem = bars->tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < nk; ++i) {
                const int slot = i % C::STAGES, use = i / C::STAGES;
                if (use > 0) mbar_wait(&bars->empty[slot], (use - 1) & 1, TTT_DEVERR_TIMEOUT_TMA);
                uint8_t* dst = ring + slot * C::STAGE;
                uint64_t* bar = &bars->full[slot];
                const int k = (k0 + i) * KB;
                mbar_expect_tx(bar, C::STAGE);
                for (int part = 0; part < 1 + C::FL; ++part, dst += OPB) {
                    if (p.kind == GRAM)
                        tma_load_3d(dst, &maps.first_k, k, bi * TM, 2 * u + part, bar);
                    else
                        load_symmetric(dst, &maps.first_k, &maps.first_mn, bi, k, 2 * u + part, bar);
                }
                for (int part = 0; part < 1 + C::SL; ++part, dst += OPB) {
                    if (p.kind == GRAM) {
                        tma_load_3d(dst, &maps.second_k, k, bj * TM, 2 * u + part, bar);
                    } else if (p.kind == POLY) {
                        load_symmetric(dst, &maps.second_k, &maps.second_mn, bj, k, 2 * u + part, bar);
                    } else {
                        tma_load_3d(dst, &maps.second_mn, bj * TM, k, 2 * u + part, bar);
                        tma_load_3d(dst + OPB / 2, &maps.second_mn, bj * TM + 64, k, 2 * u + part, bar);
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int last = -1;  // the hi hi accumulator in use
            for (int i = 0; i < nk; ++i) {
                const int slot = i % C::STAGES, t = (k0 + i) * KB / TM;
                mbar_wait(&bars->full[slot], (i / C::STAGES) & 1, TTT_DEVERR_TIMEOUT_TMA);
                tc::fence_after();
                const int fm = p.kind != GRAM && t < bi, sm = p.kind >= NEXT || (p.kind == POLY && t < bj);  // MN-major
                const uint32_t fb = smem_u32(ring + slot * C::STAGE), sb = fb + (1 + C::FL) * OPB;
                const uint64_t fh = tc::smem_desc(fb, fm ? OPB / 2 : 16, 1024, 2), sh = tc::smem_desc(sb, sm ? OPB / 2 : 16, 1024, 2);
                const uint64_t lo = OPB >> 4, fstep = fm ? 128 : 2, sstep = sm ? 128 : 2;
                const uint32_t idesc = tc::idesc_f16(128, 128, 0, 0) | (uint32_t)fm << 15 | (uint32_t)sm << 16;
                const int acc = i * C::ACC / nk;
                const uint32_t to = tmem + acc * TM, cross = tmem + C::ACC * TM;
#pragma unroll
                for (int ks = 0; ks < KB / 16; ++ks) {
                    const uint64_t f = fh + fstep * ks, s = sh + sstep * ks;
                    tc::mma_bf16(to, f, s, idesc, acc == last);
                    last = acc;
                    if (C::SL) tc::mma_bf16(cross, f, s + lo, idesc, i > 0 || ks > 0);
                    if (C::FL) tc::mma_bf16(cross, f + lo, s, idesc, C::SL || i > 0 || ks > 0);
                }
                tc::commit(&bars->empty[slot]);
            }
            tc::commit(&bars->done);
        }
    }
    const int tid = threadIdx.x - 64, q4 = warp & 3;
    const uint32_t lane_base = tmem + ((uint32_t)(q4 * 32) << 16);
    const int used = nk > 0 ? (nk - 1) * C::ACC / nk + 1 : 0;
    // columns c .. c + 15 of the accumulators' sum, in the thread's row
    auto take = [&](int c, float (&v)[16]) {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
        if (nk == 0) return;
        float x[16];
        if (C::FL || C::SL) {
            tc::ld16(lane_base + C::ACC * TM + c, x);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = x[e];
        }
        for (int a = 0; a < used; ++a) {
            tc::ld16(lane_base + a * TM + c, x);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] += x[e];
        }
    };
    if (warp >= 2) {
        if (nk > 0) {
            mbar_wait(&bars->done, 0, TTT_DEVERR_TIMEOUT_TMA);
            tc::fence_after();
        }
        if (S == 1) {
            const int row = q4 * 32 + lane;
            for (int h = 0; h < 2; ++h) {
                for (int c = 0; c < 64; c += 16) {
                    float v[16];
                    take(64 * h + c, v);
                    stage16(p, u, bi * TM + row, bj * TM + 64 * h + c, ring, TM, row, c, v);
                }
                epilogue_sync();
                flush64(p, u, bi * TM, bj * TM + 64 * h, ring, TM, tid);
                epilogue_sync();
            }
        }
    }
    if (S > 1) {
        const int R = TM / S;                          // rows of a slice
        float* buf = reinterpret_cast<float*>(ring);   // [S][128 columns][R], over the ring
        cluster_sync_all();  // every CTA's MMAs have read their operands: the rings are free
        if (warp >= 2) {
            const int row = q4 * 32 + lane;
            const uint32_t to = dsmem_map(buf + r * TM * R + row % R, row / R);
            for (int c = 0; c < TM; c += 16) {
                float v[16];
                take(c, v);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4u * R * (c + e)), "f"(v[e]) : "memory");
            }
        }
        cluster_sync_all();
        if (warp >= 2) {
            uint8_t* area = ring + TM * TM * 4;
            const int groups = 128 / R, row = tid % R, g = tid / R;  // threads of a group: the slice's rows
            for (int h = 0; h < 2; ++h) {
                for (int c = 16 * g; c < 64; c += 16 * groups) {
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = 0.f;
                    for (int s = 0; s < S; ++s)
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] += buf[(s * TM + 64 * h + c + e) * R + row];
                    stage16(p, u, bi * TM + r * R + row, bj * TM + 64 * h + c, area, R, row, c, v);
                }
                epilogue_sync();
                flush64(p, u, bi * TM + r * R, bj * TM + 64 * h, area, R, tid);
                epilogue_sync();
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) tc::dealloc(tmem, C::COLS);
}

}  // namespace orth

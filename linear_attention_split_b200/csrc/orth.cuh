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
// (result good to about 2e-6 of its norm).  bf16 ones take them too, up to the last step: the iteration
// enlarges what is lost early by up to a^5 along small singular values, so with X and P in 11 bits at every
// step a direction 30, 100 or 1000 times the rest left 0.8, 2 or 9 % of the result's norm wrong.  In the last
// step (the last ones whose slopes multiply to at most 4: orth_high_from) X and P are held as hi alone and only
// A Q is taken in full, which costs less than rounding the result to bf16, whatever the spectrum (1.5e-3 to
// 2.3e-3 in all, measured; 1024 x 4096: 238 us, with hi alone at every step 157, in full throughout 263).
// Values are bounded (|s| <= 2 throughout, checked on the host), so fixed powers of two keep them inside fp16:
// X and A are stored times 2^12, P times 2^10, Q times 2^9.
//
// product_kernel: one tile of 128 x 64, 128 or 256 of a product per cluster; the K range is split over the S
// CTAs of the cluster when there are few tiles, and the partial tiles are exchanged through
// distributed shared memory (each CTA adds one slice of rows, in rank order: deterministic).  Per CTA
// a TMA producer and two tcgen05 issuers over a ring of 64-wide K blocks, and eight epilogue warps, which
// stage what they write so that rows go out whole (straight from the accumulator's layout, one row per
// lane, a tile took 5300 cycles; staged about a third).  A, Q and P are symmetric: only tiles on or
// above the diagonal are formed, and an operand block below it is read from its mirror image as an
// MN-major operand.  The tensor cores cut what falls below the accumulator's last bit at every
// addition, about 1e-7 of the result for each: a full product therefore spreads its K blocks over
// three or seven accumulators and keeps the cross terms in another, added in fp32 in the epilogue
// (1024 x 4096, one accumulator: 1.3e-5 of the norm, now 2.7e-6), and A Q and P X take the K blocks of a tile's own rows
// last: A's and P's diagonals make their sums large, and all that is added to a large sum is cut.  (In ascending order
// 4 x 1024 x 1024 was 8.0e-6 off, 2048 x 2048 1.5e-5 and 2048 x 8192 2.2e-5; now 3.0e-6, 3.1e-6 and 3.6e-6, the same steps in
// plain fp32 2.6e-6, 3.3e-6 and 4.5e-6.)
#pragma once
#include "common.cuh"
#include <cuda_fp16.h>
#include <type_traits>

namespace orth {

constexpr int TPB = 256;
constexpr int MAX_PARTS = 512;
constexpr float SX = 4096.f, SP = 1024.f;  // scale of stored X and A, and of stored P

// part[u][p] = sum of squares of piece p of matrix u; 16 bytes a load where the matrices allow it
template <typename T>
__global__ void __launch_bounds__(TPB) square_kernel(const T* __restrict__ x, double* __restrict__ part, long long mn) {
    __shared__ double sm[TPB / 32];
    constexpr int VEC = 16 / sizeof(T);
    struct alignas(16) Lane {
        T v[VEC];
    };
    griddep_wait();
    griddep_launch();
    const T* xu = x + blockIdx.y * mn;
    const long long first = (long long)blockIdx.x * TPB + threadIdx.x, stride = (long long)gridDim.x * TPB;
    double s = 0.0;
    if (mn % VEC == 0) {
#pragma unroll 4
        for (long long i = first; i < mn / VEC; i += stride) {
            const Lane l = reinterpret_cast<const Lane*>(xu)[i];
#pragma unroll
            for (int e = 0; e < VEC; ++e) s = fma((double)to_f(l.v[e]), (double)to_f(l.v[e]), s);
        }
    } else {
#pragma unroll 4
        for (long long i = first; i < mn; i += stride) s = fma((double)to_f(xu[i]), (double)to_f(xu[i]), s);
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

// the parts' sum, the same in every thread of the block (a warp's lanes take every 32nd, in order)
__device__ __forceinline__ double sum_parts(const double* part, int parts) {
    double s = 0.0;
    for (int p = threadIdx.x & 31; p < parts; p += 32) s += part[p];
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// X [u][hi, lo][M][ld] (hi alone with halves = 1) from x, zero in columns N .. ld - 1.  Any shape, a tall x
// transposed on the way: 32 x 32 tiles through shared memory, so that both sides go along rows.
template <typename T>
__global__ void __launch_bounds__(256)
    start_kernel(const T* __restrict__ x, const double* __restrict__ part, __half* __restrict__ y, int parts, int M,
                 int N, int ld, int tall, int halves, float eps) {
    __shared__ float sm[32][33];
    griddep_wait();
    griddep_launch();
    const int u = blockIdx.z, i0 = blockIdx.y * 32, j0 = blockIdx.x * 32;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const T* xu = x + (long long)u * M * N;
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = ty + 8 * k, i = tall ? i0 + tx : i0 + r, j = tall ? j0 + r : j0 + tx;
        v[k] = i < M && j < N ? to_f(xu[tall ? (long long)j * M + i : (long long)i * N + j]) : 0.f;
    }
    const double inv = inverse_norm(sum_parts(part + (long long)u * parts, parts), eps) * SX;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = ty + 8 * k;
        const float f = (float)((double)v[k] * inv);
        if (tall)
            sm[tx][r] = f;
        else
            sm[r][tx] = f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = i0 + ty + 8 * k, j = j0 + tx;
        if (i >= M || j >= ld) continue;
        __half* yu = y + (long long)u * 2 * M * ld + (long long)i * ld + j;
        __half lo;
        split(sm[ty + 8 * k][tx], yu[0], lo);
        if (halves == 2) yu[(long long)M * ld] = lo;
    }
}
// The same for wide matrices whose size is a multiple of 8 (then ld = N and nothing is padded): eight
// adjacent values a thread.
template <typename T>
__global__ void __launch_bounds__(256)
    start8_kernel(const T* __restrict__ x, const double* __restrict__ part, __half* __restrict__ y, int parts, long long mn,
                  int halves, float eps) {
    struct alignas(16) Lane {
        T v[8];
    };
    griddep_wait();
    griddep_launch();
    const long long u = blockIdx.y, i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8;
    Lane l;
    if (i < mn) l = *reinterpret_cast<const Lane*>(x + u * mn + i);
    const double inv = inverse_norm(sum_parts(part + u * parts, parts), eps) * SX;
    if (i >= mn) return;
    __align__(16) __half hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) split((float)((double)to_f(l.v[e]) * inv), hi[e], lo[e]);
    __half* o = y + u * 2 * mn + i;
    *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(hi);
    if (halves == 2) *reinterpret_cast<uint4*>(o + mn) = *reinterpret_cast<const uint4*>(lo);
}

constexpr int TM = 128, KB = 64;                     // rows of a tile of the output, K block
constexpr int PANEL = 64 * KB * 2;                   // a K block of 64 rows or columns, 8 KB
constexpr int OPB = 2 * PANEL;                       // the first operand's K block
constexpr float SQ = 512.f;                          // scale of stored Q

enum Kind { GRAM = 0, POLY = 1, NEXT = 2, OUT_F32 = 3, OUT_BF16 = 4 };

struct PParams {
    int kblocks;             // K blocks of the whole product
    int M, tiles_n;          // rows of X, A, Q and P; tiles along the columns (NEXT, OUT)
    int ld;                  // row stride of the halves that are written (GRAM, POLY, NEXT), columns written
    int parts;               // 2: hi and lo are written, 1: hi alone
    __half* y;               // where they go, [u][hi, lo][M][ld]
    __half* y2;              // GRAM: Q, same shape
    void* out;               // OUT: [u][M][N], or [u][N][M] when tall
    int N, tall;
    float ca, cb, cc, scale;
};
constexpr int MAX_STAGES = 8;
struct PBars {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES], done;
    uint32_t tmem_base;
};
constexpr int STG = 40;                             // padded row of 32 staged halves (16-byte rows); floats: 36
__host__ __device__ constexpr int stage_area(int rows) { return rows * STG * 2 * 4; }  // of one column half: four arrays of halves
// What a product takes: FL, SL: the first / second operand's lo part as well; BN columns of a tile; ACC
// accumulators for hi hi (and one for the cross terms, if any); STAGES K blocks in flight.  One CTA on an SM.
template <bool FL_, bool SL_, int BN_, int ACC_, int STAGES_>
struct Config {
    static constexpr bool FL = FL_, SL = SL_;
    static constexpr int BN = BN_, ACC = ACC_, STAGES = STAGES_;
    static constexpr int SECOND = BN / 64 * PANEL;                 // the second operand's K block
    static constexpr int STAGE = (1 + FL) * OPB + (1 + SL) * SECOND;
    static constexpr bool CROSS = FL || SL;
    static constexpr int ACCS = ACC + CROSS;
    static constexpr int FRONT = 96, THREADS = FRONT + 256;  // producer and two issuers; eight epilogue warps
    static_assert(CROSS || (ACC == 2 && STAGES % 2 == 0), "hi hi alone: an accumulator and slots of its own for each issuer");
    static constexpr int COLS = ACCS * BN;                         // of tensor memory
    static constexpr int EXCHANGE = BN > 128 ? 0 : TM * BN * 4;    // the S partial slices of a tile
    // the ring; over it the exchange and what is staged
    static constexpr int USED = EXCHANGE + 2 * stage_area(TM / 2);
    static constexpr int RING = STAGES * STAGE > USED ? STAGES * STAGE : USED;
    static constexpr int SMEM = RING + (int)sizeof(PBars) + 1024;
    static_assert(RING >= 2 * stage_area(TM) && STAGES <= MAX_STAGES && COLS <= 512 && (COLS & (COLS - 1)) == 0, "");
    // cycles of a K block: its MMAs (measured 53, 67 and 131 for 128 x 64, 128 and 256 x 16), or its loads at
    // the 92 bytes a cycle that an SM gets
    static constexpr int MMA = 4 * (1 + FL + SL) * (BN == 64 ? 53 : BN == 128 ? 67 : 131);
    static constexpr int BLOCK = MMA > STAGE / 92 ? MMA : STAGE / 92;
};
// hi hi + hi lo + lo hi, and hi hi alone
template <int BN>
using Full = Config<true, true, BN, BN == 64 ? 7 : 3, BN == 64 ? 4 : 3>;
template <int BN>
using High = Config<false, false, BN, 2, BN == 64 ? 8 : BN == 128 ? 6 : 4>;

__device__ __forceinline__ void group_sync(int g) {
    if (g == 0)
        asm volatile("bar.sync 1, 128;" ::: "memory");
    else
        asm volatile("bar.sync 2, 128;" ::: "memory");
}
// four values as fp16 hi and lo
__device__ __forceinline__ void split4(const float (&v)[4], uint2& hi, uint2& lo) {
    const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
    const float2 fa = __half22float2(a), fb = __half22float2(b);
    const __half2 c = __floats2half2_rn(v[0] - fa.x, v[1] - fa.y), d = __floats2half2_rn(v[2] - fb.x, v[3] - fb.y);
    hi = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    lo = make_uint2(*reinterpret_cast<const uint32_t*>(&c), *reinterpret_cast<const uint32_t*>(&d));
}

// Four adjacent values of the product at (row, col) of the matrix into the staging area (`rows` rows, four
// arrays y hi, y lo, y2 hi, y2 lo): `sr` is the row there, `sc` the column of the 32 that are staged.
template <int KIND>
__device__ __forceinline__ void stage4(const PParams& p, int row, int col, uint8_t* area, int rows, int sr, int sc, const float (&v)[4]) {
    if constexpr (KIND == OUT_F32) {
        const float f = p.scale / (SX * SP);
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(area) + sr * 36 + sc) = make_float4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
    } else if constexpr (KIND == OUT_BF16) {
        const float f = p.scale / (SX * SP);
        *reinterpret_cast<uint2*>(area + (sr * STG + sc) * 2) = make_uint2(pack_bf16(v[0] * f, v[1] * f), pack_bf16(v[2] * f, v[3] * f));
    } else {
        uint8_t* o = area + (sr * STG + sc) * 2;
        const int arr = rows * STG * 2;
        uint2 hi, lo;
        float w[4];
        constexpr float m = KIND == GRAM ? 1.f / SX : KIND == NEXT ? 1.f / SP : SP / (SX * SQ);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = v[e] * m + (KIND == POLY && row == col + e ? SP * p.ca : 0.f);
        split4(w, hi, lo);
        *reinterpret_cast<uint2*>(o) = hi;
        *reinterpret_cast<uint2*>(o + arr) = lo;
        if constexpr (KIND == GRAM) {  // Q = b I + c A, of the A that was computed, not of its rounded parts
            const float f = SQ * p.cc / (SX * SX);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = v[e] * f + (row == col + e ? SQ * p.cb : 0.f);
            split4(w, hi, lo);
            *reinterpret_cast<uint2*>(o + 2 * arr) = hi;
            *reinterpret_cast<uint2*>(o + 3 * arr) = lo;
        }
    }
}
// The staged 32 columns of ROWS rows (matrix rows row0.., columns col0..) out to memory, by 128 threads
template <int KIND, int ROWS>
__device__ __forceinline__ void flush32(const PParams& p, int u, int row0, int col0, const uint8_t* area, int tid) {
    if constexpr (KIND >= OUT_F32) {
        using T = std::conditional_t<KIND == OUT_F32, float, __nv_bfloat16>;
        constexpr int per = 16 / sizeof(T), lanes = 32 / per, pitch = KIND == OUT_F32 ? 36 : STG;
        const T* s = reinterpret_cast<const T*>(area);
        T* out = static_cast<T*>(p.out) + (long long)u * p.M * p.N;
        if (p.tall) {  // out [N][M]: adjacent threads take adjacent rows of the tile
            const int r = tid % ROWS;
            T* o = out + (long long)(col0 + tid / ROWS) * p.M + row0 + r;
            if (row0 + r < p.M)
#pragma unroll 8
                for (int c = tid / ROWS; c < 32; c += 128 / ROWS, o += (long long)(128 / ROWS) * p.M)
                    if (col0 + c < p.N) *o = s[r * pitch + c];
            return;
        }
        const bool whole = p.N % per == 0;
        const int c = tid % lanes * per;
        constexpr int STEP = 128 / lanes;
        T* o = out + (long long)(row0 + tid / lanes) * p.N + col0 + c;
        if (col0 + c < p.N)
#pragma unroll
            for (int r = tid / lanes; r < ROWS; r += STEP, o += (long long)STEP * p.N) {
                if (row0 + r >= p.M) break;
                if (whole) {
                    *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(s + r * pitch + c);
                } else {
#pragma unroll
                    for (int e = 0; e < per; ++e)
                        if (col0 + c + e < p.N) o[e] = s[r * pitch + c + e];
                }
            }
    } else {
        const long long mat = (long long)p.M * p.ld;
        const int c = tid % 4 * 8, r0 = tid / 4;  // 32 rows at a time
        if (col0 + c >= p.ld) return;
        const long long at = u * 2 * mat + (long long)(row0 + r0) * p.ld + col0 + c;
#pragma unroll
        for (int a = 0; a < (KIND == GRAM ? 4 : 2); ++a) {
            if (a == 1 && KIND != GRAM && p.parts == 1) break;
            __half* y = (a < 2 ? p.y : p.y2) + at + (a & 1) * mat;
            const uint8_t* s = area + (a * ROWS * STG + r0 * STG + c) * 2;
#pragma unroll
            for (int r = 0; r < (ROWS + 31) / 32; ++r)
                if (32 * r + r0 < ROWS && row0 + 32 * r + r0 < p.M)
                    *reinterpret_cast<uint4*>(y + (long long)(32 * r) * p.ld) = *reinterpret_cast<const uint4*>(s + 32 * r * STG * 2);
        }
    }
}
// The slice of 128 / S rows that this CTA owns, columns col0 .. col0 + BN / 2 - 1: the S partials added in rank order
template <int KIND, int BN, int S>
__device__ __forceinline__ void finish_slice(const PParams& p, int u, int row0, int col0, const float* buf, uint8_t* areas, int g,
                                             int tid) {
    constexpr int R = TM / S, PW = R / 4;  // rows; a thread's columns of each 32
    uint8_t* area = areas + g * stage_area(R);
    const int sr = tid % R, sc = tid / R * PW;
#pragma unroll 1
    for (int c0 = 0; c0 < BN / 2; c0 += 32) {
        const float* b = buf + (BN / 2 * g + c0 + sc) * R + sr;
        float v[PW];
#pragma unroll
        for (int c = 0; c < PW; ++c) v[c] = b[c * R];
#pragma unroll
        for (int s = 1; s < S; ++s)
#pragma unroll
            for (int c = 0; c < PW; ++c) v[c] += b[(s * BN + c) * R];
#pragma unroll
        for (int c = 0; c < PW; c += 4)
            stage4<KIND>(p, row0 + sr, col0 + c0 + sc + c, area, R, sr, sc + c, {v[c], v[c + 1], v[c + 2], v[c + 3]});
        group_sync(g);
        flush32<KIND, R>(p, u, row0, col0 + c0, area, tid);
        group_sync(g);
    }
}

// One K block of rows at .. at + rows - 1 of a symmetric operand: K-major from its own tiles, which lie on
// or above the diagonal (in blocks of 128), or from the mirror image, MN-major in panels of 64
__device__ __forceinline__ void load_symmetric(uint8_t* dst, const CUtensorMap* km, const CUtensorMap* mn, int at, int rows, int k,
                                               int z, uint64_t* bar) {
    if (k / TM >= at / TM) {
        tma_load_3d(dst, km, k, at, z, bar);
    } else {
        for (int c = 0; c < rows; c += 64) tma_load_3d(dst + c / 64 * PANEL, mn, at + c, k, z, bar);
    }
}

// Operands' tensor maps over [2 u + part][rows][ld], by rows of K (box 64 x 128, the second's 64 x BN: k)
// and by 64 x 64 blocks (mn).  GRAM: both operands X, K-major.  POLY: A and Q, symmetric.  NEXT, OUT: P, symmetric, and X, MN-major.
struct Maps {
    CUtensorMap first_k, first_mn, second_k, second_mn;
};
template <typename C, int KIND>
__global__ void __launch_bounds__(C::THREADS, 1) product_kernel(const __grid_constant__ Maps maps, const PParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_align<1024>(smem_raw);
    PBars* bars = reinterpret_cast<PBars*>(ring + C::RING);
    const int S = gridDim.x, r = blockIdx.x, u = blockIdx.z;  // cluster (S, 1, 1)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int bi = blockIdx.y / p.tiles_n, bj = blockIdx.y % p.tiles_n;
    if (KIND <= POLY) {  // tiles on or above the diagonal, row by row
        int t = blockIdx.y;
        for (bi = 0; t >= p.tiles_n - bi * TM / C::BN; ++bi) t -= p.tiles_n - bi * TM / C::BN;
        bj = bi * TM / C::BN + t;
    }
    const int i0 = bi * TM, j0 = bj * C::BN;  // the tile's place
    const int per = (p.kblocks + S - 1) / S, k0 = min(r * per, p.kblocks), nk = min(per, p.kblocks - k0);
    // A Q and P X take the CTA's K blocks in a circle that ends with those of the tile's own rows, if they are among them
    int turn = 0;
    if (KIND >= POLY) {
        const int last = min(2 * bi + 1, p.kblocks - 1) - k0;
        if (last >= 0 && last < nk) turn = last + 1 < nk ? last + 1 : 0;
    }
    // accumulators for hi hi: `used` of them, each for a run of `len` of the 4 nk MMAs (hi hi alone: one for
    // each issuer)
    const int len = (4 * nk + C::ACC - 1) / C::ACC;
    const int used = !C::CROSS ? min(nk, 2) : nk > 0 ? (4 * nk + len - 1) / len : 0;
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&maps.first_k);
        tma_prefetch_desc(KIND <= POLY ? &maps.second_k : &maps.second_mn);
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], C::CROSS ? 2 : 1);
        }
        mbar_init(&bars->done, 2);
        mbar_fence_init();
    }
    if (warp == 1) tc::alloc(&bars->tmem_base, C::COLS);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    griddep_wait();
    griddep_launch();
    const uint32_t tmem = bars->tmem_base;

    // The MMAs of one issuing thread.  A thread spends about 300 cycles a K block on its barriers (a test of a
    // phase that is over already takes 200) while the tensor cores wait, so there are two: with cross terms the
    // first issues hi hi and the second the rest, hi hi alone they take alternate K blocks.  Either way each has
    // accumulators of its own, so nothing depends on how the two interleave (one issuer against two: 1024 x 1024
    // fp32 155 against 138 us, 1024 x 4096 bf16 180 against 163).  The issuer's number is a constant: addresses
    // that come from the thread's index cost a move to the uniform registers for each MMA (384 x 1536 fp32 113 us
    // that way, 97 so).
    auto issue = [&](auto issuer) {
        constexpr int j = decltype(issuer)::value;
        int acc = C::CROSS ? 0 : j, count = 0;  // the hi hi accumulator in use, and its MMAs so far
        bool ready = false;
        constexpr int FROM = C::CROSS ? 0 : j, STEP = C::CROSS ? 1 : 2;
        for (int i = FROM; i < nk; i += STEP) {
            const int slot = i % C::STAGES, t = (k0 + (i + turn < nk ? i + turn : i + turn - nk)) * KB / TM;
            if (!ready) mbar_wait(&bars->full[slot], (i / C::STAGES) & 1, TTT_DEVERR_TIMEOUT_TMA);
            const int n = i + STEP;  // the next block's phase is asked for ahead of this block's MMAs
            ready = n < nk && mbar_test_wait(&bars->full[n % C::STAGES], (n / C::STAGES) & 1);
            tc::fence_after();
            const int fm = KIND != GRAM && t < bi, sm = KIND >= NEXT || (KIND == POLY && t < j0 / TM);  // MN-major
            const uint32_t fb = smem_u32(ring + slot * C::STAGE), sb = fb + (1 + C::FL) * OPB;
            const uint64_t fh = tc::smem_desc(fb, fm ? PANEL : 16, 1024, 2), sh = tc::smem_desc(sb, sm ? PANEL : 16, 1024, 2);
            const uint64_t fstep = fm ? 128 : 2, sstep = sm ? 128 : 2;
            const uint32_t idesc = tc::idesc_f16(TM, C::BN, 0, 0) | (uint32_t)fm << 15 | (uint32_t)sm << 16;
            const uint32_t cross = tmem + C::ACC * C::BN;
#pragma unroll
            for (int ks = 0; ks < KB / 16; ++ks) {
                const uint64_t f = fh + fstep * ks, s = sh + sstep * ks;
                if (!C::CROSS || j == 0) {
                    if (C::CROSS && count == len) {
                        ++acc;
                        count = 0;
                    }
                    tc::mma_bf16(tmem + acc * C::BN, f, s, idesc, count++ > 0);
                } else {
                    if (C::SL) tc::mma_bf16(cross, f, s + (C::SECOND >> 4), idesc, i > 0 || ks > 0);
                    if (C::FL) tc::mma_bf16(cross, f + (OPB >> 4), s, idesc, C::SL || i > 0 || ks > 0);
                }
            }
            tc::commit(&bars->empty[slot]);
        }
        if (nk > 0) tc::commit(&bars->done);  // nobody waits for a CTA without K blocks
    };
    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < nk; ++i) {
                const int slot = i % C::STAGES, use = i / C::STAGES;
                if (use > 0) mbar_wait(&bars->empty[slot], (use - 1) & 1, TTT_DEVERR_TIMEOUT_TMA);
                uint8_t* dst = ring + slot * C::STAGE;
                uint64_t* bar = &bars->full[slot];
                const int k = (k0 + (i + turn < nk ? i + turn : i + turn - nk)) * KB;
                mbar_expect_tx(bar, C::STAGE);
                for (int part = 0; part < 1 + C::FL; ++part, dst += OPB) {
                    if (KIND == GRAM)
                        tma_load_3d(dst, &maps.first_k, k, i0, 2 * u + part, bar);
                    else
                        load_symmetric(dst, &maps.first_k, &maps.first_mn, i0, TM, k, 2 * u + part, bar);
                }
                for (int part = 0; part < 1 + C::SL; ++part, dst += C::SECOND) {
                    if (KIND == GRAM) {
                        tma_load_3d(dst, &maps.second_k, k, j0, 2 * u + part, bar);
                    } else if (KIND == POLY) {
                        load_symmetric(dst, &maps.second_k, &maps.second_mn, j0, C::BN, k, 2 * u + part, bar);
                    } else {
                        for (int c = 0; c < C::BN; c += 64)
                            tma_load_3d(dst + c / 64 * PANEL, &maps.second_mn, j0 + c, k, 2 * u + part, bar);
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) issue(std::integral_constant<int, 0>());
    } else if (warp == 2) {
        if (lane == 0) issue(std::integral_constant<int, 1>());
    }
    // Epilogue: two groups of four warps, each taking half of the columns; a warp reads the 32 lanes (rows)
    // of its quarter of tensor memory.
    constexpr int HALF = C::BN / 2;
    constexpr int FIRST = C::FRONT / 32;  // epilogue warp
    const int g = (warp - FIRST) >> 2, tid = (threadIdx.x - C::FRONT) & 127, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    // columns c .. c + 15 of the accumulators' sum, in the thread's row
    auto take = [&](int c, float (&v)[16]) {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
#pragma unroll
        for (int a0 = 0; a0 < C::ACCS; a0 += 4) {  // four accumulators' loads in flight
            float x[4][16];
#pragma unroll
            for (int a = 0; a < 4; ++a)
                if (a0 + a < C::ACCS) tc::ld16(lane_base + (a0 + a) * C::BN + c, x[a]);
            tc::wait_ld();
#pragma unroll
            for (int a = 0; a < 4; ++a)
                if (a0 + a < used || (C::CROSS && a0 + a == C::ACC && used > 0))
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] += a0 + a < C::ACCS ? x[a][e] : 0.f;
        }
    };
    if (warp >= FIRST) {
        if (nk > 0) {
            mbar_wait(&bars->done, 0, TTT_DEVERR_TIMEOUT_TMA);
            tc::fence_after();
        }
        if (S == 1) {
            uint8_t* area = ring + g * stage_area(TM);
#pragma unroll 1
            for (int c0 = HALF * g; c0 < HALF * g + HALF; c0 += 32) {
#pragma unroll
                for (int c = 0; c < 32; c += 16) {
                    float v[16];
                    take(c0 + c, v);
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        stage4<KIND>(p, i0 + row, j0 + c0 + c + e, area, TM, row, c + e, {v[e], v[e + 1], v[e + 2], v[e + 3]});
                }
                group_sync(g);
                flush32<KIND, TM>(p, u, i0, j0 + c0, area, tid);
                group_sync(g);
            }
        }
    }
    if (C::EXCHANGE > 0 && S > 1) {
        const int R = TM / S;                          // rows of a slice
        float* buf = reinterpret_cast<float*>(ring);   // [S][BN columns][R], over the ring
        cluster_sync_all();  // every CTA's MMAs have read their operands: the rings are free
        if (warp >= FIRST) {
            float* here = buf + r * C::BN * R + row % R;
            const uint32_t there = dsmem_map(here, row / R);
#pragma unroll 1
            for (int c = HALF * g; c < HALF * g + HALF; c += 16) {
                float v[16];
                take(c, v);
                if (row / R == r)
#pragma unroll
                    for (int e = 0; e < 16; ++e) here[R * (c + e)] = v[e];
                else
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there + 4u * R * (c + e)), "f"(v[e]) : "memory");
            }
        }
        cluster_sync_all();
        if (warp >= FIRST) {
            const int row0 = i0 + r * R, col0 = j0 + HALF * g;
            if (S == 2)
                finish_slice<KIND, C::BN, 2>(p, u, row0, col0, buf, ring + C::EXCHANGE, g, tid);
            else if (S == 4)
                finish_slice<KIND, C::BN, 4>(p, u, row0, col0, buf, ring + C::EXCHANGE, g, tid);
            else
                finish_slice<KIND, C::BN, 8>(p, u, row0, col0, buf, ring + C::EXCHANGE, g, tid);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) tc::dealloc(tmem, C::COLS);
}

}  // namespace orth
